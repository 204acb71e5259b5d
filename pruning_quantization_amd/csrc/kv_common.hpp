// Paged 8-bit key/value cache as the append and attention kernels see it.
//
// A pool of blocks of T tokens (T = 1 << tsh, 16..256).  Per block and kv
// head: K codes [T][D], V codes [D][T] (both reductions of attention run over
// contiguous bytes: q.k along D, p.v along the tokens), and one fp32 scale
// each.  Position p of sequence b lives in block table[b][p >> tsh], row
// p & (T - 1).  A table entry outside 0 .. blocks - 1 names no block: nothing
// is written there and attention sees no tokens in it, so bad tables never
// become addresses.
#pragma once

#include "device_common.hpp"
#include "launch_serving.hpp"

namespace sparq24 {

// Rows of the token tensors and tokens in the cache of one sequence.
struct SeqRows {
  int first, n;  // rows first .. first + n - 1
  int len;       // tokens in the cache, new ones included
};

__device__ inline SeqRows seq_rows(const KvSeqs& q, int64_t b) {
  SeqRows r;
  if (q.cu) {
    const int total = (int)q.total;
    const int lo = q.cu[b], hi = q.cu[b + 1];
    r.first = lo < 0 ? 0 : (lo > total ? total : lo);
    const int end = hi < r.first ? r.first : (hi > total ? total : hi);
    r.n = end - r.first;
  } else {
    r.first = (int)(b * q.nper);
    r.n = (int)q.nper;
  }
  const int len = q.lens[b];
  r.len = len < 0 ? 0 : len;
  return r;
}

// Inclusive sum over the wave's lanes (every lane active), by DPP: within rows of
// 16 lanes, then across them.
__device__ inline uint32_t wave_scan_sum(uint32_t v) {
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, true);   // row_shr:1
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, true);   // row_shr:2
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, true);   // row_shr:4
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, true);   // row_shr:8
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false);  // row_bcast:15
  v += (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false);  // row_bcast:31
  return v;
}

// Counts of one sequence are held below 2^26, so that 64 of them add up in 32 bits
// (the calls' size limits keep sane ones below it; offsets that do not ascend
// can ask for more, and then get fewer units than they asked for).
constexpr int64_t kMostUnits = (1 << 26) - 1;

// The sequence that holds unit `item` when sequence b has count(b) of them in
// order, and the unit's number within it; false if there are fewer units.
// Every lane of the wave takes part and gets the same answer (scalars).
template <class F>
__device__ inline bool find_sequence(int64_t seqs, int64_t item, int lane, int& seq, int& local, F&& count) {
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < seqs; b0 += 64) {
    const int64_t b = b0 + lane, n = b < seqs ? count(b) : 0;
    const uint32_t c = (uint32_t)(n < kMostUnits ? n : kMostUnits), end = wave_scan_sum(c);
    const uint64_t past = __ballot((int64_t)end > item - base);
    if (past) {
      const int src = __ffsll((unsigned long long)past) - 1;
      seq = (int)b0 + src;
      local = (int)(item - base) - __builtin_amdgcn_readlane((int)(end - c), src);
      return true;
    }
    base += (uint32_t)__builtin_amdgcn_readlane((int)end, 63);
  }
  return false;
}

// The last i of 0 .. n - 1 with reached(i), true for i = 0 and a prefix: the wave
// looks at 64 places at a time, so at most 64 need one round of loads, 4096 two.
// Every lane of the wave takes part and gets the same answer (a scalar).
template <class F>
__device__ inline int last_reached(int n, int lane, F&& reached) {
  int at = 0;
  while (n > 1) {
    const int step = (n + 63) / 64, i = lane * step;
    const int k = __popcll(__ballot(i < n && (i == 0 || reached(at + i)))) - 1;
    at += k * step;
    n = n - k * step < step ? n - k * step : step;
  }
  return at;
}

}  // namespace sparq24
