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

// Inclusive sum over the wave's lanes (every lane active).
__device__ inline int64_t wave_scan_sum(int64_t v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// The sequence that holds unit `item` when sequence b has count(b) of them in
// order, and the unit's number within it; false if there are fewer units.
// Every lane of the wave takes part and gets the same answer.
template <class F>
__device__ inline bool find_sequence(int64_t seqs, int64_t item, int lane, int64_t& seq,
                                     int64_t& local, F&& count) {
  int64_t base = 0;
  for (int64_t b0 = 0; b0 < seqs; b0 += 64) {
    const int64_t b = b0 + lane, c = b < seqs ? count(b) : 0;
    const int64_t end = base + wave_scan_sum(c, lane);
    const uint64_t past = __ballot(end > item);
    if (past) {
      const int src = __ffsll((unsigned long long)past) - 1;
      seq = b0 + src;
      local = item - __shfl(end - c, src, 64);
      return true;
    }
    base = __shfl(end, 63, 64);
  }
  return false;
}

}  // namespace sparq24
