// Work of a kv_attention launch, for both kinds of cache: which sequence, row tile and
// chunk of tokens a workgroup has, the ranges of tokens that its rows see, and the
// join of split sequences (kernels_kv_split.hip).
#pragma once

#include "dispatch.hpp"
#include "kv_common.hpp"

namespace sparq24 {

typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4v __attribute__((ext_vector_type(4)));
typedef float f32x2v __attribute__((ext_vector_type(2)));
typedef unsigned u32x4v __attribute__((ext_vector_type(4)));

constexpr int kKvTile = 64;
constexpr float kNegInf = -__builtin_inff();

// Work of one launch: item = ((sequence, chunk, row tile), kv head).
struct KvAttnArgs {
  KvAttn a;
  int g;            // query heads per kv head
  int rb;           // rows (token, head of the group) per row tile
  int above, most;  // sequences with more than `above` and at most `most` rows
  int64_t target;   // items that the launch aims at
  int64_t items;    // items that it has room for
  int64_t round;    // units that the CUs take up first, where a second round is dealt in reverse (else all)
  int cmin;         // least tiles of a chunk
  int* starts;      // [seqs + 2] or null: first unit of each sequence, all units, len (k_kv_plan)
  int* plan;        // [seqs][2]: first item / kv heads, chunks
  float* ml;        // [items][rb][2]: reference n and sum of a split row tile
  float* po;        // [items][rb][D]: its output by itself
};

// Sequences of at most so many tiles stay whole: a second launch that joins chunks costs
// more (one new token on 600: 11.9 and 13.8 us, on 1024: 13.6 and 13.9).
constexpr int kWholeTiles = 16;
constexpr int kNever = 1 << 26;  // tiles of a chunk that nothing reaches

struct KvWork {
  int rows, rt, lo, tiles;  // rows, row tiles, first tile, tiles of the visible range
};
// First position that a query at pos sees (window 0: all).
__device__ inline int first_seen(int pos, int window) {
  return window && pos >= window ? pos - window + 1 : 0;
}
__device__ inline KvWork kv_work(const KvAttnArgs& w, const SeqRows& r) {
  KvWork k;
  k.rows = r.n * w.g;
  if (k.rows <= w.above || k.rows > w.most) {
    k.rows = k.rt = k.lo = k.tiles = 0;
    return k;
  }
  k.rt = (k.rows + w.rb - 1) / w.rb;
  const int hi = (int)(r.len < w.a.q.cap ? r.len : w.a.q.cap);
  const int lo = first_seen(r.len - r.n, w.a.window);
  k.lo = lo / kKvTile;
  k.tiles = hi > lo ? (hi + kKvTile - 1) / kKvTile - k.lo : 0;
  return k;
}

// Values that are the same in every lane, for scalar registers and branches.
__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline int64_t uniform(int64_t v) {
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
  return (int64_t)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 | lo);
}

// Holds a value that is the same in all lanes in a scalar register.  The compiler knows
// that it is, but may move such arithmetic into vector registers all the same,
// here behind the divisions of kv_item: that cost the prompt kernel 20 registers,
// reloaded in its loop (a prompt of 8192 tokens took 1.4 times as long).
__device__ inline int scalar(int v) {
  v = uniform(v);
  asm("" : "+s"(v));
  return v;
}

struct KvItem {
  SeqRows r;
  KvWork k;
  int64_t slot;
  int seq, chunk, chunks, len, rt, head;  // len: tiles of a chunk
};
// Tiles of a chunk: all tiles of all row tiles over the items aimed at.
__device__ inline int chunk_tiles(const KvAttnArgs& w, int64_t all) {
  int64_t len = (all * w.a.c.heads + w.target - 1) / w.target;
  len = len < w.cmin ? w.cmin : (len + 3) / 4 * 4;  // four waves share a chunk
  return (int)(len < kNever ? len : kNever);
}
__device__ inline int64_t tiles_of(const KvWork& k) {  // bounded, so that no sum leaves 64 bits
  const int64_t c = (int64_t)k.rt * k.tiles;
  return c < (1ll << 36) ? c : 1ll << 36;
}
__device__ inline int64_t units_of(const KvWork& k, int len) {
  const int64_t ch = ((int64_t)k.tiles + len - 1) / len, n = k.rt * (ch > 1 ? ch : 1);
  return n < kMostUnits ? n : kMostUnits;
}

// A unit is a chunk of a row tile of a sequence, an item a unit and a kv head.  Where
// every sequence has as many units (same row counts, no chunks) a unit's place
// follows from its number; up to kScanned sequences every workgroup adds up what
// comes before it, in two rounds of loads; more have been added up by k_kv_plan
// (one new token each, with offsets: 128 sequences of 300 31.4 us, by k_kv_plan 35.2;
// 256 of 512 59.9 and 61.9, so the two meet somewhat above; from there on the sums of
// every workgroup grow with the square of the sequences).
constexpr int kScanned = 128;
__device__ inline bool kv_item(const KvAttnArgs& w, int64_t id, int lane, KvItem& it) {
  const int H = w.a.c.heads;
  const int64_t seqs = w.a.q.seqs, unit = id / H;
  int at;
  if (w.starts) {
    if (unit >= w.starts[seqs]) return false;
    it.len = uniform(w.starts[seqs + 1]);
    it.seq = last_reached((int)seqs, lane, [&](int b) { return w.starts[b] <= unit; });
    at = (int)unit - w.starts[it.seq];
  } else if (!w.a.q.cu && w.cmin == kNever) {
    const int rt = (int)((w.a.q.nper * w.g + w.rb - 1) / w.rb);
    it.len = kNever;
    if (unit >= seqs * rt) return false;
    // the longest of all sequences first (8 prompts of 2048: 331 us, sequence by sequence
    // 344); in a second round (`round`) the shortest first, beside the longest of the first
    const int64_t u = unit < w.round ? unit : seqs * rt - 1 - (unit - w.round);
    at = (int)(u / seqs);
    it.seq = (int)(u % seqs);
  } else {
    it.len = w.cmin;
    if (w.cmin < kNever) {
      int64_t all = 0;
      for (int64_t b0 = 0; b0 < seqs; b0 += 64) {
        const int64_t b = b0 + lane;
        const int64_t c = b < seqs ? tiles_of(kv_work(w, seq_rows(w.a.q, b))) : 0;
        // 64 sums of 2^36 in two halves of 32 bits
        all += (uint32_t)__builtin_amdgcn_readlane((int)wave_scan_sum((uint32_t)c & 0xFFFFF), 63) +
               ((int64_t)(uint32_t)__builtin_amdgcn_readlane((int)wave_scan_sum((uint32_t)(c >> 20)), 63) << 20);
      }
      it.len = uniform(chunk_tiles(w, all));
    }
    if (!find_sequence(seqs, unit, lane, it.seq, at,
                       [&](int64_t b) { return units_of(kv_work(w, seq_rows(w.a.q, b)), it.len); }))
      return false;
  }
  it.r = seq_rows(w.a.q, it.seq);
  it.r.first = uniform(it.r.first);
  it.r.n = uniform(it.r.n);
  it.r.len = uniform(it.r.len);
  it.k = kv_work(w, it.r);
  it.chunks = (it.k.tiles + it.len - 1) / it.len;
  if (it.chunks < 1) it.chunks = 1;
  it.chunk = scalar(at / it.k.rt);
  it.rt = scalar(it.k.rt - 1 - at % it.k.rt);  // the last rows see the most: first
  it.head = scalar((int)(id % H));
  it.slot = id;
  if (w.plan && at == 0 && it.head == 0 && threadIdx.x == 0) {
    w.plan[2 * it.seq] = (int)unit;
    w.plan[2 * it.seq + 1] = it.chunks;
  }
  return true;
}

__device__ inline void kv_store_out(const KvAttn& a, int64_t o, float v) {
  if (a.dtype == 1) ((__bf16*)a.out)[o] = (__bf16)v;
  else ((_Float16*)a.out)[o] = (_Float16)v;
}

// Over the four lane groups (lanes l ^ 16, l ^ 32), in every lane.
__device__ inline float groups_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  float m;
  asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(r[0]), "v"(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(m), __float_as_uint(m), false, false);
  asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(r[0]), "v"(r[1]));
  return m;
}
__device__ inline float groups_sum(float v) {
  auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ inline float kv_lse(float top, float sum) {
  return sum == 0.0f ? kNegInf : (top + __builtin_amdgcn_logf(sum)) * 0.69314718055994530942f;
}

// Tiles and limits of a row tile within its chunk.
struct KvRange {
  int t0, t1;       // tiles
  int lo, hi;       // tokens that some row sees
  int least, from;  // tokens from .. least - 1 are seen by every row
};
__device__ inline KvRange kv_range(const KvAttnArgs& p, const KvItem& it, int r0, int r1) {
  const KvAttn& a = p.a;
  const int pos0 = it.r.len - it.r.n, i0 = r0 / p.g, i1 = (r1 - 1) / p.g;
  const int hi_all = (int)(it.r.len < a.q.cap ? it.r.len : a.q.cap);
  KvRange k;
  k.hi = a.causal && pos0 + i1 + 1 < hi_all ? pos0 + i1 + 1 : hi_all;
  k.lo = first_seen(pos0 + i0, a.window);
  k.least = a.causal && pos0 + i0 + 1 < k.hi ? pos0 + i0 + 1 : k.hi;
  k.from = first_seen(pos0 + i1, a.window);
  k.t0 = it.k.lo + it.chunk * it.len;
  k.t1 = k.t0 + it.len;
  if (k.t1 > it.k.lo + it.k.tiles) k.t1 = it.k.lo + it.k.tiles;
  if (k.t0 < k.lo / kKvTile) k.t0 = k.lo / kKvTile;
  if (k.t1 > (k.hi + kKvTile - 1) / kKvTile) k.t1 = (k.hi + kKvTile - 1) / kKvTile;
  return {scalar(k.t0), scalar(k.t1), scalar(k.lo), scalar(k.hi), scalar(k.least), scalar(k.from)};
}


// Which kernels run, their row tiles and the room for split results
// (kernels_kv_split.hip).
struct KvPlan {
  KvAttnArgs few, many;
  bool run_few, run_many, split, planned;
  size_t need;
};
// few_rows: most rows of the few-rows kernel, one row tile; prompt_rows: of a prompt
// workgroup; resident: prompt workgroups that a CU holds.
KvPlan kv_plan(const KvAttn& a, char* ws, int few_rows, int prompt_rows, int resident);
// Whether the launches' grids hold it; threads: of a prompt workgroup.
bool kv_plan_fits(const KvAttn& a, const KvPlan& p, int threads);
hipError_t launch_kv_starts(const KvPlan& p, hipStream_t s);  // before the kernels, where p.planned
hipError_t launch_kv_join(const KvPlan& p, hipStream_t s);    // after them, where p.split

}  // namespace sparq24
