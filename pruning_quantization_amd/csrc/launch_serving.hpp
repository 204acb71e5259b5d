// Launchers of the 8-bit serving operators (kernels_int8.hip, kernels_kv.hip), as
// launch.hpp is for the others.  All of them only enqueue on the given stream.
#pragma once

#include "launch.hpp"

namespace sparq24 {

// y = (sum_k a b) * sa[m] * sb[n] (+ bias[n]) from INT8 codes (row strides in
// bytes) with int32 sums; dtype is a sparq24_dtype, ldc in elements.
struct Int8Gemm {
  const int8_t *a, *b;
  int64_t lda, ldb;
  const float *sa, *sb, *bias;
  int64_t M, N, K;
  void* c;
  int64_t ldc;
  int dtype;
};
hipError_t launch_int8_gemm(const Int8Gemm& g, hipStream_t s);

// Paged 8-bit key/value cache (layout: kv_common.hpp) and the sequences of one
// call: token rows cu[b] .. cu[b + 1] - 1 belong to sequence b (nper rows each
// where cu is null), lens[b] tokens of it are in the cache, the new included.
struct KvCache {
  uint8_t* k;
  float* ks;
  uint8_t* v;
  float* vs;
  int64_t blocks;
  int heads, dim, tsh;  // kv heads, head dim, log2 of the tokens per block
  bool fp8;
};
struct KvSeqs {
  const int32_t* table;
  int64_t table_stride;
  int64_t cap;  // tokens that a table row can hold (at most 2^31 - 1)
  const int32_t* lens;
  const int32_t* cu;
  int64_t seqs, total, nper;
  int slots;  // blocks that nper rows can touch
};
// One side (K or V) of the new token rows: strides in bytes.
struct KvRows {
  const char* x;
  int64_t ts, hs;
};
hipError_t launch_kv_append(const KvCache& c, const KvSeqs& q, const KvRows& k, const KvRows& v,
                            int dtype, hipStream_t s);
struct KvAttn {
  KvCache c;
  KvSeqs q;
  const char* x;    // queries, strides in bytes
  int64_t ts, hs;
  int dtype;        // SPARQ24_BF16 or SPARQ24_F16
  int heads;        // query heads
  float scale;
  int causal;
  int window;       // 0: none
  char* out;
  float* lse;       // or null
};
bool kv_append_fits(const KvCache& c, const KvSeqs& q);  // the launches' grids
bool kv_attn_fits(const KvAttn& a);
size_t kv_attn_workspace(const KvAttn& a);
hipError_t launch_kv_attn(const KvAttn& a, void* ws, hipStream_t s);

}  // namespace sparq24
