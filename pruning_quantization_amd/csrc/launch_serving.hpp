// Launchers of the serving operators (kernels_int8.hip, kernels_mxfp4.hip,
// kernels_norm.hip, kernels_kv.hip, kernels_kv4.hip), as launch.hpp is for the others.  All of them only enqueue on the given stream.
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

// y = sum_g 2^(sa[m][g] + sb[n][g] - 254) sum_{k in g} a b (+ bias[n]) over groups of
// 32 from MXFP4 codes (row strides in bytes) and dense scale bytes.
struct Mxfp4Gemm {
  const uint8_t *a, *b;
  int64_t lda, ldb;
  const uint8_t *sa, *sb;
  const float* bias;
  int64_t M, N, K;
  void* c;
  int64_t ldc;
  int dtype;
};
hipError_t launch_mxfp4_gemm(const Mxfp4Gemm& g, hipStream_t s);
bool mxfp4_gemm_fits(const Mxfp4Gemm& g);  // the launch's grid

// RMS norm of x (+ residual) rows, quantized; cfmt is a CodeFmt.
struct NormRows {  // strides in bytes; row = b * R + r
  char* x;
  int64_t R, bs, rs;
};
struct RmsNorm {
  NormRows x, res, sum;  // res.x and sum.x null: none
  const void* w;
  int dtype, wdtype;
  int64_t rows, nunits;  // units of 8 elements
  float eps;
  int cfmt;
  float qmax;
  char* codes;
  void* scales;
};
hipError_t launch_rmsnorm_quantize(const RmsNorm& n, hipStream_t s);

// Paged key/value cache (layouts: kv_common.hpp) and the sequences of one
// call: token rows cu[b] .. cu[b + 1] - 1 belong to sequence b (nper rows each
// where cu is null), lens[b] tokens of it are in the cache, the new included.
struct KvCache {
  uint8_t* k;
  float* ks;          // 8 bits: scales of a block and head
  uint8_t* v;
  float* vs;
  uint8_t *ke, *ve;   // 4 bits: exponents of a token and 32 dims
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
hipError_t launch_kv4_append(const KvCache& c, const KvSeqs& q, const KvRows& k, const KvRows& v,
                             int dtype, hipStream_t s);
bool kv_append_fits(const KvCache& c, const KvSeqs& q);  // the launches' grids
bool kv4_append_fits(const KvCache& c, const KvSeqs& q);
bool kv_attn_fits(const KvAttn& a);
size_t kv_attn_workspace(const KvAttn& a);
hipError_t launch_kv_attn(const KvAttn& a, void* ws, hipStream_t s);
bool kv4_attn_fits(const KvAttn& a);
size_t kv4_attn_workspace(const KvAttn& a);
hipError_t launch_kv4_attn(const KvAttn& a, void* ws, hipStream_t s);

}  // namespace sparq24
