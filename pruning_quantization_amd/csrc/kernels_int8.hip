// INT8 matrix product of the dense INT8 side [PD §2: the quantized side's
// operands with one scale per row]: y[m][n] = (sum_k a[m][k] b[n][k]) *
// sa[m] * sb[n] (+ bias[n]).  The sums are int32 (exact: K < 2^17), so every
// split of K gives the same bits; then one rounding to fp32, the two scale
// multiplies, the bias and the rounding to the output type.
#include "dispatch.hpp"
#include "gemm_tile.hpp"

namespace sparq24 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

__device__ inline void int8_store(const Int8Gemm& g, int64_t m, int64_t n, int acc) {
  if (m >= g.M || n >= g.N) return;
  float y = (float)acc * g.sa[m] * g.sb[n];
  if (g.bias) y += g.bias[n];
  const int64_t o = m * g.ldc + n;
  if (g.dtype == 0) ((float*)g.c)[o] = y;
  else if (g.dtype == 1) ((__bf16*)g.c)[o] = (__bf16)y;
  else ((_Float16*)g.c)[o] = (_Float16)y;
}

// Few rows: the weight is streamed once, straight into MFMA operands.  A
// workgroup owns 16 MT x 16 NT outputs, its 8 waves take 256-byte runs of K
// in turn, and their int32 sums meet in LDS.  Bound by the weight's bytes.
template <int MT, int NT>
__global__ __launch_bounds__(512) void k_int8_stream(Int8Gemm g, int64_t ntn) {
  constexpr int W = 8, RUN = 256;
  __shared__ i32x4_t red[W][MT * NT][64];
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, c = lane & 15, h = lane >> 4;
  const int64_t m0 = (blockIdx.x / ntn) * (16 * MT), n0 = (blockIdx.x % ntn) * (16 * NT);
  const int8_t* ar[MT];
  const int8_t* br[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {  // rows past the end repeat the last one, unused
    const int64_t m = m0 + 16 * i + c;
    ar[i] = g.a + (m < g.M ? m : g.M - 1) * g.lda;
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const int64_t n = n0 + 16 * j + c;
    br[j] = g.b + (n < g.N ? n : g.N - 1) * g.ldb;
  }
  i32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  for (int64_t kb = w * RUN; kb < g.K; kb += W * RUN) {
#pragma unroll
    for (int s = 0; s < RUN / 64; ++s) {
      const int64_t k = kb + 64 * s + 16 * h;
      const i32x4_t zero = {0, 0, 0, 0};
      i32x4_t af[MT], bf[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) af[i] = k < g.K ? *(const i32x4_t*)(ar[i] + k) : zero;
#pragma unroll
      for (int j = 0; j < NT; ++j) bf[j] = k < g.K ? *(const i32x4_t*)(br[j] + k) : zero;
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(af[i], bf[j], acc[i][j], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[w][i * NT + j][lane] = acc[i][j];
  __syncthreads();
  for (int t = w; t < MT * NT; t += W) {
    i32x4_t s = red[0][t][lane];
#pragma unroll
    for (int q = 1; q < W; ++q) s += red[q][t][lane];
    const int64_t m = m0 + 16 * (t / NT) + 4 * h, n = n0 + 16 * (t % NT) + c;
#pragma unroll
    for (int e = 0; e < 4; ++e) int8_store(g, m + e, n, s[e]);
  }
}

hipError_t launch_int8_gemm(const Int8Gemm& g, hipStream_t s) {
  auto go = [&]<int MT, int NT>() {
    const int64_t ntm = (g.M + 16 * MT - 1) / (16 * MT), ntn = (g.N + 16 * NT - 1) / (16 * NT);
    hipLaunchKernelGGL((k_int8_stream<MT, NT>), dim3((unsigned)(ntm * ntn)), dim3(512), 0, s, g, ntn);
    return hipGetLastError();
  };
  if (g.M <= 16) return go.template operator()<1, 1>();
  if (g.M <= 32) return go.template operator()<2, 1>();
  return go.template operator()<4, 2>();
}

}  // namespace sparq24
