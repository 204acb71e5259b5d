// MXFP4 matrix product of the dense 4-bit side [PD §3: MXFP4, one power of two per 32
// elements]: y[m][n] = sum_g 2^(sa[m][g] + sb[n][g] - 254) sum_{k in g} a[m][k] b[n][k]
// (+ bias[n]) on v_mfma_scale_f32_16x16x128_f8f6f4, which takes 32 codes (16 bytes) and
// their exponent byte from each lane: lane (c, h) holds row c of its operand and one
// group of the four that the instruction adds up.  Which group that is, is free as long
// as both operands agree.
#include "dispatch.hpp"
#include "gemm_tile.hpp"
#include "launch_serving.hpp"

namespace sparq24 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// c += b a (b's rows are c's rows, so that a lane holds four adjacent outputs of one row
// of a); byte SB of sb and byte SA of sa are the exponents.
template <int SB, int SA>
__device__ inline f32x4_t mx_product(i32x4_t b, i32x4_t a, f32x4_t c, uint32_t sb, uint32_t sa) {
  constexpr int kFp4 = 4;  // the operand's format
  const i32x8_t b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0}, a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b8, a8, c, kFp4, kFp4, SB, (int)sb, SA, (int)sa);
}

// Rows of exponents begin at any byte.
typedef uint16_t u16_any __attribute__((aligned(1)));

// Four outputs n .. n + 3 of row m: one store where all are inside (rows may begin at
// any element), else one by one.
template <class T>
__device__ inline void mx_store4(const Mxfp4Gemm& g, int64_t m, int64_t n, f32x4_t acc, const float (&bias)[4]) {
  if (m >= g.M) return;
  typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  T* c = (T*)g.c + m * g.ldc + n;
  t4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (T)(acc[e] + bias[e]);
  if (n + 4 <= g.N) {
    *(t4*)c = y;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < g.N) c[e] = y[e];
  }
}

// Few rows: the weight is streamed once.  A workgroup owns 16 MT x 16 NT outputs; each
// of its W waves takes slabs of 256 codes (128 bytes) of K in turn, with S buffers of its
// own in LDS (chunks XOR-swizzled by row) that it fills with global_load_lds S - 1 slabs
// ahead, so no wave waits for another until the sums meet in LDS, in wave order.  Of a
// slab's eight groups lane group h takes 2 h and 2 h + 1: their exponents are one
// 16-bit load.
template <int MT, int NT, int W, int S>
__global__ __launch_bounds__(64 * W) void k_mxfp4_stream(Mxfp4Gemm g, int64_t ntn) {
  constexpr int SK = 128, QA = 2 * MT, QB = 2 * NT, STAGE = (MT + NT) * 16 * SK;
  constexpr int BYTES = W * S * STAGE > W * MT * NT * 1024 ? W * S * STAGE : W * MT * NT * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t smem[BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int64_t m0 = (blockIdx.x / ntn) * (16 * MT), n0 = (blockIdx.x % ntn) * (16 * NT);
  uint8_t* mine = smem + w * S * STAGE;
  const int64_t last_m = g.M - 1 - m0, last_n = g.N - 1 - n0, groups = g.K / 32;
  const uint8_t *base_a = g.a + m0 * g.lda, *base_b = g.b + n0 * g.ldb;
  // rows r and r + 2 of a half (even or odd rows) lie in chunks of their own, and so do
  // those of the next lane group, two chunks on
  auto swizzle = [](int r) { return ((r >> 1) & 1) | (r & 4); };
  // eight rows of a slab per load; rows past the ends repeat the last, unused
  int64_t off_a[QA], off_b[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int64_t r = 8 * q + (lane >> 3);
    off_a[q] = (r < last_m ? r : last_m) * g.lda + 16 * ((lane & 7) ^ swizzle((int)r));
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int64_t r = 8 * q + (lane >> 3);
    off_b[q] = (r < last_n ? r : last_n) * g.ldb + 16 * ((lane & 7) ^ swizzle((int)r));
  }
  // this lane's rows of exponents
  const uint8_t *ea[MT], *eb[NT];
#pragma unroll
  for (int i = 0; i < MT; ++i) ea[i] = g.sa + (m0 + (16 * i + c < last_m ? 16 * i + c : last_m)) * groups;
#pragma unroll
  for (int j = 0; j < NT; ++j) eb[j] = g.sb + (n0 + (16 * j + c < last_n ? 16 * j + c : last_n)) * groups;
  uint32_t sa[S][MT], sb[S][NT];
  auto fetch = [&](int buf, int kt) {
    uint8_t* st = mine + buf * STAGE;
    const uint8_t *ka = base_a + kt * SK, *kb = base_b + kt * SK;
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const uint8_t* src = kb + off_b[q];
      __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(st + QA * 1024 + q * 1024), 16, 0, 0);
    }
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const uint8_t* src = ka + off_a[q];
      __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(st + q * 1024), 16, 0, 0);
    }
  };
  // (between the slab's loads and the next ones', as the wait below counts them)
  auto exponents = [&](uint32_t(&xa)[MT], uint32_t(&xb)[NT], int kt) {
    asm volatile("" ::: "memory");
#pragma unroll
    for (int i = 0; i < MT; ++i) xa[i] = *(const u16_any*)(ea[i] + 8 * kt + 2 * h);
#pragma unroll
    for (int j = 0; j < NT; ++j) xb[j] = *(const u16_any*)(eb[j] + 8 * kt + 2 * h);
    asm volatile("" ::: "memory");
  };
  f32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int KB = (int)(g.K / 2), nk = KB / SK;  // bytes of a row, whole slabs
  const int last = nk - 1 - (nk - 1 - w) % W;   // this wave's last slab, asked for again past the end
  if (w < nk) {
#pragma unroll
    for (int s = 0; s + 1 < S; ++s) {
      const int kt = w + s * W < last ? w + s * W : last;
      fetch(s, kt);
      exponents(sa[s], sb[s], kt);
    }
  }
  // the bias of the 16 x 16 tiles t = w + W u that this wave joins
  constexpr int U = (MT * NT + W - 1) / W;
  float bias[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int64_t n = 16 * ((w + W * u) % NT) + 4 * h;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      bias[u][e] = g.bias ? g.bias[n0 + (n + e < last_n ? n + e : last_n)] : -0.0f;  // y + -0 is y
  }
  if (w == nk % W) {  // the rest of K, zeros behind it, while the first slabs come
    for (int k = nk * SK + 16 * h; k - 16 * h < KB; k += 64) {
      const i32x4_t zero = {0, 0, 0, 0};
      i32x4_t af[MT], bf[NT];
      uint32_t xa[MT], xb[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int64_t r = 16 * i + c;
        af[i] = k < KB ? *(const i32x4_t*)(base_a + (r < last_m ? r : last_m) * g.lda + k) : zero;
        xa[i] = k < KB ? ea[i][k / 16] : 127u;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int64_t r = 16 * j + c;
        bf[j] = k < KB ? *(const i32x4_t*)(base_b + (r < last_n ? r : last_n) * g.ldb + k) : zero;
        xb[j] = k < KB ? eb[j][k / 16] : 127u;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[i][j] = mx_product<0, 0>(bf[j], af[i], acc[i][j], xb[j], xa[i]);
    }
  }
  if (w < nk) {
    for (int k0 = w; k0 < nk; k0 += S * W) {
#pragma unroll
      for (int s = 0; s < S; ++s) {
        const int kt = k0 + s * W;
        if (kt >= nk) break;
        const int next = kt + (S - 1) * W < last ? kt + (S - 1) * W : last;
        constexpr int kOthers = S - 1;
        const int to = (s + kOthers) % S;
        fetch(to, next);
        exponents(sa[to], sb[to], next);
        wait_vmcnt<(S - 1) * (QA + QB + MT + NT)>();
        asm volatile("" ::: "memory");
        const uint8_t* st = mine + s * STAGE + c * SK;
        auto step = [&]<int X>() {
          i32x4_t af[MT], bf[NT];
          const int ch = ((2 * h + X) ^ swizzle(c)) * 16;
#pragma unroll
          for (int i = 0; i < MT; ++i) af[i] = *(const i32x4_t*)(st + 16 * SK * i + ch);
#pragma unroll
          for (int j = 0; j < NT; ++j) bf[j] = *(const i32x4_t*)(st + 16 * SK * (MT + j) + ch);
#pragma unroll
          for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) acc[i][j] = mx_product<X, X>(bf[j], af[i], acc[i][j], sb[s][j], sa[s][i]);
        };
        step.template operator()<0>();
        step.template operator()<1>();
        __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read before it is filled again
        asm volatile("" ::: "memory");
      }
    }
    wait_vmcnt<0>();  // what was asked for past the end has landed
    asm volatile("" ::: "memory");
  }
  __syncthreads();  // every wave is done with its buffers
  f32x4_t* red = (f32x4_t*)smem;  // [W][MT * NT][64]
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) red[(w * MT * NT + i * NT + j) * 64 + lane] = acc[i][j];
  __syncthreads();
  auto out = [&]<class T>(T) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = w + W * u;
      if (t >= MT * NT) break;
      f32x4_t s = red[t * 64 + lane];
#pragma unroll
      for (int q = 1; q < W; ++q) s += red[(q * MT * NT + t) * 64 + lane];
      mx_store4<T>(g, m0 + 16 * (t / NT) + c, n0 + 16 * (t % NT) + 4 * h, s, bias[u]);
    }
  };
  if (g.dtype == 0) out(0.0f);
  else if (g.dtype == 1) out((__bf16)0.0f);
  else out((_Float16)0.0f);
}

hipError_t launch_mxfp4_gemm(const Mxfp4Gemm& g, hipStream_t s) {
  auto few = [&]<int MT, int NT, int W, int S>() {
    const int64_t ntm = (g.M + 16 * MT - 1) / (16 * MT), ntn = (g.N + 16 * NT - 1) / (16 * NT);
    hipLaunchKernelGGL((k_mxfp4_stream<MT, NT, W, S>), dim3((unsigned)(ntm * ntn)), dim3(64 * W), 0, s, g, ntn);
    return hipGetLastError();
  };
  if (g.M <= 16) return few.template operator()<1, 1, 8, 2>();
  return few.template operator()<4, 4, 4, 2>();
}

}  // namespace sparq24
