// INT8 matrix product of the dense INT8 side [PD §2: the quantized side's
// operands with one scale per row]: y[m][n] = (sum_k a[m][k] b[n][k]) *
// sa[m] * sb[n] (+ bias[n]).  The sums are int32 (exact: K < 2^17), so every
// split of K gives the same bits; then one rounding to fp32, the two scale
// multiplies, the bias and the rounding to the output type.
#include "dispatch.hpp"
#include "gemm_tile.hpp"
#include "launch_serving.hpp"

namespace sparq24 {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

// Four outputs n .. n + 3 of row m: one store where all are inside (rows may begin at
// any element, which global stores take: 777 x 1031 x 2064 10.8 us with the call,
// 11.6 with aligned stores only), else one by one.
template <class T>
__device__ inline void int8_store4(const Int8Gemm& g, int64_t m, int64_t n, i32x4_t acc, float sa,
                                   const float (&sb)[4], const float (&bias)[4]) {
  if (m >= g.M) return;
  typedef T t4 __attribute__((ext_vector_type(4), aligned(sizeof(T))));
  T* c = (T*)g.c + m * g.ldc + n;
  t4 y;
#pragma unroll
  for (int e = 0; e < 4; ++e) y[e] = (T)((float)acc[e] * sa * sb[e] + bias[e]);
  if (n + 4 <= g.N) {
    *(t4*)c = y;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < g.N) c[e] = y[e];
  }
}

// Few rows: the weight is streamed once.  A workgroup owns 16 MT x 16 NT
// outputs; each of its W waves takes slabs of 128 codes of K in turn, with S
// buffers of its own in LDS (chunks XOR-swizzled by row) that it fills with
// global_load_lds S - 1 slabs ahead, so no wave waits for another until the
// int32 sums meet in LDS.  Through LDS because an MFMA operand straight from
// memory gives adjacent lanes adjacent rows, which the address unit takes at one
// lane (16 bytes) a cycle: 34 GB/s per CU measured, against 64 bytes a
// cycle in row order.  Bound by the weight's bytes (48 x 14336 x 4096: 12.8 us, 5.6
// TB/s past the launch and the first slabs); of a small weight by the latter (1 x
// 4096 x 4096: 4.5 us).  The products take b first, so that a lane holds four
// adjacent outputs, and the scales are asked for before the slabs are read: with
// stores one by one and scales at the end 14.7 us, 777 x 1031 x 2064 12.4 (9.2).
template <int MT, int NT, int W, int S>
__global__ __launch_bounds__(64 * W) void k_int8_stream(Int8Gemm g, int64_t ntn) {
  constexpr int SK = 128, QA = 2 * MT, QB = 2 * NT, STAGE = (MT + NT) * 16 * SK;
  constexpr int BYTES = W * S * STAGE > W * MT * NT * 1024 ? W * S * STAGE : W * MT * NT * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t smem[BYTES];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int64_t m0 = (blockIdx.x / ntn) * (16 * MT), n0 = (blockIdx.x % ntn) * (16 * NT);
  uint8_t* mine = smem + w * S * STAGE;
  const int64_t last_m = g.M - 1 - m0, last_n = g.N - 1 - n0;
  const int8_t *base_a = g.a + m0 * g.lda, *base_b = g.b + n0 * g.ldb;
  // eight rows of a slab per load; rows past the ends repeat the last, unused
  int64_t off_a[QA], off_b[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int64_t r = 8 * q + (lane >> 3);
    off_a[q] = (r < last_m ? r : last_m) * g.lda + 16 * ((lane & 7) ^ (int)(r & 7));
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int64_t r = 8 * q + (lane >> 3);
    off_b[q] = (r < last_n ? r : last_n) * g.ldb + 16 * ((lane & 7) ^ (int)(r & 7));
  }
#define SPARQ24_INT8_FETCH(buf, k0)                                                            \
  {                                                                                            \
    uint8_t* st = mine + (buf) * STAGE;                                                        \
    const int8_t *ka = base_a + (k0), *kb = base_b + (k0);                                     \
    _Pragma("unroll") for (int q = 0; q < QB; ++q) {                                           \
      const int8_t* src = kb + off_b[q];                                                       \
      __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(st + QA * 1024 + q * 1024), 16, 0, 0); \
    }                                                                                          \
    _Pragma("unroll") for (int q = 0; q < QA; ++q) {                                           \
      const int8_t* src = ka + off_a[q];                                                       \
      __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(st + q * 1024), 16, 0, 0);           \
    }                                                                                          \
  }
  i32x4_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};
  const int K = (int)g.K, nk = K / SK;         // whole slabs
  const int last = nk - 1 - (nk - 1 - w) % W;  // this wave's last slab, asked for again past the end
  if (w < nk) {
#pragma unroll
    for (int s = 0; s + 1 < S; ++s) SPARQ24_INT8_FETCH(s, (w + s * W < last ? w + s * W : last) * SK);
  }
  // the scales and bias of the 16 x 16 tiles t = w + W u that this wave joins
  constexpr int U = (MT * NT + W - 1) / W;
  float sa[U], sb[U][4], bias[U][4];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int t = w + W * u;
    const int64_t m = 16 * (t / NT) + c, n = 16 * (t % NT) + 4 * h;
    sa[u] = g.sa[m0 + (m < last_m ? m : last_m)];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t at = n0 + (n + e < last_n ? n + e : last_n);
      sb[u][e] = g.sb[at];
      bias[u][e] = g.bias ? g.bias[at] : -0.0f;  // y + -0 is y
    }
  }
  if (w == nk % W) {  // the rest of K, zeros behind it, while the first slabs come
    for (int k = nk * SK + 16 * h; k - 16 * h < K; k += 64) {
      const i32x4_t zero = {0, 0, 0, 0};
      i32x4_t af[MT], bf[NT];
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        const int64_t r = 16 * i + c;
        af[i] = k < K ? *(const i32x4_t*)(base_a + (r < last_m ? r : last_m) * g.lda + k) : zero;
      }
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int64_t r = 16 * j + c;
        bf[j] = k < K ? *(const i32x4_t*)(base_b + (r < last_n ? r : last_n) * g.ldb + k) : zero;
      }
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[j], af[i], acc[i][j], 0, 0, 0);
    }
  }
  if (w < nk) {
    int buf = 0;
    for (int kt = w; kt < nk; kt += W) {
      const int next = kt + (S - 1) * W;
      const int to = buf == 0 ? S - 1 : buf - 1;
      SPARQ24_INT8_FETCH(to, (next < last ? next : last) * SK);
      wait_vmcnt<(S - 1) * (QA + QB)>();
      asm volatile("" ::: "memory");
      const uint8_t* st = mine + buf * STAGE + c * SK;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        i32x4_t af[MT], bf[NT];
        const int ch = ((4 * x + h) ^ (c & 7)) * 16;
#pragma unroll
        for (int i = 0; i < MT; ++i) af[i] = *(const i32x4_t*)(st + 16 * SK * i + ch);
#pragma unroll
        for (int j = 0; j < NT; ++j) bf[j] = *(const i32x4_t*)(st + 16 * SK * (MT + j) + ch);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
          for (int j = 0; j < NT; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(bf[j], af[i], acc[i][j], 0, 0, 0);
      }
      __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read before it is filled again
      asm volatile("" ::: "memory");
      buf = buf + 1 == S ? 0 : buf + 1;
    }
    wait_vmcnt<0>();  // what was asked for past the end has landed
    asm volatile("" ::: "memory");
  }
  __syncthreads();  // every wave is done with its buffers
  i32x4_t* red = (i32x4_t*)smem;  // [W][MT * NT][64]
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
      i32x4_t s = red[t * 64 + lane];
#pragma unroll
      for (int q = 1; q < W; ++q) s += red[(q * MT * NT + t) * 64 + lane];
      const int64_t m = m0 + 16 * (t / NT) + c, n = n0 + 16 * (t % NT) + 4 * h;  // outputs n .. n + 3 of row m
      int8_store4<T>(g, m, n, s, sa[u], sb[u], bias[u]);
    }
  };
  if (g.dtype == 0) out(0.0f);
  else if (g.dtype == 1) out((__bf16)0.0f);
  else out((_Float16)0.0f);
}

// Many rows: a BM x BN tile per workgroup, waves of WM x 64 on
// v_mfma_i32_16x16x64_i8.  Slabs of 128 codes go from memory straight into LDS
// (global_load_lds) into two buffers; their 16-byte chunks are XOR-swizzled by
// row.  A slab is two steps of 64 codes.  Rows past the ends repeat the last; a
// rest of K is filled up with zeros.  Two schedules:
// Mixed (small tiles, several workgroups per CU): the fragments of a step are
// read while the products of the step before run, across slabs too; between a
// slab's two steps every wave has its last fragments of it and the next slab
// has landed (one barrier), and the slab after that starts into the freed
// buffer.
// In turns (PP, eight waves, two per SIMD): waves 4..7 run half a step behind
// waves 0..3, with a barrier after every half, so on each SIMD one wave
// multiplies (at raised priority) while the other reads and requests slabs.
// With phases p between barriers, waves 0..3 read step s at p = 2 s, waves
// 4..7 at 2 s + 1.  Slab t + 1 is requested by the reads of step 2 t, when both
// groups have read all of slab t - 1 (phases up to 4 t - 1), and waited for at
// the end of phase 4 t + 3, before anyone reads it.
// 4096 x 14336 x 4096, bf16 out: mixed 267 us, in turns 229 us.  By the counters the
// matrix units are busy for 54% of the cycles and LDS for 20% (192 KB of fragments per
// slab), without conflicts: what is left are the turns' barriers and waits.
// 16 outputs n .. n + 15 of row m: 16-byte stores where `wide` says that all
// are inside (rows may begin at any element), else one by one.
template <class T>
__device__ inline void int8_store16(const Int8Gemm& g, int64_t m, int64_t n, const i32x4_t (&acc)[4], float sa,
                                    const float* sb, const float* bias, bool wide) {
  typedef T t8 __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  constexpr int V = 16 / sizeof(T);
  T* c = (T*)g.c + m * g.ldc + n;
  T y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = (T)((float)acc[e / 4][e % 4] * sa * sb[e] + bias[e]);
  if (wide) {
#pragma unroll
    for (int q = 0; q < 16 / V; ++q) {
      t8 v;
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = y[V * q + e];
      *(t8*)(c + V * q) = v;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (n + e < g.N) c[e] = y[e];
  }
}

template <int BM, int BN, int WM, bool PP>
__global__ __launch_bounds__((BM / WM) * (BN / 64) * 64) void k_int8_tile(Int8Gemm g) {
  constexpr int WN = 64, NWN = BN / WN, NT = (BM / WM) * NWN * 64;
  constexpr int TI = WM / 16, TJ = 4, SK = 128;
  constexpr int A_BYTES = BM * SK, STAGE = (BM + BN) * SK;
  constexpr int QA = BM * 8 / NT, QB = BN * 8 / NT;
  static_assert(QA * NT == BM * 8 && QB * NT == BN * 8 && TI % 4 == 0, "tile / thread mismatch");
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w / NWN, wn = w % NWN;
  // XCD-aware order: each XCD owns a contiguous run of tiles, walked in
  // groups of eight row tiles, so that its L2 serves the shared slabs
  const int64_t ntn = (g.N + BN - 1) / BN, ntm = (g.M + BM - 1) / BM, total = ntm * ntn;
  const int64_t pid = blockIdx.x, per = total / 8;
  const int64_t lid = pid < per * 8 ? (pid % 8) * per + pid / 8 : pid;
  constexpr int64_t kGroupM = 8;
  const int64_t ingroup = kGroupM * ntn, first = (lid / ingroup) * kGroupM;
  const int64_t gsz = ntm - first < kGroupM ? ntm - first : kGroupM;
  const int64_t m0 = (first + (lid % ingroup) % gsz) * BM, n0 = ((lid % ingroup) / gsz) * BN;

  // Loads of a slab: 32-bit offsets from the tile's first rows (row strides of
  // 8 MiB and more go to k_int8_stream).
  const int K = (int)g.K, rows_a = (int)(g.M - m0 < BM ? g.M - m0 : BM), rows_b = (int)(g.N - n0 < BN ? g.N - n0 : BN);
  const int8_t *base_a = g.a + m0 * g.lda, *base_b = g.b + n0 * g.ldb;
  unsigned off_a[QA], off_b[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int p = q * NT + tid, r = p >> 3, m = r < rows_a ? r : rows_a - 1;
    off_a[q] = (unsigned)m * (unsigned)g.lda + 16 * ((p & 7) ^ (r & 7));
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int p = q * NT + tid, r = p >> 3, n = r < rows_b ? r : rows_b - 1;
    off_b[q] = (unsigned)n * (unsigned)g.ldb + 16 * ((p & 7) ^ ((r & 3) | ((r >> 2) & 4)));
  }
#define SPARQ24_INT8_SLAB(buf, k0)                                                             \
  {                                                                                            \
    uint8_t* st = smem + (buf) * STAGE + w * 1024;                                             \
    const int8_t *ka = base_a + (k0), *kb = base_b + (k0);                                     \
    _Pragma("unroll") for (int q = 0; q < QA; ++q) {                                           \
      const int8_t* src = ka + off_a[q];                                                       \
      __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(st + q * NT * 16), 16, 0, 0);        \
    }                                                                                          \
    _Pragma("unroll") for (int q = 0; q < QB; ++q) {                                           \
      const int8_t* src = kb + off_b[q];                                                       \
      __builtin_amdgcn_global_load_lds(src, (lds_void_t*)(st + A_BYTES + q * NT * 16), 16, 0, 0); \
    }                                                                                          \
  }

  const int fr = lane & 15, h = lane >> 4;
  // fragment rows: A tile i row fr; B tile j row fr is weight row
  // 16 (fr / 4) + 4 j + fr % 4 (a lane then holds 16 adjacent outputs)
  const uint8_t* fa = smem + (wm * WM + fr) * SK;
  const uint8_t* fb = smem + A_BYTES + (wn * WN + 16 * (fr >> 2) + (fr & 3)) * SK;
  const int c0 = (h ^ (fr & 7)) * 16, c1 = ((4 + h) ^ (fr & 7)) * 16;
  i32x4_t acc[TI][TJ], a0[TI], b0[TJ], a1[TI], b1[TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = i32x4_t{0, 0, 0, 0};

#define SPARQ24_INT8_READ(fa_, fb_, at, c)                                                     \
  {                                                                                            \
    _Pragma("unroll") for (int j = 0; j < TJ; ++j) fb_[j] = *(const i32x4_t*)(fb + (at) + 4 * SK * j + (c)); \
    _Pragma("unroll") for (int i = 0; i < TI; ++i) fa_[i] = *(const i32x4_t*)(fa + (at) + 16 * SK * i + (c)); \
  }
#define SPARQ24_INT8_MULTIPLY(fa_, fb_)                                                        \
  {                                                                                            \
    _Pragma("unroll") for (int i = 0; i < TI; ++i) _Pragma("unroll") for (int j = 0; j < TJ; ++j) \
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fb_[j], fa_[i], acc[i][j], 0, 0, 0); \
  }
  const int nk = K / SK;  // whole slabs
  auto barrier = [] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
  };
  constexpr int kLgkm0 = 0xC07F, kAll0 = 0x0070;  // s_waitcnt lgkmcnt(0); with vmcnt(0)
  if (PP && nk) {
    const bool late = w >= 4;
    SPARQ24_INT8_SLAB(0, 0);
    SPARQ24_INT8_SLAB(1, nk > 1 ? SK : 0);  // past the end: the last one again
    wait_vmcnt<0>();
    barrier();
    if (late) barrier();
    for (int kt = 0; kt < nk; ++kt) {
      const int cur = (kt & 1) * STAGE;
      SPARQ24_INT8_READ(a0, b0, cur, c0);
      if (kt) SPARQ24_INT8_SLAB((kt & 1) ^ 1, (kt + 1 < nk ? kt + 1 : nk - 1) * SK);
      __builtin_amdgcn_s_waitcnt(kLgkm0);
      barrier();
      __builtin_amdgcn_s_setprio(1);
      SPARQ24_INT8_MULTIPLY(a0, b0);
      __builtin_amdgcn_s_setprio(0);
      barrier();
      SPARQ24_INT8_READ(a0, b0, cur, c1);
      if (late) __builtin_amdgcn_s_waitcnt(kAll0);
      else __builtin_amdgcn_s_waitcnt(kLgkm0);
      barrier();
      __builtin_amdgcn_s_setprio(1);
      SPARQ24_INT8_MULTIPLY(a0, b0);
      __builtin_amdgcn_s_setprio(0);
      if (!late) wait_vmcnt<0>();
      barrier();
    }
    if (!late) barrier();
  } else if (nk) {
    SPARQ24_INT8_SLAB(0, 0);
    SPARQ24_INT8_SLAB(1, nk > 1 ? SK : 0);  // past the end: the last one again
    wait_vmcnt<QA + QB>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    SPARQ24_INT8_READ(a0, b0, 0, c0);
    for (int kt = 0; kt < nk; ++kt) {
      const int cur = (kt & 1) * STAGE, nxt = STAGE - cur;
      SPARQ24_INT8_READ(a1, b1, cur, c1);
      SPARQ24_INT8_MULTIPLY(a0, b0);
#pragma unroll
      for (int i = 0; i < TI + TJ; ++i) {  // a read among every two or three products
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, TI * TJ / (TI + TJ), 0);
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      SPARQ24_INT8_SLAB(kt & 1, (kt + 2 < nk ? kt + 2 : nk - 1) * SK);
      SPARQ24_INT8_READ(a0, b0, nxt, c0);
      SPARQ24_INT8_MULTIPLY(a1, b1);
#pragma unroll
      for (int i = 0; i < QA + QB; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 1);
        __builtin_amdgcn_sched_group_barrier(0x020, 1, 1);
      }
#pragma unroll
      for (int i = 0; i < TI + TJ; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 1);
        __builtin_amdgcn_sched_group_barrier(0x008, (TI * TJ - QA - QB) / (TI + TJ), 1);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (nk) {
    wait_vmcnt<0>();  // the slabs requested past the end have landed
    __syncthreads();
  }
  if (K % SK) {  // the rest of K, filled up with zeros
    auto fill = [&](uint8_t* at, const int8_t* src, unsigned off, int chunk) {
      i32x4_t v = {0, 0, 0, 0};
      if (nk * SK + chunk < K) v = *(const i32x4_t*)(src + nk * SK + off);
      *(i32x4_t*)at = v;
    };
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int p = q * NT + tid;
      fill(smem + p * 16, base_a, off_a[q], 16 * ((p & 7) ^ ((p >> 3) & 7)));
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int p = q * NT + tid, r = p >> 3;
      fill(smem + A_BYTES + p * 16, base_b, off_b[q], 16 * ((p & 7) ^ ((r & 3) | ((r >> 2) & 4))));
    }
    __syncthreads();
    SPARQ24_INT8_READ(a0, b0, 0, c0);
    SPARQ24_INT8_READ(a1, b1, 0, c1);
    SPARQ24_INT8_MULTIPLY(a0, b0);
    SPARQ24_INT8_MULTIPLY(a1, b1);
  }
  // lane: row 16 i + fr, outputs 16 h + 4 j + e
  const int64_t n = n0 + wn * WN + 16 * h;
  float sb[16], bias[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int64_t c = n + e < g.N ? n + e : g.N - 1;
    sb[e] = g.sb[c];
    bias[e] = g.bias ? g.bias[c] : -0.0f;  // y + -0 is y
  }
  auto out = [&]<class T>(T) {
    const bool wide = n + 16 <= g.N;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t m = m0 + wm * WM + 16 * i + fr;
      if (m < g.M) int8_store16<T>(g, m, n, acc[i], g.sa[m], sb, bias, wide);
    }
  };
  if (g.dtype == 0) out(0.0f);
  else if (g.dtype == 1) out((__bf16)0.0f);
  else out((_Float16)0.0f);
}

hipError_t launch_int8_gemm(const Int8Gemm& g, hipStream_t s) {
  auto few = [&]<int MT, int NT, int W, int S>() {
    const int64_t ntm = (g.M + 16 * MT - 1) / (16 * MT), ntn = (g.N + 16 * NT - 1) / (16 * NT);
    hipLaunchKernelGGL((k_int8_stream<MT, NT, W, S>), dim3((unsigned)(ntm * ntn)), dim3(64 * W), 0, s, g, ntn);
    return hipGetLastError();
  };
  auto tile = [&]<int BM, int BN, int WM, bool PP>() {
    const int64_t n = ((g.M + BM - 1) / BM) * ((g.N + BN - 1) / BN);
    hipLaunchKernelGGL((k_int8_tile<BM, BN, WM, PP>), dim3((unsigned)n), dim3((BM / WM) * (BN / 64) * 64), 0, s, g);
    return hipGetLastError();
  };
  auto tiles = [&](int bm, int bn) { return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn); };
  // k_int8_stream takes about 2.4 us + 1.1 us per 16-row group of a and b that a
  // CU streams (K = 4096): (1, 1) and (1, 4) for 1 x 4096 and 1 x 14336: 4.5, 11.0;
  // (2, 2) 6.8, (2, 4) 8.0, (4, 4) 10.8 us for 64, 128, 256 x 4096.  At two rounds
  // of (4, 4) the tiles draw level (100 x 14336: 22.8 and 22.4 us, 512 x 4096: 20.9
  // and 21.6; with K = 1024, 777 x 2048: 11.4 and 9.2).
  const int cus = device_cu_count();
  const bool far_rows = g.lda >= (1 << 23) || g.ldb >= (1 << 23);  // past the tiles' 32-bit offsets
  int mt = 0, nt = 0;
  int64_t best = INT64_MAX;
  for (int i = 1; i <= 4; i *= 2)
    for (int j = 1; j <= 4; j *= 2) {
      const int64_t rounds = (tiles(16 * i, 16 * j) + cus - 1) / cus;
      if (rounds * (i + j) < best) best = rounds * (i + j), mt = i, nt = j;
    }
  if (best <= 8 || far_rows) {
    switch (mt * 8 + nt) {
      case 9: return few.template operator()<1, 1, 8, 3>();
      case 10: return few.template operator()<1, 2, 8, 2>();
      case 12: return few.template operator()<1, 4, 8, 2>();
      case 17: return few.template operator()<2, 1, 8, 2>();
      case 18: return few.template operator()<2, 2, 8, 2>();
      case 20: return few.template operator()<2, 4, 4, 2>();
      case 33: return few.template operator()<4, 1, 8, 2>();
      case 34: return few.template operator()<4, 2, 4, 2>();
      default: return few.template operator()<4, 4, 4, 2>();
    }
  }
  // The largest tile that still gives every CU one, else four small ones per CU
  // (a 64 x 64 tile takes 32 KB of LDS), else the middle.  At K = 4096, us for
  // 256 x 256 / 256 x 128 / 128 x 128 / 64 x 64: 4096 x 14336: 256 / 284 / 304 /
  // 416; 2048 x 4096: 49 / 37 / 41 / 58; 1024 x 4096: 46 / 30 / 27 / 26.
  if (tiles(256, 256) >= cus) return tile.template operator()<256, 256, 128, true>();
  if (tiles(256, 128) >= cus) return tile.template operator()<256, 128, 64, false>();
  if (tiles(64, 64) > 4 * cus) return tile.template operator()<128, 128, 64, false>();
  return tile.template operator()<64, 64, 64, false>();
}

}  // namespace sparq24
