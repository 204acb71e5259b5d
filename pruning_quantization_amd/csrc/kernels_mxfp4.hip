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

// 16 outputs n .. n + 15 of row m: 16-byte stores where `wide` says that all
// are inside (rows may begin at any element), else one by one.
template <class T>
__device__ inline void mx_store16(const Mxfp4Gemm& g, int64_t m, int64_t n, const f32x4_t (&acc)[4],
                                  const float* bias, bool wide) {
  typedef T t8 __attribute__((ext_vector_type(16 / sizeof(T)), aligned(sizeof(T))));
  constexpr int V = 16 / sizeof(T);
  T* c = (T*)g.c + m * g.ldc + n;
  T y[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = (T)(acc[e / 4][e % 4] + bias[e]);
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

// Exponent rows begin at any byte.
typedef uint32_t u32_any __attribute__((aligned(1)));
typedef __attribute__((address_space(1))) const uint8_t* global_bytes_t;
typedef __attribute__((address_space(1))) const u32_any* global_u32_any_t;
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(1)));

// Loads at a scalar base and a 32-bit offset of the lane.  The compiler would add the
// offset to the base's loop-invariant part first and keep 64-bit sums, one pair of
// registers per load of the loop (which the largest tile does not have), so the base comes
// through hidden() and the offset is widened here.
__device__ inline const uint8_t* hidden(const uint8_t* p) {
  asm("" : "+s"(p));
  return p;
}
__device__ inline unsigned lane_value(unsigned v) {
  asm("" : "+v"(v));
  return v;
}
__device__ inline global_bytes_t lane_address(const uint8_t* p, unsigned o) { return (global_bytes_t)p + lane_value(o); }
__device__ inline void load_lds16(const uint8_t* p, unsigned o, uint8_t* lds) {
  __builtin_amdgcn_global_load_lds(lane_address(p, o), (lds_void_t*)lds, 16, 0, 0);
}
__device__ inline uint32_t load_any(const uint8_t* p, unsigned o) { return *(global_u32_any_t)lane_address(p, o); }

// c += b a with byte X of both exponents, c in accumulation registers and in place: with
// the builtin the compiler gives results registers of their own, which a wave that
// accumulates in half of its registers does not have.  The compiler puts no waits around it:
// before the first product and behind the last one stands settle().
template <int X>
__device__ inline void mx_product_at(i32x4_t b, i32x4_t a, f32x4_t& c, uint32_t sb, uint32_t sa) {
#define SPARQ24_MXFP4_ASM(sel)                                                                   \
  asm volatile("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 " sel " cbsz:4 blgp:4" \
               : "+a"(c) : "v"(b), "v"(a), "v"(sb), "v"(sa))
  if constexpr (X == 0) SPARQ24_MXFP4_ASM("op_sel_hi:[0,0,0]");
  if constexpr (X == 1) SPARQ24_MXFP4_ASM("op_sel:[1,1,0] op_sel_hi:[0,0,0]");
  if constexpr (X == 2) SPARQ24_MXFP4_ASM("op_sel_hi:[1,1,0]");
  if constexpr (X == 3) SPARQ24_MXFP4_ASM("op_sel:[1,1,0] op_sel_hi:[1,1,0]");
}
// Waits until products are done, or what they start from is written.  All accumulators go
// through asm on both sides of the wait (which yields no instruction), so that neither
// copies out of them nor zeros into them can pass it.
template <int TI, int TJ>
__device__ inline void settle(f32x4_t (&c)[TI][TJ]) {
  auto hold = [&] {
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) asm volatile("" : "+a"(c[i][j]));
  };
  hold();
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
  hold();
}

// Many rows: a BM x BN tile per workgroup, waves of WM x 64.  Slabs of 256 codes go from
// memory straight into LDS (global_load_lds) into two buffers, their 16-byte chunks
// XOR-swizzled by row; the slab's eight exponents of a row go through registers.  A
// slab is two steps of 128 codes: of its eight groups lane group h takes 2 h in the
// first and 2 h + 1 in the second, so that a row's exponents of both are one 16-bit read.
// Rows past the ends repeat the last; a rest of K is filled up with zeros.  Fragments of a
// step are read while the products of the step before run, across slabs too; between a
// slab's two steps every wave has its last fragments of it and the next slab has landed
// (one barrier), and the slab after that starts into the freed buffer.
template <int BM, int BN, int WM>
__global__ __launch_bounds__((BM / WM) * (BN / 64) * 64) void k_mxfp4_tile(Mxfp4Gemm g) {
  constexpr int WN = 64, NWN = BN / WN, NT = (BM / WM) * NWN * 64;
  constexpr int TI = WM / 16, TJ = 4, SK = 128;
  constexpr int A_BYTES = BM * SK, E_AT = (BM + BN) * SK, STAGE = E_AT + (BM + BN) * 8;
  constexpr int QA = BM * 8 / NT, QB = BN * 8 / NT, NE = (BM + BN) * 2, QE = (NE + NT - 1) / NT;
  static_assert(QA * NT == BM * 8 && QB * NT == BN * 8 && NE % 64 == 0 && TI % 4 == 0, "tile / threads");
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
  // 8 MiB and more go to k_mxfp4_stream).  Swizzles: the sixteen lanes that a 16-byte
  // LDS read takes at a time (rows 0 .. 7 of a fragment, two lane groups) meet sixteen
  // chunks; the rows of a B fragment are 4 j + 0 .. 3 and 16 more.
  auto swizzle_a = [](int r) { return ((r >> 1) & 1) | (r & 4); };
  auto swizzle_b = [](int r) { return ((r >> 1) & 1) | ((r >> 2) & 4); };
  const int KB = (int)(g.K / 2), groups = (int)(g.K / 32);
  const int rows_a = (int)(g.M - m0 < BM ? g.M - m0 : BM), rows_b = (int)(g.N - n0 < BN ? g.N - n0 : BN);
  const uint8_t *base_a = g.a + m0 * g.lda, *base_b = g.b + n0 * g.ldb;
  const uint8_t *exps_a = g.sa + m0 * groups, *exps_b = g.sb + n0 * groups;
  unsigned off_a[QA], off_b[QB], off_e[QE];
#pragma unroll
  for (int q = 0; q < QA; ++q) {
    const int p = q * NT + tid, r = p >> 3, m = r < rows_a ? r : rows_a - 1;
    off_a[q] = (unsigned)m * (unsigned)g.lda + 16 * ((p & 7) ^ swizzle_a(r));
  }
#pragma unroll
  for (int q = 0; q < QB; ++q) {
    const int p = q * NT + tid, r = p >> 3, n = r < rows_b ? r : rows_b - 1;
    off_b[q] = (unsigned)n * (unsigned)g.ldb + 16 * ((p & 7) ^ swizzle_b(r));
  }
  // exponents: dword p of a slab is half p % 2 of row p / 2, the rows of A first
  auto is_a = [&](int q) { return BM * 2 % NT == 0 ? q < BM * 2 / NT : w + NT / 64 * q < BM * 2 / 64; };
#pragma unroll
  for (int q = 0; q < QE; ++q) {
    const int r = (q * NT + tid) >> 1, m = r < rows_a ? r : rows_a - 1;
    const int n = r - BM < rows_b ? r - BM : rows_b - 1;
    off_e[q] = (unsigned)(is_a(q) ? m : n) * (unsigned)groups + 4 * (tid & 1);
  }
  auto has_e = [&](int q) { return NE % NT == 0 || w + NT / 64 * q < NE / 64; };
  uint32_t ex[QE];
#define SPARQ24_MXFP4_SLAB(buf, kt)                                                            \
  {                                                                                            \
    const int t_ = __builtin_amdgcn_readfirstlane(kt);                                         \
    uint8_t* st = smem + (buf) * STAGE + w * 1024;                                             \
    const uint8_t *ka = hidden(base_a + t_ * SK), *kb = hidden(base_b + t_ * SK);              \
    const uint8_t *xa_ = hidden(exps_a + t_ * 8), *xb_ = hidden(exps_b + t_ * 8);              \
    _Pragma("unroll") for (int q = 0; q < QE; ++q) ex[q] = load_any(is_a(q) ? xa_ : xb_, off_e[q]); \
    _Pragma("unroll") for (int q = 0; q < QA; ++q) load_lds16(ka, off_a[q], st + q * NT * 16); \
    _Pragma("unroll") for (int q = 0; q < QB; ++q) load_lds16(kb, off_b[q], st + A_BYTES + q * NT * 16); \
  }
#define SPARQ24_MXFP4_EXPONENTS(buf)                                                           \
  {                                                                                            \
    _Pragma("unroll") for (int q = 0; q < QE; ++q)                                             \
        if (has_e(q)) *(uint32_t*)(smem + (buf) * STAGE + E_AT + (q * NT + tid) * 4) = ex[q];  \
  }

  const int fr = lane & 15, h = lane >> 4;
  // fragment rows: A tile i row fr; B tile j row fr is weight row
  // 16 (fr / 4) + 4 j + fr % 4 (a lane then holds 16 adjacent outputs)
  const int ra = wm * WM + fr, rb = wn * WN + 16 * (fr >> 2) + (fr & 3);
  const uint8_t *fa = smem + ra * SK, *fb = smem + A_BYTES + rb * SK;
  const uint8_t *xa = smem + E_AT + ra * 8 + 2 * h, *xb = smem + E_AT + (BM + rb) * 8 + 2 * h;
  const int ca0 = ((2 * h) ^ swizzle_a(fr)) * 16, ca1 = ca0 ^ 16;
  const int cb0 = ((2 * h) ^ swizzle_b(16 * (fr >> 2) + (fr & 3))) * 16, cb1 = cb0 ^ 16;
  f32x4_t acc[TI][TJ];
  i32x4_t a0[TI], b0[TJ], a1[TI], b1[TJ];
  uint32_t ea[TI], eb[TJ], na[TI], nb[TJ];
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#define SPARQ24_MXFP4_READ(fa_, fb_, at, ca, cb)                                               \
  {                                                                                            \
    _Pragma("unroll") for (int j = 0; j < TJ; ++j) fb_[j] = *(const i32x4_t*)(fb + (at) + 4 * SK * j + (cb)); \
    _Pragma("unroll") for (int i = 0; i < TI; ++i) fa_[i] = *(const i32x4_t*)(fa + (at) + 16 * SK * i + (ca)); \
  }
#define SPARQ24_MXFP4_READ_EXPONENTS(ea_, eb_, at)                                             \
  {                                                                                            \
    _Pragma("unroll") for (int j = 0; j < TJ; ++j) eb_[j] = *(const uint16_t*)(xb + (at) + 32 * j); \
    _Pragma("unroll") for (int i = 0; i < TI; ++i) ea_[i] = *(const uint16_t*)(xa + (at) + 128 * i); \
  }
#define SPARQ24_MXFP4_MULTIPLY(X, fa_, fb_, ea_, eb_)                                          \
  {                                                                                            \
    _Pragma("unroll") for (int i = 0; i < TI; ++i) _Pragma("unroll") for (int j = 0; j < TJ; ++j) \
        acc[i][j] = mx_product<X, X>(fb_[j], fa_[i], acc[i][j], eb_[j], ea_[i]);               \
  }
  const int nk = KB / SK;  // whole slabs
  constexpr int kLgkm0 = 0xC07F;  // s_waitcnt lgkmcnt(0)
  if (nk) {
    SPARQ24_MXFP4_SLAB(0, 0);
    SPARQ24_MXFP4_EXPONENTS(0);
    SPARQ24_MXFP4_SLAB(1, nk > 1 ? 1 : 0);  // past the end: the last one again
    wait_vmcnt<QA + QB + QE>();
    __builtin_amdgcn_s_waitcnt(kLgkm0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    SPARQ24_MXFP4_READ(a0, b0, 0, ca0, cb0);
    SPARQ24_MXFP4_READ_EXPONENTS(ea, eb, 0);
    for (int kt = 0; kt < nk; ++kt) {
      const int cur = (kt & 1) * STAGE, nxt = STAGE - cur;
      SPARQ24_MXFP4_READ(a1, b1, cur, ca1, cb1);
      SPARQ24_MXFP4_MULTIPLY(0, a0, b0, ea, eb);
      __builtin_amdgcn_sched_barrier(0);
      wait_vmcnt<0>();
      SPARQ24_MXFP4_EXPONENTS((kt & 1) ^ 1);
      __builtin_amdgcn_s_waitcnt(kLgkm0);
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
      SPARQ24_MXFP4_SLAB(kt & 1, kt + 2 < nk ? kt + 2 : nk - 1);
      SPARQ24_MXFP4_READ(a0, b0, nxt, ca0, cb0);
      SPARQ24_MXFP4_READ_EXPONENTS(na, nb, nxt);
      SPARQ24_MXFP4_MULTIPLY(1, a1, b1, ea, eb);
#pragma unroll
      for (int i = 0; i < TI; ++i) ea[i] = na[i];
#pragma unroll
      for (int j = 0; j < TJ; ++j) eb[j] = nb[j];
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (nk) {
    wait_vmcnt<0>();  // the slabs requested past the end have landed
    __syncthreads();
  }
  if (KB % SK) {  // the rest of K, filled up with zeros (codes; exponents of 1)
    auto fill = [&](uint8_t* at, const uint8_t* src, unsigned off, int chunk) {
      i32x4_t v = {0, 0, 0, 0};
      if (nk * SK + chunk < KB) v = *(const i32x4_t*)(src + nk * SK + off);
      *(i32x4_t*)at = v;
    };
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int p = q * NT + tid;
      fill(smem + p * 16, base_a, off_a[q], 16 * ((p & 7) ^ swizzle_a(p >> 3)));
    }
#pragma unroll
    for (int q = 0; q < QB; ++q) {
      const int p = q * NT + tid;
      fill(smem + A_BYTES + p * 16, base_b, off_b[q], 16 * ((p & 7) ^ swizzle_b(p >> 3)));
    }
#pragma unroll
    for (int q = 0; q < QE; ++q) {
      if (!has_e(q)) continue;
      uint32_t v = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const bool in = 8 * nk + 4 * (tid & 1) + e < groups;
        v |= (in ? ((is_a(q) ? exps_a : exps_b) + off_e[q] + 8 * nk)[e] : 127u) << (8 * e);
      }
      *(uint32_t*)(smem + E_AT + (q * NT + tid) * 4) = v;
    }
    __syncthreads();
    SPARQ24_MXFP4_READ_EXPONENTS(ea, eb, 0);
    SPARQ24_MXFP4_READ(a0, b0, 0, ca0, cb0);
    SPARQ24_MXFP4_MULTIPLY(0, a0, b0, ea, eb);
    SPARQ24_MXFP4_READ(a0, b0, 0, ca1, cb1);
    SPARQ24_MXFP4_MULTIPLY(1, a0, b0, ea, eb);
  }
  // lane: row 16 i + fr, outputs 16 h + 4 j + e
  const int64_t n = n0 + wn * WN + 16 * h;
  float bias[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) bias[e] = g.bias ? g.bias[n + e < g.N ? n + e : g.N - 1] : -0.0f;  // y + -0 is y
  auto out = [&]<class T>(T) {
    const bool wide = n + 16 <= g.N;
#pragma unroll
    for (int i = 0; i < TI; ++i) {
      const int64_t m = m0 + wm * WM + 16 * i + fr;
      if (m < g.M) mx_store16<T>(g, m, n, acc[i], bias, wide);
    }
  };
  if (g.dtype == 0) out(0.0f);
  else if (g.dtype == 1) out((__bf16)0.0f);
  else out((_Float16)0.0f);
}

// 256 x 256 tiles, four waves of 128 x 128, one per SIMD.  Slabs of 256 codes (128 bytes) go
// from memory straight into two buffers in LDS; a slab is two steps of 128 codes, of whose
// eight groups lane group h takes 2 h and 2 h + 1.  The fragments of a step are read while
// the products of the step before run; between a slab's two steps every wave has its last
// fragments of it and the next slab has landed (one barrier a slab), and the slab after
// that starts into the freed buffer.  The exponents of a row come two slabs at a time, a
// thread two rows: 16 bytes [slab][lane group][step], turned into [lane group][slab][step],
// so that a lane group gets its four in one dword, whose byte the matrix instruction
// selects.
// CHAINED, where rows end with such a pair of slabs: a workgroup walks through several
// tiles, and what is asked for behind a tile's end is the next one's first slabs, which land
// while results are stored (4096 x 14336 x 4096: 140 us, a workgroup per tile 145).
// 4096 x 14336 x 4096 140 us, 3.4 Pflop/s; at K = 8192 254 us, 3.8.  By counters the first
// takes 298000 cycles (2.13 GHz; 2.4 without load), the matrix units busy for 115000 of them
// (38%).  A slab takes 3570 (the difference of the two, over four rounds of tiles), 2048 of them
// products: the rest is the one wave of a SIMD issuing reads and loads among them and waiting
// at the barrier (26% of its cycles wait for data, 27% to issue).  A tile's start and end take
// 17000 more, and 896 tiles leave half of the CUs idle in the last of four rounds.
template <bool CHAINED>
__global__ __launch_bounds__(256, 1) void k_mxfp4_wide(Mxfp4Gemm g, unsigned tiles) {
  constexpr int BM = 256, BN = 256, NT = 256, TI = 8, TJ = 8, SK = 128;
  constexpr int A_BYTES = BM * SK, STAGE = (BM + BN) * SK, E_AT = 2 * STAGE, QA = 8, QB = 8;
  __shared__ __attribute__((aligned(16))) uint8_t smem[E_AT + (BM + BN) * 32];
  const int tid = threadIdx.x, lane = tid & 63, w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = w >> 1, wn = w & 1;
  // XCD-aware order: each XCD owns a contiguous run of tiles, walked in
  // groups of eight row tiles, so that its L2 serves the shared slabs
  const unsigned ntn = (unsigned)((g.N + BN - 1) / BN), ntm = (unsigned)((g.M + BM - 1) / BM), per = tiles / 8;
  int64_t m0, n0;
  auto place = [&](unsigned pid) {
    const unsigned lid = pid < per * 8 ? (pid % 8) * per + pid / 8 : pid;
    constexpr unsigned kGroupM = 8;
    const unsigned ingroup = kGroupM * ntn, first = (lid / ingroup) * kGroupM;
    const unsigned gsz = ntm - first < kGroupM ? ntm - first : kGroupM;
    m0 = (int64_t)__builtin_amdgcn_readfirstlane(first + (lid % ingroup) % gsz) * BM;
    n0 = (int64_t)__builtin_amdgcn_readfirstlane((lid % ingroup) / gsz) * BN;
  };

  // Swizzles: the sixteen lanes that a 16-byte LDS read takes at a time (rows 0 .. 7 of a
  // fragment, two lane groups) meet sixteen chunks; the rows of a B fragment are 4 j + 0 .. 3
  // and 16 more.
  auto swizzle_a = [](int r) { return ((r >> 1) & 1) | (r & 4); };
  auto swizzle_b = [](int r) { return ((r >> 1) & 1) | ((r >> 2) & 4); };
  const int KB = (int)(g.K / 2), groups = (int)(g.K / 32);
  const uint8_t *base_a, *base_b, *exps_a, *exps_b;
  unsigned off_a[QA], off_b[QB];
  auto aim = [&] {  // at the tile m0, n0
    const int rows_a = (int)(g.M - m0 < BM ? g.M - m0 : BM), rows_b = (int)(g.N - n0 < BN ? g.N - n0 : BN);
    const int t = (int)lane_value(tid);  // nothing of this is kept over a tile
    base_a = g.a + m0 * g.lda;
    base_b = g.b + n0 * g.ldb;
#pragma unroll
    for (int q = 0; q < QA; ++q) {
      const int p = q * NT + t, r = p >> 3;
      off_a[q] = (unsigned)(r < rows_a ? r : rows_a - 1) * (unsigned)g.lda + 16 * ((p & 7) ^ swizzle_a(r));
      off_b[q] = (unsigned)(r < rows_b ? r : rows_b - 1) * (unsigned)g.ldb + 16 * ((p & 7) ^ swizzle_b(r));
    }
    // this thread's rows of exponents: row tid of A and of B
    exps_a = g.sa + (m0 + (t < rows_a ? t : rows_a - 1)) * groups;
    exps_b = g.sb + (n0 + (t < rows_b ? t : rows_b - 1)) * groups;
  };
  // chunk c: groups 16 c .. 16 c + 15 (there are 16 at least).  The last one, where the row
  // ends in it, is put together once (exponents of 1 behind the end) and waits in LDS.
  uint8_t* rest = smem + E_AT + (BM + BN) * 16 + tid * 16;
  u32x4_t next_a, next_b;
  auto ask_chunk = [&](int c) {
    const int at = 16 * c + 16 <= groups ? 16 * c : groups - 16;
    next_a = *(const u32x4_any*)(exps_a + at);
    next_b = *(const u32x4_any*)(exps_b + at);
  };
  auto put_row = [&](u32x4_t v, int row) {
    *(u32x4_t*)(smem + E_AT + row * 16) =
        u32x4_t{__builtin_amdgcn_perm(v[2], v[0], 0x05040100u), __builtin_amdgcn_perm(v[2], v[0], 0x07060302u),
                __builtin_amdgcn_perm(v[3], v[1], 0x05040100u), __builtin_amdgcn_perm(v[3], v[1], 0x07060302u)};
  };
  auto put_chunk = [&](int c) {
    const bool ends = !CHAINED && 16 * c + 16 > groups;
    put_row(ends ? *(const u32x4_t*)rest : next_a, tid);
    put_row(ends ? *(const u32x4_t*)(rest + NT * 16) : next_b, BM + tid);
  };
  const int nk = KB / SK;  // whole slabs
  auto request = [&](int stage, int slab) {
    const int t = __builtin_amdgcn_readfirstlane(slab < nk ? slab : nk - 1);  // past the end: the last one again
    uint8_t* st = smem + stage * STAGE + w * 1024;
    const uint8_t *ka = hidden(base_a + t * SK), *kb = hidden(base_b + t * SK);
#pragma unroll
    for (int q = 0; q < QA; ++q) load_lds16(ka, off_a[q], st + q * NT * 16);
#pragma unroll
    for (int q = 0; q < QB; ++q) load_lds16(kb, off_b[q], st + A_BYTES + q * NT * 16);
  };

  const int fr = lane & 15, h = lane >> 4;
  // fragment rows: A tile i row fr; B tile j row fr is weight row 64 (j / 4) +
  // 16 (fr / 4) + 4 (j % 4) + fr % 4 (a lane then holds 16 adjacent outputs of each half)
  const int ra = wm * 128 + fr, rb = wn * 128 + 16 * (fr >> 2) + (fr & 3);
  const unsigned fa = ra * SK + 16 * ((2 * h) ^ swizzle_a(ra)), fb = A_BYTES + rb * SK + 16 * ((2 * h) ^ swizzle_b(rb));
  const unsigned xa = E_AT + ra * 16 + 4 * h, xb = E_AT + (BM + rb) * 16 + 4 * h;
  f32x4_t acc[TI][TJ];
  i32x4_t af[2][TI], bf[2][TJ];
  uint32_t ea[TI], eb[TJ];
  auto read = [&]<int X>(int stage) {  // step X of the slab in `stage`
    const unsigned a = lane_value((fa ^ (16 * X)) + stage * STAGE), b = lane_value((fb ^ (16 * X)) + stage * STAGE);
#pragma unroll
    for (int j = 0; j < TJ; ++j) bf[X][j] = *(const i32x4_t*)(smem + b + 64 * SK * (j >> 2) + 4 * SK * (j & 3));
#pragma unroll
    for (int i = 0; i < TI; ++i) af[X][i] = *(const i32x4_t*)(smem + a + 16 * SK * i);
  };
  auto read_exponents = [&] {
#pragma unroll
    for (int j = 0; j < TJ; ++j) eb[j] = *(const uint32_t*)(smem + xb + 1024 * (j >> 2) + 64 * (j & 3));
#pragma unroll
    for (int i = 0; i < TI; ++i) ea[i] = *(const uint32_t*)(smem + xa + 256 * i);
  };
  // Products p of step X of slab Y of a chunk, four at a time.
  auto multiply4 = [&]<int X, int Y>(int p) {
#pragma unroll
    for (int q = 4 * p; q < 4 * p + 4; ++q)
      mx_product_at<2 * Y + X>(bf[X][q % TJ], af[X][q / TJ], acc[q / TJ][q % TJ], eb[q % TJ], ea[q / TJ]);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto fence = [] {
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
  };
  constexpr int kLgkm0 = 0xC07F;  // s_waitcnt lgkmcnt(0)
  unsigned pid = blockIdx.x;
  place(pid);
  aim();
  if (!CHAINED && groups % 16) {
#pragma unroll 1
    for (int e = 0; e < 16; ++e) {
      const int i = groups / 16 * 16 + e;
      rest[e] = i < groups ? exps_a[i] : 127;
      rest[NT * 16 + e] = i < groups ? exps_b[i] : 127;
    }
  }
  {
    ask_chunk(0);
    request(0, 0);
    put_chunk(0);
    request(1, 1);
    wait_vmcnt<16>();
    __builtin_amdgcn_s_waitcnt(kLgkm0);
    fence();
    __builtin_amdgcn_s_barrier();
    fence();
    read_exponents();
    read.template operator()<0>(0);
  }
  for (;;) {  // the workgroup's tiles
    const int64_t out_m = m0, out_n = n0;  // m0 and n0 go on to the next tile before this one is stored
    const bool more = CHAINED && pid + gridDim.x < tiles;
#pragma unroll
    for (int i = 0; i < TI; ++i)
#pragma unroll
      for (int j = 0; j < TJ; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    settle(acc);
    // Slab s, number Y of its chunk; asks for slab `next` in its place and (Y = 0) for
    // chunk `chunk`, which is put down in Y = 1.  A read or two loads among every four
    // products.
    auto slab = [&]<int Y>(int next, int chunk) {
      constexpr int kQuads = TI * TJ / 4;
      const unsigned a1 = lane_value((fa ^ 16) + Y * STAGE), b1 = lane_value((fb ^ 16) + Y * STAGE);
      if constexpr (Y == 0) ask_chunk(chunk);
#pragma unroll
      for (int p = 0; p < kQuads; ++p) {
        if (p < TJ) bf[1][p] = *(const i32x4_t*)(smem + b1 + 64 * SK * (p >> 2) + 4 * SK * (p & 3));
        else af[1][p - TJ] = *(const i32x4_t*)(smem + a1 + 16 * SK * (p - TJ));
        multiply4.template operator()<0, Y>(p);
      }
      wait_vmcnt<0>();
      if constexpr (Y == 1) put_chunk(chunk);
      __builtin_amdgcn_s_waitcnt(kLgkm0);
      fence();
      __builtin_amdgcn_s_barrier();
      fence();
      const unsigned a0 = lane_value(fa + (1 - Y) * STAGE), b0 = lane_value(fb + (1 - Y) * STAGE);
      const int t = __builtin_amdgcn_readfirstlane(next < nk ? next : nk - 1);  // past the end: the last one again
      uint8_t* st = smem + Y * STAGE + w * 1024;
      const uint8_t *ka = hidden(base_a + t * SK), *kb = hidden(base_b + t * SK);
#pragma unroll
      for (int p = 0; p < kQuads; ++p) {
        if (p < TJ) bf[0][p] = *(const i32x4_t*)(smem + b0 + 64 * SK * (p >> 2) + 4 * SK * (p & 3));
        else af[0][p - TJ] = *(const i32x4_t*)(smem + a0 + 16 * SK * (p - TJ));
        if (p < QA / 2) {
          load_lds16(ka, off_a[2 * p], st + (2 * p) * NT * 16);
          load_lds16(ka, off_a[2 * p + 1], st + (2 * p + 1) * NT * 16);
        } else if (p < QA / 2 + QB / 2) {
          const int q = 2 * p - QA;
          load_lds16(kb, off_b[q], st + A_BYTES + q * NT * 16);
          load_lds16(kb, off_b[q + 1], st + A_BYTES + (q + 1) * NT * 16);
        }
        multiply4.template operator()<1, Y>(p);
      }
      if constexpr (Y == 1) read_exponents();
    };
    int s = 0;
    for (; s + 2 <= nk; s += 2) {
      const bool next = CHAINED && s + 2 == nk;
      if (next && more) {
        pid += gridDim.x;
        place(pid);
        aim();
      }
      const int chunk = next ? 0 : s / 2 + 1;
      slab.template operator()<0>(next ? 0 : s + 2, chunk);
      slab.template operator()<1>(next ? 1 : s + 3, chunk);
    }
    if constexpr (!CHAINED) {
      if (s < nk) slab.template operator()<0>(nk, s / 2 + 1);
    }
    settle(acc);
    if (!more) {
      wait_vmcnt<0>();  // the slabs requested past the end have landed
      __syncthreads();
    }
    if (!CHAINED && KB % SK) {  // the rest of K, filled up with zeros (codes; exponents of 1)
      auto fill = [&](uint8_t* at, const uint8_t* src, unsigned off, int chunk) {
        i32x4_t v = {0, 0, 0, 0};
        if (nk * SK + chunk < KB) v = *(const i32x4_t*)(src + nk * SK + off);
        *(i32x4_t*)at = v;
      };
#pragma unroll
      for (int q = 0; q < QA; ++q) {
        const int p = q * NT + tid;
        fill(smem + p * 16, base_a, off_a[q], 16 * ((p & 7) ^ swizzle_a(p >> 3)));
        fill(smem + A_BYTES + p * 16, base_b, off_b[q], 16 * ((p & 7) ^ swizzle_b(p >> 3)));
      }
      // the last chunk: this slab is its first or its second
      u32x4_t va = *(const u32x4_t*)rest, vb = *(const u32x4_t*)(rest + NT * 16);
      if (nk & 1) va = u32x4_t{va[2], va[3], va[2], va[3]}, vb = u32x4_t{vb[2], vb[3], vb[2], vb[3]};
      put_row(va, tid);
      put_row(vb, BM + tid);
      __syncthreads();
      read_exponents();
      read.template operator()<0>(0);
      read.template operator()<1>(0);
#pragma unroll
      for (int p = 0; p < TI * TJ / 4; ++p) {
        multiply4.template operator()<0, 0>(p);
        multiply4.template operator()<1, 0>(p);
      }
      settle(acc);
    }
    // lane: row 16 i + fr, outputs 64 half + 16 h + 4 j + e
    const int l = (int)lane_value(lane);  // row numbers are not kept over the products
    auto out = [&]<class T>(T) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int64_t n = out_n + wn * 128 + 64 * half + 16 * (l >> 4);
        float bias[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) bias[e] = g.bias ? g.bias[n + e < g.N ? n + e : g.N - 1] : -0.0f;  // y + -0 is y
        const bool wide = n + 16 <= g.N;
#pragma unroll
        for (int i = 0; i < TI; ++i) {
          const int64_t m = out_m + wm * 128 + 16 * i + (l & 15);
          const f32x4_t y[4] = {acc[i][4 * half], acc[i][4 * half + 1], acc[i][4 * half + 2], acc[i][4 * half + 3]};
          if (m < g.M) mx_store16<T>(g, m, n, y, bias, wide);
        }
      }
    };
    if (g.dtype == 0) out(0.0f);
    else if (g.dtype == 1) out((__bf16)0.0f);
    else out((_Float16)0.0f);
    if (!more) break;
  }
}

namespace {
// The kernel of a product, its tile and its launch.
struct Mxfp4Shape {
  enum { STREAM, TILE, WIDE } kernel;
  int bm, bn, threads;
  int64_t tiles;  // and workgroups, unless those walk from tile to tile
};
Mxfp4Shape shape_of(const Mxfp4Gemm& g) {
  auto tiles = [&](int bm, int bn) { return ((g.M + bm - 1) / bm) * ((g.N + bn - 1) / bn); };
  // k_mxfp4_stream takes time by the rounds of workgroups and the 16-row groups of a and b
  // that each streams (K = 4096, with the call: (1, 1) and (2, 4) for 1 x 4096 and 1 x
  // 14336: 4.1 and 8.8 us; (2, 2) 6.9, (2, 4) 8.2, (4, 4) 10.7 for 64, 128, 256 x 4096).
  // At two rounds of (4, 4) the tiles draw level (100 x 14336: 19.8 and 17.9 us).
  const int cus = device_cu_count();
  const bool far_rows = g.lda >= (1 << 23) || g.ldb >= (1 << 23);  // past the tiles' 32-bit offsets
  int mt = 0, nt = 0;
  int64_t best = INT64_MAX;
  for (int i = 1; i <= 4; i *= 2)
    for (int j = 1; j <= 4; j *= 2) {
      const int64_t rounds = (tiles(16 * i, 16 * j) + cus - 1) / cus;
      if (rounds * (i + j) < best) best = rounds * (i + j), mt = i, nt = j;
    }
  if (best <= 8 || far_rows)
    return {Mxfp4Shape::STREAM, 16 * mt, 16 * nt, mt * nt < 8 ? 512 : 256, tiles(16 * mt, 16 * nt)};
  // The largest tile that still gives every CU one, else small ones.  At K = 4096, us for
  // 256 x 256 / 256 x 128 / 128 x 128 / 64 x 64: 4096 x 14336: 141 / 168 / 193 / 278; 2048 x
  // 4096: 33 / 27 / 31 / 44; 1024 x 4096: 31 / 23 / 23 / 24.
  if (tiles(256, 256) >= cus && g.K >= 512) return {Mxfp4Shape::WIDE, 256, 256, 256, tiles(256, 256)};
  if (tiles(256, 128) >= cus) return {Mxfp4Shape::TILE, 256, 128, 512, tiles(256, 128)};
  if (tiles(64, 64) > 4 * cus) return {Mxfp4Shape::TILE, 128, 128, 256, tiles(128, 128)};
  return {Mxfp4Shape::TILE, 64, 64, 64, tiles(64, 64)};
}
}  // namespace

bool mxfp4_gemm_fits(const Mxfp4Gemm& g) {
  if (g.M <= 1 << 28 && g.N <= 1 << 28 && g.M * g.N <= 1ll << 34) return true;  // any shape's grid holds these
  const Mxfp4Shape p = shape_of(g);
  return p.tiles <= kMostThreads / p.threads;
}

hipError_t launch_mxfp4_gemm(const Mxfp4Gemm& g, hipStream_t s) {
  const Mxfp4Shape p = shape_of(g);
  auto few = [&]<int MT, int NT, int S>() {
    constexpr int W = MT * NT < 8 ? 8 : 4;
    hipLaunchKernelGGL((k_mxfp4_stream<MT, NT, W, S>), dim3((unsigned)p.tiles), dim3(64 * W), 0, s, g,
                       (g.N + 16 * NT - 1) / (16 * NT));
    return hipGetLastError();
  };
  auto tile = [&]<int BM, int BN, int WM>() {
    hipLaunchKernelGGL((k_mxfp4_tile<BM, BN, WM>), dim3((unsigned)p.tiles), dim3((BM / WM) * (BN / 64) * 64), 0, s, g);
    return hipGetLastError();
  };
  if (p.kernel == Mxfp4Shape::STREAM) {
    switch (p.bm / 16 * 8 + p.bn / 16) {
      case 9: return few.template operator()<1, 1, 2>();
      case 10: return few.template operator()<1, 2, 2>();
      case 12: return few.template operator()<1, 4, 2>();
      case 17: return few.template operator()<2, 1, 2>();
      case 18: return few.template operator()<2, 2, 2>();
      case 20: return few.template operator()<2, 4, 2>();
      case 33: return few.template operator()<4, 1, 2>();
      case 34: return few.template operator()<4, 2, 2>();
      default: return few.template operator()<4, 4, 2>();
    }
  }
  if (p.kernel == Mxfp4Shape::WIDE) {
    const unsigned n = (unsigned)p.tiles, cus = (unsigned)device_cu_count();
    // (K in whole pairs of slabs: chained tiles, one workgroup a CU)
    if (g.K % 512) hipLaunchKernelGGL(k_mxfp4_wide<false>, dim3(n), dim3(256), 0, s, g, n);
    else hipLaunchKernelGGL(k_mxfp4_wide<true>, dim3(n < cus ? n : cus), dim3(256), 0, s, g, n);
    return hipGetLastError();
  }
  if (p.bm == 256) return tile.template operator()<256, 128, 64>();
  if (p.bm == 128) return tile.template operator()<128, 128, 64>();
  return tile.template operator()<64, 64, 64>();
}

}  // namespace sparq24
