// Paged 8-bit key/value cache: append of new token rows, and attention of
// query rows over the cached tokens.  Layout and conventions: kv_common.hpp.
#include "kv_split.hpp"

namespace sparq24 {

// ---------------------------------------------------------------------------
// Append.  One workgroup per touched block, kv head and side (K, V).  With
// amax the absolute maximum of the block's new elements (the finite ones, so that an
// infinite element costs the block's other tokens nothing):
//   cand = amax < 2^-64 ? 0 : fp32(amax / qmax)
//   s    = the block begins with a new token ? cand : max(s_old, cand)
//   code = encode(fp32(x * fp32(1 / s)));  infinities saturate, NaN is coded as 0
// and where s > s_old the codes before the new ones become
//   encode(fp32(code * fp32(s_old * fp32(1 / s)))).
// Codes behind the new ones stay as they are.
//
// A thread takes 4 tokens x 8 dims at a time (16-byte loads, 8 dims of a row for
// adjacent lanes' neighbours), so that both layouts are written from packed
// dwords: K rows directly, V through LDS as [D][T] rows in 16-byte stores.  Where
// the new rows of a block fit one round of the workgroup (T * D <= 8192) they are
// read once and held; larger blocks read them again for the codes, from L2.
// Bound by HBM for prompts, by latency for single tokens.
// ---------------------------------------------------------------------------
template <bool FP8>
__device__ inline float kv_clamp(float y) {
  constexpr float q = FP8 ? 448.0f : 127.0f;
  return y == y ? __builtin_amdgcn_fmed3f(y, -q, q) : 0.0f;
}
// Codes of four fp32 values in code units, packed little-endian.
template <bool FP8>
__device__ inline uint32_t kv_encode4(float a, float b, float c, float d) {
  a = kv_clamp<FP8>(a);
  b = kv_clamp<FP8>(b);
  c = kv_clamp<FP8>(c);
  d = kv_clamp<FP8>(d);
  if constexpr (FP8) return enc_e4m3_x4(a, b, c, d);
  const uint32_t lo = __builtin_amdgcn_perm(__float_as_uint(b + kRoundMagic), __float_as_uint(a + kRoundMagic), 0x0c0c0400u);
  const uint32_t hi = __builtin_amdgcn_perm(__float_as_uint(d + kRoundMagic), __float_as_uint(c + kRoundMagic), 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
template <bool FP8>
__device__ inline float kv_decode(uint32_t c) {
  if constexpr (FP8) return dec_e4m3(c);
  else return (float)(int8_t)c;
}

template <class DT, bool FP8>
__global__ __launch_bounds__(kBlock) void k_kv_append(KvCache c, KvSeqs q, KvRows kr, KvRows vr) {
  extern __shared__ __attribute__((aligned(16))) uint8_t tile[];  // V: codes [D][T + 16]
  __shared__ float red[kBlock / 64];
  const int tid = threadIdx.x, lane = tid & 63;
  const int T = 1 << c.tsh, D = c.dim;
  // Block number j of sequence b.  Without offsets each has as many slots as its
  // rows may touch blocks; with them sequence b has those from cu[b] / T + 2 b on
  // (n rows touch at most n / T + 2 blocks), so that no lengths are needed to find it.
  int b, j;
  if (q.cu) {
    const int64_t u = blockIdx.x;
    auto slot = [&](int i) -> int64_t {
      const int at = q.cu[i];
      return (at < 0 ? 0 : (at > q.total ? q.total : at) >> c.tsh) + 2 * (int64_t)i;
    };
    b = last_reached((int)q.seqs, lane, [&](int i) { return slot(i) <= u; });
    j = (int)(u - slot(b));
  } else {
    b = (int)(blockIdx.x / (unsigned)q.slots);
    j = (int)(blockIdx.x % (unsigned)q.slots);
  }
  const SeqRows r = seq_rows(q, b);
  const int p0 = r.len > r.n ? r.len - r.n : 0;
  const int64_t cend = r.len < q.cap ? r.len : q.cap;
  if (r.n <= 0 || p0 >= cend || j < 0 || j > ((cend - 1) >> c.tsh) - (p0 >> c.tsh)) return;
  const int64_t page = (p0 >> c.tsh) + j;
  const int64_t blk = q.table[b * q.table_stride + page];
  if (blk < 0 || blk >= c.blocks) return;
  const int64_t base = page << c.tsh;
  const int o0 = base < p0 ? (int)(p0 - base) : 0;
  const int o1 = cend - base < T ? (int)(cend - base) : T;  // new codes: rows o0 .. o1 - 1
  const int head = blockIdx.y;
  const bool side_v = blockIdx.z != 0;
  const KvRows rows = side_v ? vr : kr;
  // row of the block's row o: position base + o is new token base + o - (len - n)
  const int64_t row0 = r.first + (base - ((int64_t)r.len - r.n));
  const char* x = rows.x + row0 * rows.ts + head * rows.hs;
  float* sp = (side_v ? c.vs : c.ks) + blk * c.heads + head;
  const float old = o0 ? *sp : 0.0f;
  uint8_t* codes = (side_v ? c.v : c.k) + (blk * c.heads + head) * (int64_t)T * D;

  // quad i: tokens 4 g .. 4 g + 3 (those outside o0 .. o1 - 1 left out), dims 8 d ..
  const unsigned upr = D / 8, g0 = o0 >> 2, quads = (((o1 + 3) >> 2) - g0) * upr;
  const int pitch = T + 16;
  auto load = [&](unsigned i, Unit<DT>(&u)[4]) {
    const int o = 4 * (g0 + i / upr), d = 8 * (i % upr);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (o + e >= o0 && o + e < o1) load_unit(u[e], x + (int64_t)(o + e) * rows.ts + d * DT::ESIZE);
      else zero_unit(u[e]);
    }
  };
  float am = 0.0f;
  auto widest = [&](const Unit<DT>(&u)[4], bool finite) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int f = 0; f < 8; ++f) {
        const float x = __builtin_fabsf(u[e].f(f));
        am = __builtin_fmaxf(am, finite && x == __builtin_inff() ? 0.0f : x);
      }
  };
  auto store = [&](unsigned i, const Unit<DT>(&u)[4], float inv) {
    const int o = 4 * (g0 + i / upr), d = 8 * (i % upr);
    if (side_v) {
#pragma unroll
      for (int f = 0; f < 8; ++f)
        *(uint32_t*)(tile + (d + f) * pitch + o) =
            kv_encode4<FP8>(u[0].f(f) * inv, u[1].f(f) * inv, u[2].f(f) * inv, u[3].f(f) * inv);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint2 w;
        w.x = kv_encode4<FP8>(u[e].f(0) * inv, u[e].f(1) * inv, u[e].f(2) * inv, u[e].f(3) * inv);
        w.y = kv_encode4<FP8>(u[e].f(4) * inv, u[e].f(5) * inv, u[e].f(6) * inv, u[e].f(7) * inv);
        if (o + e >= o0 && o + e < o1) *(uint2*)(codes + (o + e) * D + d) = w;
      }
    }
  };
  Unit<DT> held[4];
  const bool once = quads <= kBlock;
  auto meet = [&] {  // am over the workgroup
    am = __uint_as_float(wave_max_u32<64>(__float_as_uint(am)));
    if (lane == 0) red[tid >> 6] = am;
    __syncthreads();  // (every thread has read the old scale, too)
#pragma unroll
    for (int i = 0; i < kBlock / 64; ++i) am = __builtin_fmaxf(am, red[i]);
  };
  if (once) {
    if (tid < (int)quads) {
      load(tid, held);
      widest(held, false);
    }
  } else {
    for (unsigned i = tid; i < quads; i += kBlock) {
      load(i, held);
      widest(held, false);
    }
  }
  meet();
  if (am == __builtin_inff()) {  // once more, without the infinities
    __syncthreads();             // red has been read
    am = 0.0f;
    if (once) {
      if (tid < (int)quads) widest(held, true);
    } else {
      for (unsigned i = tid; i < quads; i += kBlock) {
        load(i, held);
        widest(held, true);
      }
    }
    meet();
  }

  const float cand = am >= 0x1p-64f ? am / (FP8 ? 448.0f : 127.0f) : 0.0f;
  const float s = cand > old ? cand : old;
  const float inv = s > 0.0f ? 1.0f / s : 0.0f;
  if (tid == 0) *sp = s;
  if (o0 && s > old) {  // code what the block held again, to the grown scale
    const float ratio = old * inv;
    for (int i = tid; i < D * o0; i += kBlock) {
      uint8_t* p = side_v ? codes + (i / o0) * T + i % o0 : codes + i;
      *p = (uint8_t)kv_encode4<FP8>(kv_decode<FP8>(*p) * ratio, 0.f, 0.f, 0.f);
    }
  }
  if (once) {
    if (tid < (int)quads) store(tid, held, inv);
  } else {
    for (unsigned i = tid; i < quads; i += kBlock) {
      load(i, held);
      store(i, held, inv);
    }
  }
  if (!side_v) return;
  __syncthreads();
  // 16-byte chunks that the new rows cover whole, bytes at the ragged ends
  const int q0 = o0 >> 4, nq = ((o1 + 15) >> 4) - q0;
  for (int i = tid; i < D * nq; i += kBlock) {
    const int d = i / nq, t = (q0 + i % nq) * 16;
    const uint8_t* from = tile + d * pitch + t;
    uint8_t* to = codes + d * T + t;
    if (t >= o0 && t + 16 <= o1) {
      *(uint4*)to = *(const uint4*)from;
    } else {
      for (int e = t < o0 ? o0 - t : 0; e < (t + 16 < o1 ? 16 : o1 - t); ++e) to[e] = from[e];
    }
  }
}

namespace {
int64_t append_blocks(const KvCache& c, const KvSeqs& q) {
  return q.cu ? (q.total >> c.tsh) + 2 * q.seqs : q.seqs * q.slots;
}
}  // namespace

bool kv_append_fits(const KvCache& c, const KvSeqs& q) { return append_blocks(c, q) <= kMostThreads / kBlock; }

hipError_t launch_kv_append(const KvCache& c, const KvSeqs& q, const KvRows& k, const KvRows& v,
                            int dtype, hipStream_t s) {
  const int64_t T = 1ll << c.tsh;
  const int64_t most = append_blocks(c, q);
  const size_t shmem = (size_t)c.dim * (size_t)(T + 16);
  const dim3 grid((unsigned)most, (unsigned)c.heads, 2);
  return with_dtype(dtype, [&]<class DT>() {
    auto go = [&](auto kern) {
      if (shmem > 65536) {
        const hipError_t e = hipFuncSetAttribute((const void*)kern,
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, (int)shmem);
        if (e != hipSuccess) return e;
      }
      hipLaunchKernelGGL(kern, grid, dim3(kBlock), shmem, s, c, q, k, v);
      return hipGetLastError();
    };
    return c.fp8 ? go(k_kv_append<DT, true>) : go(k_kv_append<DT, false>);
  });
}

// ---------------------------------------------------------------------------
// Attention.  For query row i of sequence b at position pos = len - n + i and
// kv head j = h / g (g query heads per kv head), over the visible tokens t:
//   s_t = scale * ks[blk(t)] * (q . kcode_t),  p_t = exp(s_t),
//   o = (sum_t p_t vs[blk(t)] vcode_t) / (sum_t p_t).
// Both products run on v_mfma_f32_16x16x32_f16 with the codes widened exactly
// to fp16.  Transposed throughout, so that no operand is rearranged:
//   S^T [token][row] = K Q^T    lane: row c = lane % 16, tokens 4 h + i
//   O^T [dim][row]   = V^T P^T  lane: row c, dims 4 h + i  (h = lane / 16)
// A tile is 64 tokens.  Rows of the four 16-token MFMA tiles are dealt so that
// lane group h gets the scores of tokens 16h .. 16h + 15, which are exactly
// the k slots in which it supplies P^T, and one 16-byte run of a V row.
// The block scales ride on the exponent: with w_t = p_t vs, w = exp2(s_t log2e
// + log2 vs - m) feeds the second product, and the sum of p_t is the sum of
// w / vs, so neither scale costs an instruction per score and w stays in
// fp16's range whatever the scales are.  The sum is kept over 2^n, n near the
// largest score, since a token of small values counts in it as much as any; m - n is
// a whole number, so that 2^(m - n) is exact.  (Were m itself one, the largest weight
// would not be 2^8 and lose by its rounding to fp16: errors of peaked rows 2^-12 more.)
// Where a V scale is 2^28 and more below the one that set m, w could leave fp32's range
// (2^-126) with a p_t that counts: there the sum comes from the scores themselves.
// A query row is multiplied by a power of two that puts its largest element at 2^13:
// fp16 then holds every bf16 or fp16 element down to 2^-27 of it in full and rounds
// smaller ones to 2^-38 of it, so a score is off by at most scale 2^-38 max |q| sum |K_t|.
// Scores, m, sums and O are fp32; w is rounded to fp16 (relative 2^-11, below bf16's
// own rounding and at fp16's).
// ---------------------------------------------------------------------------
// Eight codes (two dwords) as fp16, exactly.
template <bool FP8>
__device__ inline f16x8_t widen8(uint32_t a, uint32_t b) {
  f16x2_t r[4];
  if constexpr (FP8) {
    r[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, false);
    r[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(a, 1.0f, true);
    r[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, false);
    r[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(b, 1.0f, true);
  } else {
    // 0x6400 | (code + 128) is the fp16 number 1024 + 128 + code
    const f16x2_t off = {(_Float16)1152.0f, (_Float16)1152.0f};
    const uint32_t ua = a ^ 0x80808080u, ub = b ^ 0x80808080u;
    r[0] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, ua, 0x04010400u)) - off;
    r[1] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, ua, 0x04030402u)) - off;
    r[2] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, ub, 0x04010400u)) - off;
    r[3] = __builtin_bit_cast(f16x2_t, __builtin_amdgcn_perm(0x64646464u, ub, 0x04030402u)) - off;
  }
  return f16x8_t{r[0].x, r[0].y, r[1].x, r[1].y, r[2].x, r[2].y, r[3].x, r[3].y};
}

constexpr float kTopSet = 8.0f;    // a new reference puts the largest w at 2^8 ...
constexpr float kTopMost = 15.0f;  // ... and stands until one would pass 2^15
// One fma from score to exponent rounds m, not the exponent: the same factor for
// every token, harmless until the rounding itself is large.  From here on every
// tile takes the exponent as the difference of the rounded terms, so that the
// largest stays in range.
constexpr float kFarTop = 65536.0f;
// Most that a weight is multiplied by for the sum: so a p_t passes 2^n by 2^35 at most,
// and one that is lost (w < 2^-126) is below 2^-106 of it.
constexpr float kMostFactor = 0x1p20f;

// Query row r of the row tile (column c of the MFMA tiles), in fp16 times a power
// of two: elements d(j) .. d(j) + 7 of lane group h into qf[j].
struct KvRow {
  float c;       // scale * log2 e / that power of two
  int lim, low;  // last and first position seen (lim -1: no row)
};
template <int NJ, class F>
__device__ inline KvRow kv_query(const KvAttnArgs& p, const KvItem& it, int r, f16x8_t (&qf)[NJ], F&& d) {
  const KvAttn& a = p.a;
  const bool valid = r < it.k.rows;
  const int i = valid ? r / p.g : 0, hq = valid ? it.head * p.g + r % p.g : 0;
  const int pos = it.r.len - it.r.n + i;
  const int hi_all = (int)(it.r.len < a.q.cap ? it.r.len : a.q.cap);
  KvRow row;
  row.lim = !valid ? -1 : (a.causal && pos + 1 < hi_all ? pos + 1 : hi_all) - 1;
  row.low = first_seen(pos, a.window);
  const char* x = a.x + (it.r.first + (int64_t)i) * a.ts + hq * a.hs;
  u32x4v raw[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) raw[j] = *(const u32x4v*)(x + 2 * d(j));
  float am = 0.0f;
  auto at = [&](int j, int e) {
    const uint32_t v = (raw[j][e / 2] >> (16 * (e & 1))) & 0xFFFFu;
    return a.dtype == 1 ? BF16T::to_f32(v) : F16T::to_f32(v);
  };
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) am = __builtin_fmaxf(am, __builtin_fabsf(at(j, e)));
  am = groups_max(am);
  int ex = (int)(__float_as_uint(am) >> 23);  // 0: zero or subnormal, 255: inf
  // an infinite element makes every score infinite or NaN, and the softmax NaN
  const bool inf = ex > 254;
  ex = ex < 64 ? 64 : (inf ? 127 : ex);
  const float up = inf ? __builtin_nanf("") : __uint_as_float((uint32_t)(127 + 13 - (ex - 127)) << 23);
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) qf[j][e] = (_Float16)(at(j, e) * up);
  row.c = a.scale * 1.44269504088896340736f * __uint_as_float((uint32_t)(127 - 13 + (ex - 127)) << 23);
  return row;
}

// Block scales of the 16 tokens of a lane group.  A zero scale counts as 2^-80:
// its codes are zeros.  A scale that is no finite number makes every score of its
// tokens NaN, before the masks, so that it reaches the rows that see them only.
struct KvScales {
  bool there, fine;
  float ks, lv, rv;  // K scale, log2 and reciprocal of V's
};
__device__ inline KvScales kv_scales(bool there, float ks, float vs) {
  KvScales k;
  const float vse = vs < 0x1p-80f ? 0x1p-80f : vs;
  const bool fine = there && __builtin_isfinite(ks + vs);
  k.there = there;
  k.fine = fine;
  k.ks = ks;
  k.lv = fine ? __builtin_amdgcn_logf(vse) : 0.0f;
  k.rv = fine ? __builtin_amdgcn_rcpf(vse) : 1.0f;
  return k;
}

// State of a wave's rows over the tiles.
template <int QT, int NU>
struct KvState {
  float m[QT], e[QT], l[QT];  // reference of O (log2), 2^(m - n), sum of this lane group's tokens over 2^n
  f32x4v o[QT][NU];
  int far;                    // some row's reference is past kFarTop
  __device__ inline void init() {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      m[t] = kNegInf;
      e[t] = 1.0f;
      l[t] = 0.0f;
#pragma unroll
      for (int u = 0; u < NU; ++u) o[t][u] = f32x4v{0.f, 0.f, 0.f, 0.f};
    }
    far = 0;
  }
};
// log2 of a power of two, exactly.
__device__ inline float log2_exact(float e) { return (float)((int)(__float_as_uint(e) >> 23) - 127); }

// Where a factor of the weights for the sum has grown past kMostFactor: the sums'
// references rise to the largest scores, and if a V scale is still so far below,
// the tile's part of the sums comes straight from the scores.  was, up: e and m have
// been raised from e = was by 2^up (which may have left e's range).
template <int QT, int NU>
__device__ inline void kv_sum_reference(const f32x4v (&sc)[QT][4], const float (&ck)[QT], const float (&mx)[QT],
                                        float rv, const float (&was)[QT], const float (&up)[QT], KvState<QT, NU>& st,
                                        float (&f)[QT]) {
  bool apart = false;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float best = groups_max(mx[t] * ck[t]);
    const float d = log2_exact(was[t]) + up[t];                       // m - n
    float nd = __builtin_fminf(d, __builtin_rintf(st.m[t] - best));  // NaN (both infinite): as it was
    nd = __builtin_amdgcn_fmed3f(nd, -126.0f, 126.0f);
    if (st.m[t] != kNegInf) {
      st.l[t] *= __builtin_amdgcn_exp2f(nd - d);
      st.e[t] = __builtin_amdgcn_ldexpf(1.0f, (int)nd);
      f[t] = st.e[t] * rv;
    }
    apart |= f[t] > kMostFactor;
  }
  if (__any(apart)) {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const float ref = st.m[t] == kNegInf ? 0.0f : st.m[t], d = log2_exact(st.e[t]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float x = st.far ? sc[t][mt][e] * ck[t] - ref : __builtin_fmaf(sc[t][mt][e], ck[t], -ref);
          st.l[t] += __builtin_amdgcn_exp2f(x + d);
        }
      f[t] = 0.0f;
    }
  }
}

// Scores of a tile (lane: QT rows, tokens tok0 .. tok0 + 15) to weights: masks
// (where `edge`: a mask or a bad scale), the rows' references, sums (fp32: a token of a
// small V scale can have a weight that fp16 does not hold and still be most of the
// sum) and the rescaling of O.  (Taking the weights first and forming the maxima only where
// one passed 2^15 costs more than it saves as soon as scores spread: 8192 tokens took
// 1.23 times as long, the maxima of 16 rows grow in most tiles.)
template <int QT, int NU>
__device__ inline void kv_weights(f32x4v (&sc)[QT][4], const KvRow (&row)[QT], const KvScales& k, int tok0,
                                  bool edge, KvState<QT, NU>& st, f16x8_t (&pf)[QT][2]) {
  float ck[QT], mx[QT], top[QT], f[QT];  // f: factor of the weights for the sum
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    ck[t] = k.fine ? row[t].c * k.ks : 1.0f;
    ck[t] = ck[t] < 0x1p-120f ? 0x1p-120f : ck[t];
  }
  if (edge) {
    if (__any(k.there && !k.fine)) {
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) sc[t][mt] += k.there && !k.fine ? __builtin_nanf("") : 0.0f;
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      // tokens tok0 + x with first <= x <= last
      const int first = k.there ? row[t].low - tok0 : 16, last = row[t].lim - tok0;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 4 * mt + e;
          sc[t][mt][e] = x > last || x < first ? kNegInf : sc[t][mt][e];
        }
    }
  }
  bool turn = false;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    mx[t] = kNegInf;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[t] = __builtin_fmaxf(mx[t], sc[t][mt][e]);
    f[t] = st.e[t] * k.rv;
    top[t] = groups_max(__builtin_fmaf(mx[t], ck[t], k.lv));
    turn |= top[t] - st.m[t] > kTopMost;  // -inf - -inf is NaN: no new reference
    turn |= f[t] > kMostFactor;
  }
  if (__any(turn)) {
    float was[QT], up[QT];
    bool apart = false;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const bool g = top[t] - st.m[t] > kTopMost;
      float nm = top[t] - kTopSet;
      nm = top[t] - nm > kTopMost ? top[t] : nm;  // where scores have steps of 16, top - 8 may round to top - 16
      const float by = g ? nm - st.m[t] : 0.0f;
      up[t] = __builtin_rintf(by);
      was[t] = st.e[t];
      const float al = __builtin_amdgcn_exp2f(-by);
      st.l[t] *= by < __builtin_inff() ? __builtin_amdgcn_exp2f(up[t] - by) : 1.0f;  // n has m's fraction
      st.m[t] = g ? nm : st.m[t];
      st.e[t] = __builtin_amdgcn_ldexpf(st.e[t], (int)up[t]);  // infinite at the first reference
      st.far |= uniform((int)__any(__builtin_fabsf(st.m[t]) > kFarTop && st.m[t] != kNegInf));
#pragma unroll
      for (int u = 0; u < NU; ++u) st.o[t][u] *= al;
      f[t] = st.e[t] * k.rv;
      apart |= f[t] > kMostFactor;
    }
    if (__any(apart)) kv_sum_reference(sc, ck, mx, k.rv, was, up, st, f);
  }
  if (st.far) {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const float ref = st.m[t] == kNegInf ? 0.0f : st.m[t];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][mt][e] = __builtin_fmaf(sc[t][mt][e], ck[t], k.lv) - ref;
    }
  } else {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const float off = k.lv - (st.m[t] == kNegInf ? 0.0f : st.m[t]);
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][mt][e] = __builtin_fmaf(sc[t][mt][e], ck[t], off);
    }
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float sum = 0.0f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float w = __builtin_amdgcn_exp2f(sc[t][mt][e]);
        sum += w;
        pf[t][mt / 2][4 * (mt & 1) + e] = (_Float16)w;
      }
    st.l[t] = __builtin_fmaf(sum, f[t], st.l[t]);
  }
}

// e4m3 only.  A V code can be NaN, and 0 * NaN carries it to rows that do not see it.
// Where O holds a NaN that its sum does not explain, kv_nan_pass forms O of the wave's 16
// rows again, with the references and sums that stand: codes that are NaN count as
// zeros, and a second product counts those that a row sees, whose elements of O are
// NaN then.  It takes the kernel's arguments and its item anew, hidden from the
// compiler: shared with the loops before, which hardly ever need it, they took
// registers from those (8192 e4m3 tokens 654 us, shared 686).
template <int QT, int NU>
__device__ inline bool kv_nan_values(const KvState<QT, NU>& st) {  // l: over the lane groups
  bool nan = false;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    bool some = false;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) some |= st.o[t][u][e] != st.o[t][u][e];
    nan |= some && st.l[t] == st.l[t];
  }
  return nan;
}
typedef __attribute__((address_space(3))) float lds_float_t;
typedef __attribute__((address_space(4))) const KvAttnArgs const_args_t;
// Row r (column c of the wave's tile) over tiles first, first + step, .. of its range;
// m: its reference.  To LDS: O of the row; else O times inv to its place.
template <int D>
__device__ inline __attribute__((always_inline)) void kv_nan_pass(int r, int first, int step, float m, int far,
                                                                  float inv, lds_float_t* lds) {
  constexpr int NJ = D / 32;
  auto args = (const_args_t*)__builtin_amdgcn_kernarg_segment_ptr();
  int id = (int)blockIdx.x;
  asm volatile("" : "+s"(args), "+s"(id));
  const KvAttnArgs& p = *(const KvAttnArgs*)args;
  const KvAttn& a = p.a;
  const int lane = __lane_id(), c16 = lane & 15, h = lane >> 4, T = 1 << a.c.tsh;
  KvItem it;
  if (!kv_item(p, id, lane, it)) return;
  f16x8_t qf[NJ];
  const KvRow row = kv_query(p, it, r, qf, [&](int j) { return 64 * (j / 2) + 16 * h + 8 * (j & 1); });
  const int hi = (int)(it.r.len < a.q.cap ? it.r.len : a.q.cap);
  const int* table = a.q.table + (int64_t)it.seq * a.q.table_stride;
  const float ref = m == kNegInf ? 0.0f : m;
  const int r0 = it.rt * p.rb, r1 = r0 + p.rb < it.k.rows ? r0 + p.rb : it.k.rows;
  const KvRange rg = kv_range(p, it, r0, r1);
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 64) {  // 64 dims at a time: few registers
    f32x4v o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) o[u] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int tt = rg.t0 + first; tt < rg.t1; tt += step) {
      // this lane's K rows are of the 16 tokens of lane group c16 / 4, its V codes of its own
      auto block = [&](int pos) -> int64_t {
        const int b = pos < hi ? table[pos >> a.c.tsh] : -1;
        return b >= 0 && b < a.c.blocks ? b : -1;
      };
      auto place = [&](int64_t b) { return (b < 0 ? 0 : b) * a.c.heads + it.head; };
      const int b0 = tt * kKvTile, kpos = b0 + 16 * (c16 >> 2), tok0 = b0 + 16 * h;
      const int64_t kb = block(kpos), vb = block(tok0);
      const uint8_t* kp = a.c.k + place(kb) * T * D + (int64_t)((kpos & (T - 1)) + (c16 & 3)) * D + 16 * h;
      const uint8_t* vp = a.c.v + place(vb) * T * D + (int64_t)(d0 + c16) * T + (tok0 & (T - 1));
      f32x4v sc[4];
#pragma unroll
      for (int mt = 0; mt < 4; ++mt) {
        sc[mt] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NJ; j += 2) {
          const u32x4v k = *(const u32x4v*)(kp + 4 * mt * D + 32 * j);
          sc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8<true>(k[0], k[1]), qf[j], sc[mt], 0, 0, 0);
          sc[mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8<true>(k[2], k[3]), qf[j + 1], sc[mt], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      const KvScales k = kv_scales(vb >= 0, a.c.ks[place(vb)], a.c.vs[place(vb)]);
      float ck = k.fine ? row.c * k.ks : 1.0f;
      ck = ck < 0x1p-120f ? 0x1p-120f : ck;
      f16x8_t pf[2], sees[2];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const bool seen = vb >= 0 && tok0 + x >= row.low && tok0 + x <= row.lim;
        const float s = sc[x / 4][x % 4];
        const float w = far ? __builtin_fmaf(s, ck, k.lv) - ref : __builtin_fmaf(s, ck, k.lv - ref);
        pf[x / 8][x % 8] = seen ? (_Float16)__builtin_amdgcn_exp2f(w) : (_Float16)0.0f;
        sees[x / 8][x % 8] = seen ? (_Float16)1.0f : (_Float16)0.0f;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const u32x4v c = *(const u32x4v*)(vp + 16 * u * T);
        f32x4v count = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          f16x8_t v = widen8<true>(c[2 * x], c[2 * x + 1]), none;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const bool nan = v[e] != v[e];
            none[e] = nan ? (_Float16)1.0f : (_Float16)0.0f;
            v[e] = nan ? (_Float16)0.0f : v[e];
          }
          o[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v, pf[x], o[u], 0, 0, 0);
          count = __builtin_amdgcn_mfma_f32_16x16x32_f16(none, sees[x], count, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) o[u][e] = count[e] > 0.0f ? __builtin_nanf("") : o[u][e];
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (lds) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) lds[d0 + 16 * u + 4 * h + e] = o[u][e];
    } else if (r < it.k.rows) {
      const int64_t tok = it.r.first + r / p.g, hq = it.head * p.g + r % p.g;
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int d = d0 + 16 * u + 4 * h + e;
          if (it.chunks > 1) p.po[(it.slot * p.rb + (r - it.rt * p.rb)) * D + d] = o[u][e] * inv;
          else kv_store_out(a, (tok * a.heads + hq) * D + d, o[u][e] * inv);
        }
    }
  }
}

// Few rows per kv head (decoding): one tile of 16 rows, four waves that take the
// chunk's tiles in turn, K and V straight from memory into MFMA operands.  Bound by
// the cache's bytes: 64 sequences of 300..16384 tokens, 32 heads over 8 of 128, in
// 208 us (5.3 TB/s; vector instructions take a third of the cycles), 4096 of 100 in
// 345 (half of their last blocks is empty).  Three waves per SIMD there: with two,
// short sequences took 1.3 times as long.
// BIG: blocks of 64 tokens and more, so a tile lies in one block (scalar addresses
// and scales).
template <int D, bool FP8, bool BIG>
__global__ __launch_bounds__(256, BIG && D <= 128 ? 3 : 1) void k_kv_attn(KvAttnArgs p) {
  constexpr int NS = D / 64, NU = D / 16;
  const KvAttn& a = p.a;
  const int lane = threadIdx.x & 63, wv = uniform((int)threadIdx.x >> 6), c16 = lane & 15, h = lane >> 4;
  KvItem it;
  if (!kv_item(p, blockIdx.x, lane, it)) return;
  const int H = a.c.heads, tsh = a.c.tsh, T = 1 << tsh;
  f16x8_t qf[2 * NS];
  const KvRow row[1] = {kv_query(p, it, it.rt * p.rb + c16, qf,
                                 [&](int j) { return 64 * (j / 2) + 16 * h + 8 * (j & 1); })};

  KvState<1, NU> st;
  st.init();

  const int r0 = it.rt * p.rb, r1 = r0 + 16 < it.k.rows ? r0 + 16 : it.k.rows;
  const KvRange rg = kv_range(p, it, r0, r1);
  const int lo = rg.lo, hi = rg.hi;
  const int* table = a.q.table + (int64_t)it.seq * a.q.table_stride;
  const int64_t bhead = (int64_t)T * D;

  // Block of a tile (BIG) or of this lane group's 16 tokens of it, or -1: what no row
  // sees (its scales may be anything) and what has no block reads block 0, masked.
  auto block_of = [&](int tt) -> int {
    const int gp = tt * kKvTile + (BIG ? 0 : 16 * h);
    int blk = tt < rg.t1 && gp < hi && gp + (BIG ? kKvTile : 16) > lo ? table[gp >> tsh] : -1;
    if (blk >= a.c.blocks) blk = -1;
    return BIG ? scalar(blk) : blk;
  };
  u32x4v kr[4][NS], vr[NU];
  float ks = 0.0f, vs = 0.0f;
  auto place = [&](int blk) -> int64_t { return (int64_t)(blk < 0 ? 0 : blk) * H + it.head; };
  const unsigned koff = (16 * (c16 >> 2) + (c16 & 3)) * D + 16 * h, voff = c16 * T + 16 * h;
  auto load_k = [&](int tt, int blk) {
    const uint8_t* kp;
    if constexpr (BIG) {
      kp = a.c.k + place(blk) * bhead + ((tt * kKvTile) & (T - 1)) * D + koff;
    } else {
      const int src = 16 * (c16 >> 2), krow = ((tt * kKvTile + src) & (T - 1)) + (c16 & 3);
      kp = a.c.k + place(__shfl(blk, src, 64)) * bhead + (int64_t)krow * D + 16 * h;
    }
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int s = 0; s < NS; ++s) kr[mt][s] = *(const u32x4v*)(kp + 4 * mt * D + 64 * s);
  };
  auto load_v = [&](int tt, int blk) {
    const uint8_t* vb = a.c.v + place(blk) * bhead;
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      if constexpr (BIG) vr[u] = *(const u32x4v*)(vb + ((tt * kKvTile) & (T - 1)) + 16 * T * u + voff);
      else vr[u] = *(const u32x4v*)(vb + (int64_t)(c16 + 16 * u) * T + ((tt * kKvTile + 16 * h) & (T - 1)));
    }
  };
  // K of the next tile is asked for as soon as this one's is used, V likewise, the
  // table entry a tile earlier: each load has a tile's work to arrive in.
  int tt = rg.t0 + wv, blk = -1, blk1 = -1;
  if (tt < rg.t1) {
    blk = block_of(tt);
    blk1 = block_of(tt + 4);
    load_k(tt, blk);
    ks = a.c.ks[place(blk)];
    vs = a.c.vs[place(blk)];
    load_v(tt, blk);
  }
  for (; tt < rg.t1; tt += 4) {
    const int b0 = tt * kKvTile, gp = b0 + 16 * h;
    const bool there = blk >= 0 && (!BIG || (gp < hi && gp + 16 > lo)), more = tt + 4 < rg.t1;
    f32x4v sc[1][4];
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) sc[0][mt] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        const f16x8_t k0 = widen8<FP8>(kr[mt][s][0], kr[mt][s][1]);
        const f16x8_t k1 = widen8<FP8>(kr[mt][s][2], kr[mt][s][3]);
        sc[0][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[2 * s], sc[0][mt], 0, 0, 0);
        sc[0][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[2 * s + 1], sc[0][mt], 0, 0, 0);
      }

    const KvScales kk = kv_scales(there, ks, vs);
    const bool edge = __any(!kk.fine) || b0 + kKvTile > rg.least || b0 < rg.from;
    int blk2 = -1;
    if (more) {
      load_k(tt + 4, blk1);
      ks = a.c.ks[place(blk1)];
      vs = a.c.vs[place(blk1)];
      blk2 = block_of(tt + 8);
    }
    f16x8_t pf[1][2];
    kv_weights<1, NU>(sc, row, kk, gp, edge, st, pf);
    if constexpr (FP8) {
      if (edge) {  // codes that nobody sees can be NaN: 0 * NaN must not reach O
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t keep = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = gp + 4 * q + e;
            if (there && tok < hi && tok >= lo) keep |= 0xFFu << (8 * e);
          }
#pragma unroll
          for (int u = 0; u < NU; ++u) vr[u][q] &= keep;
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NU; ++u) {
      const f16x8_t v0 = widen8<FP8>(vr[u][0], vr[u][1]), v1 = widen8<FP8>(vr[u][2], vr[u][3]);
      st.o[0][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[0][0], st.o[0][u], 0, 0, 0);
      st.o[0][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[0][1], st.o[0][u], 0, 0, 0);
    }
    if (more) load_v(tt + 4, blk1);
    blk = blk1;
    blk1 = blk2;
  }

  // the four waves' parts of each row meet in LDS, in wave order
  constexpr int PITCH = D + 4;
  __shared__ float os[4][16][PITCH];
  __shared__ __attribute__((aligned(16))) float mls[4][16][4];  // m, n, sum
  st.l[0] = groups_sum(st.l[0]);
  if (h == 0) *(f32x4v*)mls[wv][c16] = f32x4v{st.m[0], st.m[0] - log2_exact(st.e[0]), st.l[0], 0.0f};
#pragma unroll
  for (int u = 0; u < NU; ++u) *(f32x4v*)&os[wv][c16][16 * u + 4 * h] = st.o[0][u];
  if constexpr (FP8) {
    if (__builtin_expect(__any(kv_nan_values(st)), 0))
      kv_nan_pass<D>(it.rt * p.rb + c16, wv, 4, st.m[0], st.far, 0.0f, (lds_float_t*)os[wv][c16]);
  }
  __syncthreads();
  const int at = 4 * wv + h, sub = c16, g = scalar(p.g);  // (held over the loop, p.g's reciprocal is spilled)
  const int r = it.rt * p.rb + at;
  if (r < it.k.rows) {
    float top = kNegInf, most = kNegInf, f[4], sum = 0.0f;  // references of O and the sum
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      top = __builtin_fmaxf(top, mls[q][at][0]);
      most = __builtin_fmaxf(most, mls[q][at][1]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f[q] = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mls[q][at][0] - top);
      sum += mls[q][at][2] * (top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mls[q][at][1] - most));
    }
    const int64_t tok = it.r.first + r / g, hq = it.head * g + r % g;
    const bool split = it.chunks > 1;
    const float inv = sum == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(top - most) / sum;
    const int64_t base = split ? (it.slot * p.rb + at) * D : (tok * a.heads + hq) * D;
#pragma unroll
    for (int e = 0; e < D / 16; ++e) {
      const int d = sub + 16 * e;
      float v = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) v += os[q][at][d] * f[q];
      if (split) p.po[base + d] = v * inv;
      else kv_store_out(a, base + d, v * inv);
    }
    if (sub == 0) {
      if (split) {
        const f32x2v ml = {sum == sum ? most : -kNegInf, sum};  // NaN has the last word in the join
        *(f32x2v*)(p.ml + (it.slot * p.rb + at) * 2) = ml;
      } else if (a.lse) {
        a.lse[tok * a.heads + hq] = kv_lse(most, sum);
      }
    }
  }
}

// Many rows per kv head (prompts): the waves of a workgroup hold 16 QT rows each and
// share every tile, which is widened once into LDS as fp16 (K [64][D], V [D][64],
// 16-byte chunks XOR-swizzled by row), one tile ahead of its use, its codes loaded
// one tile ahead of that.  Bound by the matrix and vector units in turn: per tile,
// 16 rows and head of 128 a wave issues 32 MFMAs (512 cycles of its SIMD's matrix
// unit) and 184 other vector instructions (softmax, widening), and several waves per
// SIMD overlap the one's products with the other's softmax: by the counters the
// matrix units are busy for 33% of the cycles, vector instructions (the MFMAs' issue
// among them) take 62%.  A causal prompt of 8192 tokens, 32 heads over 8: 655 us (839
// Tflop/s; such MFMAs alone reach 1985).
//
// Shapes, 128 rows a workgroup each: as many waves as the registers of D allow, but
// for D = 64, whose products are short next to the reads of a tile, two row tiles a
// wave.  8192 tokens by themselves, 32 heads over 8 (16 over 8 above 128), int8 in
// blocks of 64: D = 64 478 us (one row tile, four waves per SIMD: 1.15 times that), 128
// 703 (two row tiles, two waves: 1.05), 192 635 and 256 703 (two row tiles, one wave:
// 1.25 and 1.54).
template <int D>
struct KvPromptShape {
  // 16-row tiles of a wave, waves of a workgroup, waves per SIMD (three with D = 64 in
  // blocks of 64 and more: e4m3 410 us, with two 485; smaller blocks lose more by the
  // registers that short chunks spill: a mixed batch 49.2 instead of 47.7)
  static constexpr int QT = D == 64 ? 2 : 1, NW = D == 64 ? 4 : 8, WAVES = D == 128 ? 4 : 2;
};

// BIG: blocks of 64 tokens and more, so a tile lies in one block (scalar addresses
// and scales).
template <int D, bool FP8, bool BIG>
__global__ __launch_bounds__(64 * KvPromptShape<D>::NW, D == 64 && BIG ? 3 : KvPromptShape<D>::WAVES)
    void k_kv_prompt(KvAttnArgs p) {
  constexpr int QT = KvPromptShape<D>::QT, NJ = D / 32, NU = D / 16, KC = D / 16;
  constexpr int NT = 64 * KvPromptShape<D>::NW, C = kKvTile * KC, NQ = 2 * C / NT;  // 16-code chunks of K and V
  static_assert(C % 64 == 0 && 2 * C % NT == 0, "a wave loads K chunks or V chunks at a time");
  constexpr int K_BYTES = kKvTile * D * 2, BUF = 2 * K_BYTES;
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * BUF];
  const KvAttn& a = p.a;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, h = lane >> 4;
  KvItem it;
  if (!kv_item(p, blockIdx.x, lane, it)) return;
  const int H = a.c.heads, tsh = a.c.tsh, T = 1 << tsh;

  const int w0 = it.rt * p.rb + 16 * QT * wv;  // this wave's first row
  f16x8_t qf[QT][NJ];
  KvRow row[QT];
#pragma unroll
  for (int t = 0; t < QT; ++t)
    row[t] = kv_query(p, it, w0 + 16 * t + c16, qf[t], [&](int j) { return 32 * j + 8 * h; });
  KvState<QT, NU> st;
  st.init();
  const int r0 = it.rt * p.rb, r1 = r0 + p.rb < it.k.rows ? r0 + p.rb : it.k.rows;
  const KvRange rg = kv_range(p, it, r0, r1);
  // what this wave's own rows see (none: rows past the end)
  const int w1 = w0 + 16 * QT < it.k.rows ? w0 + 16 * QT : it.k.rows;
  KvRange mine = rg;
  if (w0 < w1) mine = kv_range(p, it, w0, w1);
  else mine.hi = 0;

  const int* table = a.q.table + (int64_t)it.seq * a.q.table_stride;
  const int64_t bhead = (int64_t)T * D;
  // Block of a tile (BIG) or of lane group h's 16 tokens of it, or -1 where no row
  // sees them or there is none; its place among blocks and heads (0's if none).
  auto block_of = [&](int tt) -> int {
    const int gp = tt * kKvTile + (BIG ? 0 : 16 * h);
    if (tt >= rg.t1 || gp >= rg.hi || (!BIG && gp + 16 <= rg.lo)) return -1;
    const int b = table[gp >> tsh];
    return b >= 0 && b < a.c.blocks ? b : -1;
  };
  auto place = [&](int blk) -> int64_t { return (int64_t)(blk < 0 ? 0 : blk) * H + it.head; };
  // whether lane group g's tokens of a tile are there
  auto is_there = [&](int tt, int blk, int g) {
    const int gp = tt * kKvTile + 16 * g;
    return blk >= 0 && (!BIG || (gp < rg.hi && gp + 16 > rg.lo));
  };
  // A 16-byte LDS access takes lanes l .. l + 7 and l + 16 .. l + 23 (two lane groups)
  // at a time, from 16 slots of 16 bytes: the xor of a row's chunks is chosen so
  // that these sixteen lanes of a fragment read meet sixteen slots (rows c % 8 =
  // r % 4 + 4 (r / 16 % 2) of K two chunks apart or, where rows are odd multiples of
  // 128 bytes, in their own half; rows d % 8 of V in halves by d % 2).
  auto k_swizzle = [](int r) {
    return D % 128 == 0 ? 2 * ((r & 3) | ((r >> 2) & 4)) : ((r & 2) | ((r >> 2) & 4));
  };
  auto v_swizzle = [](int d) { return ((d >> 2) & 1) | ((d << 1) & 4); };
  // This lane's first fragments; the others lie at fixed distances, but for address
  // bits that the swizzle turns (KX).  One register each, and not one per chunk.
  constexpr unsigned KX = D % 128 == 0 ? 255 : 127;
  const int kr = 16 * (c16 >> 2) + (c16 & 3);
  const unsigned kat = kr * (2 * D) + (h ^ k_swizzle(kr)) * 16;
  const unsigned vat = K_BYTES + c16 * 128 + ((2 * h) ^ v_swizzle(c16)) * 16;
  // Chunk i = tid + NT q of a tile: of K for i < C (row i / KC, 16 elements), of V
  // above (dim (i - C) / 4, tokens 16 (i % 4)).
  u32x4v cr[NQ];
  auto is_k = [&](int q) { return C % NT == 0 ? q < C / NT : wv + NT / 64 * q < C / 64; };
  const int koff = tid * 16, voff = ((tid - C % NT) >> 2) * T + 16 * (tid & 3);
  auto fetch = [&](int tt, int blk) {
    if constexpr (BIG) {
      const int64_t safe = place(blk);
      const int o = (tt * kKvTile) & (T - 1);
      const uint8_t *kb = a.c.k + safe * bhead + o * D, *vb = a.c.v + safe * bhead + o;
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        if (is_k(q)) cr[q] = *(const u32x4v*)(kb + koff + q * (NT * 16));
        else cr[q] = *(const u32x4v*)(vb + voff + (q - C / NT) * (NT / 4) * T);
      }
    } else {
#pragma unroll
      for (int q = 0; q < NQ; ++q) {
        const int i = tid + NT * q;
        if (is_k(q)) {
          const int r = i / KC;
          const int64_t b = place(__shfl(blk, 16 * (r >> 4), 64));
          cr[q] = *(const u32x4v*)(a.c.k + b * bhead + (int64_t)(r & (T - 1)) * D + 16 * (i % KC));
        } else {
          const int64_t b = place(__shfl(blk, 16 * (tid & 3), 64));
          cr[q] = *(const u32x4v*)(a.c.v + b * bhead + (int64_t)((i - C) / 4) * T + ((16 * (tid & 3)) & (T - 1)));
        }
      }
    }
  };
  auto widen = [&](int tt, int blk, uint8_t* buf) {
    if constexpr (FP8) {  // codes that nobody sees can be NaN: 0 * NaN must not reach O
      const int tok = tt * kKvTile + 16 * (tid & 3);
      const bool none = BIG ? !is_there(tt, blk, tid & 3) : (bool)__shfl((int)(blk < 0), 16 * (tid & 3), 64);
      if (none || tok + 16 > rg.hi || tok < rg.lo) {
#pragma unroll
        for (int d = 0; d < 4; ++d) {
          uint32_t keep = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!none && tok + 4 * d + e < rg.hi && tok + 4 * d + e >= rg.lo) keep |= 0xFFu << (8 * e);
#pragma unroll
          for (int q = 0; q < NQ; ++q)
            if (!is_k(q)) cr[q][d] &= keep;
        }
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int i = tid + NT * q;
      const f16x8_t x0 = widen8<FP8>(cr[q][0], cr[q][1]), x1 = widen8<FP8>(cr[q][2], cr[q][3]);
      if (is_k(q)) {
        const int r = i / KC, c = 2 * (i % KC), z = k_swizzle(r);
        uint8_t* k = buf + r * (2 * D);
        *(f16x8_t*)(k + (c ^ z) * 16) = x0;
        *(f16x8_t*)(k + ((c + 1) ^ z) * 16) = x1;
      } else {
        const int d = (i - C) / 4, x = 2 * (tid & 3);
        uint8_t* v = buf + K_BYTES + d * 128;
        *(f16x8_t*)(v + (x ^ v_swizzle(d)) * 16) = x0;
        *(f16x8_t*)(v + ((x + 1) ^ v_swizzle(d)) * 16) = x1;
      }
    }
  };

  if (rg.t0 < rg.t1) {
    int blk = block_of(rg.t0), blk1 = block_of(rg.t0 + 1);
    fetch(rg.t0, blk);
    widen(rg.t0, blk, smem);
    float ks = a.c.ks[place(blk)], vs = a.c.vs[place(blk)];
    fetch(rg.t0 + 1, blk1);  // past the end: block 0, unused
    int blk2 = block_of(rg.t0 + 2);
    __syncthreads();
    for (int tt = rg.t0; tt < rg.t1; ++tt) {
      const unsigned buf = ((tt - rg.t0) & 1) * BUF;
      const int b0 = tt * kKvTile;
      const float ks1 = a.c.ks[place(blk1)], vs1 = a.c.vs[place(blk1)];
      if (b0 < mine.hi && b0 + kKvTile > mine.lo) {
        __builtin_amdgcn_s_setprio(1);
        f32x4v sc[QT][4];
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) sc[t][mt] = f32x4v{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int mt = 0; mt < 4; ++mt) {
            // row r = 16 (c16 / 4) + 4 mt + c16 % 4, chunk 4 j + h
            const f16x8_t kf = *(const f16x8_t*)(smem + ((buf + kat) ^ (64 * j & KX)) + (64 * j & ~KX) + mt * (8 * D));
#pragma unroll
            for (int t = 0; t < QT; ++t)
              sc[t][mt] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qf[t][j], sc[t][mt], 0, 0, 0);
          }
        __builtin_amdgcn_s_setprio(0);
        const bool there = is_there(tt, blk, h);
        const KvScales kk = kv_scales(there, ks, vs);
        const bool edge = __any(!kk.fine) || b0 + kKvTile > mine.least || b0 < mine.from;
        f16x8_t pf[QT][2];
        kv_weights<QT, NU>(sc, row, kk, b0 + 16 * h, edge, st, pf);
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            // dim 16 u + c16, chunk 2 h + x
            const f16x8_t vf = *(const f16x8_t*)(smem + ((buf + vat) ^ (16 * x)) + u * 2048);
#pragma unroll
            for (int t = 0; t < QT; ++t)
              st.o[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pf[t][x], st.o[t][u], 0, 0, 0);
          }
        __builtin_amdgcn_s_setprio(0);
      }
      if (tt + 1 < rg.t1) {
        widen(tt + 1, blk1, smem + ((tt + 1 - rg.t0) & 1) * BUF);
        fetch(tt + 2, blk2);
        blk = blk1;
        blk1 = blk2;
        blk2 = block_of(tt + 3);
        ks = ks1;
        vs = vs1;
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) st.l[t] = groups_sum(st.l[t]);
  const bool again = FP8 && __any(kv_nan_values(st));  // (the queries may lie where the output goes)
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const int r = w0 + 16 * t + c16;
    if (r >= it.k.rows) continue;
    const int64_t tok = it.r.first + r / p.g, hq = it.head * p.g + r % p.g;
    const float inv = st.l[t] == 0.0f ? 0.0f : st.e[t] / st.l[t], most = st.m[t] - log2_exact(st.e[t]);
    if (it.chunks > 1) {
      const int64_t at = it.slot * p.rb + (r - r0);
      if (!again) {
#pragma unroll
        for (int u = 0; u < NU; ++u) *(f32x4v*)(p.po + at * D + 16 * u + 4 * h) = st.o[t][u] * inv;
      }
      const f32x2v ml = {st.l[t] == st.l[t] ? most : -kNegInf, st.l[t]};  // NaN has the last word in the join
      if (h == 0) *(f32x2v*)(p.ml + at * 2) = ml;
    } else {
      const int64_t at = (tok * a.heads + hq) * D;
      if (!again) {
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) kv_store_out(a, at + 16 * u + 4 * h + e, st.o[t][u][e] * inv);
      }
      if (a.lse && h == 0) a.lse[tok * a.heads + hq] = kv_lse(most, st.l[t]);
    }
  }
  if constexpr (FP8) {
    if (__builtin_expect(again, 0)) {
#pragma unroll
      for (int t = 0; t < QT; ++t)
        kv_nan_pass<D>(w0 + 16 * t + c16, 0, 1, st.m[t], st.far, st.l[t] == 0.0f ? 0.0f : st.e[t] / st.l[t],
                       nullptr);
    }
  }
}

namespace {
// Row shapes of the prompt kernel by head dim (KvPromptShape).
template <int D>
constexpr int kPromptRows = 16 * KvPromptShape<D>::QT * KvPromptShape<D>::NW;
int prompt_rows(int dim) {
  return dim == 64 ? kPromptRows<64> : dim == 128 ? kPromptRows<128> : dim == 192 ? kPromptRows<192> : kPromptRows<256>;
}

KvPlan plan_of(const KvAttn& a, void* ws) {
  return kv_plan(a, (char*)ws, 16, prompt_rows(a.c.dim), a.c.dim <= 128 ? 2 : 1);
}

}  // namespace

bool kv_attn_fits(const KvAttn& a) {
  return kv_plan_fits(a, plan_of(a, nullptr),
                      a.c.dim == 64 ? 64 * KvPromptShape<64>::NW : 64 * KvPromptShape<128>::NW);
}

size_t kv_attn_workspace(const KvAttn& a) { return plan_of(a, nullptr).need; }

hipError_t launch_kv_attn(const KvAttn& a, void* ws, hipStream_t s) {
  const KvPlan p = plan_of(a, ws);
  if (p.planned) {
    const hipError_t e = launch_kv_starts(p, s);
    if (e != hipSuccess) return e;
  }
  auto dim = [&]<int D>() {
    if (p.run_many) {
      auto k = a.c.tsh >= 6 ? (a.c.fp8 ? k_kv_prompt<D, true, true> : k_kv_prompt<D, false, true>)
                            : (a.c.fp8 ? k_kv_prompt<D, true, false> : k_kv_prompt<D, false, false>);
      hipLaunchKernelGGL(k, dim3((unsigned)p.many.items), dim3(64 * KvPromptShape<D>::NW), 0, s, p.many);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (p.run_few) {
      auto k = a.c.tsh >= 6 ? (a.c.fp8 ? k_kv_attn<D, true, true> : k_kv_attn<D, false, true>)
                            : (a.c.fp8 ? k_kv_attn<D, true, false> : k_kv_attn<D, false, false>);
      hipLaunchKernelGGL(k, dim3((unsigned)p.few.items), dim3(256), 0, s, p.few);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    return p.split ? launch_kv_join(p, s) : hipSuccess;
  };
  switch (a.c.dim) {
    case 64: return dim.template operator()<64>();
    case 128: return dim.template operator()<128>();
    case 192: return dim.template operator()<192>();
    case 256: return dim.template operator()<256>();
    default: return hipErrorInvalidValue;
  }
}

}  // namespace sparq24
