// Paged 4-bit key/value cache (MXFP4 along the head dim): append of new token rows,
// and attention of query rows over the cached tokens.  Layout: kv_common.hpp.
#include "kv_split.hpp"

namespace sparq24 {

// ---------------------------------------------------------------------------
// Append.  A wave takes whole tokens, a lane 8 dims of one head at a time, four lanes
// a group of 32 dims: amax over its finite elements, the exponent byte of
// mx_exponent, E2M1 codes.  A token's codes depend on it alone, so nothing is read
// back from the cache.  One token on 64 sequences, 8 heads of 128: 4.3 us, the launch and
// loads that depend on each other (length, block); 256 tokens 25.9, 3.3 TB/s, 4096 on 16
// sequences 83, 4.1 TB/s: vector instructions and single bytes of scales beside the rows.
// ---------------------------------------------------------------------------
template <class DT>
__global__ __launch_bounds__(kBlock) void k_kv4_append(KvCache c, KvSeqs q, KvRows kr, KvRows vr, int tokens) {
  const int lane = threadIdx.x & 63;
  const int64_t wave = (int64_t)blockIdx.x * (kBlock / 64) + (threadIdx.x >> 6);
  const int64_t tok0 = wave * tokens;
  if (tok0 >= q.total) return;
  const int upr = c.dim / 8, units = c.heads * upr;  // of a token
  const int all = (int)((q.total - tok0 < tokens ? q.total - tok0 : tokens) * units);
  const int b0 = q.cu ? last_reached((int)q.seqs, lane, [&](int i) { return q.cu[i] <= tok0; }) : 0;
  const int T = 1 << c.tsh;
  // The block that a token goes to (-1: none) and its place there.
  struct Spot {
    int64_t blk;
    int o;
  };
  auto spot = [&](int64_t tok) {
    int64_t b = b0;
    if (q.cu) {
      while (b + 1 < q.seqs && q.cu[b + 1] <= tok) ++b;
    } else {
      b = (uint32_t)tok / (uint32_t)q.nper;  // (both fit: there are at most 2^31 - 1 tokens)
    }
    const SeqRows r = seq_rows(q, b);
    const int64_t pos = (int64_t)r.len - r.n + (tok - r.first);
    const bool mine = tok >= r.first && tok < (int64_t)r.first + r.n && pos >= 0 && pos < q.cap;
    const int64_t blk = mine ? q.table[b * q.table_stride + (pos >> c.tsh)] : -1;
    return Spot{blk < c.blocks ? blk : -1, (int)(pos & (T - 1))};
  };
  // A token that is the wave's only one is placed once: divisions and searches took most
  // of the vector unit's time (256 tokens on 64 sequences, 8 heads of 128: 29.2 us, now 25.9).
  const Spot only = tokens == 1 ? spot(tok0) : Spot{-1, 0};
  for (int i0 = 0; i0 < all; i0 += 64) {
    const int i = i0 + lane, at = i < all ? i : 0;
    const int64_t tok = tokens == 1 ? tok0 : tok0 + at / units;
    const int unit = tokens == 1 ? at : at % units, head = unit / upr, u = unit % upr;
    const Spot to = tokens == 1 ? only : spot(tok);
    const int64_t blk = i < all ? to.blk : -1;
    const int o = to.o;
    Unit<DT> kv[2];  // both asked for before either's codes are stored
    load_unit(kv[0], kr.x + tok * kr.ts + head * kr.hs + u * (8 * DT::ESIZE));
    load_unit(kv[1], vr.x + tok * vr.ts + head * vr.hs + u * (8 * DT::ESIZE));
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const Unit<DT>& x = kv[side];
      uint32_t am = 0;
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = x.f(e);
        const uint32_t a = __float_as_uint(y[e]) & 0x7FFFFFFFu;
        am = a < 0x7F800000u && a > am ? a : am;
      }
      uint32_t w = xor_lane32<1>(am);
      am = am > w ? am : w;
      w = xor_lane32<2>(am);
      am = am > w ? am : w;
      const int ex = mx_exponent(am);
#pragma unroll
      for (int e = 0; e < 8; ++e)  // (8: above the largest code, for infinities)
        y[e] = y[e] == y[e] ? __builtin_amdgcn_fmed3f(__builtin_ldexpf(y[e], -ex), -8.0f, 8.0f) : 0.0f;
      const uint32_t pk = enc_e2m1_x8(y);
      if (blk >= 0) {
        const int64_t at = blk * c.heads + head;
        *(uint32_t*)((side ? c.v : c.k) + (at * T + o) * (c.dim / 2) + 4 * u) = pk;
        if ((u & 3) == 0) (side ? c.ve : c.ke)[(at * (c.dim / 32) + (u >> 2)) * T + o] = (uint8_t)(ex + 127);
      }
    }
  }
}

namespace {
// Tokens of a wave: so many that its lanes are busy.
int append_tokens(const KvCache& c) {
  const int units = c.heads * (c.dim / 8);
  return units >= 64 ? 1 : 64 / units;
}
int64_t append_groups(const KvCache& c, const KvSeqs& q) {
  const int64_t per = (kBlock / 64) * append_tokens(c);
  return (q.total + per - 1) / per;
}
}  // namespace

bool kv4_append_fits(const KvCache& c, const KvSeqs& q) {
  return append_groups(c, q) <= kMostThreads / kBlock && (int64_t)c.heads * c.dim <= INT32_MAX / 64;
}

hipError_t launch_kv4_append(const KvCache& c, const KvSeqs& q, const KvRows& k, const KvRows& v,
                             int dtype, hipStream_t s) {
  return with_dtype(dtype, [&]<class DT>() {
    hipLaunchKernelGGL((k_kv4_append<DT>), dim3((unsigned)append_groups(c, q)), dim3(kBlock), 0, s, c, q, k, v,
                       append_tokens(c));
    return hipGetLastError();
  });
}

// ---------------------------------------------------------------------------
// Attention.  For query row i of sequence b at position pos = len - n + i and kv head
// j = h / g (g query heads per kv head), over the visible tokens t:
//   s_t = scale * (q . K_t),  p_t = exp(s_t),  o = (sum_t p_t V_t) / (sum_t p_t).
// Both products run on v_mfma_f32_16x16x32, the first in the queries' type (bf16 or fp16),
// the second in fp16 (outside_fp16 below), which the codes enter through
// v_cvt_scalef32_pk_*_fp4: two codes times their power of two an instruction, exact in bf16
// and, within its range, in fp16.  (The power's operand
// counts by its exponent field alone, so an exponent byte is put there by one shift,
// whatever lies around it.)  Transposed throughout:
//   S^T [token][row] = K Q^T    lane: row c = lane % 16, tokens of lane group h = lane / 16
//   O^T [dim][row]   = V^T P^T  lane: row c
// A tile is 64 tokens; row 4 q + i of MFMA tile mt of K is token 16 q + 4 i + mt, so that
// lane group h gets the scores of its 16 tokens 16 h + 4 i + mt in slots 4 mt + i, and a
// lane's four K rows are adjacent tokens: their exponents are one dword.  V's operand
// has the dims as rows: row c of tile u is dim 8 c + u of a span of 128 dims (4 c + u of
// one of 64), so that a lane reads 8 (4) adjacent dims of its group's 16 tokens, whose
// exponents are 16 adjacent bytes; pairs of tokens are put together by byte permutes.
// Scores, maxima, sums and O are fp32; p_t is rounded to V's type, for P V only.
// ---------------------------------------------------------------------------
typedef __bf16 bf16x2v __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8v __attribute__((ext_vector_type(8)));

constexpr float kTopSet4 = 8.0f;    // a new reference puts the largest weight at 2^8 ...
constexpr float kTopMost4 = 15.0f;  // ... and stands until one would pass 2^15 (fp16's range)
// One fma from score to exponent rounds the reference, not the exponent: the same factor
// for every token, harmless until the rounding itself is large.  From here on every
// tile takes the difference of the rounded terms, so that the largest stays in range.
constexpr float kFarTop4 = 65536.0f;

template <bool F16>
struct Kv4Type {
  // the largest exponent byte whose codes stay finite
  static constexpr uint32_t kMost = F16 ? 140u : 252u;
  // codes of byte B of w times the power whose exponent field is in s
  template <int B>
  static __device__ inline uint32_t widen(uint32_t w, uint32_t s) {
    if constexpr (F16) return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, __uint_as_float(s), B));
    else return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, __uint_as_float(s), B));
  }
  static __device__ inline u32x4v widen8(uint32_t w, uint32_t s) {
    return u32x4v{widen<0>(w, s), widen<1>(w, s), widen<2>(w, s), widen<3>(w, s)};
  }
  static __device__ inline f32x4v mfma(u32x4v a, u32x4v b, f32x4v c) {
    if constexpr (F16)
      return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
    else
      return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
  }
  static __device__ inline uint32_t pack(float x, float y) {
    if constexpr (F16) return __builtin_bit_cast(uint32_t, f16x2_t{(_Float16)x, (_Float16)y});
    else return __builtin_bit_cast(uint32_t, bf16x2v{(__bf16)x, (__bf16)y});
  }
  static constexpr uint32_t kNan = F16 ? 0x7E007E00u : 0x7FC07FC0u;
  static constexpr uint32_t kExp = F16 ? 0x7C00u : 0x7F80u;  // exponent field
};

// Exponent byte B of w in a float's exponent field.
template <int B>
__device__ inline uint32_t exponent_field(uint32_t w) {
  if constexpr (B == 3) return w >> 1;
  else return w << (23 - 8 * B);
}

// Exponent bytes of w: those above `most` become it; 255 (NaN) becomes `nan`.  bad
// gets a bit per byte that was 255.
__device__ inline uint32_t tame_exponents(uint32_t w, uint32_t most, uint32_t nan, uint32_t& bad) {
  uint32_t r = 0;
  bad = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (w >> (8 * i)) & 0xFFu;
    r |= (b == 255 ? nan : (b > most ? most : b)) << (8 * i);
    bad |= (b == 255 ? 1u : 0u) << i;
  }
  return r;
}

// Bit 7 of the bytes of w that are above MOST (128 to 254).
template <uint32_t MOST>
__device__ inline uint32_t above(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + (255 - MOST) * 0x01010101u) & w & 0x80808080u;
}

// V enters its product in fp16 whatever the queries' type, so that the weights keep fp16's
// eleven bits (rounded to bf16's eight they were the largest error of a result: 8192 tokens
// 1.8e-3 off, the output's own rounding 1.5e-3).  Codes times 2^-23 to 2^8 are exact there: bits
// 7 to 5 of a byte are set where an exponent is outside of that (in the lowest such byte of a
// word for certain: nothing is borrowed from it).  With bf16 queries, where a tile has such an
// exponent, the wave (the prompt kernel's workgroup) goes through all of its tiles again in
// bf16, in a loop of its own.  (Both types in one loop: registers spilled at every use, decoding
// 6 to 35% slower.  The second loop recomputes what it needs, so that the first keeps nothing
// for it.  Prompts with heads of 256 pay for it all the same: 734 us, all in bf16 657.  Where every
// tile has such exponents, 64 sequences of 300..16384 take 133 us for 128, but two row tiles a wave
// and prompts, which do not end their first loop early, twice the time: 8192 tokens 1110 us.)
__device__ inline uint32_t outside_fp16(uint32_t w) { return (w - 0x68686868u) & 0xE0E0E0E0u; }

// Whether exponents w of four tokens leave fp16, but for those of tokens whose codes are zero
// or that are not within first .. last (0: the first of the four): no one sees them.
__device__ inline bool leaves_fp16(uint32_t w, uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, int first, int last) {
  const uint32_t c[4] = {c0, c1, c2, c3};
  bool leaves = false;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t b = (w >> (8 * i)) & 0xFFu;
    leaves |= outside_fp16(b | 0x80808000u) & 0xE0u && b != 255 && c[i] & 0x77777777u && i >= first && i <= last;
  }
  return leaves;
}

// Over lanes l and l ^ 32, in both.
__device__ inline float halves_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  float m;
  asm("v_max_f32 %0, %1, %2" : "=v"(m) : "v"(r[0]), "v"(r[1]));
  return m;
}
__device__ inline float halves_sum(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Query row r of the row tile (column c of the MFMA tiles): elements d(j) .. d(j) + 7 of
// this lane into qf[j].  A row with an element that is no finite number is all NaN.
struct Kv4Row {
  int lim, low;  // last and first position seen (lim -1: no row)
};
template <bool F16, int LANES, int NJ, class F>  // LANES of a row: four lane groups of 16, or two of 32
__device__ inline Kv4Row kv4_query(const KvAttnArgs& p, const KvItem& it, int r, u32x4v (&qf)[NJ], F&& d) {
  const KvAttn& a = p.a;
  const bool valid = r < it.k.rows;
  const int i = valid ? r / p.g : 0, hq = valid ? it.head * p.g + r % p.g : 0;
  const int pos = it.r.len - it.r.n + i;
  const int hi_all = (int)(it.r.len < a.q.cap ? it.r.len : a.q.cap);
  Kv4Row row;
  row.lim = !valid ? -1 : (a.causal && pos + 1 < hi_all ? pos + 1 : hi_all) - 1;
  row.low = first_seen(pos, a.window);
  const char* x = a.x + (it.r.first + (int64_t)i) * a.ts + hq * a.hs;
#pragma unroll
  for (int j = 0; j < NJ; ++j) qf[j] = *(const u32x4v*)(x + 2 * d(j));
  constexpr uint32_t E = Kv4Type<F16>::kExp;
  bool bad = false;
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e) bad |= (qf[j][e] & E) == E || (qf[j][e] & (E << 16)) == (E << 16);
  if (__any(bad)) {
    const float b = LANES == 4 ? groups_max(bad ? 1.0f : 0.0f) : halves_max(bad ? 1.0f : 0.0f);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) qf[j][e] = b > 0.0f ? Kv4Type<F16>::kNan : qf[j][e];
  }
  return row;
}

// State of a wave's rows over the tiles.
template <int QT, int NU>
struct Kv4State {
  float m[QT], l[QT];  // reference (log2), sum of this lane group's weights
  f32x4v o[QT][NU];
  int far;             // some row's reference is past kFarTop4
  __device__ inline void init() {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      m[t] = kNegInf;
      l[t] = 0.0f;
#pragma unroll
      for (int u = 0; u < NU; ++u) o[t][u] = f32x4v{0.f, 0.f, 0.f, 0.f};
    }
    far = 0;
  }
};

// Scores of a tile to weights in VX's type: lane: QT rows, slot 4 mt + i is token tok(mt, i)
// of the lane group's 16 (tok0 = its first).  edge: some token is not seen by some row, or is
// NaN (bad: by slot).  The sum is of the weights before their rounding.
template <class VX, int QT, int NU>
__device__ inline void kv4_weights(f32x4v (&sc)[QT][4], const Kv4Row (&row)[QT], float c, bool there, int tok0,
                                   bool edge, uint32_t bad, Kv4State<QT, NU>& st, u32x4v (&pf)[QT][2]) {
  auto token = [](int mt, int i) { return 4 * i + mt; };  // of slot (mt, i)
  if (edge) {
    if (__any(bad != 0)) {
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            sc[t][mt][e] = (bad >> token(mt, e)) & 1 ? __builtin_nanf("") : sc[t][mt][e];
    }
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      // tokens tok0 + x with first <= x <= last
      const int first = there ? row[t].low - tok0 : 16, last = row[t].lim - tok0;
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sc[t][mt][e] = token(mt, e) > last || token(mt, e) < first ? kNegInf : sc[t][mt][e];
    }
  }
  float top[QT];
  bool turn = false;
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    float mx = kNegInf;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx = __builtin_fmaxf(mx, sc[t][mt][e]);
    top[t] = groups_max(mx) * c;
    turn |= top[t] - st.m[t] > kTopMost4;  // -inf - -inf is NaN: no new reference
  }
  if (__any(turn)) {
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const bool g = top[t] - st.m[t] > kTopMost4;
      float nm = top[t] - kTopSet4;
      nm = top[t] - nm > kTopMost4 ? top[t] : nm;  // where scores have steps of 16, top - 8 may round to top - 16
      const float al = g ? __builtin_amdgcn_exp2f(st.m[t] - nm) : 1.0f;
      st.m[t] = g ? nm : st.m[t];
      st.l[t] *= al;
      st.far |= uniform((int)__any(__builtin_fabsf(st.m[t]) > kFarTop4 && st.m[t] != kNegInf));
#pragma unroll
      for (int u = 0; u < NU; ++u) st.o[t][u] *= al;
    }
  }
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    const float ref = st.m[t] == kNegInf ? 0.0f : st.m[t];
    if (st.far) {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][mt][e] = sc[t][mt][e] * c - ref;
    } else {
#pragma unroll
      for (int mt = 0; mt < 4; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[t][mt][e] = __builtin_fmaf(sc[t][mt][e], c, -ref);
    }
    float sum = 0.0f;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[t][mt][e] = __builtin_amdgcn_exp2f(sc[t][mt][e]);
        sum += sc[t][mt][e];
      }
      pf[t][mt / 2][2 * (mt & 1)] = VX::pack(sc[t][mt][0], sc[t][mt][1]);
      pf[t][mt / 2][2 * (mt & 1) + 1] = VX::pack(sc[t][mt][2], sc[t][mt][3]);
    }
    st.l[t] += sum;
  }
}

// Few rows per kv head (decoding): QT tiles of 16 rows, four waves that take the
// chunk's tiles in turn, K and V straight from memory into MFMA operands.
// BIG: blocks of 64 tokens and more, so a tile lies in one block (scalar addresses).
// The cache's bytes bound it, where the waves hide their latency: 64 sequences of 300 to
// 16384 tokens, 8 kv heads of 128, 128 us, 4.6 TB/s (6.5 in a large copy), heads of 64 82, of
// 192 116, of 256 on 300 to 8192 136.  A third wave a SIMD took 148 us to 134, a second at heads
// of 192 and 256 171 to 127 and 188 to 144; block numbers asked for two tiles ahead, before
// loads that are not due yet, 165 to 148; exponents looked at byte by byte only where the type
// does not hold them, and not from 128 on, 130 to 128 (heads of 64 89 to 82).  With two row
// tiles every widened operand serves two products; they take half of the waves' registers
// more, and a wave less a SIMD (heads of 64 keep 18 to 23 registers in scratch, of 256 50).
template <int D, int QT>
constexpr int Kv4FewWaves = QT == 1 ? (D == 64 ? 4 : D == 128 ? 3 : 2) : (D == 64 ? 3 : D == 128 ? 2 : 1);  // per SIMD
template <int D, bool F16, bool BIG, int QT>
__global__ __launch_bounds__(256, (Kv4FewWaves<D, QT>)) void k_kv4_attn(KvAttnArgs p) {
  using X = Kv4Type<F16>;
  // spans of 128 dims (16 bytes of a K row a lane) and of 64 (8 bytes)
  constexpr int S128 = D / 128, S64 = D % 128 / 64, NS = S128 + S64, NJ = D / 32, NU = D / 16, G = D / 32;
  const KvAttn& a = p.a;
  const int lane = threadIdx.x & 63, wv = uniform((int)threadIdx.x >> 6);
  int c16 = lane & 15, h = lane >> 4;
  KvItem it;
  if (!kv_item(p, blockIdx.x, lane, it)) return;
  const int H = a.c.heads, tsh = a.c.tsh, T = 1 << tsh;
  u32x4v qf[QT][NJ];
  Kv4Row row[QT];
  auto query = [&] {
#pragma unroll
    for (int t = 0; t < QT; ++t)
      row[t] = kv4_query<F16, 4>(p, it, it.rt * p.rb + 16 * t + c16, qf[t], [&](int j) {
        return j / 4 < S128 ? 128 * (j / 4) + 32 * h + 8 * (j % 4) : 128 * S128 + 16 * h + 8 * (j % 4);
      });
  };
  query();
  const float c = a.scale * 1.44269504088896340736f;
  Kv4State<QT, NU> st;

  const int r0 = it.rt * p.rb, r1 = r0 + 16 * QT < it.k.rows ? r0 + 16 * QT : it.k.rows;
  const KvRange rg = kv_range(p, it, r0, r1);
  const int lo = rg.lo, hi = rg.hi;
  const int* table = a.q.table + (int64_t)it.seq * a.q.table_stride;

  // Block of a tile (BIG) or of this lane group's 16 tokens of it, or -1: what no row
  // sees and what has no block reads block 0, masked.  `entry` is asked for before the
  // loads that `known` must not wait for.
  auto entry = [&](int tt) -> int {
    const int gp = tt * kKvTile + (BIG ? 0 : 16 * h);
    if (tt >= rg.t1 || gp >= hi || gp + (BIG ? kKvTile : 16) <= lo) return -1;
    return table[gp >> tsh];
  };
  auto known = [&](int blk) -> int {
    if (blk >= a.c.blocks) blk = -1;
    return BIG ? scalar(blk) : blk;
  };
  auto place = [&](int blk) -> int64_t { return (int64_t)(blk < 0 ? 0 : blk) * H + it.head; };
  // K: rows 4 c16 .. 4 c16 + 3 of the tile; V: rows 16 h .. 16 h + 15
  u32x4v kr[4][S128 ? S128 : 1], vs[NS];
  uint2 k8[4];
  uint32_t vr[16][S128 ? S128 : 1], ks[NS];
  uint16_t v2[16];
  auto load_k = [&](int tt, int blk) {
    const int row0 = (tt * kKvTile + 4 * c16) & (T - 1);
    const int64_t at = place(BIG ? blk : __shfl(blk, 16 * (c16 >> 2), 64));
    const uint8_t* kp = a.c.k + (at * T + row0) * (D / 2);
    const uint8_t* ep = a.c.ke + at * G * T + row0;
#pragma unroll
    for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
      for (int s = 0; s < S128; ++s) kr[mt][s] = *(const u32x4v*)(kp + mt * (D / 2) + 64 * s + 16 * h);
      if constexpr (S64) k8[mt] = *(const uint2*)(kp + mt * (D / 2) + 64 * S128 + 8 * h);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) ks[s] = *(const uint32_t*)(ep + (4 * s + (s < S128 ? h : h >> 1)) * T);
  };
  auto load_v = [&](int tt, int blk) {
    const int row0 = (tt * kKvTile + 16 * h) & (T - 1);
    const int64_t at = place(blk);
    const uint8_t* vp = a.c.v + (at * T + row0) * (D / 2);
    const uint8_t* ep = a.c.ve + at * G * T + row0;
#pragma unroll
    for (int e = 0; e < 16; ++e) {
#pragma unroll
      for (int s = 0; s < S128; ++s) vr[e][s] = *(const uint32_t*)(vp + e * (D / 2) + 64 * s + 4 * c16);
      if constexpr (S64) v2[e] = *(const uint16_t*)(vp + e * (D / 2) + 64 * S128 + 2 * c16);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) vs[s] = *(const u32x4v*)(ep + (4 * s + (s < S128 ? c16 >> 2 : c16 >> 3)) * T);
  };
  bool gone = false;  // V left fp16
  auto run = [&]<class VX>() __attribute__((always_inline)) {  // with V in VX's type
    constexpr bool kMayLeave = !F16 && __is_same(VX, Kv4Type<true>);
    st.init();
    int tt = rg.t0 + wv, blk = -1, blk1 = -1, ahead = -1;
    if (tt < rg.t1) {
      const int e0 = entry(tt), e1 = entry(tt + 4);
      ahead = entry(tt + 8);
      blk = known(e0);
      blk1 = known(e1);
      load_k(tt, blk);
      load_v(tt, blk);
    }
    for (; tt < rg.t1; tt += 4) {
      const int b0 = tt * kKvTile, gp = b0 + 16 * h;
      const bool there = blk >= 0 && (!BIG || (gp < hi && gp + 16 > lo)), more = tt + 4 < rg.t1;
      // Exponents that the types do not hold are rare: only then are their bytes looked at
      // one by one.
      uint32_t high = 0, bad = 0;
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        high |= above<X::kMost>(ks[s]);
#pragma unroll
        for (int i = 0; i < 4; ++i) high |= kMayLeave ? outside_fp16(vs[s][i]) : above<VX::kMost>(vs[s][i]);
      }
      if (__builtin_expect(__any(high), 0)) {
        if constexpr (kMayLeave) {
          bool leaves = false;
#pragma unroll
          for (int s = 0; s < NS; ++s) {
            auto codes = [&](int e) { return s < S128 ? vr[e][s < S128 ? s : 0] : (uint32_t)v2[e]; };
#pragma unroll
            for (int i = 0; i < 4; ++i)
              leaves |= leaves_fp16(vs[s][i], codes(4 * i), codes(4 * i + 1), codes(4 * i + 2), codes(4 * i + 3),
                                    lo - gp - 4 * i, hi - 1 - gp - 4 * i);
          }
          if (__any(leaves)) {
            gone = true;
            if constexpr (QT == 1) return;  // (with two, at heads of 256, this took 151 us to 179)
          }
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
          uint32_t none;
          ks[s] = tame_exponents(ks[s], X::kMost, 255, none);  // K's NaN makes the score NaN
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t b;
            vs[s][i] = tame_exponents(vs[s][i], VX::kMost, 0, b);
            bad |= b << (4 * i);
          }
        }
        bad |= (uint32_t)__shfl_xor((int)bad, 4, 64);  // the other groups of dims
        bad |= (uint32_t)__shfl_xor((int)bad, 8, 64);
      }
      f32x4v sc[QT][4];
#pragma unroll
      for (int t = 0; t < QT; ++t)
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) sc[t][mt] = f32x4v{0.f, 0.f, 0.f, 0.f};
      auto scores = [&]<int MT>() {
#pragma unroll
        for (int s = 0; s < S128; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const u32x4v k = X::widen8(kr[MT][s][j], exponent_field<MT>(ks[s]));
#pragma unroll
            for (int t = 0; t < QT; ++t) sc[t][MT] = X::mfma(k, qf[t][4 * s + j], sc[t][MT]);
          }
        if constexpr (S64) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const u32x4v k = X::widen8(j ? k8[MT].y : k8[MT].x, exponent_field<MT>(ks[S128]));
#pragma unroll
            for (int t = 0; t < QT; ++t) sc[t][MT] = X::mfma(k, qf[t][4 * S128 + j], sc[t][MT]);
          }
        }
      };
      scores.template operator()<0>();
      scores.template operator()<1>();
      scores.template operator()<2>();
      scores.template operator()<3>();
      const bool edge = __any(bad != 0 || !there) || b0 + kKvTile > rg.least || b0 < rg.from;
      int blk2 = -1;
      if (more) {
        blk2 = known(ahead);
        ahead = entry(tt + 12);
        load_k(tt + 4, blk1);
      }
      u32x4v pf[QT][2];
      kv4_weights<VX, QT, NU>(sc, row, c, there, gp, edge, bad, st, pf);
      // slot 4 mt + i of V is token 4 i + mt: byte mt of exponent dword i
      auto out = [&]<int U0, int NB>(auto&& word, const u32x4v& ex) {  // NB bytes: 2 NB dims a lane
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          uint32_t w[8][NB];  // slots 8 x ..: dims 2 b and 2 b + 1
          auto slot = [&]<int MT>() {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const uint32_t v = word(4 * i + 2 * x + MT), s = x ? exponent_field<2 + MT>(ex[i]) : exponent_field<MT>(ex[i]);
              w[4 * MT + i][0] = VX::template widen<0>(v, s);
              w[4 * MT + i][1] = VX::template widen<1>(v, s);
              if constexpr (NB == 4) {
                w[4 * MT + i][2] = VX::template widen<2>(v, s);
                w[4 * MT + i][3] = VX::template widen<3>(v, s);
              }
            }
          };
          slot.template operator()<0>();
          slot.template operator()<1>();
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            u32x4v even, odd;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              even[j] = __builtin_amdgcn_perm(w[2 * j + 1][b], w[2 * j][b], 0x05040100u);
              odd[j] = __builtin_amdgcn_perm(w[2 * j + 1][b], w[2 * j][b], 0x07060302u);
            }
#pragma unroll
            for (int t = 0; t < QT; ++t) {
              st.o[t][U0 + 2 * b] = VX::mfma(even, pf[t][x], st.o[t][U0 + 2 * b]);
              st.o[t][U0 + 2 * b + 1] = VX::mfma(odd, pf[t][x], st.o[t][U0 + 2 * b + 1]);
            }
          }
        }
      };
      if constexpr (S128 > 0) out.template operator()<0, 4>([&](int e) { return vr[e][0]; }, vs[0]);
      if constexpr (S128 > 1) out.template operator()<8, 4>([&](int e) { return vr[e][1]; }, vs[1]);
      if constexpr (S64 > 0) out.template operator()<8 * S128, 2>([&](int e) { return (uint32_t)v2[e]; }, vs[S128]);
      if (more) load_v(tt + 4, blk1);
      blk = blk1;
      blk1 = blk2;
    }
  };
  run.template operator()<Kv4Type<true>>();
  if constexpr (!F16) {
    if (__builtin_expect(gone, 0)) {
      asm volatile("" : "+v"(c16), "+v"(h));  // nothing of the first loop is kept for the second
      if constexpr (QT == 1) query();
      run.template operator()<Kv4Type<false>>();
    }
  }

  // the four waves' parts of each row meet in LDS, in wave order
  constexpr int PITCH = D + 4;
  __shared__ float os[4][16][PITCH];
  __shared__ __attribute__((aligned(16))) float mls[4][16][2];  // reference, sum
#pragma unroll
  for (int t = 0; t < QT; ++t) {
    if (t) __syncthreads();  // the rows before are out
    st.l[t] = groups_sum(st.l[t]);
    if (h == 0) *(f32x2v*)mls[wv][c16] = f32x2v{st.m[t], st.l[t]};
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int s = u / 8, d = s < S128 ? 128 * s + 8 * (4 * h + i) + u % 8 : 128 * S128 + 4 * (4 * h + i) + u % 8;
        os[wv][c16][d] = st.o[t][u][i];
      }
    __syncthreads();
    const int at = 4 * wv + h, sub = c16, g = scalar(p.g);
    const int r = it.rt * p.rb + 16 * t + at;
    if (r < it.k.rows) {
      float top = kNegInf, f[4], sum = 0.0f;
#pragma unroll
      for (int q = 0; q < 4; ++q) top = __builtin_fmaxf(top, mls[q][at][0]);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        f[q] = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(mls[q][at][0] - top);
        // a wave whose scores are all NaN has no reference, and a NaN sum
        f[q] = mls[q][at][1] == mls[q][at][1] ? f[q] : __builtin_nanf("");
        sum += mls[q][at][1] * f[q];
      }
      const int64_t tok = it.r.first + r / g, hq = it.head * g + r % g;
      const bool split = it.chunks > 1;
      const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
      const int64_t base = split ? (it.slot * p.rb + 16 * t + at) * D : (tok * a.heads + hq) * D;
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
          const f32x2v ml = {sum == sum ? top : -kNegInf, sum};  // NaN has the last word in the join
          *(f32x2v*)(p.ml + (it.slot * p.rb + 16 * t + at) * 2) = ml;
        } else if (a.lse) {
          a.lse[tok * a.heads + hq] = kv_lse(top, sum);
        }
      }
    }
  }
}

// Many rows per kv head (prompts): the waves of a workgroup hold 32 rows each and share
// every tile of 64 tokens, which is widened once into LDS (K [64][D], V transposed to
// [D][64], 16-byte chunks XOR-swizzled by row), one tile ahead of its use, its codes
// loaded one tile ahead of that.  Products on v_mfma_f32_32x32x16, transposed as above:
//   S^T  lane: row c = lane % 32, tokens 32 mt + 8 (i / 4) + 4 h + i % 4  (h = lane / 32)
//   O^T  lane: row c, dims 32 u + 8 (i / 4) + 4 h + i % 4
// The tokens that a lane has of each 16 are its k slots in the second product; V's
// tokens are stored in that order (quads 0, 2 | 1, 3 of each 16).
// What bounds it: the exponentials, the sums and the widening on the vector unit (about
// 1300 cycles per 32 rows and 64 tokens of 128 dims, the products 1024), LDS reads (half of
// its rate) and the clock, 2.0 GHz under this load.  8192 tokens, 32 heads over 8 of 128:
// 549 us, 1.0 Pflop/s (1.4 in a large product); 549 to 650 us by card and run.  Taken and not
// taken, each pair on one card: 4 waves and two workgroups a CU (8 waves that multiply and
// weight in turns: level, 476 us for 434 at heads of 192, and 58 for 43 where prompts are
// short); a tile's scores formed while the one before is weighted: 660 for 628; waves
// without rows that share the others' tokens: 640 for 575; codes asked for two tiles ahead:
// level.
// Heads of 64 have registers for a third wave a SIMD: 349 us, two 387 (334 now that V is in
// fp16).  At 192 and 256 the scores of 64 tokens beside the sums pass 256 registers, so they
// are formed 32 at a time, and 8 waves share a tile, the only workgroup of its CU: 431 and 773
// us (16 heads over 8; now 440 and 734), for 498 of 64 tokens at a time and 995 of 4 waves with
// twice the registers.  Heads of 256 still keep 49 to 54 registers in scratch (bf16, over both
// loops, 118 to 129), up to four of the sixteen query fragments among them, which are read back
// for every 32 tokens; of 192 2 to 21, of 64 4 to 28, few of them inside the loop.
template <int D>
struct Kv4PromptShape {
  static constexpr int NW = D >= 192 ? 8 : 4, WAVES = D == 64 ? 3 : 2;  // waves of a workgroup, per SIMD
  static constexpr int ROWS = 32 * NW;
};
typedef float f32x16v __attribute__((ext_vector_type(16)));

template <bool F16>
__device__ inline f32x16v kv4_mfma32(u32x4v a, u32x4v b, f32x16v c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8v, a), __builtin_bit_cast(bf16x8v, b), c, 0, 0, 0);
}
template <int D, bool F16, bool BIG>
__global__ __launch_bounds__(64 * Kv4PromptShape<D>::NW, Kv4PromptShape<D>::WAVES) void k_kv4_prompt(KvAttnArgs p) {
  using X = Kv4Type<F16>;
  constexpr int NW = Kv4PromptShape<D>::NW, NJ = D / 16, NU = D / 32, G = D / 32;
  constexpr int WK = D / 32, NQ = (2 * WK + NW - 1) / NW;  // 64-unit loads of K (and of V), a wave's share
  constexpr int K_BYTES = kKvTile * D * 2, BUF = 2 * K_BYTES;
  __shared__ __attribute__((aligned(16))) uint8_t smem[2 * BUF];
  __shared__ uint32_t nan_tokens[3][2];  // tokens whose V exponent is NaN, by tile
  __shared__ uint32_t gone;              // V left fp16
  const KvAttn& a = p.a;
  const int wv = uniform((int)threadIdx.x >> 6);
  int tid = threadIdx.x, lane = tid & 63, c32 = lane & 31, h = lane >> 5;
  KvItem it;
  if (!kv_item(p, blockIdx.x, lane, it)) return;
  const int H = a.c.heads, tsh = a.c.tsh, T = 1 << tsh;

  const int w0 = it.rt * p.rb + 32 * wv;  // this wave's first row
  // Query fragments in LDS, as many as it has room for, where the registers do not hold all:
  // heads of 256 773 us (16 heads over 8, fp16), with two in LDS 675, with three 637.
  constexpr int QL = D == 256 ? 3 : 0, NR = NJ - QL;
  __shared__ u32x4v q_last[QL ? NW * QL * 64 : 1];
  u32x4v qf[NJ];
  Kv4Row row;
  auto query = [&] {
    row = kv4_query<F16, 2>(p, it, w0 + c32, qf, [&](int j) { return 16 * j + 8 * h; });
  };
  query();
#pragma unroll
  for (int j = 0; j < QL; ++j) q_last[(wv * QL + j) * 64 + lane] = qf[NR + j];
  const float c = a.scale * 1.44269504088896340736f;
  float m = kNegInf, l = 0.0f;
  f32x16v o[NU];
#pragma unroll
  for (int u = 0; u < NU; ++u)
#pragma unroll
    for (int e = 0; e < 16; ++e) o[u][e] = 0.0f;
  int far = 0;
  const int r0 = it.rt * p.rb, r1 = r0 + p.rb < it.k.rows ? r0 + p.rb : it.k.rows;
  const KvRange rg = kv_range(p, it, r0, r1);
  // what this wave's own rows see (none: rows past the end)
  const int w1 = w0 + 32 < it.k.rows ? w0 + 32 : it.k.rows;
  KvRange mine = rg;
  if (w0 < w1) mine = kv_range(p, it, w0, w1);
  else mine.hi = 0;

  const int* table = a.q.table + (int64_t)it.seq * a.q.table_stride;
  // Block of a tile (BIG) or, in lanes 16 g .., of its 16 tokens g, or -1 where no row
  // sees them or there is none; its place among blocks and heads (0's if none).
  // `entry` is asked for a tile before `known` uses it, and without a branch, behind
  // which the value would be copied and so waited for at once.
  auto first_of = [&](int tt) { return tt * kKvTile + (BIG ? 0 : 16 * (lane >> 4)); };
  auto entry = [&](int tt) -> int {
    const int gp = first_of(tt);
    return table[(gp < rg.hi ? gp : rg.hi - 1) >> tsh];  // (hi > 0 where there is a tile)
  };
  auto known = [&](int b, int tt) -> int {
    const int gp = first_of(tt);
    const bool none = tt >= rg.t1 || gp >= rg.hi || (!BIG && gp + 16 <= rg.lo) || b < 0 || b >= a.c.blocks;
    b = none ? -1 : b;
    return BIG ? uniform(b) : b;
  };
  auto place = [&](int blk) -> int64_t { return (int64_t)(blk < 0 ? 0 : blk) * H + it.head; };
  // A 16-byte LDS access takes lanes l .. l + 7 and l + 16 .. l + 23 at a time: rows 0 .. 7
  // and 16 .. 23 of a fragment (or eight later) have to meet sixteen slots of 16 bytes.
  // Rows of 256 and 512 bytes: all slots by row bits 0, 1, 2, 4; rows of odd multiples of
  // 128: the half by bit 0, the slot in it by bits 1, 2, 4.  The order of the bits and
  // V's bits 3, 5, 6 spread the writes (of rows 8 apart, for V).
  auto k_swizzle = [](int r) {
    return D % 128 == 0 ? (r & 1) | ((r >> 1) & 2) | ((r << 1) & 4) | ((r >> 1) & 8)
                        : ((r >> 1) & 1) | ((r >> 1) & 2) | ((r >> 2) & 4);
  };
  auto v_swizzle = [](int d) {
    return (((d << 1) & 4) ^ ((d >> 3) & 4)) | (((d >> 1) & 2) ^ ((d >> 5) & 2)) | (((d >> 4) & 1) ^ ((d >> 3) & 1));
  };

  // This lane's first fragments; the others lie at fixed distances, but for address bits
  // that the swizzle turns (KX).  One register each, and not one per chunk.
  constexpr unsigned KX = D % 128 == 0 ? 255 : 127;
  unsigned kat, vat;
  auto first_fragments = [&] {
    kat = c32 * (2 * D) + (h ^ k_swizzle(c32)) * 16;
    vat = K_BYTES + c32 * 128 + (h ^ v_swizzle(c32)) * 16;
  };
  first_fragments();

  // Unit i = 64 wc + lane of a tile, wc = wv + NW q.  Of K (wc < WK): 32 dims i % G of token
  // i / G.  Of V: dims 8 o .. 8 o + 7 of tokens 4 t .. 4 t + 3, o = i % (D / 8), t = i / (D / 8).
  auto is_k = [&](int q) { return WK % NW == 0 ? q < WK / NW : wv + NW * q < WK; };
  auto has = [&](int q) { return 2 * WK % NW == 0 || wv + NW * q < 2 * WK; };
  u32x4v cr[NQ];
  uint32_t ex[NQ];
  auto fetch_v = [&](int q, int tt, int blk, u32x4v& codes, uint32_t& exps) {
    const int j = 64 * (wv + NW * q) + lane - 64 * WK, od = j % (D / 8), t = j / (D / 8);
    const int64_t at = place(BIG ? blk : __shfl(blk, (4 * t) & 48, 64));
    const int o = (tt * kKvTile + 4 * t) & (T - 1);
    const uint8_t* vp = a.c.v + (at * T + o) * (D / 2) + 4 * od;
#pragma unroll
    for (int e = 0; e < 4; ++e) codes[e] = *(const uint32_t*)(vp + e * (D / 2));
    exps = *(const uint32_t*)(a.c.ve + (at * G + (od >> 2)) * T + o);
  };
  auto fetch = [&](int tt, int blk) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (!has(q)) continue;
      const int i = 64 * (wv + NW * q) + lane;
      if (is_k(q)) {
        const int r = i / G, g = i % G;
        const int64_t at = place(BIG ? blk : __shfl(blk, r & 48, 64));
        const int o = (tt * kKvTile + r) & (T - 1);
        cr[q] = *(const u32x4v*)(a.c.k + (at * T + o) * (D / 2) + 16 * g);
        ex[q] = a.c.ke[(at * G + g) * T + o];
      } else {
        fetch_v(q, tt, blk, cr[q], ex[q]);
      }
    }
  };
  // V's unit into a buffer, in VX's type
  auto put_v = [&]<class VX>(int q, const u32x4v& codes, uint32_t e, uint8_t* buf) {
    const int j = 64 * (wv + NW * q) + lane - 64 * WK, od = j % (D / 8), t = j / (D / 8);
    uint32_t w[4][4];
    auto one = [&]<int B>() {
      w[0][B] = VX::template widen<B>(codes[0], exponent_field<0>(e));
      w[1][B] = VX::template widen<B>(codes[1], exponent_field<1>(e));
      w[2][B] = VX::template widen<B>(codes[2], exponent_field<2>(e));
      w[3][B] = VX::template widen<B>(codes[3], exponent_field<3>(e));
    };
    one.template operator()<0>();
    one.template operator()<1>();
    one.template operator()<2>();
    one.template operator()<3>();
    const int chunk = 2 * (t >> 2) + (t & 1), half = (t >> 1) & 1;
#pragma unroll
    for (int d = 0; d < 8; ++d) {
      const uint32_t sel = d & 1 ? 0x07060302u : 0x05040100u;
      uint2 v;
      v.x = __builtin_amdgcn_perm(w[1][d / 2], w[0][d / 2], sel);
      v.y = __builtin_amdgcn_perm(w[3][d / 2], w[2][d / 2], sel);
      const int dim = 8 * od + d;
      *(uint2*)(buf + K_BYTES + dim * 128 + (chunk ^ v_swizzle(dim)) * 16 + 8 * half) = v;
    }
  };
  auto widen = [&]<bool V16>(int tt, uint8_t* buf) {
    constexpr bool kMayLeave = !F16 && V16;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      if (!has(q)) continue;
      const int i = 64 * (wv + NW * q) + lane;
      if (is_k(q)) {
        uint32_t e = ex[q];
        e = e > X::kMost && e != 255 ? X::kMost : e;
        const int r = i / G, g = i % G, z = k_swizzle(r);
        uint8_t* k = buf + r * (2 * D);
#pragma unroll
        for (int x = 0; x < 4; ++x) *(u32x4v*)(k + ((4 * g + x) ^ z) * 16) = X::widen8(cr[q][x], e << 23);
      } else {
        uint32_t e = ex[q];
        if (__builtin_expect(__any(kMayLeave ? outside_fp16(e) : above<Kv4Type<V16>::kMost>(e)), 0)) {
          int l = lane;
          if constexpr (kMayLeave) asm volatile("" : "+v"(l));  // nothing of this is kept over the loop
          const int t = (64 * (wv + NW * q) + l - 64 * WK) / (D / 8);
          if constexpr (kMayLeave) {
            const int tok = tt * kKvTile + 4 * t;
            if (leaves_fp16(e, cr[q][0], cr[q][1], cr[q][2], cr[q][3], rg.lo - tok, rg.hi - 1 - tok)) gone = 1;
          }
          uint32_t bad;
          e = tame_exponents(e, Kv4Type<V16>::kMost, 0, bad);
          if (bad) atomicOr(&nan_tokens[tt % 3][t >> 3], bad << ((4 * t) & 31));
        }
        put_v.template operator()<Kv4Type<V16>>(q, cr[q], e, buf);
      }
    }
  };

  auto run = [&]<bool V16>() __attribute__((always_inline)) {  // with V in fp16 or bf16
    m = kNegInf, l = 0.0f, far = 0;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[u][e] = 0.0f;
    int blk = known(entry(rg.t0), rg.t0), blk1 = known(entry(rg.t0 + 1), rg.t0 + 1), ahead = entry(rg.t0 + 2);
    fetch(rg.t0, blk);
    if (tid < 6) nan_tokens[tid >> 1][tid & 1] = 0;
    if (V16 && tid == 0) gone = 0;
    __syncthreads();
    widen.template operator()<V16>(rg.t0, smem);
    fetch(rg.t0 + 1, blk1);  // past the end: block 0, unused
    __syncthreads();
    for (int tt = rg.t0; tt < rg.t1; ++tt) {
      const unsigned buf = ((tt - rg.t0) & 1) * BUF;
      const int b0 = tt * kKvTile;
      if (b0 < mine.hi && b0 + kKvTile > mine.lo) {
        const uint64_t some = BIG ? (blk >= 0 ? ~0ull : 0ull) : __ballot(blk >= 0);
        const uint32_t nan0 = nan_tokens[tt % 3][0], nan1 = nan_tokens[tt % 3][1];
        const bool whole = some == ~0ull, bad = (nan0 | nan1) != 0;
        // the tokens 32 M .. of the tile, in MT parts of 32
        auto part = [&]<int M, int MT>() {
          f32x16v sc[MT];
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[mt][e] = 0.0f;
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
              // row 32 (M + mt) + c32, chunk 2 j + h
              const u32x4v kf =
                  *(const u32x4v*)(smem + ((buf + kat) ^ (32 * j & KX)) + (32 * j & ~KX) + (M + mt) * (64 * D));
              sc[mt] = kv4_mfma32<F16>(kf, j < NR ? qf[j] : q_last[(wv * QL + j - NR) * 64 + lane], sc[mt]);
            }
          // slot (mt, i): token 32 (M + mt) + 8 (i / 4) + 4 h + i % 4
          if (!whole || bad || b0 + kKvTile > mine.least || b0 < mine.from) {
            const int first = row.low - b0 - 4 * h, last = row.lim - b0 - 4 * h;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int x = 32 * (M + mt) + 8 * (e >> 2) + (e & 3);  // + 4 h
                const bool there = (some >> (16 * (x >> 4))) & 1;
                if (bad) sc[mt][e] = ((x < 32 ? nan0 : nan1) >> ((x & 31) + 4 * h)) & 1 ? __builtin_nanf("") : sc[mt][e];
                sc[mt][e] = x > last || x < first || !there ? kNegInf : sc[mt][e];
              }
          }
          float mx = kNegInf;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int e = 0; e < 16; ++e) mx = __builtin_fmaxf(mx, sc[mt][e]);
          const float top = halves_max(mx) * c;
          const bool turn = top - m > kTopMost4;  // -inf - -inf is NaN: no new reference
          if (__any(turn)) {
            float nm = top - kTopSet4;
            nm = top - nm > kTopMost4 ? top : nm;  // where scores have steps of 16, top - 8 may round to top - 16
            const float al = turn ? __builtin_amdgcn_exp2f(m - nm) : 1.0f;
            m = turn ? nm : m;
            l *= al;
            far |= uniform((int)__any(__builtin_fabsf(m) > kFarTop4 && m != kNegInf));
#pragma unroll
            for (int u = 0; u < NU; ++u) o[u] *= al;
          }
          if constexpr (D > 128) __builtin_amdgcn_sched_barrier(0);
          const float ref = m == kNegInf ? 0.0f : m;
          if (far) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 16; ++e) sc[mt][e] = sc[mt][e] * c - ref;
          } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int e = 0; e < 16; ++e) sc[mt][e] = __builtin_fmaf(sc[mt][e], c, -ref);
          }
          u32x4v pf[MT][2];
          float sum = 0.0f;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int d = 0; d < 4; ++d) {
                const float w0 = __builtin_amdgcn_exp2f(sc[mt][8 * x + 2 * d]);
                const float w1 = __builtin_amdgcn_exp2f(sc[mt][8 * x + 2 * d + 1]);
                sum += w0;
                sum += w1;
                pf[mt][x][d] = Kv4Type<V16>::pack(w0, w1);
              }
          l += sum;
          if constexpr (D > 128) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
              for (int u = 0; u < NU; ++u) {
                // row 32 u + c32, chunk 4 (M + mt) + 2 x + h
                const u32x4v vf = *(const u32x4v*)(smem + ((buf + vat) ^ (16 * ((4 * (M + mt) + 2 * x) ^ v_swizzle(32 * u)))) + 4096 * u);
                o[u] = kv4_mfma32<V16>(vf, pf[mt][x], o[u]);
              }
        };
        if constexpr (D <= 128) {
          part.template operator()<0, 2>();
        } else {  // the scores of 64 tokens do not fit the registers
          part.template operator()<0, 1>();
          part.template operator()<1, 1>();
        }
      }
      if (tid < 2) nan_tokens[(tt + 2) % 3][tid] = 0;
      if (tt + 1 < rg.t1) {
        widen.template operator()<V16>(tt + 1, smem + ((tt + 1 - rg.t0) & 1) * BUF);
        blk = blk1;
        blk1 = known(ahead, tt + 2);
        ahead = entry(tt + 3);
        fetch(tt + 2, blk1);
      }
      __syncthreads();
    }
  };
  if (rg.t0 < rg.t1) {
    run.template operator()<true>();
    if constexpr (!F16) {
      if (__builtin_expect(uniform((int)gone), 0)) {
        asm volatile("" : "+v"(tid));  // nothing of the first loop is kept for the second
        lane = tid & 63, c32 = lane & 31, h = lane >> 5;
        first_fragments();
        if constexpr (D == 256) query();
        run.template operator()<false>();
      }
    }
  }
  l = halves_sum(l);
  const int r = w0 + c32;
  if (r >= it.k.rows) return;
  const int64_t tok = it.r.first + r / p.g, hq = it.head * p.g + r % p.g;
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  if (it.chunks > 1) {
    const int64_t at = it.slot * p.rb + (r - r0);
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(f32x4v*)(p.po + at * D + 32 * u + 8 * q + 4 * h) =
            f32x4v{o[u][4 * q] * inv, o[u][4 * q + 1] * inv, o[u][4 * q + 2] * inv, o[u][4 * q + 3] * inv};
    const f32x2v ml = {l == l ? m : -kNegInf, l};  // NaN has the last word in the join
    if (h == 0) *(f32x2v*)(p.ml + at * 2) = ml;
  } else {
    char* out = a.out + 2 * (tok * a.heads + hq) * D;
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *(uint2*)(out + 2 * (32 * u + 8 * q + 4 * h)) =
            uint2{X::pack(o[u][4 * q] * inv, o[u][4 * q + 1] * inv), X::pack(o[u][4 * q + 2] * inv, o[u][4 * q + 3] * inv)};
    if (a.lse && h == 0) a.lse[tok * a.heads + hq] = kv_lse(m, l);
  }
}

namespace {
int prompt4_rows(int dim) {
  return dim == 64 ? Kv4PromptShape<64>::ROWS : dim == 128 ? Kv4PromptShape<128>::ROWS
         : dim == 192 ? Kv4PromptShape<192>::ROWS : Kv4PromptShape<256>::ROWS;
}
// (three workgroups a CU with heads of 64: a mixed batch of 24 sequences 41.5 us, aimed at two 43.9)
KvPlan plan_of(const KvAttn& a, void* ws) {
  // Two row tiles a wave where sequences have 17 to 32 rows each, or do on average (8 tokens
  // on 64 sequences of 300..8192, 32 heads over 8: 95 us, by the prompt kernel 200; with one
  // token on every other sequence 93 and 228; on 16 of 4096, 4 kv heads: 25.5 and 30.4).  The
  // host knows only the average, and pays where single tokens have it from a long prompt
  // beside them (63 and one of 400 tokens on such sequences: 155 us, with one row tile 140).
  const int64_t rows = a.q.total * (a.heads / a.c.heads), seqs = a.q.seqs;  // (seqs: at least one)
  return kv_plan(a, (char*)ws, rows > 16 * seqs && rows <= 32 * seqs ? 32 : 16, prompt4_rows(a.c.dim), a.c.dim == 64 ? 3 : a.c.dim == 128 ? 2 : 1);
}
}  // namespace

bool kv4_attn_fits(const KvAttn& a) {
  return kv_plan_fits(a, plan_of(a, nullptr), 2 * prompt4_rows(a.c.dim));
}

size_t kv4_attn_workspace(const KvAttn& a) { return plan_of(a, nullptr).need; }

hipError_t launch_kv4_attn(const KvAttn& a, void* ws, hipStream_t s) {
  const KvPlan p = plan_of(a, ws);
  if (p.planned) {
    const hipError_t e = launch_kv_starts(p, s);
    if (e != hipSuccess) return e;
  }
  auto dim = [&]<int D>() {
    const bool f16 = a.dtype == 2;
    if (p.run_many) {
      auto k = a.c.tsh >= 6 ? (f16 ? k_kv4_prompt<D, true, true> : k_kv4_prompt<D, false, true>)
                            : (f16 ? k_kv4_prompt<D, true, false> : k_kv4_prompt<D, false, false>);
      hipLaunchKernelGGL(k, dim3((unsigned)p.many.items), dim3(64 * Kv4PromptShape<D>::NW), 0, s, p.many);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    if (p.run_few) {
      auto kernel = [&]<int QT>() {
        return a.c.tsh >= 6 ? (f16 ? k_kv4_attn<D, true, true, QT> : k_kv4_attn<D, false, true, QT>)
                            : (f16 ? k_kv4_attn<D, true, false, QT> : k_kv4_attn<D, false, false, QT>);
      };
      auto k = p.few.rb == 16 ? kernel.template operator()<1>() : kernel.template operator()<2>();
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
