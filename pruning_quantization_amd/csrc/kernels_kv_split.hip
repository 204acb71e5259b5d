// Sequences that are split along their tokens: the plan of the chunks, and the join
// of their partial results, for both kinds of key/value cache.
#include "kv_split.hpp"

namespace sparq24 {

// First units of more than kScanned sequences, a workgroup for each kernel: that each
// of their workgroups added them up took it a round of loads per 64 sequences, twice
// (4096 sequences of 100 tokens, one new each, with offsets: 2264 us, so 551).
__global__ __launch_bounds__(1024) void k_kv_plan(KvAttnArgs few, KvAttnArgs many) {
  const KvAttnArgs& w = blockIdx.x ? many : few;
  if (!w.starts) return;
  __shared__ int64_t part[1024];
  const int tid = threadIdx.x;
  const int64_t seqs = w.a.q.seqs, per = (seqs + 1023) / 1024;
  const int64_t b0 = tid * per < seqs ? tid * per : seqs, b1 = b0 + per < seqs ? b0 + per : seqs;
  auto scan = [&](int64_t v) {  // inclusive, over the workgroup
    part[tid] = v;
    for (int o = 1; o < 1024; o <<= 1) {
      __syncthreads();
      const int64_t u = tid >= o ? part[tid - o] : 0;
      __syncthreads();
      part[tid] += u;
    }
    __syncthreads();
    return part[tid];
  };
  int len = w.cmin;
  if (w.cmin < kNever) {
    int64_t c = 0;
#pragma unroll 4
    for (int64_t b = b0; b < b1; ++b) c += tiles_of(kv_work(w, seq_rows(w.a.q, b)));
    scan(c);
    len = chunk_tiles(w, part[1023]);
    __syncthreads();  // part is read before it is used again
  }
  int64_t n = 0;
#pragma unroll 4
  for (int64_t b = b0; b < b1; ++b) n += units_of(kv_work(w, seq_rows(w.a.q, b)), len);
  int64_t at = scan(n) - n;
  for (int64_t b = b0; b < b1; ++b) {
    w.starts[b] = (int)(at < INT32_MAX ? at : INT32_MAX);
    at += units_of(kv_work(w, seq_rows(w.a.q, b)), len);
  }
  if (tid == 1023) {
    w.starts[seqs] = (int)(at < INT32_MAX ? at : INT32_MAX);
    w.starts[seqs + 1] = len;
  }
}

// Joins the chunks of split sequences.  Few rows (W = 4), and so long chains of
// chunks: a workgroup per (token, query head), the chunks dealt to its four waves,
// whose sums meet in wave order.  Many (W = 0): 16 lanes per row, so that one round
// of waves holds them all (17500 rows of 64: 7.2 us, with a wave per row 14.6).
template <int D, int W>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs few, KvAttnArgs many) {
  constexpr int L = W == 4 ? 64 : 16, V = D / L, F = W == 4 ? V : 4;  // lanes of a row, elements of a lane, in runs of F
  const KvAttn& a = few.a;
  const int tid = threadIdx.x, wv = W == 4 ? uniform(tid >> 6) : 0, l = tid & (L - 1);
  const int64_t id = W == 4 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 16 + (tid >> 4);
  if (W != 4 && id >= a.q.total * a.heads) return;
  const int64_t tok = id / a.heads;
  const int hq = (int)(id % a.heads);
  int64_t seq = 0;
  if (a.q.cu) {  // last sequence that begins at or before the token
    int64_t lo = 0, hi = a.q.seqs;
    while (hi - lo > 1) {
      const int64_t mid = (lo + hi) / 2;
      if (a.q.cu[mid] <= tok) lo = mid;
      else hi = mid;
    }
    seq = lo;
  } else {
    seq = tok / a.q.nper;
  }
  const SeqRows r = seq_rows(a.q, seq);
  if (tok < r.first || tok >= (int64_t)r.first + r.n) return;  // in no sequence
  const KvAttnArgs& p = r.n * few.g <= few.most ? few : many;
  const int chunks = p.plan[2 * seq + 1];
  if (chunks < 2) return;
  const int row = (int)(tok - r.first) * p.g + hq % p.g;
  const int nrt = (r.n * p.g + p.rb - 1) / p.rb, rt = row / p.rb, rr = row % p.rb;
  const int head = hq / p.g;
  const int64_t first = p.plan[2 * seq];
  // Offsets that do not ascend can ask for more items than there is room for.  A sequence
  // that got none has no entry in the plan: what stands there is any number, also where
  // nothing was split.
  if (!p.ml || first < 0 || chunks > p.items) return;
  const int64_t units = first + (int64_t)chunks * nrt;
  if (units > p.items || units * a.c.heads > p.items) return;
  const int64_t at0 = ((first + nrt - 1 - rt) * a.c.heads + head) * p.rb + rr;
  const int64_t step = (int64_t)nrt * a.c.heads * p.rb;
  // the common reference: the largest sum's own exponent, so that no chunk's weight passes 2
  float top = kNegInf;
  for (int c = l; c < chunks; c += L) {
    const f32x2v ml = *(const f32x2v*)(p.ml + (at0 + c * step) * 2);
    top = __builtin_fmaxf(top, ml[0] + (float)((int)(__float_as_uint(ml[1]) >> 23) - 127));
  }
#pragma unroll
  for (int x = 1; x < L; x <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x, 64));
  float sum = 0.0f, v[V];
#pragma unroll
  for (int e = 0; e < V; ++e) v[e] = 0.0f;
  auto at = [&](int e) { return F * L * (e / F) + F * l + e % F; };
  if (top != kNegInf) {
#pragma unroll 4
    for (int c = wv; c < chunks; c += W == 4 ? 4 : 1) {
      const int64_t s = at0 + c * step;
      const f32x2v ml = *(const f32x2v*)(p.ml + s * 2);
      const float f = ml[1] * __builtin_amdgcn_exp2f(ml[0] - top);
      sum += f;
#pragma unroll
      for (int e = 0; e < V; ++e) v[e] = __builtin_fmaf(p.po[s * D + at(e)], f, v[e]);
    }
  }
  if constexpr (W == 4) {
    __shared__ float part[4][D], sums[4];
#pragma unroll
    for (int e = 0; e < V; ++e) part[wv][at(e)] = v[e];
    if (l == 0) sums[wv] = sum;
    __syncthreads();
    sum = sums[0] + sums[1] + sums[2] + sums[3];
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
    for (int d = tid; d < D; d += 256)
      kv_store_out(a, id * D + d, (part[0][d] + part[1][d] + part[2][d] + part[3][d]) * inv);
  } else {
    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
    for (int e = 0; e < V; ++e) kv_store_out(a, id * D + at(e), v[e] * inv);
  }
  if (a.lse && wv == 0 && l == 0) a.lse[id] = kv_lse(top, sum);
}

// Which kernels run, their row tiles and the room for split results, from what
// the host knows (shapes; lengths and offsets stay on the device).  Sequences of
// at most few_rows rows per kv head (query tokens times heads of the group) go to the
// few-rows kernel, the others to the prompt kernel; without offsets all have the
// same count, with offsets both may be needed.  (8 bits, 16 sequences of 4096 tokens, 4 kv
// heads of 128: 32 rows 32 us in the prompt kernel, 60 in the other with two row tiles a
// wave; 64 rows 39, and 108 with four.)
KvPlan kv_plan(const KvAttn& a, char* ws, int few_rows, int prompt_rows, int resident) {
  KvPlan p;
  const int g = a.heads / a.c.heads;
  const int64_t H = a.c.heads, rows = a.q.nper * g, cus = device_cu_count();
  p.run_few = a.q.cu || rows <= few_rows;
  p.run_many = a.q.cu ? a.q.total * g > few_rows : rows > few_rows;
  const int64_t tiles = (a.q.cap + kKvTile - 1) / kKvTile;
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  size_t off = up((size_t)a.q.seqs * 8);
  p.split = p.planned = false;
  auto lay = [&](KvAttnArgs& w, bool run, int rb, int above, int most, int cmin, int64_t target, int64_t rt) {
    w.a = a;
    w.g = g;
    w.rb = rb;
    w.above = above;
    w.most = most;
    w.target = target;
    const bool split = run && tiles > kWholeTiles && (most == few_rows || rt * H < target);
    w.cmin = split ? cmin : kNever;
    w.items = rt * H;
    w.plan = (int*)ws;
    w.starts = nullptr;
    w.round = INT64_MAX;
    if (run && a.q.seqs > kScanned && (a.q.cu || split)) {
      w.starts = (int*)(ws + off);
      off += up((size_t)(a.q.seqs + 2) * 4);
      p.planned = true;
    }
    if (split) {
      const int64_t all = rt * H * ((tiles + cmin - 1) / cmin);
      w.items = all < target + rt * H ? all : target + rt * H;
      w.ml = (float*)(ws + off);
      off += up((size_t)w.items * rb * 8);
      w.po = (float*)(ws + off);
      off += up((size_t)w.items * rb * a.c.dim * 4);
      p.split = true;
    } else {
      w.ml = w.po = nullptr;
    }
  };
  const int rbf = few_rows, rbm = prompt_rows;
  int64_t rtf = a.q.seqs * ((rows + rbf - 1) / rbf), rtm = a.q.seqs * ((rows + rbm - 1) / rbm);
  if (a.q.cu) {  // n rows make at most n / rb + 1 tiles
    rtf = a.q.total * g / rbf + a.q.seqs;
    const int64_t most = a.q.seqs, longer = a.q.total * g / few_rows;
    if (rtf > most) rtf = most;
    rtm = a.q.total * g / rbm + (longer < a.q.seqs ? longer : a.q.seqs);
  }
  // chunks even out ragged lengths, but the join walks them: at most 64 of a
  // sequence and head, at most eight items per CU (64 sequences of 300..16384
  // tokens: 248 / 227 / 219 us at two / four / eight; one of 131071: 61 / 65 / 80)
  int64_t aim = 64 * a.q.seqs * H;
  // Two row tiles a wave: three a CU (8 tokens on 64 sequences of 300..8192, 32 heads over 8,
  // MXFP4: 105 us, with two 119, with eight 113; on 32 of 2048: 37, 30, 57).
  const int64_t per = few_rows > 16 ? 3 : 8;
  aim = aim < 2 * cus ? 2 * cus : (aim > per * cus ? per * cus : aim);
  // A chunk has one tile a wave at least, and four where unsplit sequences fill the
  // card twice (64 sequences of 1024: 26 and 48 us with one; 8 of 2048: 21 and 17).  Two
  // where that still gives every CU two (16 sequences of 4096, 4 kv heads of 128: MXFP4 18.7
  // us, with one 21.2, e4m3 23.0 and 26.5; one of 8192, 8 heads: 14.0 and 13.1, 16.1 and
  // 14.7), and with two row tiles a wave (5 tokens, the 16 sequences: 23.9 and 31.9).
  const int64_t seen = a.window && a.window / kKvTile + 2 < tiles ? a.window / kKvTile + 2 : tiles;
  const int least = rtf * H >= 2 * cus ? 16 : (few_rows > 16 || rtf * H * seen >= 16 * cus ? 8 : 4);
  lay(p.few, p.run_few, rbf, 0, few_rows, least, aim, rtf);
  lay(p.many, p.run_many, rbm, few_rows, INT32_MAX, 4, resident * cus, rtm);
  // Causal row tiles that are all resident at once: a CU's second is dealt from the
  // shortest up (two prompts of 1024 tokens, 32 heads over 8 of 128, in MXFP4 and FP8: 34
  // and 44 us; the longest of the rest first, sequence by sequence, 45 and 60).
  if (!a.q.cu && p.many.cmin == kNever && rtm * H > cus && rtm * H <= resident * cus && cus % H == 0)
    p.many.round = cus / H;
  p.need = p.split || p.planned ? off : 0;
  if (!p.split) p.few.plan = p.many.plan = nullptr;
  return p;
}

bool kv_plan_fits(const KvAttn& a, const KvPlan& p, int threads) {
  return (!p.run_few || p.few.items <= kMostThreads / 256) && (!p.run_many || p.many.items <= kMostThreads / threads) &&
         (!p.split || a.q.total * a.heads <= kMostThreads / 16);
}

hipError_t launch_kv_starts(const KvPlan& p, hipStream_t s) {
  hipLaunchKernelGGL(k_kv_plan, dim3(2), dim3(1024), 0, s, p.few, p.many);
  return hipGetLastError();
}

hipError_t launch_kv_join(const KvPlan& p, hipStream_t s) {
  const KvAttn& a = p.few.a;
  const int64_t rows = a.q.total * a.heads;
  auto dim = [&]<int D>() {
    if (rows <= 16 * device_cu_count())
      hipLaunchKernelGGL((k_kv_join<D, 4>), dim3((unsigned)rows), dim3(256), 0, s, p.few, p.many);
    else
      hipLaunchKernelGGL((k_kv_join<D, 0>), dim3((unsigned)((rows + 15) / 16)), dim3(256), 0, s, p.few, p.many);
    return hipGetLastError();
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
