// Root-mean-square norm of rows, with the residual's addition in front and the
// quantizer of the next product behind it: what every projection of a layer starts
// from [PD §2: the quantized side pays its online quantization].
//   h = x (+ residual, rounded once to their type, and written)
//   r = fp32(1 / sqrt(sum h^2 / K + eps)), fp64 inside
//   y = fp32(fp32(h r) w), quantized as kernels_quant.hip does
// The squares are exact in fp64 (fp32's 48 bits too) and their sum is as good as
// exact, so the codes do not depend on how a row is dealt out.
#include "dispatch.hpp"
#include "launch_serving.hpp"

namespace sparq24 {

__device__ inline char* norm_row(const NormRows& n, int64_t row) {
  if (n.bs == n.R * n.rs) return n.x + row * n.rs;
  const int64_t b = row / n.R;
  return n.x + b * n.bs + (row - b * n.R) * n.rs;
}

// fp32(a + b) of the elements, rounded to the storage type.
template <class DT>
__device__ inline Unit<DT> add_units(const Unit<DT>& a, const Unit<DT>& b) {
  Unit<DT> s;
  if constexpr (DT::ESIZE == 4) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s.w[i] = __float_as_uint(a.f(i) + b.f(i));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float lo = a.f(2 * i) + b.f(2 * i), hi = a.f(2 * i + 1) + b.f(2 * i + 1);
      if constexpr (DT::IS_BF16) {
        typedef __bf16 t2 __attribute__((ext_vector_type(2)));
        s.w[i] = __builtin_bit_cast(uint32_t, t2{(__bf16)lo, (__bf16)hi});
      } else {
        typedef _Float16 t2 __attribute__((ext_vector_type(2)));
        s.w[i] = __builtin_bit_cast(uint32_t, t2{(_Float16)lo, (_Float16)hi});
      }
    }
  }
  return s;
}

template <class DT>
__device__ inline void store_unit(void* p, const Unit<DT>& u) {
  st4(p, u.w[0], u.w[1], u.w[2], u.w[3]);
  if constexpr (DT::W == 8) st4((char*)p + 16, u.w[4], u.w[5], u.w[6], u.w[7]);
}

constexpr uint32_t kInfBits = 0x7F800000u;  // bits of |y| from here on: no finite number

// A team of TEAM lanes holds a row in registers from its one read to its codes, UPL units of
// 8 elements a lane; the weights are read again for the codes, from cache.  The rows' bytes
// bound it: 16384 x 4096 in bf16 with a residual to e4m3, 470 MB, 80 us, 5.85 TB/s; to MXFP4,
// 439 MB, 72 us.  One such row takes 3.5 us: the launch and a chain of loads, each waited for
// before the next is asked for: the row, its residual unit by unit, and behind each of the two
// reductions the weights unit by unit (MXFP4 has one), though they do not depend on the row.
template <class DT, class WT, int TEAM, int UPL>
__global__ __launch_bounds__(kBlock) void k_rmsnorm(RmsNorm n) {
  __shared__ double sums[kBlock / 64];
  __shared__ uint32_t red[kBlock / 64];
  const int t = threadIdx.x % TEAM;
  const int64_t at = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * (kBlock / TEAM) + threadIdx.x / TEAM;
  const bool act = at < n.rows;
  const int64_t row = act ? at : n.rows - 1;  // teams past the end run along
  const char* x = norm_row(n.x, row);
  const char* res = n.res.x ? norm_row(n.res, row) : nullptr;
  auto place = [&](int j) { return (int64_t)j * TEAM + t; };
  Unit<DT> h[UPL];
#pragma unroll
  for (int j = 0; j < UPL; ++j) {
    if (place(j) < n.nunits) load_unit(h[j], x + place(j) * (8 * DT::ESIZE));
    else zero_unit(h[j]);
  }
  if (res) {
    char* sum = norm_row(n.sum, row);
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      if (place(j) >= n.nunits) continue;
      Unit<DT> r;
      load_unit(r, res + place(j) * (8 * DT::ESIZE));
      h[j] = add_units(h[j], r);
    }
#pragma unroll
    for (int j = 0; j < UPL; ++j)
      if (act && place(j) < n.nunits) store_unit(sum + place(j) * (8 * DT::ESIZE), h[j]);
  }
  double ss = 0.0;
#pragma unroll
  for (int j = 0; j < UPL; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = h[j].f(e);
      ss = __builtin_fma(v, v, ss);
    }
  ss = team_sum_f64<TEAM>(ss, sums);
  const double mean = ss / (double)(8 * n.nunits) + (double)n.eps;
  // an element that is no finite number makes the row NaN
  float r = mean > 0.0 ? (float)(1.0 / __builtin_sqrt(mean)) : 0.0f;
  r = __builtin_isfinite(mean) ? r : __builtin_nanf("");

  auto value = [&](int j, const Unit<WT>& w, float(&y)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = h[j].f(e) * r * w.f(e);
  };
  auto largest = [](const float(&y)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t a = __float_as_uint(y[e]) & 0x7FFFFFFFu;
      m = m > a ? m : a;
    }
    return m;
  };
  auto weight = [&](int j) {
    Unit<WT> w;
    const char* p = (const char*)n.w + (place(j) < n.nunits ? place(j) : 0) * (8 * WT::ESIZE);
#pragma unroll
    for (int i = 0; i < WT::W / 4; ++i) {  // read by every row: no streaming hint
      const uint4 v = *(const uint4*)(p + 16 * i);
      w.w[4 * i] = v.x, w.w[4 * i + 1] = v.y, w.w[4 * i + 2] = v.z, w.w[4 * i + 3] = v.w;
    }
    return w;
  };
  if (n.cfmt == CF_MX) {
#pragma unroll
    for (int j = 0; j < UPL; ++j) {
      float y[8];
      value(j, weight(j), y);
      uint32_t am = largest(y), w = xor_lane32<1>(am);
      am = am > w ? am : w;
      w = xor_lane32<2>(am);
      am = am > w ? am : w;
      const bool fine = am < kInfBits;
      const int e = fine ? mx_exponent(am) : 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = fine ? __builtin_ldexpf(y[i], -e) : 0.0f;
      const uint32_t pk = enc_e2m1_x8(y);
      if (act && place(j) < n.nunits) {
        st((uint32_t*)n.codes + row * n.nunits + place(j), pk);
        if ((t & 3) == 0)
          st((uint8_t*)n.scales + row * (n.nunits / 4) + (place(j) >> 2), (uint8_t)(fine ? e + 127 : 255));
      }
    }
    return;
  }
  uint32_t am = 0;
#pragma unroll
  for (int j = 0; j < UPL; ++j) {
    float y[8];
    value(j, weight(j), y);
    const uint32_t a = place(j) < n.nunits ? largest(y) : 0;
    am = am > a ? am : a;
  }
  am = team_max_u32<TEAM>(am, red);
  const bool fine = am < kInfBits;
  float s, inv;
  row_scale(fine ? __uint_as_float(am) : 0.0f, n.qmax, s, inv);
#pragma unroll
  for (int j = 0; j < UPL; ++j) {
    if (!act || place(j) >= n.nunits) continue;
    float y[8];
    value(j, weight(j), y);
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = fine ? y[e] * inv : 0.0f;
    uint32_t lo, hi;
    if (n.cfmt == CF_FP8) {
      lo = enc_e4m3_x4(y[0], y[1], y[2], y[3]);
      hi = enc_e4m3_x4(y[4], y[5], y[6], y[7]);
    } else {
      uint32_t c[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) c[e] = __float_as_uint(int_round_magic(y[e], n.qmax));
      lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[3], c[2], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u), 0x05040100u);
      hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(c[7], c[6], 0x0c0c0400u),
                                 __builtin_amdgcn_perm(c[5], c[4], 0x0c0c0400u), 0x05040100u);
    }
    st2(n.codes + (row * n.nunits + place(j)) * 8, lo, hi);
  }
  if (act && t == 0) ((float*)n.scales)[row] = fine ? s : __builtin_nanf("");
}

hipError_t launch_rmsnorm_quantize(const RmsNorm& n, hipStream_t s) {
  return with_dtype(n.dtype, [&]<class DT>() {
    auto go = [&]<class WT, int TEAM, int UPL>() {
      // more workgroups than a grid has along x (64 heads of 1M tokens) in as many lines as it takes
      const int64_t per = kBlock / TEAM, all = (n.rows + per - 1) / per, most = kMostThreads / kBlock;
      const int64_t lines = (all + most - 1) / most;
      hipLaunchKernelGGL((k_rmsnorm<DT, WT, TEAM, UPL>), dim3((unsigned)((all + lines - 1) / lines), (unsigned)lines),
                         dim3(kBlock), 0, s, n);
      return hipGetLastError();
    };
    // Up to 1024 elements a wave per row, from there on a workgroup: with a residual to e4m3,
    // 16384 rows / one of 512 elements 13.7 / 2.4 us by a wave and 29.8 / 2.6 by a workgroup,
    // of 1024 23.6 / 3.2 and 34.3 / 2.7, of 2048 44.0 / 4.6 and 45.9 / 2.8, of 4096 99.3 / 7.6
    // and 79.6 / 3.6.
    auto shape = [&]<class WT>() {
      if (n.nunits <= 64) return go.template operator()<WT, 64, 1>();
      if (n.nunits <= 128) return go.template operator()<WT, 64, 2>();
      if (n.nunits <= 256) return go.template operator()<WT, 256, 1>();
      if (n.nunits <= 512) return go.template operator()<WT, 256, 2>();
      if (n.nunits <= 1024) return go.template operator()<WT, 256, 4>();
      if (n.nunits <= 2048) return go.template operator()<WT, 256, 8>();
      if (n.nunits <= 4096) return go.template operator()<WT, 256, 16>();
      return hipErrorInvalidValue;
    };
    if constexpr (DT::ESIZE == 2) {
      if (n.wdtype == n.dtype) return shape.template operator()<DT>();
    }
    return shape.template operator()<F32T>();
  });
}

}  // namespace sparq24
