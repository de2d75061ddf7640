// Rows of bf16 features in registers, 16 features (one scale's block) a lane,
// D/16 lanes a row: what appending keys and folding queries have in common.
#pragma once
#include "bca_kv4.cuh"

namespace magi {
namespace kv4 {

// Sine and cosine of an angle of up to 10^9.  Cody and Waite's reduction by
// multiples of pi/2 (in two fp32 constants below 10^5, where k pi/2's first
// product leaves an exact difference; in fp64 above), then the Taylor series up
// to r^9 and r^10 on |r| <= pi/4 (remainders 2e-9 and 1.2e-10).  Off by less than
// 2^-23.  A third of the instructions of sincosf, and no branches the warp has
// to reconverge after.
__device__ __forceinline__ void sincos_quarter(float r, uint32_t quadrant, float& sn, float& cs) {
  const float z = r * r;
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);
  s = fmaf(z, s, 8.3333333e-3f);
  s = fmaf(z, s, -1.6666667e-1f);
  s = fmaf(z * r, s, r);
  float c = fmaf(z, -2.7557319e-7f, 2.4801587e-5f);
  c = fmaf(z, c, -1.3888889e-3f);
  c = fmaf(z, c, 4.1666667e-2f);
  c = fmaf(z, c, -0.5f);
  c = fmaf(z, c, 1.f);
  const bool odd = quadrant & 1u;
  const float a = odd ? c : s, b = odd ? s : c;
  sn = __uint_as_float(__float_as_uint(a) ^ ((quadrant & 2u) << 30));
  cs = __uint_as_float(__float_as_uint(b) ^ (((quadrant + 1u) & 2u) << 30));
}

template <int N>
__device__ __forceinline__ void sincos_row(const float (&x)[N], float (&sn)[N], float (&cs)[N]) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e) top = fmaxf(top, fabsf(x[e]));
  if (__all_sync(0xffffffffu, top < 1e5f)) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float t = fmaf(x[e], 0.636619772f, 12582912.f);   // 2/pi, and 1.5 * 2^23
      const float k = t - 12582912.f;
      const float r = fmaf(-k, -4.37113883e-8f, fmaf(-k, 1.57079637f, x[e]));
      sincos_quarter(r, __float_as_uint(t), sn[e], cs[e]);
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const double k = rint((double)x[e] * 0.63661977236758134308);
      const double r = fma(-k, 6.123233995736766e-17, fma(-k, 1.5707963267948966, (double)x[e]));
      sincos_quarter((float)r, (uint32_t)(int64_t)k, sn[e], cs[e]);
    }
  }
}

// The same in fp64 (Taylor up to r^19 and r^18: remainders below 1e-18).
__device__ __forceinline__ void sincos_f64(double x, double& sn, double& cs) {
  const double k = rint(x * 0.63661977236758134308);
  const double r = fma(-k, 6.123233995736766e-17, fma(-k, 1.5707963267948966, x));
  const double z = r * r;
  double s = -1. / 121645100408832000., c = -1. / 6402373705728000.;   // 1/19!, 1/18!
  s = fma(s, z, 1. / 355687428096000.);
  c = fma(c, z, 1. / 20922789888000.);
  s = fma(s, z, -1. / 1307674368000.);
  c = fma(c, z, -1. / 87178291200.);
  s = fma(s, z, 1. / 6227020800.);
  c = fma(c, z, 1. / 479001600.);
  s = fma(s, z, -1. / 39916800.);
  c = fma(c, z, -1. / 3628800.);
  s = fma(s, z, 1. / 362880.);
  c = fma(c, z, 1. / 40320.);
  s = fma(s, z, -1. / 5040.);
  c = fma(c, z, -1. / 720.);
  s = fma(s, z, 1. / 120.);
  c = fma(c, z, 1. / 24.);
  s = fma(s, z, -1. / 6.);
  c = fma(c, z, -1. / 2.);
  s = fma(s * z, r, r);
  c = fma(c, z, 1.);
  const int64_t q = (int64_t)k;
  const double a = (q & 1) ? c : s, b = (q & 1) ? s : c;
  sn = (q & 2) ? -a : a;
  cs = ((q + 1) & 2) ? -b : b;
}

// Lane li of a row's D/16: features 16 li .. 16 li + 15.
template <int D>
struct RowLanes {
  static constexpr int kLanes = D / 16;
  static constexpr int kRows = 32 / kLanes;   // rows a warp holds
};

__device__ __forceinline__ void load_block(const uint16_t* src, float (&x)[16]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 w = *(reinterpret_cast<const uint4*>(src) + i);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[8 * i + 2 * k] = bf16_lo(v[k]);
      x[8 * i + 2 * k + 1] = bf16_hi(v[k]);
    }
  }
}

// The row's angles that the lane's features turn by.
template <int D>
__device__ __forceinline__ void load_angles(const float* row, int li, float (&a)[16]) {
  const float4* src = reinterpret_cast<const float4*>(row + li % (D / 32) * 16);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = *(src + i);
    a[4 * i] = v.x; a[4 * i + 1] = v.y; a[4 * i + 2] = v.z; a[4 * i + 3] = v.w;
  }
}

// 1 / RMS of the row, in all its lanes (at most 9 roundings in the sum).
template <int D>
__device__ __forceinline__ float row_rms_inv(const float (&x)[16], float eps) {
  float s[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] = x[i] * x[i];
#pragma unroll
  for (int i = 4; i < 16; ++i) s[i & 3] = fmaf(x[i], x[i], s[i & 3]);
  float t = (s[0] + s[1]) + (s[2] + s[3]);
#pragma unroll
  for (int o = 1; o < RowLanes<D>::kLanes; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return rms_inv<D>(t, eps);
}

// x turned by the angles; mag (|a| + |b| of each pair) bounds the rounding.
template <int D>
__device__ __forceinline__ void rope_block(float (&x)[16], const float (&sn)[16], const float (&cs)[16], int li,
                                           float (&mag)[16]) {
  constexpr int half = D / 32;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const float o = __shfl_xor_sync(0xffffffffu, x[e], half);   // the other feature of the pair
    mag[e] = fabsf(x[e]) + fabsf(o);
    x[e] = fmaf(li < half ? -o : o, sn[e], x[e] * cs[e]);
  }
}

}  // namespace kv4
}  // namespace magi
