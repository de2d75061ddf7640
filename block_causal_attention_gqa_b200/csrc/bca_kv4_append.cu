// Writing to the 4-bit key/value cache, and reading a range of it back.
//
// Mathematics.  K^ = rot(k) / sqrt(mean_d k^2 + eps) and v are cut into blocks
// of 16 features; s = RN(max|x| / 6), c = RN(x / s) (bca_kv4.cuh).
//
// A code is a decision, so it must not hang on the last bits of the
// arithmetic.  For values it never does: v is bf16, max|v| / 6 and v / s are
// correctly rounded fp32 quotients, and no fp32 quotient of such operands
// rounds onto a border it does not lie on.  A key comes out of a rotation and a
// square root, so its fp32 value carries an error, which is bounded below by
// 2^-20 (|a| + |b|) r for the pair (a, b) that was rotated (sine and cosine are
// off by 2 ulp, the three roundings of the rotation by half an ulp of a
// product each, r by less than 8 ulp).  A row in which some x +- that bound
// falls on two codes, or some block maximum on two scales, is done again in
// fp64 by the whole warp; about one row in 300 is.  The codes are those of the
// exact definition but for values within 1e-14 of a border.
//
// Layout.  One warp takes a row of the value cache, which holds two tokens,
// for one head: their two keys and two values, lane l the features [l*E,
// l*E + E), E = D/32, as the key pre-pass of the forward does; a block's
// maximum is then over 16/E lanes.  With rotary angles a warp takes several
// heads, so that a sine and cosine serve them all.
//
// Bound: bytes (4 D read, D + D/8 written per token and head) for chunks;
// launch latency for single tokens.
#include <algorithm>

#include "bca_kv4.cuh"

namespace magi {
namespace kv4 {
namespace {

constexpr float kKeyErr = 9.5367431640625e-07f;   // 2^-20

template <int E>
__device__ __forceinline__ float block_max(float v) {
#pragma unroll
  for (int o = kBlock / E / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

template <int E>
__device__ __forceinline__ void load_row(const uint16_t* src, int lane, float (&x)[E]) {
  if constexpr (E == 4) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(src + lane * 4));
    x[0] = bf16_lo(w.x); x[1] = bf16_hi(w.x); x[2] = bf16_lo(w.y); x[3] = bf16_hi(w.y);
  } else {
    const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(src + lane * 2));
    x[0] = bf16_lo(w); x[1] = bf16_hi(w);
  }
}

// x / s, correctly rounded, from r = RN(1 / s) (Markstein's division: a
// quotient estimate and one residual step; the scale has 4 significant bits).
__device__ __forceinline__ float div_by_scale(float x, float s, float r) {
  const float q = x * r;
  return fmaf(fmaf(-q, s, x), r, q);
}

// NaN -> 0, and into the range the format holds.
__device__ __forceinline__ float tame(float x) {
  return x == x ? fminf(fmaxf(x, -kTopValue), kTopValue) : 0.f;
}

// Codes of a lane's E features (E/2 bytes) and the block's scale byte, from
// features that are exact (values).
template <int E>
__device__ __forceinline__ uint32_t encode_exact(const float (&x)[E], uint32_t& scale_byte) {
  float m = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) m = fmaxf(m, fabsf(x[e]));
  scale_byte = encode_scale(block_max<E>(m) / 6.f);
  const float s = scale_value(scale_byte);
  if (scale_byte == 0) return 0;
  const float r = __frcp_rn(s);
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < E; e += 2)
    codes |= encode2(div_by_scale(x[e], s, r), div_by_scale(x[e + 1], s, r)) << (4 * e);
  return codes;
}

// A key row in fp64 (by the whole warp; x holds the raw row): the rare rows
// whose codes the fp32 arithmetic cannot settle.
template <int D>
__device__ __noinline__ uint32_t encode_key_f64(const float* x, const float* ang, int lane, float eps,
                                                uint32_t* scale_byte) {
  constexpr int E = D / 32;
  double ss = 0.;
#pragma unroll
  for (int e = 0; e < E; ++e) ss += (double)x[e] * (double)x[e];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const double norm = sqrt(ss / D + (double)eps);
  double y[E], m = 0.;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    double v = x[e];
    const double other = __shfl_xor_sync(0xffffffffu, v, 16);
    if (ang != nullptr) {
      double sn, cs;
      sincos((double)__ldg(ang + (lane & 15) * E + e), &sn, &cs);
      v = lane < 16 ? v * cs - other * sn : v * cs + other * sn;
    }
    v /= norm;
    y[e] = v == v ? fmin(fmax(v, (double)-kTopValue), (double)kTopValue) : 0.;
    m = fmax(m, fabs(y[e]));
  }
#pragma unroll
  for (int o = kBlock / E / 2; o > 0; o >>= 1) m = fmax(m, __shfl_xor_sync(0xffffffffu, m, o));
  // the scale: round m / 6 to 4 significant bits, steps of 2^-17 below 2^-14
  const double want = m / 6.;
  uint32_t byte;
  if (want < 6.103515625e-05) {
    byte = (uint32_t)__double2int_rn(want * 131072.);
  } else {
    const int ex = ilogb(want);                              // 2^ex <= want
    const int mant = __double2int_rn(scalbn(want, 3 - ex));  // 8 .. 16
    byte = min((uint32_t)((ex + 15) * 8 + (mant - 8)), kTopScaleByte);
  }
  *scale_byte = byte;
  if (byte == 0) return 0;
  const double s = (double)scale_value(byte);
  uint32_t codes = 0;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const double a = fabs(y[e]) / s;
    const double step = a < 2. ? 0.5 : a < 4. ? 1. : 2.;
    const double t = fmin(rint(a / step) * step, 6.);
    const uint32_t c = t < 2. ? (uint32_t)(t * 2.) : t < 4. ? (uint32_t)t + 2u : (uint32_t)(t * 0.5) + 4u;
    codes |= (c | (y[e] < 0. ? 8u : 0u)) << (4 * e);
  }
  return codes;
}

// Codes and scale byte of one raw key row x (lane's E features); cs, sn: the
// lane's cosines and sines (rope only).
template <int D, bool kRope>
__device__ __forceinline__ uint32_t encode_key(const float (&x)[D / 32], const float (&cs)[D / 32],
                                               const float (&sn)[D / 32], const float* ang, int lane, float eps,
                                               uint32_t& scale_byte) {
  constexpr int E = D / 32;
  const float r = rms_inv<D>(warp_sumsq_row<E>(x), eps);
  float y[E], err[E], m = 0.f, me = 0.f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    float v = x[e], mag = fabsf(v);
    if constexpr (kRope) {
      const float o = __shfl_xor_sync(0xffffffffu, v, 16);
      mag += fabsf(o);
      v = lane < 16 ? rope_first(v, o, cs[e], sn[e]) : rope_second(o, v, cs[e], sn[e]);
    }
    y[e] = tame(v * r);
    err[e] = mag * r * kKeyErr;
    m = fmaxf(m, fabsf(y[e]));
    me = fmaxf(me, err[e]);
  }
  m = block_max<E>(m);
  me = block_max<E>(me);
  scale_byte = encode_scale(m / 6.f);
  // a row that is not finite ends here: r is 0 or NaN, y and err 0 or NaN
  bool unsure = encode_scale(fmaxf(m - me, 0.f) / 6.f) != encode_scale((m + me) / 6.f);
  const float s = scale_value(scale_byte);
  const float rs = scale_byte != 0 ? __frcp_rn(s) : 0.f;
  uint32_t codes = 0, low = 0, high = 0;
#pragma unroll
  for (int e = 0; e < E; e += 2) {
    const float q0 = y[e] * rs, q1 = y[e + 1] * rs, d0 = err[e] * rs, d1 = err[e + 1] * rs;
    codes |= encode2(q0, q1) << (4 * e);
    low |= encode2(q0 - d0, q1 - d1) << (4 * e);
    high |= encode2(q0 + d0, q1 + d1) << (4 * e);
  }
  // +0 and -0 stand for the same value
  unsure = unsure || (low != high && ((low ^ high) & 0x77777777u) != 0);
  if (__any_sync(0xffffffffu, unsure)) {
    codes = encode_key_f64<D>(x, kRope ? ang : nullptr, lane, eps, &scale_byte);
  }
  return scale_byte != 0 ? codes : 0u;
}

template <int D, bool kRope>
__global__ void __launch_bounds__(256) kv4_append_kernel(const AppendParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.z;
  const int n = p.counts != nullptr ? min(max(__ldg(p.counts + b), 0), p.n) : p.n;
  const int start = __ldg(p.start + b);
  const int H = p.c.heads, cap = p.c.cap;
  const int pair_of_warp = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5);
  // tokens t0, t0 + 1 of the call land in the two halves of cache row `row`
  const int64_t first_row = start >= 0 ? start / 2 : -((1 - (int64_t)start) / 2);   // floor
  const int64_t row = first_row + pair_of_warp;
  const int64_t t0 = 2 * row - start;
  bool live[2];
  bool outside = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t t = t0 + i, at = 2 * row + i;
    live[i] = t >= 0 && t < n;
    if (live[i] && (at < 0 || at >= cap)) {
      outside = true;
      live[i] = false;
    }
  }
  if (outside && lane == 0 && blockIdx.y == 0) atomicCAS(p.status, 0, (int)kErrPosition);
  if (!live[0] && !live[1]) return;

  float cs[2][E] = {}, sn[2][E] = {};
  const float* ang[2] = {nullptr, nullptr};
  if constexpr (kRope) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      ang[i] = p.rope + (int64_t)b * p.rope_stride + (live[i] ? t0 + i : t0 + 1 - i) * (D / 2);
#pragma unroll
      for (int e = 0; e < E; ++e) sincosf(__ldg(ang[i] + (lane & 15) * E + e), &sn[i][e], &cs[i][e]);
    }
  }
  const int h0 = blockIdx.y * p.heads_per_warp, h1 = min(h0 + p.heads_per_warp, H);
  for (int h = h0; h < h1; ++h) {
    float k[2][E], v[2][E];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // a half that is not written reads the other half's token
      const int64_t src = (((int64_t)b * p.n + (live[i] ? t0 + i : t0 + 1 - i)) * H + h) * D;
      load_row<E>(p.k + src, lane, k[i]);
      load_row<E>(p.v + src, lane, v[i]);
    }
    const int64_t bh = (int64_t)b * H + h;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t sb;
      const uint32_t codes = encode_key<D, kRope>(k[i], cs[i], sn[i], ang[i], lane, p.eps, sb);
      if (live[i]) {   // warp-uniform
        const int64_t at = bh * cap + 2 * row + i;
        if constexpr (E == 4)
          reinterpret_cast<uint16_t*>(p.c.kc + at * (D / 2))[lane] = (uint16_t)codes;
        else
          (p.c.kc + at * (D / 2))[lane] = (uint8_t)codes;
        if (lane % (kBlock / E) == 0) (p.c.ks + at * (D / kBlock))[lane / (kBlock / E)] = (uint8_t)sb;
      }
    }
    uint32_t vcodes[2], vsb[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = tame(v[i][e]);
      vcodes[i] = encode_exact<E>(v[i], vsb[i]);
    }
    // byte of feature e: token 2 row in the low half, token 2 row + 1 in the high half
    const int64_t vrow = bh * (cap / 2) + row;
    uint8_t* dst = p.c.vc + vrow * D + lane * E;
    uint8_t* sdst = p.c.vs + (vrow * (D / kBlock) + lane / (kBlock / E)) * 2;
    uint32_t bytes = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      bytes |= ((vcodes[0] >> (4 * e)) & 15u) << (8 * e);
      bytes |= ((vcodes[1] >> (4 * e)) & 15u) << (8 * e + 4);
    }
    const uint32_t keep = live[0] && live[1] ? 0u : live[0] ? 0xf0f0f0f0u : 0x0f0f0f0fu;
    if constexpr (E == 4) {
      uint32_t* d = reinterpret_cast<uint32_t*>(dst);
      *d = keep == 0 ? bytes : (*d & keep) | (bytes & ~keep);
    } else {
      uint16_t* d = reinterpret_cast<uint16_t*>(dst);
      *d = (uint16_t)(keep == 0 ? bytes : (*d & keep) | (bytes & ~keep));
    }
    if (lane % (kBlock / E) == 0) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        if (live[i]) sdst[i] = (uint8_t)vsb[i];
    }
  }
}

// bf16 values of E codes (E/2 bytes) of one scale.
template <int E>
__device__ __forceinline__ void store_values(uint16_t* dst, uint32_t codes, uint32_t scale, int lane) {
  if constexpr (E == 4) {
    uint2 w;
    w.x = f16x2_to_bf16x2(hmul2(codes_f16x2(codes & 0xffu), scale));
    w.y = f16x2_to_bf16x2(hmul2(codes_f16x2((codes >> 8) & 0xffu), scale));
    reinterpret_cast<uint2*>(dst)[lane] = w;
  } else {
    reinterpret_cast<uint32_t*>(dst)[lane] = f16x2_to_bf16x2(hmul2(codes_f16x2(codes & 0xffu), scale));
  }
}

// One warp per (batch element, token, head); a position outside the cache
// gives zeros.
template <int D>
__global__ void __launch_bounds__(256) kv4_read_kernel(const ReadParams p) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int H = p.c.heads, cap = p.c.cap;
  const int64_t rows = (int64_t)p.c.batch * p.n * H;
  const int64_t warps = (int64_t)gridDim.x * (blockDim.x / 32);
  for (int64_t r = (int64_t)blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); r < rows; r += warps) {
    const int h = (int)(r % H);
    const int64_t bt = r / H;
    const int b = (int)(bt / p.n);
    const int64_t at = (p.start != nullptr ? (int64_t)__ldg(p.start + b) : 0) + bt % p.n;
    uint32_t kc = 0, vc = 0, ks = 0, vs = 0;
    if (at >= 0 && at < cap) {
      const int64_t krow = ((int64_t)b * H + h) * cap + at, vrow = ((int64_t)b * H + h) * (cap / 2) + at / 2;
      const int blk = lane / (kBlock / E), half = (int)(at & 1);
      ks = p.c.ks[krow * (D / kBlock) + blk];
      vs = p.c.vs[(vrow * (D / kBlock) + blk) * 2 + half];
      if constexpr (E == 4) {
        kc = reinterpret_cast<const uint16_t*>(p.c.kc + krow * (D / 2))[lane];
        const uint32_t w = (reinterpret_cast<const uint32_t*>(p.c.vc + vrow * D)[lane] >> (4 * half)) & 0x0f0f0f0fu;
        vc = (w | (w >> 4)) & 0x00ff00ffu;   // codes 0, 1 in byte 0, codes 2, 3 in byte 2
        vc = (vc | (vc >> 8)) & 0xffffu;
      } else {
        kc = (p.c.kc + krow * (D / 2))[lane];
        const uint32_t w = (reinterpret_cast<const uint16_t*>(p.c.vc + vrow * D)[lane] >> (4 * half)) & 0x0f0fu;
        vc = (w | (w >> 4)) & 0xffu;
      }
    }
    store_values<E>(p.k + r * D, kc, scale_dup(ks), lane);
    store_values<E>(p.v + r * D, vc, scale_dup(vs), lane);
  }
}

}  // namespace

cudaError_t launch_append(const AppendParams& p0, cudaStream_t s) {
  AppendParams p = p0;
  if (p.n <= 0) return cudaSuccess;
  const int pairs = p.n / 2 + 1;   // rows of two tokens that n tokens can touch
  // A warp that takes several heads saves sines and cosines; with few tokens the
  // heads are spread over warps instead, for latency.
  p.heads_per_warp = p.rope != nullptr && (int64_t)pairs * p.c.batch >= 2048 ? 4 : 1;
  const dim3 grid((pairs + 7) / 8, (p.c.heads + p.heads_per_warp - 1) / p.heads_per_warp, p.c.batch);
  const bool rope = p.rope != nullptr;
  if (p.c.dim == 128) {
    if (rope) kv4_append_kernel<128, true><<<grid, 256, 0, s>>>(p);
    else kv4_append_kernel<128, false><<<grid, 256, 0, s>>>(p);
  } else {
    if (rope) kv4_append_kernel<64, true><<<grid, 256, 0, s>>>(p);
    else kv4_append_kernel<64, false><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

cudaError_t launch_read(const ReadParams& p, cudaStream_t s) {
  const int64_t rows = (int64_t)p.c.batch * p.n * p.c.heads;
  if (rows <= 0) return cudaSuccess;
  const int blocks = (int)std::min<int64_t>((rows + 7) / 8, 148 * 64);
  if (p.c.dim == 128) kv4_read_kernel<128><<<blocks, 256, 0, s>>>(p);
  else kv4_read_kernel<64><<<blocks, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace kv4
}  // namespace magi
