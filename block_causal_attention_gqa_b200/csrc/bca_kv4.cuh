// The number format of the 4-bit key/value cache, on the device.
//
// A value is c * s.  c is e2m1 (sign, 2 exponent bits, 1 mantissa bit; 0, 0.5,
// 1, 1.5, 2, 3, 4, 6), s the scale of its 16 neighbouring features in 8 bits:
// 5 exponent and 3 mantissa bits with fp16's exponent bias and no sign, so
// that (bits << 7) is the scale as an fp16 number, subnormals included.  A
// scale is at most 10240, so |c * s| <= 61440, and c * s has at most 6
// significant bits and is a multiple of 2^-18: every cached value is exact in
// fp16 and in bf16.  The attention kernels therefore read fp16 operands that
// carry no rounding of their own.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

#include "bca_kv4.h"
#include "bca_norm.cuh"
#include "sm100.cuh"

namespace magi {
namespace kv4 {

// Programmatic dependent launch.  A kernel launched with launch_early() may start
// while the kernel before it on the stream is ending, and waits for that
// kernel's end (and with it for all before) itself, before it reads or writes
// anything that the kernel before touches.  What the kernel before wrote may therefore change while the grid
// is on the device, so nothing is read through the read-only path (no __ldg).
// Not for kernels whose CTAs share the work out in equal parts: started into the
// gaps of a running kernel they land unevenly on the SMs (the weights of 4 x
// 92160 tokens took 61 us so, against 48).
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

constexpr int kBlock = 16;             // features that share a scale
constexpr float kTopScale = 10240.f;   // largest scale
constexpr uint32_t kTopScaleByte = 226;
constexpr float kTopValue = 6.f * kTopScale;

// Two codes (a byte; low half first) as an fp16 pair.
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t}\n" : "=r"(r) : "r"(byte));
  return r;
}

// The eight codes of a word as four fp16 pairs (byte i -> pair i).
__device__ __forceinline__ void codes_f16x8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3]) : "r"(w));
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// a times the low (high) half of s, which the multiplication takes as an operand modifier.
__device__ __forceinline__ uint32_t hmul2_low(uint32_t a, uint32_t s) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 t;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b32 t, {lo, lo};\n\tmul.rn.f16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(s));
  return r;
}
__device__ __forceinline__ uint32_t hmul2_high(uint32_t a, uint32_t s) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 t;\n\tmov.b32 {lo, hi}, %2;\n\tmov.b32 t, {hi, hi};\n\tmul.rn.f16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(a), "r"(s));
  return r;
}

// One scale byte in both halves of an fp16 pair.
__device__ __forceinline__ uint32_t scale_dup(uint32_t byte) { return byte * (0x10001u << 7); }

// The two scale bytes of a 16-bit word (low byte in the low half) as an fp16 pair.
__device__ __forceinline__ uint32_t scale_pair(uint32_t b2) { return __byte_perm(b2, 0, 0x4140) << 7; }

// fp16 pair -> bf16 pair; exact for cached values.
__device__ __forceinline__ uint32_t f16x2_to_bf16x2(uint32_t h) {
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&h));
  return sm100::pack_bf16x2(f.x, f.y);
}

// Two values -> two codes (lo in the low half of the byte), to nearest, ties
// to even, saturating at 6.
__device__ __forceinline__ uint32_t encode2(float lo, float hi) {
  uint32_t r;
  asm("{\n\t.reg .b8 t, z;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\t"
      "mov.b32 %0, {t, t, t, t};\n\t}\n" : "=r"(r) : "f"(lo), "f"(hi));
  return r & 0xffu;
}

// The scale byte of max|x| / 6 (v >= 0, finite), to nearest, ties to even.
// fp32 division followed by this rounding gives the correctly rounded
// quotient: the midpoints between scales have 5 significant bits, and an fp32
// numerator that is not 6 times such a midpoint has a quotient that differs
// from it by more than half an fp32 ulp.
__device__ __forceinline__ uint32_t encode_scale(float v) {
  if (v < 6.103515625e-05f) return (uint32_t)__float2int_rn(v * 131072.f);   // below 2^-14: steps of 2^-17
  const uint32_t b = __float_as_uint(v);
  const uint32_t r = (b + 0x7ffffu + ((b >> 20) & 1u)) >> 20;                 // exponent and 3 mantissa bits
  return min(r - (112u << 3), kTopScaleByte);
}

__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// `all` steps in n parts, the first all % n of them a step longer.  No more
// parts than get kLeast steps each.
template <int kLeast>
struct Parts {
  int n, size, longer;
  __device__ __forceinline__ Parts(int all, int ctas) {
    n = min(ctas, (all + kLeast - 1) / kLeast);
    size = n > 0 ? all / n : 0;
    longer = all - n * size;
  }
  __device__ __forceinline__ int begin(int i) const { return i >= n ? n * size + longer : i * size + min(i, longer); }
  __device__ __forceinline__ int of(int x) const {   // the part that holds step x
    const int head = longer * (size + 1);
    return x < head ? x / (size + 1) : longer + (x - head) / size;
  }
};

}  // namespace kv4
}  // namespace magi
