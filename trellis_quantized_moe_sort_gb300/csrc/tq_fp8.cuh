// 8-bit block-scaled values: the block's scale and the codes.
//
// 128 consecutive values of a row (or 128 rows x 128 of a matrix) share a 32-bit
// scale s = max|x| / 448, 448 the largest E4M3 value; a value is kept as e4m3(x / s).
// Both quotients are rounded to fp32 as a division rounds them, and the conversion
// to nearest even: 16-bit values often lie on a border of the E4M3 grid, where a
// product with a reciprocal falls to the other side.  NaN is kept as NaN and does
// not count for the maximum; an infinity counts as the largest finite number and is
// kept as 448.  In a block whose scale is 0 (no value but zeros, NaN or ones whose
// quotient by 448 underflows) all but NaN is kept as 0.
#pragma once
#include <cfloat>

#include "tq_device.cuh"
#include "tq_types.cuh"

namespace tq {

constexpr int kFp8Block = 128;
constexpr float kFp8Most = 448.f;

// Largest magnitude (fmaxf passes over NaN).
template <int kCount>
__device__ __forceinline__ float fp8_top(const float (&v)[kCount]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kCount; ++i) top = fmaxf(top, fabsf(v[i]));
  return fminf(top, FLT_MAX);
}

// a / b rounded to nearest from r = 1 / b: q0 = a r is within an ulp of the quotient,
// a - q0 b exact in an FMA, and q0 + r (a - q0 b) the rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// That holds while nothing under- or overflows on the way: b within 2^-80 .. 2^100,
// and quotients, here at most 449, that matter for E4M3 (2^-11 and more) then have
// remainders of at least 2^-137, above fp32's smallest 2^-149.  Infinities come with
// b = FLT_MAX / 448 and take the division.
struct Fp8Scale {
  float s, r;
  bool fast;
  __device__ __forceinline__ explicit Fp8Scale(float top) {
    s = __fdiv_rn(top, kFp8Most);
    r = __frcp_rn(s);
    fast = s >= 0x1p-80f && s <= 0x1p100f;
  }
  __device__ __forceinline__ float divide(float v) const {
    if (fast) {
      const float q = __fmul_rn(v, r);
      return __fmaf_rn(__fmaf_rn(-q, s, v), r, q);
    }
    return s > 0.f ? __fdiv_rn(v, s) : v == v ? 0.f : v;
  }
};

// Four E4M3 codes, the first lowest (saturating; NaN is 0x7f).
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n\t"
      "mov.b32 %0, {l, h};\n\t}"
      : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Two E4M3 codes (low byte first) as fp32.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(two)));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The codes of 16 values.
__device__ __forceinline__ uint4 fp8_codes16(const float* v, const Fp8Scale& s) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = e4m3x4(s.divide(v[4 * i]), s.divide(v[4 * i + 1]), s.divide(v[4 * i + 2]), s.divide(v[4 * i + 3]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace tq
