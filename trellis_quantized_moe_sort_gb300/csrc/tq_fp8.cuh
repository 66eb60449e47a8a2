// 8-bit block-scaled values: the block's scale and the codes.
//
// 128 consecutive values of a row (or 128 rows x 128 of a matrix) share a 32-bit
// scale s = max|x| / 448, 448 the largest E4M3 value; a value is kept as e4m3(x / s).
// Both quotients are rounded to fp32 as a division rounds them, and the conversion
// to nearest even: 16-bit values often lie on a border of the E4M3 grid, where a
// product with a reciprocal falls to the other side.  NaN is kept as NaN and does
// not count for the maximum; an infinity counts as the largest finite number and is
// kept as 448.  Zeros, and values that round to 0, keep their sign.  In a block whose scale
// is 0 (no value but zeros, NaN or ones whose quotient by 448 underflows) all but NaN is
// kept as 0.
#pragma once
#include <cfloat>

#include "tq_device.cuh"
#include "tq_types.cuh"

namespace tq {

constexpr int kFp8Block = 128;
constexpr float kFp8Most = 448.f;

// Two fp32 operations an instruction, each rounded by itself.
__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __ffma2_rn(b, make_float2(-1.f, -1.f), a); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 fma2_down(float2 a, float2 b, float2 c) { return __ffma2_rd(a, b, c); }

// Largest magnitude; NaN is passed over.
template <int kCount>
__device__ __forceinline__ float fp8_top(const float (&v)[kCount]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kCount; i += 2)
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(v[i]), "f"(v[i + 1]));
  return fminf(top, FLT_MAX);
}

// a / b rounded to nearest from r = 1 / b (rounded): q0 = a r is within an ulp of the quotient,
// a - q0 b exact in an FMA, and q0 + r (a - q0 b) the rounded quotient (Markstein,
// "Computation of elementary functions on the IBM RISC System/6000 processor", 1990).
// That holds while nothing under- or overflows on the way: b within 2^-80 .. 2^100,
// and quotients, here at most 449, that matter for E4M3 (2^-11 and more) then have
// remainders of at least 2^-137, above fp32's smallest 2^-149.  Infinities come with
// b = FLT_MAX / 448 and take the division.  A remainder of 0 is -0 by its rounding down,
// which leaves a quotient of -0 its sign.
__device__ __forceinline__ float fp8_divide(float a, float b, float r) {
  const float q = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rd(-q, b, a), r, q);
}
struct Fp8Scale {
  float s, r;
  bool fast;
  __device__ __forceinline__ explicit Fp8Scale(float top) {
    constexpr float kInverse = 1.f / 448.f;   // rounded to nearest
    s = top >= 0x1p-70f && top <= 0x1p100f ? fp8_divide(top, kFp8Most, kInverse) : __fdiv_rn(top, kFp8Most);
    r = __frcp_rn(s);
    fast = s >= 0x1p-80f && s <= 0x1p100f;
  }
};

// Four values over the scale by divisions.
static __device__ __noinline__ float4 fp8_divide_slow(float4 v, float s) {
  float q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll 1
  for (int i = 0; i < 4; ++i) q[i] = s > 0.f ? __fdiv_rn(q[i], s) : q[i] == q[i] ? 0.f : q[i];
  return make_float4(q[0], q[1], q[2], q[3]);
}

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
  if (s.fast) {
    const float2 r = make_float2(s.r, s.r), minus = make_float2(-s.s, -s.s);
    float2 q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {   // fp8_divide, two at a time
      const float2 a = make_float2(v[2 * i], v[2 * i + 1]);
      q[i] = mul2(a, r);
      q[i] = fma2(fma2_down(q[i], minus, a), r, q[i]);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = e4m3x4(q[2 * i].x, q[2 * i].y, q[2 * i + 1].x, q[2 * i + 1].y);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 q = fp8_divide_slow(make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]), s.s);
      w[i] = e4m3x4(q.x, q.y, q.z, q.w);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace tq
