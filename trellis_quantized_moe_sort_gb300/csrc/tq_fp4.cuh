// 4-bit microscaled values: the block quantiser and the layouts it writes.
//
// A block of B values along a row (16 for TQ_FP4_NV, 32 for TQ_FP4_MX) shares
// one 8-bit scale; a value is kept as E2M1 (0, .5, 1, 1.5, 2, 3, 4, 6 and a
// sign), two to a byte, the even one in the low half.
//   NV: scale s = e4m3(max|x| / (6 g)), g a 32-bit scale of the whole tensor;
//       value = e2m1(x / (s g)).
//   MX: scale s = 2^(floor(log2 max|x|) - 2) as E8M0; value = e2m1(x / s).
// Roundings are to nearest even and saturate.  NaN is kept as 0 and does not
// count for the maximum; an infinity counts as the largest finite number.  A
// block whose scale is 0 (all zeros, below E4M3's range, or g not positive) is
// kept as zeros.
#pragma once
#include "tq_device.cuh"
#include "tq_types.cuh"

namespace tq {

constexpr int kFp4Step = 256;   // values of a row per pipeline step: one 128-byte swizzle row

__host__ __device__ constexpr int fp4_block(int fmt) { return fmt == TQ_FP4_NV ? 16 : 32; }
// Bytes of block scales that 128 rows take per kFp4Step values, in the tiled
// layout: 512-byte tiles of 128 rows x 4 blocks, byte (row % 32) * 16 +
// (row / 32) * 4 + block % 4 -- what one 32 x 128-bit copy into tensor memory
// takes and the block-scaled MMA reads.
__host__ __device__ constexpr int fp4_scale_step_bytes(int fmt) { return 128 * (kFp4Step / fp4_block(fmt)); }
// Tensor-memory columns of a step's scales: 4 a tile for the weights, 8 for up
// to 256 activation rows.
__host__ __device__ constexpr int fp4_scale_columns(int fmt) { return fp4_scale_step_bytes(fmt) / 512 * 12; }
__host__ __device__ constexpr int fp4_steps(int K) { return (K - 1) / kFp4Step + 1; }   // K >= 1, up to 2^31 - 1

// Offset of block `b`'s scale of row `r` inside a tiled scale matrix of
// 128-row groups with `steps` steps each.
__host__ __device__ constexpr size_t fp4_tiled_offset(int fmt, int steps, long long r, int b) {
  return static_cast<size_t>(r / 128) * steps * fp4_scale_step_bytes(fmt) + static_cast<size_t>(b / 4) * 512 +
         (r % 32) * 16 + ((r % 128) / 32) * 4 + b % 4;
}

// Eight E2M1 codes of v[0..8) in a word, v[0] lowest.
__device__ __forceinline__ uint32_t e2m1x8(const float* v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

__device__ __forceinline__ uint32_t to_e4m3(float v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(v));
  return r & 0xffu;
}
__device__ __forceinline__ float from_e4m3(uint32_t byte) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
  return __half2float(__ushort_as_half(static_cast<uint16_t>(h & 0xffffu)));
}
// 2^(byte - 127), byte 0 the subnormal 2^-127, byte 255 NaN; through bf16, which
// has fp32's exponents.
__device__ __forceinline__ float from_e8m0(uint32_t byte) {
  uint32_t two;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(byte)));
  return __uint_as_float(two << 16);
}
template <int kFmt>
__device__ __forceinline__ float fp4_scale_value(uint32_t byte) {
  return kFmt == TQ_FP4_NV ? from_e4m3(byte) : from_e8m0(byte);
}

// NaN to 0, infinities to the largest finite number.
__device__ __forceinline__ float finite(float v) {
  return v == v ? fminf(fmaxf(v, -3.402823466e38f), 3.402823466e38f) : 0.f;
}

// Largest magnitude of 16 values after `finite`; the values are only rewritten
// when one of them is not finite.
__device__ __forceinline__ float fp4_max16(float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);   // orders magnitudes, NaN highest
  if (m >= 0x7f800000u) {
    m = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      v[i] = finite(v[i]);
      m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    }
  }
  return __uint_as_float(m);
}

// 16 consecutive values of a row (16-byte aligned) as they are in memory, and their fp32 form with the largest
// magnitude.  16-bit types find it two values at a time, as integers.
template <typename T>
struct Piece {
  uint4 raw[sizeof(T)];
};
template <typename T>
__device__ __forceinline__ Piece<T> load_piece(const T* __restrict__ p) {
  Piece<T> r;
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)); ++i) r.raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  return r;
}
template <typename T>
__device__ __forceinline__ float open_piece(const Piece<T>& r, float (&v)[16]) {
  const T* const t = reinterpret_cast<const T*>(r.raw);
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = widen(t[i]);
  if constexpr (sizeof(T) == 2) {
    constexpr uint32_t kInf = std::is_same_v<T, __half> ? 0x7c00u : 0x7f80u;
    const uint32_t* const w = reinterpret_cast<const uint32_t*>(r.raw);
    uint32_t m = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __vmaxu2(m, w[i] & 0x7fff7fffu);
    const uint32_t top = max(m & 0xffffu, m >> 16);
    if (top >= kInf) return fp4_max16(v);
    const uint16_t bits = static_cast<uint16_t>(top);
    T value;
    memcpy(&value, &bits, 2);
    return widen(value);
  } else {
    return fp4_max16(v);
  }
}

// a / b rounded to nearest, r = 1 / b rounded to nearest.  q0 = a r is within an
// ulp of the quotient, its remainder a - q0 b exact in an FMA, and q0 + r (a - q0
// b) the correctly rounded quotient (Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990).  That wants no over-
// or underflow on the way: b well inside the exponent range and a quotient that
// is not huge (`fits`).  A remainder that underflows belongs to a quotient far
// below anything that the roundings after it can tell from 0.
__device__ __forceinline__ bool divides_fast(float largest, float b) {
  return b >= 0x1p-100f && b <= 0x1p100f && largest <= 0x1p20f * b;
}
__device__ __forceinline__ float divide_fast(float a, float b, float r) {
  const float q0 = __fmul_rn(a, r);
  return __fmaf_rn(__fmaf_rn(-q0, b, a), r, q0);
}

// The global scale as the quantisers use it: g, 6 g and 1 / (6 g).  Where g is
// not positive (of an all-zero tensor it is often 0, and 0 / 0 would be NaN) an
// infinite divisor makes every block scale 0.
struct GlobalScale {
  float g, six, r_six;
  __device__ __forceinline__ explicit GlobalScale(const float* p) : g(p ? *p : 1.f) {
    six = g > 0.f ? __fmul_rn(6.f, g) : INFINITY;
    r_six = __frcp_rn(six);
  }
};

// Scale byte of a block whose largest magnitude is `top`; *d = the divisor of
// its values, *r its reciprocal.
template <int kFmt>
__device__ __forceinline__ uint32_t fp4_block_scale(float top, const GlobalScale& g, float* d, float* r) {
  if (kFmt == TQ_FP4_NV) {
    const uint32_t byte =
        to_e4m3(divides_fast(top, g.six) ? divide_fast(top, g.six, g.r_six) : __fdiv_rn(top, g.six));
    *d = __fmul_rn(from_e4m3(byte), g.g);
    *r = __frcp_rn(*d);
    return byte;
  }
  // floor(log2 top) from the exponent field; the smallest scale serves all
  // subnormals and everything below 2^-125
  const int e = static_cast<int>(__float_as_uint(top) >> 23);
  const uint32_t byte = static_cast<uint32_t>(max(e - 2, 0));
  *d = from_e8m0(byte);
  *r = __uint_as_float((254u - byte) << 23);   // byte <= 252
  return byte;
}

// 16 codes of v / d (d = 0: zeros), |v| <= top, r = 1 / d, each quotient rounded
// as a division rounds it.  MX: d is a power of two and v r exact (a product
// below the normal range is far below the first midpoint).
template <int kFmt>
__device__ __forceinline__ uint2 fp4_codes16(const float (&v)[16], float d, float r, float top) {
  if (!(d > 0.f)) return make_uint2(0u, 0u);
  float q[16];
  if (kFmt == TQ_FP4_MX) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = v[i] * r;
  } else if (divides_fast(top, d)) {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = divide_fast(v[i], d, r);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) q[i] = __fdiv_rn(v[i], d);
  }
  return make_uint2(e2m1x8(q), e2m1x8(q + 8));
}

}  // namespace tq
