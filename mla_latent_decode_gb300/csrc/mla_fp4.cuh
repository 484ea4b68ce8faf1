// mla_fp4.cuh -- the 4-bit latent row (MLA_KV_FP4_E2M1 in include/mla_decode.h)
// and the conversions between its codes and fp32 / f16 values.
//
// A row of MLA_FP4_ROW_BYTES = 352 bytes:
//   [0, 256)    E2M1 codes of c_kv, element 2i in the low half of byte i
//   [256, 288)  E4M3 scales, one per block of 16 elements
//   [288, 352)  E4M3 codes of the RoPE key
// An E2M1 code times an E4M3 scale has at most 6 significant bits and a
// magnitude in [2^-10, 2688], and an E4M3 code 4 bits in [2^-9, 448]: both are
// exact in f16, so the tensor cores multiply exactly what is stored and the
// pool's fp32 factor g stays outside the contractions.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "mla_internal.h"

namespace mla {

constexpr int kFp4ScaleOff = MLA_NOPE_DIM / 2;                    // 256
constexpr int kFp4RopeOff = kFp4ScaleOff + MLA_NOPE_DIM / 16;     // 288
constexpr int kFp4RowBytes = MLA_FP4_ROW_BYTES;
static_assert(kFp4RopeOff + MLA_ROPE_DIM == kFp4RowBytes, "row layout");
static_assert(kFp4RowBytes % 16 == 0, "rows keep 16-byte alignment");

// Eight fp32 values -> eight E2M1 codes (round to nearest even, saturated to
// +-6), value i in bits 4i..4i+3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]),
        "f"(x[6]), "f"(x[7]));
  return r;
}

// Eight E2M1 codes -> four pairs of f16 (exact), pair i = elements 2i, 2i+1.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

// Two fp32 values -> two E4M3 codes (nearest even, saturated), low byte = a.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b) {
  uint16_t h;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(h) : "f"(a), "f"(b));
  return h;
}

// Two E4M3 codes -> two f16 (exact; NaN codes give NaN), low half = low byte.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return h;
}

__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ float2 h2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The larger of two values, NaN where either is: a maximum that dropped a NaN
// would store a broken row as zeros with scale 0.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// RMS norms of rows whose squares leave fp32's range: above about 2^60 a value
// their sum overflows, and without an eps it loses its bits below 2^-50.  Such a
// row is divided by the power of two of its largest value (exact) and takes eps
// by that power's square: the norm is the same.
__device__ __forceinline__ bool squares_leave_range(float mean, float eps) {
  return !(mean < INFINITY) || (mean < 0x1p-100f && eps == 0.f);
}
// 2^-e of the largest value top = m 2^e, kept a normal number; 1 for a row of
// zeros and for one that is not finite.
__device__ __forceinline__ float unit_factor(float top) {
  const int e = (int)(__float_as_uint(top) >> 23);  // biased; top >= 0
  return top > 0.f && top < INFINITY ? __uint_as_float((uint32_t)max(1, min(254 - e, 253)) << 23)
                                     : 1.f;
}

// Quotients by one divisor b > 0: a / b from y = RN(1 / b) and one Markstein
// correction (P. Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", IBM J. Res. Dev. 34(1), 1990): three
// instructions instead of a full division, off by at most one unit in the last
// place and exact for quotients of few bits, so a code's tie stays a tie.
// Divisors whose reciprocal leaves the normal range divide directly, and so do
// those by which the largest dividend's quotient overflows (its correction would
// be inf - inf); b = 0 gives 0, and NaN of a NaN.
struct Divisor {
  float b, y;
  bool direct;
  __device__ __forceinline__ Divisor(float d, float largest)
      : b(d), y(0.f), direct(!(d >= 0x1p-90f && d <= 0x1p+120f)) {
    if (!direct) {
      y = __frcp_rn(d);
      direct = !(__fmul_rn(largest, y) < INFINITY);
    }
  }
  __device__ __forceinline__ float operator()(float a) const {
    if (direct) return b != 0.f ? __fdiv_rn(a, b) : a == a ? 0.f : a;
    const float q = __fmul_rn(a, y);
    return __fmaf_rn(__fmaf_rn(-q, b, a), y, q);
  }
};

}  // namespace mla
