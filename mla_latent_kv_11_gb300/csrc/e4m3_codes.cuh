// Values to and from floats, and e4m3 codes of quotients (each rounded once): shared by the kernels
// that write quantised cache rows.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace mla {
namespace {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// x / s as a float32 that rounds to the same code as the quotient itself: rounded toward zero, with
// the last bit set where that lost something. (Rounded to nearest it could land on the middle of two
// codes, which a quotient beside it then rounds as: with bf16 values that is not rare, a 448 / top
// times a short value being off a middle only by the rounding of the scale.) r is 1 / s correctly
// rounded, and the steps Markstein's (IBM J. Res. Dev. 34, 1990): x * r is within two units in the
// last place; the remainder of a quotient that near is exact in one fused multiply-add, a step with
// it makes a neighbour of the quotient, and the neighbour's remainder says on which side that lies.
// No remainder of a quotient near a middle (2^-10 and up) may underflow: s is at least 2^-80 here, x
// finite or NaN. (An exact remainder needs no more: a code's middle has 5 bits, so a quotient that is
// none is 2^-29 of itself away from it at least.)
// The remainders are rounded down. That changes none that is exact, but makes a remainder of zero -0: for
// x = -0 each later sum then adds two zeros of its sign and the quotient is -0; for x = +0 it adds zeros of
// different signs, which to nearest and toward zero is +0. (Rounded to nearest, -0 came out as +0.) Where
// a remainder underflows, |x| is below 2^-125 and the quotient below 2^-45, whose code is a zero of x's
// sign: the last step, with a remainder near x where the steps before cancelled, still gives that sign.
// Two quotients at a time, in paired instructions: ns and r hold -s and 1 / s twice.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  return (uint64_t)__float_as_uint(b) << 32 | __float_as_uint(a);
}
__device__ __forceinline__ float odd(uint32_t bits, uint32_t rem) {
  asm("{\n\t.reg .pred p;\n\tsetp.neu.f32 p, %1, 0f00000000;\n\t@p or.b32 %0, %0, 1;\n\t}"
      : "+r"(bits) : "f"(__uint_as_float(rem)));
  return __uint_as_float(bits);
}
__device__ __forceinline__ void divide2(float x0, float x1, uint64_t ns, uint64_t r, float& y0, float& y1) {
  const uint64_t x = pair(x0, x1);
  uint64_t q, a, rem, t;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(q) : "l"(x), "l"(r));
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(a) : "l"(q), "l"(ns), "l"(x));
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(a) : "l"(a), "l"(r), "l"(q));
  asm("fma.rm.f32x2 %0, %1, %2, %3;" : "=l"(rem) : "l"(a), "l"(ns), "l"(x));
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(rem), "l"(r), "l"(a));
  y0 = odd((uint32_t)t, (uint32_t)rem);
  y1 = odd((uint32_t)(t >> 32), (uint32_t)(rem >> 32));
}

// The codes of two quotients: to nearest even, saturating.
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

}  // namespace
}  // namespace mla
