// Values to and from floats, and e4m3 codes of quotients (each rounded once): shared by the kernels
// that write quantised cache rows.
#pragma once

#include <cfloat>

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <cstdint>

#include "sm100_ptx.cuh"

namespace mla {
namespace {

constexpr float kE4m3Max = 448.f;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Sixteen consecutive values as floats: 32 bytes a load where `wide` (32-byte aligned), else 16.
__device__ __forceinline__ void load_words(const void* p, uint32_t (&w)[8], bool wide) {
  if (wide) {
    ptx::ld_global_32B(p, w);
  } else {
    const uint4 a = reinterpret_cast<const uint4*>(p)[0], b = reinterpret_cast<const uint4*>(p)[1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
  }
}
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&x)[16], bool wide) {
  uint32_t w[8];
  load_words(p, w, wide);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ void load16(const float* p, float (&x)[16], bool wide) {
  uint32_t w[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    load_words(p + 8 * h, w, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[8 * h + i] = __uint_as_float(w[i]);
  }
}
// Two consecutive values.
__device__ __forceinline__ float2 load2(const __nv_bfloat16* p) {
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(p));
}
__device__ __forceinline__ float2 load2(const float* p) { return *reinterpret_cast<const float2*>(p); }

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

// A group of 128 values, sixteen in each of eight consecutive lanes: the codes of this lane's, and the group's
// scale, its largest magnitude / 448 (an infinity counts as the largest float32, a NaN not at all), at least
// 2^-126 so that the division stays among normal numbers.
__device__ __forceinline__ float quantise_group(float (&x)[16], uint32_t (&w)[4]) {
  float top = 0.f;
#pragma unroll
  for (int k = 0; k < 16; ++k) top = fmaxf(top, fabsf(x[k]));   // fmaxf passes a NaN over
  const bool finite = top <= FLT_MAX;
  top = fminf(top, FLT_MAX);
#pragma unroll
  for (int m = 1; m < 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
  const float scale = fmaxf(__fdiv_rn(top, kE4m3Max), FLT_MIN);
  float by = scale;
  if (by < 0x1p-80f) {           // the same quotients, out of the way of underflow
    by *= 0x1p64f;
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] *= 0x1p64f;
  }
  if (!finite) {                 // the scale is FLT_MAX / 448 then: a code of +-448
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = fabsf(x[k]) > FLT_MAX ? copysignf(FLT_MAX, x[k]) : x[k];
  }
  const float inv = __frcp_rn(by);
  const uint64_t r = pair(inv, inv), ns = pair(-by, -by);
#pragma unroll
  for (int k = 0; k < 4; ++k) w[k] = 0;
#pragma unroll
  for (int k = 0; k < 16; k += 2) {
    float a, b;
    divide2(x[k], x[k + 1], ns, r, a, b);
    w[k >> 2] |= codes2(a, b) << (8 * (k & 2));
  }
  return scale;
}

}  // namespace
}  // namespace mla
