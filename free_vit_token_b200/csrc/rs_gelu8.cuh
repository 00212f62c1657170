// rs_gelu8.cuh -- the GELU of the 8-bit products' epilogues.
#pragma once

#include <cstdint>

#include "rs_fp8.cuh"
#include "rs_gelu_logit.h"

namespace rs {

__device__ __forceinline__ uint64_t pair_of(float c) { return f2pack(c, c); }

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// GELU of two fp32 lanes through a logistic form of the normal CDF (rs_gelu_logit.h): within
// 2^-18 of its value for z >= -4.4 and within 3e-8 below, with the approximate 2^x and reciprocal.
// Nothing bounds the exponent: 2^x overflows where GELU vanishes, and infinities and NaN go where
// z Phi(z) sends them. So each lane takes a reciprocal of its own: one for both (1/(ab)) needs a
// bound, which leaves far negative z at a multiple of z. Against a degree of 3 and one reciprocal,
// 1.4e-5 off, 50432 x 384 -> 1536 takes 68 us for 62, 25104 x 1024 -> 4096 to blocks 121 for 111.
__device__ __forceinline__ uint64_t gelu2_logit(uint64_t z2) {
  const uint64_t t = mul2(z2, z2);
  uint64_t q = pair_of(-RS_GELU_LOGIT_Q9);
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q8));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q7));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q6));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q5));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q4));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q3));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q2));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q1));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q0));
  const float2 x = f2unpack(mul2(q, z2));
  const float2 d = f2unpack(fadd2(f2pack(ex2_approx(x.x), ex2_approx(x.y)), pair_of(1.f)));
  return mul2(z2, f2pack(rcp_approx(d.x), rcp_approx(d.y)));
}

}  // namespace rs
