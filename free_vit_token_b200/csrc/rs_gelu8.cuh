// rs_gelu8.cuh -- the GELU of the 8-bit products' epilogues.
#pragma once

#include <cstdint>

#include "rs_fp8.cuh"
#include "rs_gelu_logit.h"

namespace rs {

__device__ __forceinline__ uint64_t pair_of(float c) { return f2pack(c, c); }

// GELU of two fp32 lanes through a logistic form of the normal CDF (rs_gelu_logit.h, max
// |error| 1.5e-5 with the approximate 2^x and reciprocal). Against the polynomials of
// rs_gelu.cuh it takes half the FMAs, three instructions of the exponential unit a pair (one
// reciprocal serves both lanes: 1/a = b / (ab)) and no choice by range: 50432 x 384 -> 1536 on
// values past the short polynomial's range 92 -> 73 us a call.
__device__ __forceinline__ uint64_t gelu2_logit(uint64_t z2) {
  const float2 s = f2unpack(mul2(z2, z2));
  const uint64_t t = f2pack(fminf(s.x, RS_GELU_LOGIT_T), fminf(s.y, RS_GELU_LOGIT_T));
  uint64_t q = pair_of(-RS_GELU_LOGIT_Q3);
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q2));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q1));
  q = ffma2(q, t, pair_of(-RS_GELU_LOGIT_Q0));
  const float2 x = f2unpack(mul2(q, z2));
  // up to 2^60, so that the product of two stays finite: past it GELU is z 2^-60 where it should
  // vanish (below 1e-12 for z > -1e6; -inf stays -inf). A degree-4 fit without the bound on t and
  // with this one on z instead takes one more FMA and measured 6% slower.
  const float2 d = f2unpack(
      fadd2(f2pack(ex2_approx(fminf(x.x, 60.f)), ex2_approx(fminf(x.y, 60.f))), pair_of(1.f)));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(d.x * d.y));
  return mul2(z2, f2pack(r * d.y, r * d.x));
}

}  // namespace rs
