// mx_gate.cuh -- the gated SiLU of a pair of fp32 values, forward and backward, as the
// element-wise kernels and the products' epilogues compute it:
//
//   h  = g sg u,  sg = 1 / (1 + exp(-g))
//   dg = dh u sg (1 + g (1 - sg)),  du = dh g sg
//
// The exponential and the division go through the fast hardware functions, whose error
// (a few units of 2^-22) is far below the rounding of the results to 16 or 8 bits.
#pragma once

#include "mx_common.cuh"

namespace mx {

// 1 / (1 + exp(-g)) of a gate that is not low.
__device__ __forceinline__ float sigmoid(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

// Low gates.  Below g = -87.3 the sigmoid leaves fp32's normal range, and from -88.7
// down exp(-g) overflows, while g sg u may be an ordinary number.  From kLow down sg is
// exp(g), to fp32: the results of kLow's sigmoid, to which they are proportional, are
// multiplied by exp(g - kLow), in two halves that stay in range.
constexpr float kLow = -80.0f;

__device__ __forceinline__ float low_result(float v, float g) {
  float f;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(f) : "f"((g - kLow) * (0.5f * 1.4426950408889634f)));
  return v * f * f;
}

__device__ __forceinline__ float low_gated(float g, float u) {
  return low_result(g * sigmoid(kLow) * u, g);
}

__device__ __forceinline__ void gated_back(float d, float g, float u, float& dg, float& du) {
  const bool low = g < kLow;
  const float s = sigmoid(low ? kLow : g);
  const float a = g * s;
  du = d * a;
  dg = d * u * (s + a * (1.0f - s));
  if (low) {
    du = low_result(du, g);
    dg = low_result(dg, g);
  }
}

// h of any gate.
__device__ __forceinline__ float gated(float g, float u) {
  return g < kLow ? low_gated(g, u) : g * sigmoid(g) * u;
}

}  // namespace mx
