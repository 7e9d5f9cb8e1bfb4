// mx_gate.cuh -- the gated SiLU of a pair of fp32 values, forward and backward, as the
// element-wise kernels and the products' epilogues compute it:
//
//   h  = g sg u,  sg = 1 / (1 + exp(-g))
//   dg = dh u sg (1 + g (1 - sg)),  du = dh g sg
//
// The exponential and the division go through the fast hardware functions, whose error
// (a few units of 2^-22, and |g| 2^-24 as the exponent is rounded) is far below the rounding
// of the results to 16 or 8 bits.
#pragma once

#include "mx_rows.cuh"

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

__device__ __forceinline__ f32x2 sigmoid2(f32x2 g) {
  float lo, hi;
  unpair(g, lo, hi);
  return pair(sigmoid(lo), sigmoid(hi));
}

// The largest of words of two bf16 gates each, halves apart.  As unsigned numbers the
// negative ones lie above the positive ones, in order of their size.
__device__ __forceinline__ uint32_t lowest2(const uint4& w) {
  return __vmaxu2(__vmaxu2(w.x, w.y), __vmaxu2(w.z, w.w));
}
__device__ __forceinline__ bool any_low(uint32_t lowest) {
  constexpr uint32_t kBits = 0xC2A0u << 16;              // kLow
  return lowest > (kBits | 0xFFFFu) || lowest << 16 > kBits;
}

// Whether a block with this scale byte can hold a gate below kLow: at 2^-3 its largest
// magnitude, 448, stands for 56.
__device__ __forceinline__ bool may_be_low(uint32_t sbyte) { return sbyte >= 127 - 2; }

// The products' epilogues take the sigmoid of no less than kLow, which leaves the results of
// low gates to be multiplied by this twice (1 for other gates), if there are any: no second
// copy of the formulas in the code.
__device__ __forceinline__ f32x2 low_factor2(f32x2 g) {
  constexpr float kHalf = 0.5f * 1.4426950408889634f;
  float lo, hi;
  unpair(g, lo, hi);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(lo) : "f"((fminf(lo, kLow) - kLow) * kHalf));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(hi) : "f"((fminf(hi, kLow) - kLow) * kHalf));
  return pair(lo, hi);
}

__device__ __forceinline__ f32x2 sigmoid2_from_low(f32x2 g, float& lowest) {
  float lo, hi;
  unpair(g, lo, hi);
  lowest = fminf(lowest, fminf(lo, hi));
  return pair(sigmoid(fmaxf(lo, kLow)), sigmoid(fmaxf(hi, kLow)));
}

// Eight gates and ups -> h in bf16.
__device__ __forceinline__ uint4 gated8(const f32x2 (&g)[4], const f32x2 (&u)[4]) {
  f32x2 h[4];
  float lowest = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) h[j] = mul2(mul2(g[j], sigmoid2_from_low(g[j], lowest)), u[j]);
  if (lowest < kLow) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 f = low_factor2(g[j]);
      h[j] = mul2(mul2(h[j], f), f);
    }
  }
  return pack_pairs(h);
}

// Eight dh, gates and ups -> dg and du in bf16; low: one of the gates may be below kLow.
__device__ __forceinline__ void gated_back8(const f32x2 (&d)[4], const f32x2 (&g)[4], const f32x2 (&u)[4],
                                            bool low, uint4& dg, uint4& du) {
  const f32x2 one = pair(1.0f, 1.0f), minus = pair(-1.0f, -1.0f);
  f32x2 a[4], b[4];
  auto back = [&](int j, f32x2 s) {
    const f32x2 t = mul2(g[j], s);
    a[j] = mul2(mul2(d[j], u[j]), fma2(t, fma2(s, minus, one), s));    // s (1 + g (1 - s))
    b[j] = mul2(d[j], t);
  };
#pragma unroll
  for (int j = 0; j < 4; ++j) back(j, sigmoid2(g[j]));
  if (low) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float lowest;
      back(j, sigmoid2_from_low(g[j], lowest = 0.0f));
      const f32x2 f = low_factor2(g[j]);
      a[j] = mul2(mul2(a[j], f), f);
      b[j] = mul2(mul2(b[j], f), f);
    }
  }
  dg = pack_pairs(a);
  du = pack_pairs(b);
}

}  // namespace mx
