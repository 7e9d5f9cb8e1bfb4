// mx_rows.cuh -- what the layer norm and gated SiLU kernels share: row pieces
// of 8, 2 or 1 bf16 values in registers, the MX cast of a row held by a warp
// group, MX values back from their bytes, and sums over a warp group.
#pragma once

#include "mx_common.cuh"

namespace mx {

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A piece of VEC bf16 values as it lies in memory (tensors here are read once:
// no L1 allocation).
template <int VEC>
struct Piece;

template <>
struct Piece<8> {
  uint4 w;
  __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                 : "l"(p));
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf_lo(w.x); v[1] = bf_hi(w.x); v[2] = bf_lo(w.y); v[3] = bf_hi(w.y);
    v[4] = bf_lo(w.z); v[5] = bf_hi(w.z); v[6] = bf_lo(w.w); v[7] = bf_hi(w.w);
  }
};

template <>
struct Piece<2> {
  uint32_t w;
  __device__ __forceinline__ void zero() { w = 0; }
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.nc.L1::no_allocate.u32 %0, [%1];" : "=r"(w) : "l"(p));
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf_lo(w);
    v[1] = bf_hi(w);
  }
};

template <>
struct Piece<1> {
  uint16_t w;
  __device__ __forceinline__ void zero() { w = 0; }
  __device__ __forceinline__ void load(const uint16_t* p) {
    asm volatile("ld.global.nc.u16 %0, [%1];" : "=h"(w) : "l"(p));
  }
  __device__ __forceinline__ void get(float* v) const {
    v[0] = __uint_as_float(static_cast<uint32_t>(w) << 16);
  }
};

template <int VEC>
__device__ __forceinline__ void store_bf16(uint16_t* p, const float* v, const Span& sp) {
  if (!in_span(sp, p, 2 * VEC)) return;
  if constexpr (VEC == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  else if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
  else
    *p = static_cast<uint16_t>(pack_bf16(v[0], 0.0f));
}

// VEC parameters (fp32 or bf16) as floats; read by every row, so through L1.
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, float* v) {
  if constexpr (VEC == 8) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(p));
    const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else if constexpr (VEC == 2) {
    const float2 a = __ldg(reinterpret_cast<const float2*>(p));
    v[0] = a.x; v[1] = a.y;
  } else {
    v[0] = __ldg(p);
  }
}

template <int VEC>
__device__ __forceinline__ void load_param(const uint16_t* p, float* v) {
  if constexpr (VEC == 8) {
    Piece<8> w;
    w.w = __ldg(reinterpret_cast<const uint4*>(p));
    w.get(v);
  } else if constexpr (VEC == 2) {
    const uint32_t a = __ldg(reinterpret_cast<const uint32_t*>(p));
    v[0] = bf_lo(a); v[1] = bf_hi(a);
  } else {
    v[0] = __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
  }
}

// MX cast of one 32-block held as eight values by each of four neighbouring
// lanes: this lane's eight e4m3 bytes and the block's scale byte (the same in
// the four lanes).  Every lane of the warp takes part.
__device__ __forceinline__ uint2 mx_cast_piece(const uint4& w, uint32_t& sbyte) {
  uint32_t m = absmax2(absmax2(w.x, w.y), absmax2(w.z, w.w));
  m = max(mag_lo(m), mag_hi(m));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  float mult;
  mx_scale(m, sbyte, mult);
  return make_uint2(e4m3x4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y), mult),
                    e4m3x4(bf_lo(w.z), bf_hi(w.z), bf_lo(w.w), bf_hi(w.w), mult));
}

// 2^(s - 127) of a scale byte; 0xFF is NaN.
__device__ __forceinline__ float scale_mult(uint32_t s) {
  return __uint_as_float(s == 0 ? 0x00400000u : s == 255 ? 0x7FC00000u : s << 23);
}

// Two e4m3 bytes -> two floats (exact: through f16, whose range holds e4m3's).
__device__ __forceinline__ void e4m3x2_get(uint32_t pair, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

// Eight saved values: e4m3 bytes times their block's scale.
__device__ __forceinline__ void mx_get8(const uint2& q, uint32_t sbyte, float* v) {
  const float m = scale_mult(sbyte);
  e4m3x2_get(q.x & 0xFFFFu, v[0], v[1]);
  e4m3x2_get(q.x >> 16, v[2], v[3]);
  e4m3x2_get(q.y & 0xFFFFu, v[4], v[5]);
  e4m3x2_get(q.y >> 16, v[6], v[7]);
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = mul_rn(v[j], m);
}

__device__ __forceinline__ uint2 ld_q8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over a group of `warps` warps that meet at named barrier `id`.  `red`
// holds two slots of 32 pairs, used in turn (`phase`), so that one barrier a
// sum is enough: a slot is written again only after the other slot's barrier,
// which every thread reaches after its reads of this one.  The order of the
// additions is fixed.
struct Group {
  float2* red;
  int id, warps, warp, lane;
  int phase;
  __device__ __forceinline__ float2 sum2(float a, float b) {
    a = warp_sum(a);
    b = warp_sum(b);
    if (warps == 1) return make_float2(a, b);
    float2* r = red + 32 * phase;
    phase ^= 1;
    if (lane == 0) r[warp] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory");
    const float2 v = lane < warps ? r[lane] : make_float2(0.0f, 0.0f);
    return make_float2(warp_sum(v.x), warp_sum(v.y));
  }
  __device__ __forceinline__ float sum(float a) { return sum2(a, 0.0f).x; }
};

}  // namespace mx
