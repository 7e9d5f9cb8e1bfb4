// mx_rows.cuh -- what the layer norm and gated SiLU kernels share: row pieces
// of 8, 2 or 1 bf16 values in registers, fp32 arithmetic on pairs, the MX cast of
// blocks held by four lanes, MX values back from their bytes, and sums over a
// group of warps.
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
  if constexpr (VEC == 2)
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(v[0], v[1]);
  else
    *p = static_cast<uint16_t>(pack_bf16(v[0], 0.0f));
}

// One parameter (fp32 or bf16).
__device__ __forceinline__ float load_param(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_param(const uint16_t* p) {
  return __uint_as_float(static_cast<uint32_t>(__ldg(p)) << 16);
}

// 2^(s - 127) of a scale byte; 0xFF is NaN.  The exponent field, but for s = 0 a
// subnormal's bit, and for 0xFF the quiet bit too.
__device__ __forceinline__ float scale_mult(uint32_t s) {
  return __uint_as_float(max(s << 23, 0x00400000u) | ((s + 1) >> 8) << 22);
}

// Two e4m3 bytes -> two floats (exact: through f16, whose range holds e4m3's).
__device__ __forceinline__ void e4m3x2_get(uint32_t pair, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(pair)));
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

__device__ __forceinline__ uint2 ld_q8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// ---- pairs of fp32 values (one instruction a pair) --------------------------------

using f32x2 = unsigned long long;

__device__ __forceinline__ f32x2 pair(float lo, float hi) {
  f32x2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}

__device__ __forceinline__ void unpair(f32x2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}

__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ f32x2 fma2(f32x2 a, f32x2 b, f32x2 c) {
  f32x2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// The two bf16 halves of a word.
__device__ __forceinline__ f32x2 bf_pair(uint32_t w) { return pair(bf_lo(w), bf_hi(w)); }

__device__ __forceinline__ uint32_t pack_pair(f32x2 v) {
  float lo, hi;
  unpair(v, lo, hi);
  return pack_bf16(lo, hi);
}

__device__ __forceinline__ float sum_pair(f32x2 v) {
  float lo, hi;
  unpair(v, lo, hi);
  return lo + hi;
}

__device__ __forceinline__ void get_pairs(const uint4& w, f32x2* v) {
  v[0] = bf_pair(w.x);
  v[1] = bf_pair(w.y);
  v[2] = bf_pair(w.z);
  v[3] = bf_pair(w.w);
}

__device__ __forceinline__ uint4 pack_pairs(const f32x2* v) {
  return make_uint4(pack_pair(v[0]), pack_pair(v[1]), pack_pair(v[2]), pack_pair(v[3]));
}

// Eight parameters (fp32 or bf16) as pairs, from global memory.
__device__ __forceinline__ void load_param_pairs(const float* p, f32x2* v) {
  const ulonglong2 a = __ldg(reinterpret_cast<const ulonglong2*>(p));
  const ulonglong2 b = __ldg(reinterpret_cast<const ulonglong2*>(p) + 1);
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

__device__ __forceinline__ void load_param_pairs(const uint16_t* p, f32x2* v) {
  get_pairs(__ldg(reinterpret_cast<const uint4*>(p)), v);
}

// D parameters in shared memory as fp32, from place `lead` on (ODD; otherwise 0),
// zeros before and up to `pitch`; the first and the last four of every eight in
// halves of their own: a warp's 16-byte reads of neighbouring pieces are then
// free of bank conflicts.
template <bool ODD, typename W>
__device__ __forceinline__ void stage_params(float* dst, const W* src, int lead, int D, int pitch) {
  const int threads = static_cast<int>(blockDim.x);
  auto put = [&](int c, const f32x2* v) {
    reinterpret_cast<ulonglong2*>(dst)[c] = make_ulonglong2(v[0], v[1]);
    reinterpret_cast<ulonglong2*>(dst)[pitch / 8 + c] = make_ulonglong2(v[2], v[3]);
  };
  if constexpr (ODD) {
    for (int c = threadIdx.x; c < pitch / 8; c += threads) {
      f32x2 v[4];
      float f[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int e = 8 * c + j - lead;
        f[j] = e >= 0 && e < D ? load_param(src + e) : 0.0f;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = pair(f[2 * j], f[2 * j + 1]);
      put(c, v);
    }
  } else {
    const int n = D >> 3;
    const f32x2 zero[4] = {0, 0, 0, 0};
    for (int c = n + threadIdx.x; c < pitch / 8; c += threads) put(c, zero);
    // Two pieces' loads at a time, without a condition (past the end: the last).
    constexpr int kAtOnce = 2;
    for (int c = threadIdx.x; c < n; c += kAtOnce * threads) {
      f32x2 v[kAtOnce][4];
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k) load_param_pairs(src + 8 * min(c + k * threads, n - 1), v[k]);
#pragma unroll
      for (int k = 0; k < kAtOnce; ++k)
        if (c + k * threads < n) put(c + k * threads, v[k]);
    }
  }
}

__device__ __forceinline__ void staged_pairs(const float* src, int pitch, int c, f32x2* v) {
  const ulonglong2 a = reinterpret_cast<const ulonglong2*>(src)[c];
  const ulonglong2 b = reinterpret_cast<const ulonglong2*>(src)[pitch / 8 + c];
  v[0] = a.x;
  v[1] = a.y;
  v[2] = b.x;
  v[3] = b.y;
}

__device__ __forceinline__ uint32_t e4m3_pair(f32x2 v) {
  float lo, hi;
  unpair(v, lo, hi);
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// MX cast of one 32-block held as eight values by each of four neighbouring
// lanes (w, and v, the same as pairs): this lane's eight e4m3 bytes and the
// block's scale byte (the same in the four lanes).  Every lane of the warp takes
// part.
__device__ __forceinline__ uint2 mx_cast_pairs(const uint4& w, const f32x2* v, uint32_t& sbyte) {
  uint32_t m = absmax2(absmax2(w.x, w.y), absmax2(w.z, w.w));
  m = max(mag_lo(m), mag_hi(m));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  float mult;
  mx_scale(m, sbyte, mult);
  const f32x2 m2 = pair(mult, mult);
  return make_uint2(e4m3_pair(mul2(v[0], m2)) | (e4m3_pair(mul2(v[1], m2)) << 16),
                    e4m3_pair(mul2(v[2], m2)) | (e4m3_pair(mul2(v[3], m2)) << 16));
}

// Eight saved values as pairs.
__device__ __forceinline__ void mx_get_pairs(const uint2& q, uint32_t sbyte, f32x2* v) {
  const float m = scale_mult(sbyte);
  const f32x2 m2 = pair(m, m);
  const uint32_t w[4] = {q.x & 0xFFFFu, q.x >> 16, q.y & 0xFFFFu, q.y >> 16};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float lo, hi;
    e4m3x2_get(w[j], lo, hi);
    v[j] = mul2(pair(lo, hi), m2);
  }
}

// ---- sums over a group of warps ------------------------------------------------

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sums over a group of `warps` <= 16 warps that meet at named barrier `id`.
// `red` holds two slots of 64 floats, zero at the start and used in turn, so that
// one barrier a sum is enough: a slot is written again only after the other
// slot's barrier, which every thread reaches after its reads of this one.  Two
// sums travel together, one in either half of a warp after the first exchange.
// The order of the additions is fixed.
struct Group {
  float* red;
  int id, warps, warp, lane;
  int phase;
  __device__ __forceinline__ void meet() const {
    if (warps == 1)
      __syncwarp();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(32 * warps) : "memory");
  }
  // The sum of v[0..16), in every lane.
  __device__ __forceinline__ float across(const float* v) const {
    float a = v[lane & 15];
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    return a;
  }
  __device__ __forceinline__ float2 sum2(float a, float b) {
    const bool low = lane < 16;
    float v = low ? a : b;
    v += __shfl_xor_sync(0xffffffffu, low ? b : a, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (warps > 1) {
      float* r = red + 64 * phase + (low ? 0 : 32);
      phase ^= 1;
      if ((lane & 15) == 0) r[warp] = v;
      meet();
      v = across(r);
    }
    const float w = __shfl_xor_sync(0xffffffffu, v, 16);
    return low ? make_float2(v, w) : make_float2(w, v);
  }
  __device__ __forceinline__ float sum(float a) {
    a = warp_sum(a);
    if (warps == 1) return a;
    float* r = red + 64 * phase;
    phase ^= 1;
    if (lane == 0) r[warp] = a;
    meet();
    return across(r);
  }
};

}  // namespace mx
