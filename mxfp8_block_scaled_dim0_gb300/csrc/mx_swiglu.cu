// mx_swiglu.cu -- gated SiLU of bf16 rows [gate | up], forward and backward,
// with its input saved as MX-FP8 for the backward pass.
//
//   h  = g sg u,  sg = 1 / (1 + exp(-g))
//   dg = dh u sg (1 + g (1 - sg)),  du = dh g sg
//
// A warp works on 32 pieces of a row's gate half and the same pieces of its up
// half (256 columns where the width is a multiple of 8).  Every byte is read
// and written once; the exponential and the division go through the fast
// hardware functions, whose error (a few units of 2^-22) is far below the
// bf16 rounding of the results.
#include <cuda_runtime.h>

#include "mx_kernels.h"
#include "mx_rows.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;

struct SwigluParams {
  const uint16_t* gu;
  const uint16_t* dh;
  uint16_t* out;        // h, or the gradient of gu
  uint8_t* q;
  uint8_t* s;
  int64_t M, rows, tasks;
  int F, runs;          // runs: warps' pieces of a row
  int s_cols4;          // scales of a row, padded to four
  Span sp_out, sp_q, sp_s;
};

__device__ __forceinline__ float sigmoid(float g) { return __fdividef(1.0f, 1.0f + __expf(-g)); }

template <int VEC, bool SAVE>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       t < p.tasks; t += warps) {
    const int64_t r = t / p.runs;
    const int c = (static_cast<int>(t - r * p.runs) * 32 + lane) * VEC;
    const bool live = r < p.M && c < p.F;
    Piece<VEC> pg, pu;
    pg.zero();
    pu.zero();
    if (live) {
      pg.load(p.gu + r * 2 * p.F + c);
      pu.load(p.gu + r * 2 * p.F + p.F + c);
    }
    if constexpr (SAVE) {
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t sb;
        const uint2 q = mx_cast_piece(half ? pu.w : pg.w, sb);
        const int col = half * p.F + c;
        uint8_t* qp = p.q + r * 2 * p.F + col;
        if (live && in_span(p.sp_q, qp, 8)) *reinterpret_cast<uint2*>(qp) = q;
        if (c < p.F && (lane & 3) == 0) {
          uint8_t* sp = p.s + blocked_offset(r, col >> 5, p.s_cols4);
          if (in_span(p.sp_s, sp, 1)) *sp = static_cast<uint8_t>(r < p.M ? sb : 0);
        }
      }
      // Columns of scales past the row: zero.
      const int pad = p.s_cols4 - p.F / 16;
      if (c == 0 && pad > 0)
        for (int k = 0; k < pad; ++k) {
          uint8_t* sp = p.s + blocked_offset(r, p.F / 16 + k, p.s_cols4);
          if (in_span(p.sp_s, sp, 1)) *sp = 0;
        }
    }
    if (!live) continue;
    float g[VEC], u[VEC], h[VEC];
    pg.get(g);
    pu.get(u);
#pragma unroll
    for (int j = 0; j < VEC; ++j) h[j] = g[j] * sigmoid(g[j]) * u[j];
    store_bf16<VEC>(p.out + r * p.F + c, h, p.sp_out);
  }
}

template <int VEC, bool SAVE>
__global__ void __launch_bounds__(kThreads) swiglu_back_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t warps = static_cast<int64_t>(gridDim.x) * (kThreads / 32);
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
       t < p.tasks; t += warps) {
    const int64_t r = t / p.runs;
    const int c = (static_cast<int>(t - r * p.runs) * 32 + lane) * VEC;
    if (c >= p.F) continue;
    Piece<VEC> pd;
    pd.load(p.dh + r * p.F + c);
    float g[VEC], u[VEC], d[VEC], dg[VEC], du[VEC];
    if constexpr (SAVE) {
      const uint8_t* qp = p.q + r * 2 * p.F + c;
      const uint2 qg = ld_q8(qp), qu = ld_q8(qp + p.F);
      const uint32_t sg = __ldg(p.s + blocked_offset(r, c >> 5, p.s_cols4));
      const uint32_t su = __ldg(p.s + blocked_offset(r, (p.F + c) >> 5, p.s_cols4));
      mx_get8(qg, sg, g);
      mx_get8(qu, su, u);
    } else {
      Piece<VEC> pg, pu;
      pg.load(p.gu + r * 2 * p.F + c);
      pu.load(p.gu + r * 2 * p.F + p.F + c);
      pg.get(g);
      pu.get(u);
    }
    pd.get(d);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float sg = sigmoid(g[j]);
      const float a = g[j] * sg;
      du[j] = d[j] * a;
      dg[j] = d[j] * u[j] * (sg + a * (1.0f - sg));
    }
    store_bf16<VEC>(p.out + r * 2 * p.F + c, dg, p.sp_out);
    store_bf16<VEC>(p.out + r * 2 * p.F + p.F + c, du, p.sp_out);
  }
}

template <typename K>
int run(K kernel, const SwigluParams& p, int num_sms, cudaStream_t stream) {
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, 0) != cudaSuccess ||
      per < 1)
    per = 1;
  const int64_t want = (p.tasks + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = static_cast<int64_t>(num_sms) * per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p));
}

SwigluParams params(const SwigluArgs& a, int vec, bool padded) {
  SwigluParams p = {};
  p.gu = static_cast<const uint16_t*>(a.gu);
  p.dh = static_cast<const uint16_t*>(a.dh);
  p.out = static_cast<uint16_t*>(a.out);
  p.q = static_cast<uint8_t*>(a.q);
  p.s = static_cast<uint8_t*>(a.s);
  p.M = a.M;
  p.rows = padded ? (a.M + 127) / 128 * 128 : a.M;
  p.F = static_cast<int>(a.F);
  p.runs = static_cast<int>((a.F + 32 * vec - 1) / (32 * vec));
  p.tasks = p.rows * p.runs;
  p.s_cols4 = static_cast<int>((a.F / 16 + 3) / 4 * 4);
  const uint64_t n = static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.F);
  p.sp_out = make_span(a.out, a.dh ? 4 * n : 2 * n);
  p.sp_q = make_span(a.q, 2 * n);
  p.sp_s = make_span(a.s, static_cast<uint64_t>((a.M + 127) / 128 * 128) * p.s_cols4);
  return p;
}

int vec_of(int64_t F) { return F % 8 == 0 ? 8 : F % 2 == 0 ? 2 : 1; }

}  // namespace

int launch_swiglu(const SwigluArgs& a, int num_sms, cudaStream_t stream) {
  const int v = vec_of(a.F);
  const SwigluParams p = params(a, v, a.q != nullptr);
  if (a.q) return run(swiglu_kernel<8, true>, p, num_sms, stream);
  if (v == 8) return run(swiglu_kernel<8, false>, p, num_sms, stream);
  if (v == 2) return run(swiglu_kernel<2, false>, p, num_sms, stream);
  return run(swiglu_kernel<1, false>, p, num_sms, stream);
}

int launch_swiglu_backward(const SwigluArgs& a, int num_sms, cudaStream_t stream) {
  const int v = vec_of(a.F);
  const SwigluParams p = params(a, v, false);
  if (a.q) return run(swiglu_back_kernel<8, true>, p, num_sms, stream);
  if (v == 8) return run(swiglu_back_kernel<8, false>, p, num_sms, stream);
  if (v == 2) return run(swiglu_back_kernel<2, false>, p, num_sms, stream);
  return run(swiglu_back_kernel<1, false>, p, num_sms, stream);
}

int out_of_bounds_swiglu(bool clear) { return read_out_of_bounds(clear); }

}  // namespace mx
