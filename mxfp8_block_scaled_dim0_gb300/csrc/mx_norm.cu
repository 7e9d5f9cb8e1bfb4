// mx_norm.cu -- layer norm of bf16 rows, forward and backward, with its input
// saved as MX-FP8 for the backward pass.
//
//   mean = (1/D) sum x, rstd = (eps + (1/D) sum (x - mean)^2)^(-1/2)
//   y    = (x - mean) rstd w + b
//   xh   = (x - mean) rstd, g = dy w
//   dx   = rstd (g - (1/D) sum g - xh (1/D) sum g xh)
//   dw   = sum over rows of dy xh, db = sum over rows of dy
//
// A group of warps holds a row in registers, 16 values a thread, in pieces of
// 8, 2 or 1 neighbouring values (by the row length's alignment); the next
// row's loads are issued before the present row is worked on.  The backward
// kernel keeps dw and db of its threads' columns in registers over all its
// rows, adds the groups of a CTA up at its end, and leaves one partial sum per
// CTA in the workspace, which norm_grad_kernel adds up in a fixed order.
#include <cuda_runtime.h>

#include "mx_kernels.h"
#include "mx_rows.cuh"

namespace mx {
namespace {

constexpr int kPer = 16;                     // values a thread holds of a row
constexpr int kMaxThreads = 1024;

struct NormParams {
  const uint16_t* x;
  const void* w;
  const void* b;
  uint16_t* y;
  float* mean;
  float* rstd;
  uint8_t* q;
  uint8_t* s;
  int64_t M, rows;     // rows: M, or M padded to 128 where scales are written
  int D, warps, groups;
  int s_words;         // 128x4 scale tiles of a row
  float eps;
  Span sp_y, sp_mean, sp_rstd, sp_q, sp_s;
};

// Rows of a multiple of 8 values: 32 values a thread, as 16 pairs.
constexpr int kWide = 32;

template <bool SAVE, typename W>
__global__ void __launch_bounds__(640, 1) norm_rows8_kernel(const NormParams p) {
  constexpr int V = kWide / 8;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ __align__(16) float2 red[8 * 64];
  for (int i = threadIdx.x; i < 8 * 64; i += blockDim.x) red[i] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / p.warps;
  Group grp{red + 64 * g, g + 1, p.warps, warp - g * p.warps, lane, 0};
  const int T = 32 * p.warps, tid = grp.warp * 32 + lane;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  const float inv = 1.0f / static_cast<float>(p.D);
  const W* w = static_cast<const W*>(p.w) + tid * 8;
  const W* b = p.b ? static_cast<const W*>(p.b) + tid * 8 : nullptr;

  Piece<8> nxt[V];
  auto fetch = [&](int64_t r) {
    const uint16_t* x = p.x + r * p.D + tid * 8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      nxt[i].zero();
      if (r < p.M && (i * T + tid) * 8 < p.D) nxt[i].load(x + i * T * 8);
    }
  };
  int64_t r = static_cast<int64_t>(blockIdx.x) * p.groups + g;
  fetch(r);
  for (; r < p.rows; r += step) {
    f32x2 x[kWide / 2];
    f32x2 s2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      get_pairs(nxt[i].w, x + 4 * i);
      s2 = add2(s2, add2(add2(x[4 * i], x[4 * i + 1]), add2(x[4 * i + 2], x[4 * i + 3])));
    }
    if constexpr (SAVE) {
      uint8_t* q = p.q + r * p.D + tid * 8;
      uint8_t* s = p.s + blocked_offset(r, 0, 4 * p.s_words) + (lane >> 2 & 3);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * T + tid) * 8;
        uint32_t sb;
        const uint2 v = mx_cast_pairs(nxt[i].w, x + 4 * i, sb);
        if (c < p.D && r < p.M && in_span(p.sp_q, q + i * T * 8, 8))
          *reinterpret_cast<uint2*>(q + i * T * 8) = v;
        // One lane of a block's four.  Blocks past the row and rows past the
        // matrix are zero and give 0, the padding of the blocked layout.
        if ((lane & 3) == 0 && (c >> 7) < p.s_words && in_span(p.sp_s, s + (c >> 7) * 512, 1))
          s[(c >> 7) * 512] = static_cast<uint8_t>(sb);
      }
    }
    fetch(r + step);
    if (SAVE && r >= p.M) continue;
    const float mean = grp.sum(sum_pair(s2)) * inv;
    const f32x2 m2 = pair(-mean, -mean);
    s2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((i * T + tid) * 8 >= p.D) continue;
#pragma unroll
      for (int j = 4 * i; j < 4 * i + 4; ++j) {
        x[j] = add2(x[j], m2);
        s2 = fma2(x[j], x[j], s2);
      }
    }
    const float rstd = 1.0f / sqrtf(grp.sum(sum_pair(s2)) * inv + p.eps);
    if (tid == 0) {
      if (in_span(p.sp_mean, p.mean + r, 4)) p.mean[r] = mean;
      if (in_span(p.sp_rstd, p.rstd + r, 4)) p.rstd[r] = rstd;
    }
    const f32x2 r2 = pair(rstd, rstd);
    uint16_t* y = p.y + r * p.D + tid * 8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((i * T + tid) * 8 >= p.D) continue;
      f32x2 wv[4], bv[4] = {0, 0, 0, 0};
      load_param_pairs(w + i * T * 8, wv);
      if (b) load_param_pairs(b + i * T * 8, bv);
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[j] = fma2(mul2(x[4 * i + j], r2), wv[j], bv[j]);
      if (in_span(p.sp_y, y + i * T * 8, 16)) *reinterpret_cast<uint4*>(y + i * T * 8) = pack_pairs(wv);
    }
  }
}

// Other rows, in pieces of two values or one.
template <int VEC, typename W>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const NormParams p) {
  constexpr int V = kPer / VEC;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ __align__(16) float2 red[8 * 64];
  for (int i = threadIdx.x; i < 8 * 64; i += blockDim.x) red[i] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / p.warps;
  Group grp{red + 64 * g, g + 1, p.warps, warp - g * p.warps, lane, 0};
  const int T = 32 * p.warps, tid = grp.warp * 32 + lane;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  const float inv = 1.0f / static_cast<float>(p.D);
  const W* w = static_cast<const W*>(p.w);
  const W* b = static_cast<const W*>(p.b);

  Piece<VEC> cur[V], nxt[V];
  auto fetch = [&](int64_t r, Piece<VEC>(&d)[V]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      d[i].zero();
      const int c = (i * T + tid) * VEC;
      if (r < p.M && c < p.D) d[i].load(p.x + r * p.D + c);
    }
  };
  int64_t r = static_cast<int64_t>(blockIdx.x) * p.groups + g;
  fetch(r, nxt);
  for (; r < p.M; r += step) {
#pragma unroll
    for (int i = 0; i < V; ++i) cur[i] = nxt[i];
    fetch(r + step, nxt);
    float x[kPer];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      cur[i].get(x + i * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) sum += x[i * VEC + j];
    }
    const float mean = grp.sum(sum) * inv;
    float sq = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool live = (i * T + tid) * VEC < p.D;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        x[i * VEC + j] = live ? x[i * VEC + j] - mean : 0.0f;
        sq += x[i * VEC + j] * x[i * VEC + j];
      }
    }
    const float rstd = 1.0f / sqrtf(grp.sum(sq) * inv + p.eps);
    if (tid == 0) {
      if (in_span(p.sp_mean, p.mean + r, 4)) p.mean[r] = mean;
      if (in_span(p.sp_rstd, p.rstd + r, 4)) p.rstd[r] = rstd;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * T + tid) * VEC;
      if (c >= p.D) continue;
      float wv[VEC], bv[VEC], y[VEC];
      load_param<VEC>(w + c, wv);
#pragma unroll
      for (int j = 0; j < VEC; ++j) bv[j] = 0.0f;
      if (b) load_param<VEC>(b + c, bv);
#pragma unroll
      for (int j = 0; j < VEC; ++j) y[j] = x[i * VEC + j] * rstd * wv[j] + bv[j];
      store_bf16<VEC>(p.y + r * p.D + c, y, p.sp_y);
    }
  }
}

struct NormBackParams {
  const uint16_t* dy;
  const uint16_t* x;
  const uint8_t* q;
  const uint8_t* s;
  const void* w;
  const float* mean;
  const float* rstd;
  uint16_t* dx;
  float* parts;        // [grid][2][D]
  int64_t M;
  int D, warps, groups, stages;
  int s_words;
  Span sp_dx, sp_parts;
  int64_t stall_at;
  uint64_t stall_ns;
};

// Rows of a multiple of 8 values.  The rows of dy and of x (or its saved bytes)
// come into shared memory by bulk copies, `stages` rows of a group ahead, so
// that what is in flight does not take registers; a stage is filled again once
// the row's sums are known, for by then every thread of the group has read it.
// EPT values a thread: 16, or 32 where 512 threads would not hold a row; then
// what the second pass needs is worked out again from the row's words.
// Every wait is bounded: one that runs out raises the abort flag, the threads go
// on to the end without waiting, and the watchdog word is set.
__device__ int g_norm_watchdog = 0;

constexpr int kBackThreads = 640;
constexpr int kBackMaxGroups = 20;
constexpr int kBackMaxStages = 4;
constexpr int kBackRing = 192 * 1024;

template <bool SAVE, typename W, int EPT>
__global__ void __launch_bounds__(EPT == 16 ? kBackThreads : 512, 1)
    norm_back_rows8_kernel(const NormBackParams p) {
  constexpr int V = EPT / 8;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ __align__(16) float2 red[kBackMaxGroups * 64];
  __shared__ __align__(8) uint64_t full[kBackMaxGroups * kBackMaxStages];
  __shared__ __align__(8) uint64_t stall_bar;   // diagnostic: never completed
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / p.warps;
  Group grp{red + 64 * g, g + 1, p.warps, warp - g * p.warps, lane, 0};
  const int T = 32 * p.warps, tid = grp.warp * 32 + lane;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  for (int i = threadIdx.x; i < kBackMaxGroups * 64; i += blockDim.x) red[i] = make_float2(0.0f, 0.0f);
  if (threadIdx.x == 0) {
    for (int i = 0; i < p.groups * p.stages; ++i) mbar_init(&full[i], 1);
    mbar_init(&stall_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();

  const int dy_bytes = 2 * p.D, x_bytes = SAVE ? p.D : 2 * p.D;
  const int stage_bytes = dy_bytes + x_bytes;
  uint8_t* mine = ring + g * p.stages * stage_bytes;
  uint64_t* bars = full + g * p.stages;
  volatile int* aborted = &abort_flag;
  auto issue = [&](int st, int64_t r) {
    mbar_arrive_expect_tx(&bars[st], stage_bytes);
    bulk_load(mine + st * stage_bytes, p.dy + r * p.D, dy_bytes, &bars[st]);
    if (SAVE)
      bulk_load(mine + st * stage_bytes + dy_bytes, p.q + r * p.D, x_bytes, &bars[st]);
    else
      bulk_load(mine + st * stage_bytes + dy_bytes, p.x + r * p.D, x_bytes, &bars[st]);
  };
  // Groups of a CTA are a grid apart, so that few rows spread over all CTAs.
  const int64_t r0 = static_cast<int64_t>(g) * gridDim.x + blockIdx.x;
  int issued = 0;
  if (tid == 0)
    for (; issued < p.stages && r0 + issued * step < p.M; ++issued) {
      if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
        mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
        break;
      }
      issue(issued, r0 + issued * step);
    }

  const float inv = 1.0f / static_cast<float>(p.D);
  const W* w = static_cast<const W*>(p.w) + tid * 8;
  f32x2 dw[EPT / 2] = {}, db[EPT / 2] = {};
  uint32_t ps[V], ps_next[V];
  float mean_next = 0.0f, rstd_next = 0.0f;
  auto fetch = [&](int64_t r) {              // what the copies do not bring
    if (r >= p.M) return;
    mean_next = __ldg(p.mean + r);
    rstd_next = __ldg(p.rstd + r);
    if (SAVE) {
      const uint8_t* s = p.s + blocked_offset(r, 0, 4 * p.s_words) + (lane >> 2 & 3);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * T + tid) * 8;
        if (c < p.D) ps_next[i] = __ldg(s + (c >> 7) * 512);
      }
    }
  };
#pragma unroll
  for (int i = 0; i < V; ++i) ps_next[i] = 127;
  fetch(r0);
  int st = 0;
  uint32_t parity = 0;
  for (int64_t r = r0; r < p.M; r += step) {
    const float mean = mean_next, rstd = rstd_next;
#pragma unroll
    for (int i = 0; i < V; ++i) ps[i] = ps_next[i];
    fetch(r + step);
    mbar_wait(&bars[st], parity, aborted);
    const uint8_t* sd = mine + st * stage_bytes + tid * 16;
    const uint8_t* sx = mine + st * stage_bytes + dy_bytes + tid * (SAVE ? 8 : 16);
    const f32x2 rs = pair(rstd, rstd), ms = pair(-mean, -mean);
    uint4 wd[V];
    uint4 wx[V];                              // saved bytes: in .x and .y
    f32x2 xh[EPT == 16 ? EPT / 2 : 4], gr[EPT == 16 ? EPT / 2 : 4];
    f32x2 s1 = 0, s2 = 0;
    // xh and g of piece i from its words.
    auto piece = [&](int i, f32x2* xv, f32x2* gv, f32x2* d) {
      get_pairs(wd[i], d);
      if constexpr (SAVE) mx_get_pairs(make_uint2(wx[i].x, wx[i].y), ps[i], xv);
      else get_pairs(wx[i], xv);
      f32x2 wv[4];
      load_param_pairs(w + i * T * 8, wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        xv[j] = mul2(add2(xv[j], ms), rs);
        gv[j] = mul2(d[j], wv[j]);
      }
    };
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((i * T + tid) * 8 >= p.D) continue;
      wd[i] = *reinterpret_cast<const uint4*>(sd + i * T * 16);
      if constexpr (SAVE) {
        const uint2 v = *reinterpret_cast<const uint2*>(sx + i * T * 8);
        wx[i] = make_uint4(v.x, v.y, 0, 0);
      } else {
        wx[i] = *reinterpret_cast<const uint4*>(sx + i * T * 16);
      }
      f32x2 d[4];
      f32x2* xv = xh + (EPT == 16 ? 4 * i : 0);
      f32x2* gv = gr + (EPT == 16 ? 4 * i : 0);
      piece(i, xv, gv, d);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s1 = add2(s1, gv[j]);
        s2 = fma2(gv[j], xv[j], s2);
        dw[4 * i + j] = fma2(d[j], xv[j], dw[4 * i + j]);
        db[4 * i + j] = add2(db[4 * i + j], d[j]);
      }
    }
    const float2 t = grp.sum2(sum_pair(s1), sum_pair(s2));
    if (p.warps == 1) __syncwarp();
    if (tid == 0 && r + p.stages * step < p.M && !*aborted) {
      if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
        mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
      } else {
        issue(st, r + p.stages * step);
        ++issued;
      }
    }
    // dx = rstd g - rstd c1 - xh rstd c2
    const float c1 = -rstd * (t.x * inv), c2 = -rstd * (t.y * inv);
    const f32x2 k1 = pair(c1, c1), k2 = pair(c2, c2);
    uint16_t* dx = p.dx + r * p.D + tid * 8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if ((i * T + tid) * 8 >= p.D) continue;
      f32x2* xv = xh + (EPT == 16 ? 4 * i : 0);
      f32x2* gv = gr + (EPT == 16 ? 4 * i : 0);
      if constexpr (EPT != 16) {
        f32x2 d[4];
        piece(i, xv, gv, d);
      }
      f32x2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fma2(xv[j], k2, fma2(gv[j], rs, k1));
      if (in_span(p.sp_dx, dx + i * T * 8, 16)) *reinterpret_cast<uint4*>(dx + i * T * 8) = pack_pairs(o);
    }
    if (++st == p.stages) {
      st = 0;
      parity ^= 1;
    }
  }
  if (tid == 0 && abort_flag) {
    // Gave up: the copies still in flight land (bounded) before the CTA ends.
    for (int j = issued > p.stages ? issued - p.stages : 0; j < issued; ++j)
      mbar_drain(&bars[j % p.stages], static_cast<uint32_t>((j / p.stages) & 1), 100000000ull);
    atomicOr(&g_norm_watchdog, 1);
  }
  // This CTA's partial sums: its groups' in order, through shared memory.
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  if (p.groups > 1) {
    float* sums = reinterpret_cast<float*>(ring);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < EPT / 2; ++k) {
      float lo, hi;
      unpair(dw[k], lo, hi);
      sums[(g * 2 * EPT + 2 * k) * T + tid] = lo;
      sums[(g * 2 * EPT + 2 * k + 1) * T + tid] = hi;
      unpair(db[k], lo, hi);
      sums[(g * 2 * EPT + EPT + 2 * k) * T + tid] = lo;
      sums[(g * 2 * EPT + EPT + 2 * k + 1) * T + tid] = hi;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < 2 * EPT * T; k += blockDim.x) {
      const int v = k / T, id = k - v * T;                // value v of thread id
      const int c = (((v % EPT) >> 3) * T + id) * 8 + (v & 7);
      if (c >= p.D) continue;
      float a = 0.0f;
      for (int h = 0; h < p.groups; ++h) a += sums[h * 2 * EPT * T + k];
      float* at = part + (v < EPT ? 0 : p.D) + c;
      if (in_span(p.sp_parts, at, 4)) *at = a;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * T + tid) * 8;
    if (c >= p.D || !in_span(p.sp_parts, part + p.D + c, 32)) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      *reinterpret_cast<ulonglong2*>(part + c + 4 * j) = make_ulonglong2(dw[4 * i + 2 * j], dw[4 * i + 2 * j + 1]);
      *reinterpret_cast<ulonglong2*>(part + p.D + c + 4 * j) = make_ulonglong2(db[4 * i + 2 * j], db[4 * i + 2 * j + 1]);
    }
  }
}

// Other rows, in pieces of two values or one.  MAXT: 512 threads with the
// registers they need, or 1024 for rows of more than 8192 values.
template <int VEC, typename W, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_back_kernel(const NormBackParams p) {
  constexpr int V = kPer / VEC;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ float sums[];            // groups > 1: 2 x padded row
  __shared__ __align__(16) float2 red[8 * 64];
  for (int i = threadIdx.x; i < 8 * 64; i += blockDim.x) red[i] = make_float2(0.0f, 0.0f);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / p.warps;
  Group grp{red + 64 * g, g + 1, p.warps, warp - g * p.warps, lane, 0};
  const int T = 32 * p.warps, tid = grp.warp * 32 + lane;
  const int64_t step = static_cast<int64_t>(gridDim.x) * p.groups;
  const float inv = 1.0f / static_cast<float>(p.D);
  const W* w = static_cast<const W*>(p.w);
  float dw[kPer] = {}, db[kPer] = {};
  for (int64_t r = static_cast<int64_t>(blockIdx.x) * p.groups + g; r < p.M; r += step) {
    float xh[kPer], dy[kPer], gr[kPer];
    const float mean = __ldg(p.mean + r), rstd = __ldg(p.rstd + r);
    float s1 = 0.0f, s2 = 0.0f;
    Piece<VEC> pd[V], px[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * T + tid) * VEC;
      pd[i].zero();
      px[i].zero();
      if (c >= p.D) continue;
      pd[i].load(p.dy + r * p.D + c);
      px[i].load(p.x + r * p.D + c);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * T + tid) * VEC;
      const bool live = c < p.D;
      float wv[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j) wv[j] = 0.0f;
      if (live) load_param<VEC>(w + c, wv);
      pd[i].get(dy + i * VEC);
      px[i].get(xh + i * VEC);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const int k = i * VEC + j;
        xh[k] = live ? (xh[k] - mean) * rstd : 0.0f;
        gr[k] = dy[k] * wv[j];
        s1 += gr[k];
        s2 += gr[k] * xh[k];
        dw[k] += dy[k] * xh[k];
        db[k] += dy[k];
      }
    }
    const float2 t = grp.sum2(s1, s2);
    const float c1 = t.x * inv, c2 = t.y * inv;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * T + tid) * VEC;
      if (c >= p.D) continue;
      float d[VEC];
#pragma unroll
      for (int j = 0; j < VEC; ++j)
        d[j] = rstd * (gr[i * VEC + j] - c1 - xh[i * VEC + j] * c2);
      store_bf16<VEC>(p.dx + r * p.D + c, d, p.sp_dx);
    }
  }
  // Groups of the CTA in order into group 0, then this CTA's partial sums.
  for (int k = 1; k < p.groups; ++k) {
    __syncthreads();
    if (g == k)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        sums[i * T + tid] = dw[i];
        sums[(kPer + i) * T + tid] = db[i];
      }
    __syncthreads();
    if (g == 0)
#pragma unroll
      for (int i = 0; i < kPer; ++i) {
        dw[i] += sums[i * T + tid];
        db[i] += sums[(kPer + i) * T + tid];
      }
  }
  if (g != 0) return;
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (i * T + tid) * VEC;
    if (c >= p.D || !in_span(p.sp_parts, part + p.D + c, 4 * VEC)) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      part[c + j] = dw[i * VEC + j];
      part[p.D + c + j] = db[i * VEC + j];
    }
  }
}

// dw and db: 32 columns a CTA; 32 runs of partial sums, then the runs in order.
template <typename W>
__global__ void __launch_bounds__(1024) norm_grad_kernel(const float* parts, int n, int D, W* dw,
                                                         W* db, Span sp_dw, Span sp_db) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float2 run[32][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float2 v = make_float2(0.0f, 0.0f);
  if (c < D)
    for (int i = k; i < n; i += 32) {
      v.x += __ldcg(parts + static_cast<int64_t>(i) * 2 * D + c);
      v.y += __ldcg(parts + static_cast<int64_t>(i) * 2 * D + D + c);
    }
  run[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k != 0 || c >= D) return;
  float a = 0.0f, b = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a += run[i][threadIdx.x].x;
    b += run[i][threadIdx.x].y;
  }
  auto put = [](W* p, float f, const Span& sp) {
    if (!in_span(sp, p, sizeof(W))) return;
    if constexpr (sizeof(W) == 4) *p = f;
    else *p = static_cast<W>(pack_bf16(f, 0.0f));
  };
  put(dw + c, a, sp_dw);
  if (db) put(db + c, b, sp_db);
}

template <typename... A>
int launch(void (*kernel)(A...), int grid, int threads, int smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Warps of a row's group of `per` values a thread, and groups of a CTA: `most`
// warps' worth.
void shape_of(int64_t D, int per, int most, int* warps, int* groups) {
  *warps = static_cast<int>((D + 32 * per - 1) / (32 * per));
  *groups = *warps < most ? most / *warps : 1;
}

template <typename K>
int run_norm(K kernel, NormParams p, int per_thread, int num_sms, cudaStream_t stream) {
  shape_of(p.D, per_thread, per_thread == kWide ? 4 : 8, &p.warps, &p.groups);
  const int threads = 32 * p.warps * p.groups;
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess ||
      per < 1)
    per = 1;
  const int64_t want = (p.rows + p.groups - 1) / p.groups;
  const int64_t most = static_cast<int64_t>(num_sms) * per;
  return launch(kernel, static_cast<int>(want < most ? want : most), threads, 0, stream, p);
}

template <int VEC, typename W>
int run_norm_back(NormBackParams p, int num_sms, int* grid, cudaStream_t stream) {
  shape_of(p.D, kPer, 8, &p.warps, &p.groups);
  const int threads = 32 * p.warps * p.groups;
  const int smem = p.groups > 1 ? 2 * kPer * 32 * p.warps * 4 : 0;
  const int64_t want = (p.M + p.groups - 1) / p.groups;
  int64_t most = 2 * static_cast<int64_t>(num_sms);
  if (most > kNormMaxParts) most = kNormMaxParts;
  *grid = static_cast<int>(want < most ? want : most);
  return threads <= 512 ? launch(norm_back_kernel<VEC, W, 512>, *grid, threads, smem, stream, p)
                        : launch(norm_back_kernel<VEC, W, 1024>, *grid, threads, smem, stream, p);
}

template <bool SAVE, typename W, int EPT>
int run_norm_back_rows8(NormBackParams p, int num_sms, int* grid, cudaStream_t stream) {
  shape_of(p.D, EPT, EPT == 16 ? kBackThreads / 32 : 16, &p.warps, &p.groups);
  if (p.warps > 1 && p.groups > 15) p.groups = 15;   // named barriers
  const int64_t stage = static_cast<int64_t>(p.D) * (SAVE ? 3 : 4);
  p.stages = static_cast<int>(kBackRing / (p.groups * stage));
  if (p.stages > kBackMaxStages) p.stages = kBackMaxStages;
  if (p.stages < 1) p.stages = 1;
  int64_t smem = p.groups * p.stages * stage;
  const int64_t sums = p.groups > 1 ? int64_t{2} * EPT * 32 * p.warps * 4 * p.groups : 0;
  if (smem < sums) smem = sums;
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(norm_back_rows8_kernel<SAVE, W, EPT>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kBackRing));
  });
  if (attr != 0) return attr;
  int64_t most = num_sms;
  if (most > kNormMaxParts) most = kNormMaxParts;
  *grid = static_cast<int>(p.M < most ? p.M : most);
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  return launch(norm_back_rows8_kernel<SAVE, W, EPT>, *grid, 32 * p.warps * p.groups,
                static_cast<int>(smem), stream, p);
}

template <typename W>
int run_back(const NormBackParams& p, int num_sms, int* grid, cudaStream_t stream) {
  const bool wide = p.D > 16 * 512;
  if (p.q)
    return wide ? run_norm_back_rows8<true, W, 32>(p, num_sms, grid, stream)
                : run_norm_back_rows8<true, W, 16>(p, num_sms, grid, stream);
  if (p.D % 8 == 0)
    return wide ? run_norm_back_rows8<false, W, 32>(p, num_sms, grid, stream)
                : run_norm_back_rows8<false, W, 16>(p, num_sms, grid, stream);
  return p.D % 2 == 0 ? run_norm_back<2, W>(p, num_sms, grid, stream)
                      : run_norm_back<1, W>(p, num_sms, grid, stream);
}

template <typename W>
int run_forward(const NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.q) return run_norm(norm_rows8_kernel<true, W>, p, kWide, num_sms, stream);
  if (p.D % 8 == 0) return run_norm(norm_rows8_kernel<false, W>, p, kWide, num_sms, stream);
  return p.D % 2 == 0 ? run_norm(norm_kernel<2, W>, p, kPer, num_sms, stream)
                      : run_norm(norm_kernel<1, W>, p, kPer, num_sms, stream);
}

}  // namespace

int64_t norm_back_parts(int64_t M) { return M < kNormMaxParts ? M : kNormMaxParts; }

int launch_layer_norm(const LayerNormArgs& a, int num_sms, cudaStream_t stream) {
  NormParams p = {};
  p.x = static_cast<const uint16_t*>(a.x);
  p.w = a.w;
  p.b = a.b;
  p.y = static_cast<uint16_t*>(a.y);
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.q = static_cast<uint8_t*>(a.q);
  p.s = static_cast<uint8_t*>(a.s);
  p.M = a.M;
  p.rows = a.q ? (a.M + 127) / 128 * 128 : a.M;
  p.D = static_cast<int>(a.D);
  p.s_words = static_cast<int>((a.D + 127) / 128);
  p.eps = a.eps;
  const uint64_t n = static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.D);
  p.sp_y = make_span(a.y, 2 * n);
  p.sp_mean = make_span(a.mean, 4 * static_cast<uint64_t>(a.M));
  p.sp_rstd = make_span(a.rstd, 4 * static_cast<uint64_t>(a.M));
  p.sp_q = make_span(a.q, n);
  p.sp_s = make_span(a.s, static_cast<uint64_t>(p.rows) * 4 * p.s_words);
  return a.w_f32 ? run_forward<float>(p, num_sms, stream) : run_forward<uint16_t>(p, num_sms, stream);
}

int launch_layer_norm_backward(const LayerNormBackArgs& a, int num_sms, cudaStream_t stream) {
  NormBackParams p = {};
  p.dy = static_cast<const uint16_t*>(a.dy);
  p.x = static_cast<const uint16_t*>(a.x);
  p.q = static_cast<const uint8_t*>(a.q);
  p.s = static_cast<const uint8_t*>(a.s);
  p.w = a.w;
  p.mean = a.mean;
  p.rstd = a.rstd;
  p.dx = static_cast<uint16_t*>(a.dx);
  p.parts = a.work;
  p.M = a.M;
  p.D = static_cast<int>(a.D);
  p.s_words = static_cast<int>((a.D + 127) / 128);
  p.sp_dx = make_span(a.dx, 2 * static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.D));
  p.sp_parts = make_span(a.work, static_cast<uint64_t>(norm_back_parts(a.M)) * 8 * a.D);
  int grid = 0;
  const int rc = a.w_f32 ? run_back<float>(p, num_sms, &grid, stream)
                         : run_back<uint16_t>(p, num_sms, &grid, stream);
  if (rc) return rc;
  const int blocks = (p.D + 31) / 32;
  const uint64_t wb = static_cast<uint64_t>(a.D) * (a.w_f32 ? 4 : 2);
  if (a.w_f32)
    return launch(norm_grad_kernel<float>, blocks, 1024, 0, stream,
                  static_cast<const float*>(a.work), grid, p.D, static_cast<float*>(a.dw),
                  static_cast<float*>(a.db), make_span(a.dw, wb), make_span(a.db, wb));
  return launch(norm_grad_kernel<uint16_t>, blocks, 1024, 0, stream,
                static_cast<const float*>(a.work), grid, p.D, static_cast<uint16_t*>(a.dw),
                static_cast<uint16_t*>(a.db), make_span(a.dw, wb), make_span(a.db, wb));
}

int out_of_bounds_norm(bool clear) { return read_out_of_bounds(clear); }

int read_norm_watchdog(int* out, bool clear) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_norm_watchdog, sizeof(int));
  if (e != cudaSuccess) return static_cast<int>(e);
  if (clear && v) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_norm_watchdog, &z, sizeof(int));
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  *out = v;
  return 0;
}

}  // namespace mx
