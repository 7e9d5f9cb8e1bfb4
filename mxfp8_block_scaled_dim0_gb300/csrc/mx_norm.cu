// mx_norm.cu -- layer norm of bf16 rows, forward and backward, with its input
// saved as MX-FP8 for the backward pass.
//
//   mean = (1/D) sum x, rstd = (eps + (1/D) sum (x - mean)^2)^(-1/2)
//   y    = (x - mean) rstd w + b
//   xh   = (x - mean) rstd, g = dy w
//   dx   = rstd (g - (1/D) sum g - xh (1/D) sum g xh)
//   dw   = sum over rows of dy xh, db = sum over rows of dy
//
// A group of warps works on a row.  Rows of a multiple of 8 values come into
// shared memory by bulk copies, a ring of rows for every group, so that what is
// in flight takes no registers and no instruction waits for memory; each SM runs
// one CTA of several groups, which share w and b in shared memory.  A row's
// place in shared memory is padded with zeros to the group's whole width, so
// that the arithmetic needs no conditions.  (Rows loaded a row ahead into
// registers, four CTAs an SM: 94 us forward and 159 us backward at 16640 x 5120
// with the 8-bit save.)  Other rows go through registers in pieces of two values
// or one.
//
// The backward kernel keeps dw and db of its threads' columns in registers over
// all its rows, adds the groups of a CTA up at its end, and leaves one partial
// sum per CTA in the workspace, which norm_grad_kernel adds up in a fixed order.
#include <cuda_runtime.h>

#include "mx_kernels.h"
#include "mx_rows.cuh"

namespace mx {
namespace {

constexpr int kPer = 16;                     // values a thread holds of a row
constexpr int kMaxThreads = 1024;

// Every wait is bounded: one that runs out raises the abort flag, the threads go
// on to the end without waiting, and the watchdog word is set.
__device__ int g_norm_watchdog = 0;

constexpr int kRingThreads = 640;           // forward
constexpr int kBackThreads = 512;
constexpr int kMaxGroups = 20;
constexpr int kMaxStages = 4;
constexpr int kRingBytes = 212 * 1024;       // rings, w and b

// How rows of a multiple of 8 values are shared out.
struct RowShape {
  int warps;           // of a group
  int groups;          // of a CTA
  int stages;          // rows of a group's ring
  int pitch;           // values a group holds: 32 warps EPT >= D
};

// Clears the rings' padding (all of it, once) and sets up the barriers.
__device__ __forceinline__ void ring_setup(uint8_t* ring, int bytes, uint64_t* full, int n,
                                           uint64_t* stall_bar, int* abort_flag, float* red) {
  for (int i = threadIdx.x; i < bytes / 16; i += blockDim.x)
    reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
  for (int i = threadIdx.x; i < kMaxGroups * 128; i += blockDim.x) red[i] = 0.0f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < n; ++i) mbar_init(&full[i], 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  fence_proxy_async_smem();                  // the copies write what was cleared
}

struct NormParams {
  const uint16_t* x;
  const void* w;
  const void* b;
  uint16_t* y;
  float* mean;
  float* rstd;
  uint8_t* q;
  uint8_t* s;
  int64_t M;
  int D, warps, groups;
  RowShape shape;
  int s_words;         // 128x4 scale tiles of a row
  int staged;          // w and b are read from shared memory
  float eps;
  Span sp_y, sp_mean, sp_rstd, sp_q, sp_s;
  int64_t stall_at;
  uint64_t stall_ns;
};

// EPT values a thread, as pairs.
template <bool SAVE, typename W, int EPT>
__global__ void __launch_bounds__(kRingThreads, 1) norm_rows8_kernel(const NormParams p) {
  constexpr int V = EPT / 8;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[kMaxGroups * 128];
  __shared__ __align__(8) uint64_t full[kMaxGroups * kMaxStages];
  __shared__ __align__(8) uint64_t stall_bar;   // diagnostic: never completed
  __shared__ int abort_flag;
  const RowShape& sh = p.shape;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / sh.warps;
  Group<16> grp{red + 128 * g, g + 1, sh.warps, warp - g * sh.warps, lane, 0};
  const int T = 32 * sh.warps, tid = grp.warp * 32 + lane;
  const int stage_bytes = 2 * sh.pitch;
  const int ring_bytes = sh.groups * sh.stages * stage_bytes;
  ring_setup(ring, ring_bytes, full, sh.groups * sh.stages, &stall_bar, &abort_flag, red);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* params = reinterpret_cast<float*>(ring + ring_bytes);   // w, then b
  if (p.staged) {
    stage_params(params, static_cast<const W*>(p.w), p.D, sh.pitch);
    stage_params(params + sh.pitch, static_cast<const W*>(p.b), p.b ? p.D : 0, sh.pitch);
  }
  __syncthreads();

  uint8_t* mine = ring + g * sh.stages * stage_bytes;
  uint64_t* bars = full + g * sh.stages;
  volatile int* aborted = &abort_flag;
  auto issue = [&](int st, int64_t r) {
    mbar_arrive_expect_tx(&bars[st], 2 * p.D);
    bulk_load(mine + st * stage_bytes, p.x + r * p.D, 2 * p.D, &bars[st]);
  };
  // Groups of a CTA are a grid apart, so that few rows spread over all CTAs.
  const int64_t r0 = static_cast<int64_t>(g) * gridDim.x + blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * sh.groups;
  int issued = 0;
  if (tid == 0)
    for (; issued < sh.stages && r0 + issued * step < p.M; ++issued) {
      if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
        mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
        break;
      }
      issue(issued, r0 + issued * step);
    }

  const float inv = 1.0f / static_cast<float>(p.D);
  // Piece i of this thread is piece first + 32 i of the row (a warp's pieces lie
  // together, so that their distances are constants).  One lane of a block's
  // four writes its scale; blocks past the row are zero and give 0, the padding
  // of the blocked layout.
  const int first = grp.warp * 32 * V + lane;
  const int pieces = (p.D >> 3) - first;       // live: 32 i < pieces
  const int scaled = SAVE && (lane & 3) == 0 ? 16 * p.s_words - first : 0;
  int st = 0;
  uint32_t parity = 0;
  for (int64_t r = r0; r < p.M; r += step) {
    mbar_wait(&bars[st], parity, aborted);
    const uint8_t* row = mine + st * stage_bytes + first * 16;
    uint8_t* q = SAVE ? p.q + r * p.D + first * 8 : nullptr;
    uint8_t* s = SAVE ? p.s + blocked_offset(r, 0, 4 * p.s_words) + (first >> 4) * 512 +
                            (first >> 2 & 3)
                      : nullptr;
    f32x2 x[EPT / 2];
    f32x2 s2 = 0, s3 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint4 v = *reinterpret_cast<const uint4*>(row + i * 512);
      get_pairs(v, x + 4 * i);
      s2 = add2(s2, add2(x[4 * i], x[4 * i + 1]));
      s3 = add2(s3, add2(x[4 * i + 2], x[4 * i + 3]));
      if constexpr (SAVE) {
        uint32_t sb;
        const uint2 o = mx_cast_pairs(v, x + 4 * i, sb);
        if (32 * i < pieces && in_span(p.sp_q, q + i * 256, 8))
          *reinterpret_cast<uint2*>(q + i * 256) = o;
        if (32 * i < scaled && in_span(p.sp_s, s + i * 1024, 1))
          s[i * 1024] = static_cast<uint8_t>(sb);
      }
    }
    const float mean = grp.sum(sum_pair(add2(s2, s3))) * inv;
    if (sh.warps == 1) __syncwarp();
    // Every thread of the group has read the row: fill its place again.
    if (tid == 0 && r + sh.stages * step < p.M && !*aborted) {
      if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
        mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
      } else {
        issue(st, r + sh.stages * step);
        ++issued;
      }
    }
    s2 = s3 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float m = 32 * i < pieces ? -mean : 0.0f;      // padding stays 0
      const f32x2 m2 = pair(m, m);
#pragma unroll
      for (int j = 4 * i; j < 4 * i + 4; j += 2) {
        x[j] = add2(x[j], m2);
        x[j + 1] = add2(x[j + 1], m2);
        s2 = fma2(x[j], x[j], s2);
        s3 = fma2(x[j + 1], x[j + 1], s3);
      }
    }
    const float rstd = rsqrtf(grp.sum(sum_pair(add2(s2, s3))) * inv + p.eps);
    if (tid == 0) {
      if (in_span(p.sp_mean, p.mean + r, 4)) p.mean[r] = mean;
      if (in_span(p.sp_rstd, p.rstd + r, 4)) p.rstd[r] = rstd;
    }
    const f32x2 r2 = pair(rstd, rstd);
    uint16_t* y = p.y + r * p.D + first * 8;
    auto put = [&](int i, const f32x2* wv, const f32x2* bv) {
      f32x2 o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fma2(mul2(x[4 * i + j], r2), wv[j], bv[j]);
      if (32 * i < pieces && in_span(p.sp_y, y + i * 256, 16))
        *reinterpret_cast<uint4*>(y + i * 256) = pack_pairs(o);
    };
    if (p.staged) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f32x2 wv[4], bv[4];
        staged_pairs(params, sh.pitch, first + 32 * i, wv);
        staged_pairs(params + sh.pitch, sh.pitch, first + 32 * i, bv);
        put(i, wv, bv);
      }
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f32x2 wv[4] = {0, 0, 0, 0}, bv[4] = {0, 0, 0, 0};
        if (32 * i < pieces) {
          load_param_pairs(static_cast<const W*>(p.w) + (first + 32 * i) * 8, wv);
          if (p.b) load_param_pairs(static_cast<const W*>(p.b) + (first + 32 * i) * 8, bv);
        }
        put(i, wv, bv);
      }
    }
    if (++st == sh.stages) {
      st = 0;
      parity ^= 1;
    }
  }
  if (SAVE && blockIdx.x == 0) {
    // Rows of scales past the matrix: zero.
    const int64_t n = ((p.M + 127) / 128 * 128 - p.M) * p.s_words;
    for (int64_t i = threadIdx.x; i < n; i += blockDim.x) {
      uint8_t* s = p.s + blocked_offset(p.M + i / p.s_words, (i % p.s_words) * 4, 4 * p.s_words);
      if (in_span(p.sp_s, s, 4)) *reinterpret_cast<uint32_t*>(s) = 0;
    }
  }
  if (tid == 0 && abort_flag) {
    // Gave up: the copies still in flight land (bounded) before the CTA ends.
    for (int j = issued > sh.stages ? issued - sh.stages : 0; j < issued; ++j)
      mbar_drain(&bars[j % sh.stages], static_cast<uint32_t>((j / sh.stages) & 1), 100000000ull);
    atomicOr(&g_norm_watchdog, 1);
  }
}

// Other rows, in pieces of two values or one.
template <int VEC, typename W>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const NormParams p) {
  constexpr int V = kPer / VEC;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float red[8 * 128];
  for (int i = threadIdx.x; i < 8 * 128; i += blockDim.x) red[i] = 0.0f;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / p.warps;
  Group<32> grp{red + 128 * g, g + 1, p.warps, warp - g * p.warps, lane, 0};
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
    const float rstd = rsqrtf(grp.sum(sq) * inv + p.eps);
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
  int D, warps, groups;
  RowShape shape;
  int s_words;
  Span sp_dx, sp_parts;
  int64_t stall_at;
  uint64_t stall_ns;
};

// EPT values a thread.  The second pass reads the row from shared memory again:
// with dw and db in 2 EPT registers there is no room for more of the row (16
// values a thread, held from the first pass: 117 us where this takes 85).
template <bool SAVE, typename W, int EPT>
__global__ void __launch_bounds__(kBackThreads, 1) norm_back_rows8_kernel(const NormBackParams p) {
  constexpr int V = EPT / 8;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[kMaxGroups * 128];
  __shared__ __align__(8) uint64_t full[kMaxGroups * kMaxStages];
  __shared__ __align__(8) uint64_t stall_bar;   // diagnostic: never completed
  __shared__ int abort_flag;
  const RowShape& sh = p.shape;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / sh.warps;
  Group<16> grp{red + 128 * g, g + 1, sh.warps, warp - g * sh.warps, lane, 0};
  const int T = 32 * sh.warps, tid = grp.warp * 32 + lane;
  const int x_at = 2 * sh.pitch, stage_bytes = (SAVE ? 3 : 4) * sh.pitch;
  const int ring_bytes = sh.groups * sh.stages * stage_bytes;
  ring_setup(ring, ring_bytes, full, sh.groups * sh.stages, &stall_bar, &abort_flag, red);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* params = reinterpret_cast<float*>(ring + ring_bytes);   // w
  stage_params(params, static_cast<const W*>(p.w), p.D, sh.pitch);
  __syncthreads();

  uint8_t* mine = ring + g * sh.stages * stage_bytes;
  uint64_t* bars = full + g * sh.stages;
  volatile int* aborted = &abort_flag;
  auto issue = [&](int st, int64_t r) {
    uint8_t* to = mine + st * stage_bytes;
    mbar_arrive_expect_tx(&bars[st], (SAVE ? 3 : 4) * p.D);
    bulk_load(to, p.dy + r * p.D, 2 * p.D, &bars[st]);
    if (SAVE)
      bulk_load(to + x_at, p.q + r * p.D, p.D, &bars[st]);
    else
      bulk_load(to + x_at, p.x + r * p.D, 2 * p.D, &bars[st]);
  };
  // Groups of a CTA are a grid apart, so that few rows spread over all CTAs.
  const int64_t r0 = static_cast<int64_t>(g) * gridDim.x + blockIdx.x;
  const int64_t step = static_cast<int64_t>(gridDim.x) * sh.groups;
  int issued = 0;
  if (tid == 0)
    for (; issued < sh.stages && r0 + issued * step < p.M; ++issued) {
      if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
        mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
        break;
      }
      issue(issued, r0 + issued * step);
    }

  const float inv = 1.0f / static_cast<float>(p.D);
  f32x2 dw[EPT / 2] = {}, db[EPT / 2] = {};
  // Piece i of this thread is piece first + 32 i of the row (a warp's pieces lie
  // together, so that their distances are constants).
  const int first = grp.warp * 32 * V + lane;
  const int pieces = (p.D >> 3) - first;       // live: 32 i < pieces
  // What the copies do not bring, a row ahead; without a condition, for loads
  // under one are waited for where it ends.  A warp's scales are 2 V words of
  // four, one to a lane (past the row its last word: the values there are 0).
  uint32_t words_next;
  const int word = min(grp.warp * 2 * V + (lane & (2 * V - 1)), p.s_words - 1) * 512;
  const int byte = (lane >> 2 & 3) * 8;
  float mean_next, rstd_next;
  auto fetch = [&](int64_t r) {
    r = r < p.M ? r : p.M - 1;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(mean_next) : "l"(p.mean + r));
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(rstd_next) : "l"(p.rstd + r));
    if constexpr (SAVE) {
      asm volatile("ld.global.nc.u32 %0, [%1];"
                   : "=r"(words_next)
                   : "l"(p.s + blocked_offset(r, 0, 4 * p.s_words) + word));
    }
  };
  fetch(r0);
  int st = 0;
  uint32_t parity = 0;
  for (int64_t r = r0; r < p.M; r += step) {
    const float rstd = rstd_next;
    const f32x2 rs = pair(rstd, rstd), ms = pair(-mean_next, -mean_next);
    float mult[V];
    if constexpr (SAVE) {
#pragma unroll
      for (int i = 0; i < V; ++i)
        mult[i] = scale_mult(
            __shfl_sync(0xffffffffu, words_next, 2 * i + (lane >> 4)) >> byte & 0xFFu);
    }
    fetch(r + step);
    mbar_wait(&bars[st], parity, aborted);
    const uint8_t* sd = mine + st * stage_bytes + first * 16;
    const uint8_t* sx = mine + st * stage_bytes + x_at + first * (SAVE ? 8 : 16);
    // x - mean of piece i.
    auto get_x = [&](int i, f32x2* xv) {
      if constexpr (SAVE) {
        const uint2 q = *reinterpret_cast<const uint2*>(sx + i * 256);
        const uint32_t w[4] = {q.x, q.x >> 16, q.y, q.y >> 16};
        const f32x2 m = pair(mult[i], mult[i]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float lo, hi;
          e4m3x2_get(w[j], lo, hi);
          xv[j] = fma2(pair(lo, hi), m, ms);
        }
      } else {
        get_pairs(*reinterpret_cast<const uint4*>(sx + i * 512), xv);
#pragma unroll
        for (int j = 0; j < 4; ++j) xv[j] = add2(xv[j], ms);
      }
    };
    f32x2 s1 = 0, s2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f32x2 xv[4], d[4], wv[4];
      get_x(i, xv);
      get_pairs(*reinterpret_cast<const uint4*>(sd + i * 512), d);
      staged_pairs(params, sh.pitch, first + 32 * i, wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const f32x2 gv = mul2(d[j], wv[j]);
        xv[j] = mul2(xv[j], rs);
        s1 = add2(s1, gv);
        s2 = fma2(gv, xv[j], s2);
        dw[4 * i + j] = fma2(d[j], xv[j], dw[4 * i + j]);
        db[4 * i + j] = add2(db[4 * i + j], d[j]);
      }
    }
    const float2 t = grp.sum2(sum_pair(s1), sum_pair(s2));
    asm volatile("" ::: "memory");           // the second pass reads anew
    // dx = rstd g - rstd c1 - (x - mean) rstd^2 c2
    const float c1 = -rstd * (t.x * inv), c2 = -rstd * (t.y * inv) * rstd;
    const f32x2 k1 = pair(c1, c1), k2 = pair(c2, c2);
    uint16_t* dx = p.dx + r * p.D + first * 8;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f32x2 xv[4], d[4], wv[4];
      get_x(i, xv);
      get_pairs(*reinterpret_cast<const uint4*>(sd + i * 512), d);
      staged_pairs(params, sh.pitch, first + 32 * i, wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = fma2(xv[j], k2, fma2(mul2(d[j], wv[j]), rs, k1));
      if (32 * i < pieces && in_span(p.sp_dx, dx + i * 256, 16))
        *reinterpret_cast<uint4*>(dx + i * 256) = pack_pairs(d);
    }
    grp.meet();
    // Every thread of the group has read the row: fill its place again.
    if (tid == 0 && r + sh.stages * step < p.M && !*aborted) {
      if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
        mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
      } else {
        issue(st, r + sh.stages * step);
        ++issued;
      }
    }
    if (++st == sh.stages) {
      st = 0;
      parity ^= 1;
    }
  }
  if (tid == 0 && abort_flag) {
    // Gave up: the copies still in flight land (bounded) before the CTA ends.
    for (int j = issued > sh.stages ? issued - sh.stages : 0; j < issued; ++j)
      mbar_drain(&bars[j % sh.stages], static_cast<uint32_t>((j / sh.stages) & 1), 100000000ull);
    atomicOr(&g_norm_watchdog, 1);
  }
  // This CTA's partial sums: its groups' in order, through shared memory.
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * p.D;
  if (sh.groups > 1) {
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
      const int c = ((id >> 5) * 32 * V + ((v % EPT) >> 3) * 32 + (id & 31)) * 8 + (v & 7);
      if (c >= p.D) continue;
      float a = 0.0f;
      for (int h = 0; h < sh.groups; ++h) a += sums[h * 2 * EPT * T + k];
      float* at = part + (v < EPT ? 0 : p.D) + c;
      if (in_span(p.sp_parts, at, 4)) *at = a;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = (first + 32 * i) * 8;
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
  __shared__ float red[8 * 128];
  for (int i = threadIdx.x; i < 8 * 128; i += blockDim.x) red[i] = 0.0f;
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / p.warps;
  Group<32> grp{red + 128 * g, g + 1, p.warps, warp - g * p.warps, lane, 0};
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

// dw (blockIdx.y == 0) and db: 32 columns a CTA, in pieces of VEC; each of its
// threads adds up a run of the partial sums, eight under way at a time, then the
// runs are added up in order.
template <int VEC, typename W>
__global__ void __launch_bounds__(256) norm_grad_kernel(const float* parts, int n, int D, W* dw,
                                                        W* db, Span sp_dw, Span sp_db) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  constexpr int kCols = 32 / VEC, kRuns = 256 / kCols;
  __shared__ float run[kRuns][33];
  const int l = threadIdx.x % kCols, k = threadIdx.x / kCols;
  const int c = blockIdx.x * 32 + l * VEC;
  const float* src = parts + (blockIdx.y ? D : 0) + c;
  float v[VEC] = {};
  if (c < D)
    for (int i = k; i < n; i += 8 * kRuns) {
      float u[8][VEC];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int q = i + j * kRuns;
        if constexpr (VEC == 4) {
          const float4 f = q < n ? __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(q) * 2 * D))
                                 : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          u[j][0] = f.x; u[j][1] = f.y; u[j][2] = f.z; u[j][3] = f.w;
        } else {
          u[j][0] = q < n ? __ldcg(src + static_cast<int64_t>(q) * 2 * D) : 0.0f;
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] += u[j][e];
    }
#pragma unroll
  for (int e = 0; e < VEC; ++e) run[k][l * VEC + e] = v[e];
  __syncthreads();
  const int o = blockIdx.x * 32 + threadIdx.x;
  if (threadIdx.x >= 32 || o >= D) return;
  float a = 0.0f;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) a += run[i][threadIdx.x];
  W* at = (blockIdx.y ? db : dw) + o;
  if (!in_span(blockIdx.y ? sp_db : sp_dw, at, sizeof(W))) return;
  if constexpr (sizeof(W) == 4) *at = a;
  else *at = static_cast<W>(pack_bf16(a, 0.0f));
}

template <typename... A>
int launch(void (*kernel)(A...), dim3 grid, int threads, int smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
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
int run_norm(K kernel, NormParams p, int num_sms, cudaStream_t stream) {
  shape_of(p.D, kPer, 8, &p.warps, &p.groups);
  const int threads = 32 * p.warps * p.groups;
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, 0) != cudaSuccess ||
      per < 1)
    per = 1;
  const int64_t want = (p.M + p.groups - 1) / p.groups;
  const int64_t most = static_cast<int64_t>(num_sms) * per;
  return launch(kernel, static_cast<int>(want < most ? want : most), threads, 0, stream, p);
}

// The shape for M rows of D values, `row` bytes a padded value of a stage and
// `param` bytes a value of the parameters: as many groups as fit in `threads` and
// have rows to work on, as many stages as fit.
RowShape ring_shape(int64_t M, int64_t D, int ept, int threads, int row, int param, int num_sms) {
  RowShape s = {};
  shape_of(D, ept, threads / 32, &s.warps, &s.groups);
  const int64_t rows = (M + num_sms - 1) / num_sms;
  if (s.groups > rows) s.groups = static_cast<int>(rows);
  if (s.warps > 1 && s.groups > 15) s.groups = 15;   // named barriers
  s.pitch = 32 * s.warps * ept;
  const int64_t room = kRingBytes - static_cast<int64_t>(param) * s.pitch;
  s.stages = static_cast<int>(room / (static_cast<int64_t>(s.groups) * row * s.pitch));
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  return s;
}

template <typename K>
int allow_ring(K kernel) {
  return static_cast<int>(cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes));
}

template <bool SAVE, typename W, int EPT>
int run_norm_rows8(NormParams p, int num_sms, cudaStream_t stream) {
  // With a row or two a group, w and b are not worth a copy of their own.
  p.staged = p.M > 8 * static_cast<int64_t>(num_sms);
  const int param = p.staged ? 8 : 0;
  p.shape = ring_shape(p.M, p.D, EPT, kRingThreads, 2, param, num_sms);
  const int64_t smem = static_cast<int64_t>(p.shape.pitch) *
                       (p.shape.groups * p.shape.stages * 2 + param);
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] { return allow_ring(norm_rows8_kernel<SAVE, W, EPT>); });
  if (attr != 0) return attr;
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  return launch(norm_rows8_kernel<SAVE, W, EPT>, static_cast<int>(p.M < num_sms ? p.M : num_sms),
                32 * p.shape.warps * p.shape.groups, static_cast<int>(smem), stream, p);
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
  p.shape = ring_shape(p.M, p.D, EPT, kBackThreads, SAVE ? 3 : 4, 4, num_sms);
  const RowShape& s = p.shape;
  int64_t smem = static_cast<int64_t>(s.pitch) * (s.groups * s.stages * (SAVE ? 3 : 4) + 4);
  const int64_t sums = s.groups > 1 ? int64_t{8} * s.pitch * s.groups : 0;
  if (smem < sums) smem = sums;
  static DeviceCache attr_cache;
  const int attr =
      attr_cache.get([] { return allow_ring(norm_back_rows8_kernel<SAVE, W, EPT>); });
  if (attr != 0) return attr;
  int64_t most = num_sms;
  if (most > kNormMaxParts) most = kNormMaxParts;
  *grid = static_cast<int>(p.M < most ? p.M : most);
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  return launch(norm_back_rows8_kernel<SAVE, W, EPT>, *grid, 32 * s.warps * s.groups,
                static_cast<int>(smem), stream, p);
}

// 32 values a thread; fewer where one warp then holds the row all the same.
template <bool SAVE, typename W>
int pick_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.D <= 256) return run_norm_rows8<SAVE, W, 8>(p, num_sms, stream);
  if (p.D <= 512) return run_norm_rows8<SAVE, W, 16>(p, num_sms, stream);
  return run_norm_rows8<SAVE, W, 32>(p, num_sms, stream);
}

template <bool SAVE, typename W>
int pick_norm_back(const NormBackParams& p, int num_sms, int* grid, cudaStream_t stream) {
  if (p.D <= 256) return run_norm_back_rows8<SAVE, W, 8>(p, num_sms, grid, stream);
  if (p.D <= 512) return run_norm_back_rows8<SAVE, W, 16>(p, num_sms, grid, stream);
  return run_norm_back_rows8<SAVE, W, 32>(p, num_sms, grid, stream);
}

template <typename W>
int run_back(const NormBackParams& p, int num_sms, int* grid, cudaStream_t stream) {
  if (p.q) return pick_norm_back<true, W>(p, num_sms, grid, stream);
  if (p.D % 8 == 0) return pick_norm_back<false, W>(p, num_sms, grid, stream);
  return p.D % 2 == 0 ? run_norm_back<2, W>(p, num_sms, grid, stream)
                      : run_norm_back<1, W>(p, num_sms, grid, stream);
}

template <typename W>
int run_forward(const NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.q) return pick_norm<true, W>(p, num_sms, stream);
  if (p.D % 8 == 0) return pick_norm<false, W>(p, num_sms, stream);
  return p.D % 2 == 0 ? run_norm(norm_kernel<2, W>, p, num_sms, stream)
                      : run_norm(norm_kernel<1, W>, p, num_sms, stream);
}

template <typename W>
int run_grad(const LayerNormBackArgs& a, int D, int n, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((D + 31) / 32), a.db ? 2 : 1);
  const uint64_t bytes = static_cast<uint64_t>(D) * sizeof(W);
  return launch(D % 4 == 0 ? norm_grad_kernel<4, W> : norm_grad_kernel<1, W>, grid, 256, 0, stream,
                static_cast<const float*>(a.work), n, D, static_cast<W*>(a.dw),
                static_cast<W*>(a.db), make_span(a.dw, bytes), make_span(a.db, bytes));
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
  p.D = static_cast<int>(a.D);
  p.s_words = static_cast<int>((a.D + 127) / 128);
  p.eps = a.eps;
  const uint64_t n = static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.D);
  p.sp_y = make_span(a.y, 2 * n);
  p.sp_mean = make_span(a.mean, 4 * static_cast<uint64_t>(a.M));
  p.sp_rstd = make_span(a.rstd, 4 * static_cast<uint64_t>(a.M));
  p.sp_q = make_span(a.q, n);
  p.sp_s = make_span(a.s, static_cast<uint64_t>((a.M + 127) / 128 * 128) * 4 * p.s_words);
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
  return a.w_f32 ? run_grad<float>(a, p.D, grid, stream) : run_grad<uint16_t>(a, p.D, grid, stream);
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
