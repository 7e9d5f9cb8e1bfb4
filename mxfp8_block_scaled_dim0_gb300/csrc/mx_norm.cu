// mx_norm.cu -- layer norm of bf16 rows, forward and backward, with its input
// saved as MX-FP8 for the backward pass.
//
//   mean = (1/D) sum x, rstd = (eps + (1/D) sum (x - mean)^2)^(-1/2)
//   y    = (x - mean) rstd w + b
//   xh   = (x - mean) rstd, g = dy w
//   dx   = rstd (g - (1/D) sum g - xh (1/D) sum g xh)
//   dw   = sum over rows of dy xh, db = sum over rows of dy
//
// A group of warps works on a row.  Rows come into shared memory by bulk copies,
// a ring of rows for every group, so that what is in flight takes no registers
// and no instruction waits for memory; each SM runs one CTA of several groups,
// which share w and b in shared memory.  A row's place in shared memory is padded
// with zeros to the group's whole width, so that the arithmetic needs no
// conditions.  (Rows loaded a row ahead into registers, four CTAs an SM: 94 us
// forward and 159 us backward at 16640 x 5120 with the 8-bit save.)
//
// Every tensor crosses the memory bus once: 5 bytes a value forward with the save
// and backward from it, 6 backward from bf16.  16640 x 5120: forward with the save
// 72 us (6.0 TB/s), backward from 8 bits 89 us (4.8 TB/s, the gradient kernel's
// 5 us in it), from bf16 86 us (5.9 TB/s); 1 x 4096 forward 2.4 us.  Forward is
// bound by the way through shared memory (waits for its loads, 52% of the issue
// slots taken), backward by issue and by the few warps that dw and db leave room for.
//
// Bulk copies and 16-byte accesses want 16-byte boundaries.  Where the row length
// is no multiple of 8 values, rows r and r + 8 begin at the same distance from
// one: the grid is a multiple of 8, so that all rows of a CTA have the same
// distance, `lead` values, and the CTA works on rows that begin `lead` values
// early, on the boundary, its w and b shifted by as much.  What a copy brings of
// the neighbouring rows (in the first and the last piece) is cleared by the
// thread that reads it (backward, which reads twice, in shared memory: 16640 x 4099
// 125 -> 94 us, 16640 x 500 17.2 -> 18.3), and those two pieces are stored value by value.
//
// The backward kernel keeps dw and db of its threads' columns in registers over
// all its rows, adds the groups of a CTA up at its end, and leaves one partial
// sum per CTA in the workspace, which norm_grad_kernel adds up in a fixed order.
#include <cuda_runtime.h>

#include "mx_kernels.h"
#include "mx_rows.cuh"

namespace mx {
namespace {

// Every wait is bounded: one that runs out raises the abort flag, the threads go
// on to the end without waiting, and the watchdog word is set.
__device__ int g_norm_watchdog = 0;

constexpr int kRingThreads = 640;           // forward
constexpr int kBackThreads = 512;
constexpr int kMaxGroups = 20;
constexpr int kMaxStages = 4;
constexpr int kRingBytes = 212 * 1024;       // rings, w and b

// How rows are shared out.
struct RowShape {
  int warps;           // of a group
  int groups;          // of a CTA
  int stages;          // rows of a group's ring
  int pitch;           // values a group holds: 32 warps EPT >= D (and the lead)
};

// Sets up the barriers and the sums' slots.
__device__ __forceinline__ void ring_setup(uint64_t* full, int n, uint64_t* stall_bar,
                                           int* abort_flag, float* red) {
  for (int i = threadIdx.x; i < kMaxGroups * 128; i += blockDim.x) red[i] = 0.0f;
  if (threadIdx.x == 0) {
    for (int i = 0; i < n; ++i) mbar_init(&full[i], 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
}

// Zeros in bytes [from, to) of `n` places `stride` bytes apart: the padding that
// no copy writes.  Multiples of 8.
__device__ __forceinline__ void clear_padding(uint8_t* at, int n, int stride, int from, int to) {
  const int words = (to - from) >> 3;
  for (int i = threadIdx.x; i < n * words; i += blockDim.x) {
    const int k = i / words;
    *reinterpret_cast<uint2*>(at + k * stride + from + 8 * (i - k * words)) = make_uint2(0, 0);
  }
}

// A CTA's rows: `lead` values early (ODD: the row length is no multiple of 8),
// in `total` pieces of 8 values.
template <bool ODD>
struct RowSpan {
  int lead, width, total;
  __device__ __forceinline__ explicit RowSpan(int D) {
    lead = ODD ? static_cast<int>((blockIdx.x * static_cast<unsigned>(D)) & 7u) : 0;
    width = D + lead;
    total = (width + 7) >> 3;
  }
  __device__ __forceinline__ bool edge(int c) const { return ODD && (c == 0 || c == total - 1); }
  __device__ __forceinline__ bool holds(int e) const { return e >= lead && e < width; }
  // Bit i: piece first + 32 i, of `n` that a thread works on, is the row's first or
  // last.
  __device__ __forceinline__ uint32_t edges(int first, int n) const {
    uint32_t m = 0;
    if (ODD)
      for (int i = 0; i < n; ++i)
        if (edge(first + 32 * i)) m |= 1u << i;
    return m;
  }
  // Clears what piece c, an edge, holds of the neighbouring rows.
  __device__ __forceinline__ void clear(uint4& v, int c) const {
    uint32_t* w = &v.x;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      w[k] &= (holds(8 * c + 2 * k) ? 0xFFFFu : 0u) | (holds(8 * c + 2 * k + 1) ? 0xFFFF0000u : 0u);
  }
  // The same in the row's place (at: piece `first`) for its later reads, all by
  // this thread.
  __device__ __forceinline__ void clear_place(uint8_t* at, int first, uint32_t edges) const {
    for (; edges; edges &= edges - 1) {
      const int i = __ffs(edges) - 1;
      uint4* place = reinterpret_cast<uint4*>(at + i * 512);
      uint4 v = *place;
      clear(v, first + 32 * i);
      *place = v;
    }
  }
  // Stores piece c of the row that begins at `row` (lead included).
  __device__ __forceinline__ void store(uint16_t* row, int c, const f32x2* v, const Span& sp) const {
    if (c >= total) return;
    const uint4 w = pack_pairs(v);
    uint16_t* at = row + 8 * c;
    if (!edge(c)) {
      if (in_span(sp, at, 16)) *reinterpret_cast<uint4*>(at) = w;
      return;
    }
    const uint32_t* h = &w.x;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (holds(8 * c + j) && in_span(sp, at + j, 2))
        at[j] = static_cast<uint16_t>(h[j >> 1] >> (16 * (j & 1)));
  }
  // Bytes of a row's copy, and what of them lies before the end of the M rows.
  __device__ __forceinline__ int copy_bytes(int64_t r, int64_t M, int D) const {
    if (!ODD) return 2 * D;
    const int64_t room = 2 * (M * D - (r * D - lead));
    return room < 16 * total ? static_cast<int>(room & ~int64_t{15}) : 16 * total;
  }
  // The last values of the matrix, where no 16 bytes are left.
  __device__ __forceinline__ void copy_tail(uint8_t* to, const uint16_t* row, int bytes) const {
    if (!ODD || bytes == 16 * total) return;
    uint16_t* d = reinterpret_cast<uint16_t*>(to);
    for (int e = bytes / 2; e < width; ++e) d[e] = row[e];
    fence_proxy_async_smem();
  }
};

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
  int D;
  RowShape shape;
  int s_words;         // 128x4 scale tiles of a row
  int staged;          // w and b are read from shared memory
  float eps;
  Span sp_y, sp_mean, sp_rstd, sp_q, sp_s;
  int64_t stall_at;
  uint64_t stall_ns;
};

// EPT values a thread, as pairs, and R rows a turn, which share a reading of w and b
// and the reductions' barriers.
template <bool SAVE, bool ODD, typename W, int EPT, int R>
__global__ void __launch_bounds__(R == 1 ? kRingThreads : kBackThreads, 1)
    norm_kernel(const NormParams p) {
  constexpr int V = EPT / 8;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[kMaxGroups * 128];
  __shared__ __align__(8) uint64_t full[kMaxGroups * kMaxStages];
  __shared__ __align__(8) uint64_t stall_bar;   // diagnostic: never completed
  __shared__ int abort_flag;
  const RowShape& sh = p.shape;
  const RowSpan<ODD> span(p.D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / sh.warps;
  Group grp{red + 128 * g, g + 1, sh.warps, warp - g * sh.warps, lane, 0};
  const int T = 32 * sh.warps, tid = grp.warp * 32 + lane;
  const int stage_bytes = 2 * sh.pitch;
  const int places = sh.groups * sh.stages;
  ring_setup(full, places, &stall_bar, &abort_flag, red);
  clear_padding(ring, places, stage_bytes, 16 * span.total, 2 * sh.pitch);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* params = reinterpret_cast<float*>(ring + places * stage_bytes);   // w, then b
  auto stage = [&] {
    if (!p.staged) return;
    stage_params<ODD>(params, static_cast<const W*>(p.w), span.lead, p.D, sh.pitch);
    stage_params<ODD>(params + sh.pitch, static_cast<const W*>(p.b), span.lead, p.b ? p.D : 0,
                      sh.pitch);
  };
  const bool early = ODD || sh.warps < 4;      // see below
  if (early) stage();
  __syncthreads();

  uint8_t* mine = ring + g * sh.stages * stage_bytes;
  uint64_t* bars = full + g * sh.stages;
  volatile int* aborted = &abort_flag;
  auto issue = [&](int st, int64_t r) {
    uint8_t* to = mine + st * stage_bytes;
    const uint16_t* x = p.x + r * p.D - span.lead;
    const int bytes = span.copy_bytes(r, p.M, p.D);
    span.copy_tail(to, x, bytes);
    mbar_arrive_expect_tx(&bars[st], bytes);
    if (!ODD || bytes > 0) bulk_load(to, x, bytes, &bars[st]);
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

  // While the first rows come: the parameters (16640 x 5120 60.2 -> 55.3 us, with the
  // save 74.0 -> 71.9).  Their loads first are quicker for short rows (16640 x 1024
  // with the save 15.7 and 16.9 us), with a lead (16640 x 4099 64.0 and 66.7), and
  // backward (16640 x 5120 88.3 and 94.7).
  if (!early) stage();
  if constexpr (SAVE) {
    // Zeros for the scales of rows past the matrix.  16 bytes of a scale tile hold
    // rows c, c + 32, c + 64 and c + 96.  (At the kernel's end and by one CTA, a
    // word at a time: 8 x 13344 11.7 us, 4.6 so.)
    const int m = static_cast<int>(p.M & 127);
    uint8_t* s = p.s + (p.M >> 7) * 512 * p.s_words;
    if (m)
      for (int i = blockIdx.x * blockDim.x + threadIdx.x; i < 32 * p.s_words;
           i += gridDim.x * blockDim.x) {
        const int c = i & 31;
        if (c >= m) {
          if (in_span(p.sp_s, s + 16 * i, 16)) *reinterpret_cast<uint4*>(s + 16 * i) = make_uint4(0, 0, 0, 0);
          continue;
        }
#pragma unroll
        for (int g = 1; g < 4; ++g)
          if (c + 32 * g >= m && in_span(p.sp_s, s + 16 * i + 4 * g, 4))
            *reinterpret_cast<uint32_t*>(s + 16 * i + 4 * g) = 0;
      }
  }
  if (!early) __syncthreads();

  const float inv = 1.0f / static_cast<float>(p.D);
  // Piece i of this thread is piece first + 32 i of the row (a warp's pieces lie
  // together, so that their distances are constants).  One lane of a block's
  // four writes its scale; blocks past the row are zero and give 0, the padding
  // of the blocked layout.
  const int first = grp.warp * 32 * V + lane;
  const int pieces = span.total - first;       // live: 32 i < pieces
  const int scaled = SAVE && (lane & 3) == 0 ? 16 * p.s_words - first : 0;
  auto group_sums = [&](float (&v)[R]) {
    if constexpr (R == 1) {
      v[0] = grp.sum(v[0]);
    } else {
      const float2 s = grp.sum2(v[0], v[1]);
      v[0] = s.x;
      v[1] = s.y;
    }
  };
  int st = 0;
  uint32_t parity = 0;
  for (int64_t r = r0; r < p.M; r += R * step) {
    f32x2 x[R][EPT / 2];
    float mean[R], rstd[R];
#pragma unroll
    for (int k = 0; k < R; ++k) {
      mean[k] = 0.0f;
      if (k > 0 && r + k * step >= p.M) continue;
      const int64_t rk = r + k * step;
      mbar_wait(&bars[st], parity, aborted);
      const uint8_t* row = mine + st * stage_bytes + first * 16;
      if (++st == sh.stages) {
        st = 0;
        parity ^= 1;
      }
      uint8_t* q = SAVE ? p.q + rk * p.D + first * 8 : nullptr;
      uint8_t* s = SAVE ? p.s + blocked_offset(rk, 0, 4 * p.s_words) + (first >> 4) * 512 +
                              (first >> 2 & 3)
                        : nullptr;
      f32x2 s2 = 0, s3 = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f32x2* xi = x[k] + 4 * i;
        uint4 v = *reinterpret_cast<const uint4*>(row + i * 512);
        if (span.edge(first + 32 * i)) span.clear(v, first + 32 * i);
        get_pairs(v, xi);
        s2 = add2(s2, add2(xi[0], xi[1]));
        s3 = add2(s3, add2(xi[2], xi[3]));
        if constexpr (SAVE) {
          uint32_t sb;
          const uint2 o = mx_cast_pairs(v, xi, sb);
          if (32 * i < pieces && in_span(p.sp_q, q + i * 256, 8))
            *reinterpret_cast<uint2*>(q + i * 256) = o;
          if (32 * i < scaled && in_span(p.sp_s, s + i * 1024, 1))
            s[i * 1024] = static_cast<uint8_t>(sb);
        }
      }
      mean[k] = sum_pair(add2(s2, s3));
    }
    group_sums(mean);
    if (sh.warps == 1) __syncwarp();
    // Every thread of the group has read the rows: fill their places again.
    if (tid == 0) {
      for (int64_t k = r + sh.stages * step; k < r + (sh.stages + R) * step && k < p.M && !*aborted;
           k += step) {
        if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
          mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
        } else {
          issue(issued % sh.stages, k);
          ++issued;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < R; ++k) {
      rstd[k] = 0.0f;
      if (k > 0 && r + k * step >= p.M) continue;
      mean[k] *= inv;
      f32x2 s2 = 0, s3 = 0;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        f32x2* xi = x[k] + 4 * i;
        const float m = 32 * i < pieces ? -mean[k] : 0.0f;      // padding stays 0
        const f32x2 m2 = pair(m, m);
#pragma unroll
        for (int j = 0; j < 4; ++j) xi[j] = add2(xi[j], m2);
        if (span.edge(first + 32 * i)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float lo, hi;
            unpair(xi[j], lo, hi);
            const int e = 8 * (first + 32 * i) + 2 * j;
            xi[j] = pair(span.holds(e) ? lo : 0.0f, span.holds(e + 1) ? hi : 0.0f);
          }
        }
        s2 = fma2(xi[0], xi[0], s2);
        s3 = fma2(xi[1], xi[1], s3);
        s2 = fma2(xi[2], xi[2], s2);
        s3 = fma2(xi[3], xi[3], s3);
      }
      rstd[k] = sum_pair(add2(s2, s3));
    }
    group_sums(rstd);
#pragma unroll
    for (int k = 0; k < R; ++k) {
      rstd[k] = rsqrtf(rstd[k] * inv + p.eps);
      const int64_t rk = r + k * step;
      if (tid == 0 && (k == 0 || rk < p.M)) {
        if (in_span(p.sp_mean, p.mean + rk, 4)) p.mean[rk] = mean[k];
        if (in_span(p.sp_rstd, p.rstd + rk, 4)) p.rstd[rk] = rstd[k];
      }
    }
    auto put = [&](int i, const f32x2* wv, const f32x2* bv) {
#pragma unroll
      for (int k = 0; k < R; ++k) {
        if (k > 0 && r + k * step >= p.M) continue;
        const f32x2 r2 = pair(rstd[k], rstd[k]);
        f32x2 o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = fma2(mul2(x[k][4 * i + j], r2), wv[j], bv[j]);
        span.store(p.y + (r + k * step) * p.D - span.lead, first + 32 * i, o, p.sp_y);
      }
    };
    if (ODD || p.staged) {
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
  }
  if (tid == 0 && abort_flag) {
    // Gave up: the copies still in flight land (bounded) before the CTA ends.
    for (int j = issued > sh.stages ? issued - sh.stages : 0; j < issued; ++j)
      mbar_drain(&bars[j % sh.stages], static_cast<uint32_t>((j / sh.stages) & 1), 100000000ull);
    atomicOr(&g_norm_watchdog, 1);
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
  float* parts;        // [grid][2][D padded to 4]
  int64_t M;
  int D;
  RowShape shape;
  int s_words;
  uint32_t last_blocks;   // of a row's last word of scales, the bytes that belong to blocks
  Span sp_dx, sp_parts;
  int64_t stall_at;
  uint64_t stall_ns;
};

// EPT values a thread.  The second pass reads the row from shared memory again:
// with dw and db in 2 EPT registers there is no room for more of the row (16
// values a thread, held from the first pass, are no quicker: 70 us against 71 at
// 16640 x 4096, 111 us against 94 at 16640 x 5120, with the 8-bit save).
template <bool SAVE, bool ODD, typename W, int EPT>
__global__ void __launch_bounds__(kBackThreads, 1) norm_back_kernel(const NormBackParams p) {
  constexpr int V = EPT / 8;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[kMaxGroups * 128];
  __shared__ __align__(8) uint64_t full[kMaxGroups * kMaxStages];
  __shared__ __align__(8) uint64_t stall_bar;   // diagnostic: never completed
  __shared__ int abort_flag;
  const RowShape& sh = p.shape;
  const RowSpan<ODD> span(p.D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = warp / sh.warps;
  Group grp{red + 128 * g, g + 1, sh.warps, warp - g * sh.warps, lane, 0};
  const int T = 32 * sh.warps, tid = grp.warp * 32 + lane;
  const int x_at = 2 * sh.pitch, stage_bytes = (SAVE ? 3 : 4) * sh.pitch;
  const int places = sh.groups * sh.stages;
  ring_setup(full, places, &stall_bar, &abort_flag, red);
  clear_padding(ring, places, stage_bytes, 16 * span.total, 2 * sh.pitch);
  clear_padding(ring + x_at, places, stage_bytes, SAVE ? p.D : 16 * span.total,
                SAVE ? sh.pitch : 2 * sh.pitch);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float* params = reinterpret_cast<float*>(ring + places * stage_bytes);   // w
  stage_params<ODD>(params, static_cast<const W*>(p.w), span.lead, p.D, sh.pitch);
  __syncthreads();

  uint8_t* mine = ring + g * sh.stages * stage_bytes;
  uint64_t* bars = full + g * sh.stages;
  volatile int* aborted = &abort_flag;
  auto issue = [&](int st, int64_t r) {
    uint8_t* to = mine + st * stage_bytes;
    if (SAVE) {
      mbar_arrive_expect_tx(&bars[st], 3 * p.D);
      bulk_load(to, p.dy + r * p.D, 2 * p.D, &bars[st]);
      bulk_load(to + x_at, p.q + r * p.D, p.D, &bars[st]);
      return;
    }
    const int64_t at = r * p.D - span.lead;
    const int bytes = span.copy_bytes(r, p.M, p.D);
    span.copy_tail(to, p.dy + at, bytes);
    span.copy_tail(to + x_at, p.x + at, bytes);
    mbar_arrive_expect_tx(&bars[st], 2 * bytes);
    if (ODD && bytes == 0) return;
    bulk_load(to, p.dy + at, bytes, &bars[st]);
    bulk_load(to + x_at, p.x + at, bytes, &bars[st]);
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
  const uint32_t edges = span.edges(first, V);
  // What the copies do not bring, a row ahead; without a condition, for loads
  // under one are waited for where it ends.  A warp's scales are 2 V words of
  // four, one to a lane (past the row its last word: the values there are 0).
  uint32_t words_next;
  const int word = min(grp.warp * 2 * V + min(lane, 2 * V - 1), p.s_words - 1) * 512;
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
  // The bytes that pad the row's last word may be anything, 0xFF too, which is NaN
  // times the zeros there.  Taken off after the sums, when the next row's word has long
  // arrived: 88.3 -> 88.9 us at 16640 x 5120 (90.3 where the word is used).
  auto drop_padding = [&]() {
    if (SAVE && word == (p.s_words - 1) * 512) words_next &= p.last_blocks;
  };
  fetch(r0);
  drop_padding();
  // Fills the place of row r, which every thread of the group has read.  From 8
  // bits, where three rows at least fit, this waits for the barrier of the next
  // row's sums, and a row needs no second one (16640 x 5120 95.1 -> 88.7 us, 4096 x
  // 16384 79.6 -> 73.7), and for odd lengths (16640 x 4099 94.0 -> 91.8 us, 4096 x
  // 16383 140 -> 121.5).  For bf16 rows it is too late where only two fit (8192 x
  // 8192 68.4 us, 82.2 so; 16640 x 5120, three rows, 85.6 and 84.1), and a choice at
  // run time costs what it gains.
  constexpr bool late = SAVE || ODD;
  auto refill = [&](int64_t r) {
    r += sh.stages * step;
    if (r >= p.M || *aborted) return;
    if (kDiagStall && blockIdx.x == 0 && g == 0 && issued == p.stall_at) {
      mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
      return;
    }
    issue(issued % sh.stages, r);
    ++issued;
  };
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
    uint8_t* sd = mine + st * stage_bytes + first * 16;
    uint8_t* sx = mine + st * stage_bytes + x_at + first * (SAVE ? 8 : 16);
    if (ODD && edges) {
      span.clear_place(sd, first, edges);
      span.clear_place(sx, first, edges);
    }
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
    auto get_dy = [&](int i, f32x2* d) {
      get_pairs(*reinterpret_cast<const uint4*>(sd + i * 512), d);
    };
    f32x2 s1 = 0, s2 = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f32x2 xv[4], d[4], wv[4];
      get_x(i, xv);
      get_dy(i, d);
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
    if (sh.warps == 1) __syncwarp();
    asm volatile("" ::: "memory");           // the second pass reads anew
    // Every thread of the group is past the row before this one.
    if (late && tid == 0 && r > r0) refill(r - step);
    drop_padding();
    // dx = rstd g - rstd c1 - (x - mean) rstd^2 c2
    const float c1 = -rstd * (t.x * inv), c2 = -rstd * (t.y * inv) * rstd;
    const f32x2 k1 = pair(c1, c1), k2 = pair(c2, c2);
    uint16_t* dx = p.dx + r * p.D - span.lead;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      f32x2 xv[4], d[4], wv[4];
      get_x(i, xv);
      get_dy(i, d);
      staged_pairs(params, sh.pitch, first + 32 * i, wv);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[j] = fma2(xv[j], k2, fma2(mul2(d[j], wv[j]), rs, k1));
      span.store(dx, first + 32 * i, d, p.sp_dx);
    }
    if (ODD && edges) fence_proxy_async_smem();   // what was cleared, before the next copies
    if (!late) {
      grp.meet();
      if (tid == 0) refill(r);
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
  const int pitch = (p.D + 3) & ~3;
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * 2 * pitch;
  // Value v of thread tid at (v T' + tid), T' = T + 4: the writes by v and the
  // reads by column (eight values of a thread, then the next thread's) are both
  // free of bank conflicts, and the partial sums leave in whole lines.
  float* sums = reinterpret_cast<float*>(ring);
  const int stride = T + 4, all = 2 * EPT * stride;
  __syncthreads();
  float* to = sums + g * all + tid;
#pragma unroll
  for (int k = 0; k < EPT / 2; ++k) {
    unpair(dw[k], to[2 * k * stride], to[(2 * k + 1) * stride]);
    unpair(db[k], to[(EPT + 2 * k) * stride], to[(EPT + 2 * k + 1) * stride]);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < span.width; e += blockDim.x) {
    if (!span.holds(e)) continue;
    const int c = e >> 3;                                 // piece: warp, i, lane
    const int v = (c >> 5) % V * 8 + (e & 7), id = (c >> 5) / V * 32 + (c & 31);
    const float* s = sums + v * stride + id;
    float a = 0.0f, b = 0.0f;
    for (int h = 0; h < sh.groups; ++h, s += all) {
      a += s[0];
      b += s[EPT * stride];
    }
    float* at = part + e - span.lead;
    if (in_span(p.sp_parts, at, 4)) *at = a;
    if (in_span(p.sp_parts, at + pitch, 4)) at[pitch] = b;
  }
}

// dw (blockIdx.y == 0) and db: 32 columns a CTA, four to a thread; each thread
// adds up a run of the partial sums, six under way at a time, then the runs are
// added up in order.
template <typename W>
__global__ void __launch_bounds__(256) norm_grad_kernel(const float* parts, int n, int D, W* dw,
                                                        W* db, Span sp_dw, Span sp_db) {
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kRuns = 32, kAtOnce = 6;
  __shared__ float run[kRuns][33];
  const int l = threadIdx.x & 7, k = threadIdx.x >> 3;
  const int pitch = (D + 3) & ~3, c = blockIdx.x * 32 + l * 4;
  const float* src = parts + (blockIdx.y ? pitch : 0) + c;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (c < D)
    for (int i = k; i < n; i += kAtOnce * kRuns) {
      float4 u[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int q = i + j * kRuns;
        u[j] = q < n ? __ldcg(reinterpret_cast<const float4*>(src + static_cast<int64_t>(q) * 2 * pitch))
                     : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        v.x += u[j].x;
        v.y += u[j].y;
        v.z += u[j].z;
        v.w += u[j].w;
      }
    }
  run[k][4 * l] = v.x;
  run[k][4 * l + 1] = v.y;
  run[k][4 * l + 2] = v.z;
  run[k][4 * l + 3] = v.w;
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

// The shape for M rows of `width` values (the largest lead included), EPT values a
// thread, `row` bytes a padded value of a stage and `param` bytes a value of the
// parameters: as many groups as fit in `threads` and have rows to work on, as many
// stages as fit.
RowShape ring_shape(int64_t M, int64_t width, int ept, int threads, int row, int param,
                    int num_sms) {
  RowShape s = {};
  s.warps = static_cast<int>((width + 32 * ept - 1) / (32 * ept));
  s.groups = s.warps < threads / 32 ? threads / 32 / s.warps : 1;
  const int64_t rows = (M + num_sms - 1) / num_sms;
  if (s.groups > rows) s.groups = static_cast<int>(rows);
  s.pitch = 32 * s.warps * ept;
  const int64_t room = kRingBytes - static_cast<int64_t>(param) * s.pitch;
  s.stages = static_cast<int>(room / (static_cast<int64_t>(s.groups) * row * s.pitch));
  if (s.stages > kMaxStages) s.stages = kMaxStages;
  return s;
}

// CTAs: one an SM, no more than rows; with a lead, a multiple of 8.
int grid_of(int64_t M, bool odd, int num_sms) {
  int64_t most = num_sms < kNormMaxParts ? num_sms : kNormMaxParts;
  if (!odd) return static_cast<int>(M < most ? M : most);
  most = most < 8 ? 8 : most & ~int64_t{7};
  const int64_t want = (M + 7) & ~int64_t{7};
  return static_cast<int>(want < most ? want : most);
}

template <typename K>
int allow_ring(K kernel) {
  return static_cast<int>(cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes));
}

template <bool SAVE, bool ODD, typename W, int EPT, int R = 1>
int run_norm(NormParams p, int num_sms, cudaStream_t stream) {
  // With a row or two a group, w and b are not worth a copy of their own.
  p.staged = ODD || p.M > 8 * static_cast<int64_t>(num_sms);
  const int param = p.staged ? 8 : 0;
  p.shape = ring_shape(p.M, p.D + (ODD ? 7 : 0), EPT, R == 1 ? kRingThreads : kBackThreads, 2,
                       param, num_sms);
  if (p.shape.stages < R) return static_cast<int>(cudaErrorInvalidConfiguration);   // no width is
  const int64_t smem = static_cast<int64_t>(p.shape.pitch) *
                       (p.shape.groups * p.shape.stages * 2 + param);
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] { return allow_ring(norm_kernel<SAVE, ODD, W, EPT, R>); });
  if (attr != 0) return attr;
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  return launch(norm_kernel<SAVE, ODD, W, EPT, R>, dim3(grid_of(p.M, ODD, num_sms)),
                32 * p.shape.warps * p.shape.groups, static_cast<int>(smem), stream, p);
}

template <bool SAVE, bool ODD, typename W, int EPT>
int run_norm_back(NormBackParams p, int num_sms, int* grid, cudaStream_t stream) {
  constexpr int kRow = SAVE ? 3 : 4;
  p.shape = ring_shape(p.M, p.D + (ODD ? 7 : 0), EPT, kBackThreads, kRow, 4, num_sms);
  const RowShape& s = p.shape;
  // No width is: 3 x 16384 bytes and 4 x 16384 of parameters fit three times, 4 x twice.
  if (s.stages < (SAVE ? 3 : 2)) return static_cast<int>(cudaErrorInvalidConfiguration);
  int64_t smem = static_cast<int64_t>(s.pitch) * (s.groups * s.stages * kRow + 4);
  const int64_t sums = int64_t{8} * EPT * (32 * s.warps + 4) * s.groups;
  if (smem < sums) smem = sums;
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] { return allow_ring(norm_back_kernel<SAVE, ODD, W, EPT>); });
  if (attr != 0) return attr;
  *grid = grid_of(p.M, ODD, num_sms);
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  return launch(norm_back_kernel<SAVE, ODD, W, EPT>, dim3(*grid), 32 * s.warps * s.groups,
                static_cast<int>(smem), stream, p);
}

// Values a thread holds of a row.  32 carry the most rows at a time (a group of 16
// warps holds 16384); few values for an SM are spread over more threads (values:
// an SM's rows times the width).  Backward, 32 / 16 / 8 values: 1031 x 1021 11.0 /
// 9.0 / 8.1 us, 600 x 4096 10.2 / 9.5 / 10.1, 2400 x 4096 17.0 / 17.7 / 21.4;
// forward: 1 x 4096 2.9 / 2.5 / 2.4 us, 1200 x 1024 3.3 / 3.1 / 3.6, 2400 x 1024
// 3.9 / 4.3 / 5.6.  With a lead, 40 for the few widths that need them and where they
// carry many more rows, as past 1024 and 8192: backward, 32 / 40 values, 16640 x
// 1021 44.5 / 34.0 us, 8000 x 8190 108 / 95.8, 16640 x 2050 60.4 / 54.4 (1.6 times
// the rows), but 4000 x 6001 38.2 / 42.5 (1.5 times); forward 30.0 / 19.6, 80.4 /
// 63.1, 40.1 / 33.4, 25.0 / 23.3.  24 where they take no more warps: with the save,
// forward, 16640 x 768 14.7 -> 12.5 us, 16640 x 1536 29.2 -> 24.3, backward 22.8 ->
// 19.2, 40.4 -> 33.7; but 16640 x 2560, four warps and not three, 41.0 -> 45.4.
int values_of(int width, int64_t M, int num_sms, int64_t few, bool odd) {
  if (width > kNormMaxWidth) return 40;
  const int64_t values = (M + num_sms - 1) / num_sms * width;
  if (width <= 256 || (width <= 4096 && values < 8192)) return 8;
  if (width <= 512 || (width <= 8192 && values < few)) return 16;
  auto warps = [width](int n) { return (width + 32 * n - 1) / (32 * n); };
  if (odd && 5 * (16 / warps(40)) >= 8 * (16 / warps(32))) return 40;
  return warps(24) == warps(32) ? 24 : 32;
}

template <bool SAVE, bool ODD, typename W>
int pick_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int n = values_of(p.D + (ODD ? 7 : 0), p.M, num_sms, 16384, ODD);
  if (n == 8) return run_norm<SAVE, ODD, W, 8>(p, num_sms, stream);
  if (n == 16) return run_norm<SAVE, ODD, W, 16>(p, num_sms, stream);
  if constexpr (ODD)
    if (n == 40)
      // Two rows a turn where a row has a group of many warps: 8000 x 8190 63.1 ->
      // 59.7 us, 4096 x 16383 70.8 -> 63.0, but 16640 x 1021 19.6 -> 20.2.
      return p.D > 8000 ? run_norm<SAVE, ODD, W, 40, 2>(p, num_sms, stream)
                        : run_norm<SAVE, ODD, W, 40>(p, num_sms, stream);
  if (n == 24) return run_norm<SAVE, ODD, W, 24, 2>(p, num_sms, stream);
  return run_norm<SAVE, ODD, W, 32, 2>(p, num_sms, stream);
}

template <bool SAVE, bool ODD, typename W>
int pick_norm_back(const NormBackParams& p, int num_sms, int* grid, cudaStream_t stream) {
  const int n = values_of(p.D + (ODD ? 7 : 0), p.M, num_sms, 40000, ODD);
  if (n == 8) return run_norm_back<SAVE, ODD, W, 8>(p, num_sms, grid, stream);
  if (n == 16) return run_norm_back<SAVE, ODD, W, 16>(p, num_sms, grid, stream);
  if constexpr (ODD)
    if (n == 40) return run_norm_back<SAVE, ODD, W, 40>(p, num_sms, grid, stream);
  if (n == 24) return run_norm_back<SAVE, ODD, W, 24>(p, num_sms, grid, stream);
  return run_norm_back<SAVE, ODD, W, 32>(p, num_sms, grid, stream);
}

template <typename W>
int run_back(const NormBackParams& p, int num_sms, int* grid, cudaStream_t stream) {
  if (p.q) return pick_norm_back<true, false, W>(p, num_sms, grid, stream);
  return p.D % 8 == 0 ? pick_norm_back<false, false, W>(p, num_sms, grid, stream)
                      : pick_norm_back<false, true, W>(p, num_sms, grid, stream);
}

template <typename W>
int run_forward(const NormParams& p, int num_sms, cudaStream_t stream) {
  if (p.q) return pick_norm<true, false, W>(p, num_sms, stream);
  return p.D % 8 == 0 ? pick_norm<false, false, W>(p, num_sms, stream)
                      : pick_norm<false, true, W>(p, num_sms, stream);
}

template <typename W>
int run_grad(const LayerNormBackArgs& a, int D, int n, cudaStream_t stream) {
  const dim3 grid(static_cast<unsigned>((D + 31) / 32), a.db ? 2 : 1);
  const uint64_t bytes = static_cast<uint64_t>(D) * sizeof(W);
  return launch(norm_grad_kernel<W>, grid, 256, 0, stream,
                static_cast<const float*>(a.work), n, D, static_cast<W*>(a.dw),
                static_cast<W*>(a.db), make_span(a.dw, bytes), make_span(a.db, bytes));
}

}  // namespace

int64_t norm_back_work_floats(int64_t M, int64_t D) {
  const int64_t ctas = D % 8 == 0 ? M : (M + 7) & ~int64_t{7};
  return (ctas < kNormMaxParts ? ctas : kNormMaxParts) * 2 * ((D + 3) & ~int64_t{3});
}

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
  p.last_blocks = 0xFFFFFFFFu >> (8 * ((4 - p.D / 32 % 4) % 4));
  p.sp_dx = make_span(a.dx, 2 * static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.D));
  p.sp_parts = make_span(a.work, 4 * static_cast<uint64_t>(norm_back_work_floats(a.M, a.D)));
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
