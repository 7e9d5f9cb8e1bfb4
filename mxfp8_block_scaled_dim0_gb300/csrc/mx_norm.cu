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

template <int VEC, bool SAVE, typename W>
__global__ void __launch_bounds__(kMaxThreads, 1) norm_kernel(const NormParams p) {
  constexpr int V = kPer / VEC;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float2 red[8 * 64];
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
  for (; r < p.rows; r += step) {
#pragma unroll
    for (int i = 0; i < V; ++i) cur[i] = nxt[i];
    fetch(r + step, nxt);
    if (SAVE) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * T + tid) * 8;
        uint32_t sb = 0;
        uint2 q = make_uint2(0, 0);
        if constexpr (VEC == 8) q = mx_cast_piece(cur[i].w, sb);
        if (c < p.D && r < p.M && in_span(p.sp_q, p.q + r * p.D + c, 8))
          *reinterpret_cast<uint2*>(p.q + r * p.D + c) = q;
        // Scales of four neighbouring blocks (16 lanes) as one word; pieces
        // past the row give 0, the padding of the blocked layout.
        uint32_t word = sb << (8 * ((lane >> 2) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
        word |= __shfl_xor_sync(0xffffffffu, word, 8);
        if ((lane & 15) == 0 && (c >> 7) < p.s_words) {
          uint8_t* at = p.s + blocked_offset(r, c >> 5, 4 * p.s_words);
          if (in_span(p.sp_s, at, 4)) *reinterpret_cast<uint32_t*>(at) = word;
        }
      }
      if (r >= p.M) continue;
    }
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
  int D, warps, groups;
  int s_words;
  Span sp_dx, sp_parts;
};

// MAXT: 512 threads with the registers they need, or 1024 for rows of more
// than 8192 values.
template <int VEC, bool SAVE, typename W, int MAXT>
__global__ void __launch_bounds__(MAXT, 1) norm_back_kernel(const NormBackParams p) {
  constexpr int V = kPer / VEC;
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  extern __shared__ float sums[];            // groups > 1: 2 x padded row
  __shared__ float2 red[8 * 64];
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
    uint2 pq[V];
    uint32_t ps[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * T + tid) * VEC;
      pd[i].zero();
      px[i].zero();
      pq[i] = make_uint2(0, 0);
      ps[i] = 127;
      if (c >= p.D) continue;
      pd[i].load(p.dy + r * p.D + c);
      if (SAVE) {
        pq[i] = ld_q8(p.q + r * p.D + c);
        ps[i] = __ldg(p.s + blocked_offset(r, c >> 5, 4 * p.s_words));
      } else {
        px[i].load(p.x + r * p.D + c);
      }
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
      if constexpr (SAVE && VEC == 8) mx_get8(pq[i], ps[i], xh + i * VEC);
      else px[i].get(xh + i * VEC);
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

// Warps of a row's group, and groups of a CTA: eight warps where a row takes
// fewer.
void shape_of(int64_t D, int* warps, int* groups) {
  *warps = static_cast<int>((D + 32 * kPer - 1) / (32 * kPer));
  *groups = *warps < 8 ? 8 / *warps : 1;
}

int vec_of(int64_t D) { return D % 8 == 0 ? 8 : D % 2 == 0 ? 2 : 1; }

template <int VEC, bool SAVE, typename W>
int run_norm(const NormParams& p, int num_sms, cudaStream_t stream) {
  const int threads = 32 * p.warps * p.groups;
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, norm_kernel<VEC, SAVE, W>, threads, 0) !=
          cudaSuccess ||
      per < 1)
    per = 1;
  const int64_t want = (p.rows + p.groups - 1) / p.groups;
  const int64_t most = static_cast<int64_t>(num_sms) * per;
  return launch(norm_kernel<VEC, SAVE, W>, static_cast<int>(want < most ? want : most), threads, 0,
                stream, p);
}

template <int VEC, bool SAVE, typename W>
int run_norm_back(const NormBackParams& p, int grid, cudaStream_t stream) {
  const int threads = 32 * p.warps * p.groups;
  const int smem = p.groups > 1 ? 2 * kPer * 32 * p.warps * 4 : 0;
  return threads <= 512 ? launch(norm_back_kernel<VEC, SAVE, W, 512>, grid, threads, smem, stream, p)
                        : launch(norm_back_kernel<VEC, SAVE, W, 1024>, grid, threads, smem, stream, p);
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
  shape_of(a.D, &p.warps, &p.groups);
  const uint64_t n = static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.D);
  p.sp_y = make_span(a.y, 2 * n);
  p.sp_mean = make_span(a.mean, 4 * static_cast<uint64_t>(a.M));
  p.sp_rstd = make_span(a.rstd, 4 * static_cast<uint64_t>(a.M));
  p.sp_q = make_span(a.q, n);
  p.sp_s = make_span(a.s, static_cast<uint64_t>(p.rows) * 4 * p.s_words);
  const int v = vec_of(a.D);
  if (a.q)
    return a.w_f32 ? run_norm<8, true, float>(p, num_sms, stream)
                   : run_norm<8, true, uint16_t>(p, num_sms, stream);
  if (v == 8)
    return a.w_f32 ? run_norm<8, false, float>(p, num_sms, stream)
                   : run_norm<8, false, uint16_t>(p, num_sms, stream);
  if (v == 2)
    return a.w_f32 ? run_norm<2, false, float>(p, num_sms, stream)
                   : run_norm<2, false, uint16_t>(p, num_sms, stream);
  return a.w_f32 ? run_norm<1, false, float>(p, num_sms, stream)
                 : run_norm<1, false, uint16_t>(p, num_sms, stream);
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
  shape_of(a.D, &p.warps, &p.groups);
  const int64_t want = (a.M + p.groups - 1) / p.groups;
  int64_t most = 2 * static_cast<int64_t>(num_sms);
  if (most > kNormMaxParts) most = kNormMaxParts;
  const int grid = static_cast<int>(want < most ? want : most);
  p.sp_dx = make_span(a.dx, 2 * static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.D));
  p.sp_parts = make_span(a.work, static_cast<uint64_t>(norm_back_parts(a.M)) * 8 * a.D);
  const int v = vec_of(a.D);
  int rc = 0;
  if (a.q)
    rc = a.w_f32 ? run_norm_back<8, true, float>(p, grid, stream)
                 : run_norm_back<8, true, uint16_t>(p, grid, stream);
  else if (v == 8)
    rc = a.w_f32 ? run_norm_back<8, false, float>(p, grid, stream)
                 : run_norm_back<8, false, uint16_t>(p, grid, stream);
  else if (v == 2)
    rc = a.w_f32 ? run_norm_back<2, false, float>(p, grid, stream)
                 : run_norm_back<2, false, uint16_t>(p, grid, stream);
  else
    rc = a.w_f32 ? run_norm_back<1, false, float>(p, grid, stream)
                 : run_norm_back<1, false, uint16_t>(p, grid, stream);
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

}  // namespace mx
