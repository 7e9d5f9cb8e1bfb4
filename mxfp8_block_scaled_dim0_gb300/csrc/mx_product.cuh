// mx_product.cuh -- products of two MX operands on the block-scaled tensor cores whose
// results do not go out as they are (mx_matmul_swiglu.cu) or whose operands have 4 bits
// (mx_matmul_fp4.cu):
//
//   P[m][n] = sum_k (qa[m][k] 2^(sa[m][k/32] - 127)) (qb[n][k] 2^(sb[n][k/32] - 127))
//
// Both operands have their contraction dimension contiguous.  A stage of the rings is
// 128 bytes of every row: 128 steps of e4m3, with one 128x4 blocked scale tile an
// operand and 128 rows, or 256 steps of e2m1 with two.  An MMA takes 32 bytes a row: 32
// steps and one scale (kind::mxf8f6f4), or 64 steps and two (kind::mxf4, at twice the
// rate).  Loads, scales and tensor memory go as in mx_matmul.cu, which has the reasons:
//
// pair_kernel: persistent CTA pairs, 256 x 256 results at a time, five stages of loads
// ahead of the MMAs; the epilogue warps take a tile's results into registers at once, and
// the next tile's MMAs run while they work on them.
// tile_kernel: 128 x 128 (or 64) results by a cluster of S CTAs that share the
// contraction; each sums and finishes 128 / S of the tile's rows, in rank order.
//
// What happens to the results (EPI):
//   kPlain       out = P in bf16 or fp32
//   kSwiglu      B is two operands, gate and up: a tile is as many columns of gate as the up
//                columns that belong to them, and goes out as h = g u / (1 + exp(-g)), with
//                gate and up themselves saved as MX-FP8 if wanted
//   kSwigluBack  P is the gradient of h: out is that of [gate | up], from the saved gate
//                and up (MX-FP8 or bf16)
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx_common.cuh"
#include "mx_gate.cuh"
#include "mx_kernels.h"
#include "mx_rows.cuh"
#include "mx_tensor.cuh"

namespace mx {
namespace {

__device__ int g_product_watchdog = 0;

constexpr int kBoxRows = 128;               // rows of one operand box
constexpr int kBoxCols = 128;               // bytes of a row of one stage
constexpr int kBoxBytes = kBoxRows * kBoxCols;
constexpr int kSfBytes = 512;               // one 128x4 blocked scale tile
constexpr int kStageOut = 4096;             // a warp's results on their way out

enum Epilogue { kPlain, kSwiglu, kSwigluBack };

template <bool FP4, int EPI>
struct Shape {
  static constexpr int kSteps = FP4 ? 256 : 128;        // contraction steps of a stage
  static constexpr int kSf = FP4 ? 2 : 1;               // scale tiles of 128 rows in a stage
  // One row tile of A's scales, two of B's.
  static constexpr int kPairBytes = 2 * kBoxBytes + 3 * kSf * kSfBytes;
  static constexpr int kPairStride = (kPairBytes + 1023) / 1024 * 1024;
  // B's row tiles of scales in the tile kernel: one, or gate's and up's.
  static constexpr int kTileSfRows = EPI == kSwiglu ? 2 : 1;
  static constexpr int kTileBytes = 2 * kBoxBytes + (1 + kTileSfRows) * kSf * kSfBytes;
  static constexpr int kTileStride = (kTileBytes + 1023) / 1024 * 1024;
};

struct ProductParams {
  void* out;
  int64_t M, N;        // N: columns of the results (kSwiglu: of h)
  int k_blocks;        // stages
  int last_mmas;       // of the last stage, 1..4
  int m_tiles, n_tiles;
  int split;           // CTAs of a cluster along the contraction (tile kernel)
  int out_f32;
  int run;             // stages summed in tensor memory at a time, at most
  int band;            // M-tiles of a band (pair kernel)
  int mapped;          // maps.out describes the result's rows
  int load_bytes;      // of a stage (tile kernel)
  int cols;            // of a tile, 64 or 128 (tile kernel; kSwiglu: 128, gate and up)
  // The gated SiLU's saved input: written (kSwiglu, or null) or read (kSwigluBack: q and s,
  // or gu).
  uint8_t* q;
  uint8_t* s;
  const uint16_t* gu;
  int64_t s_cols4;     // scales of a row, padded to four
  Span sp_out, sp_q, sp_s;
  int64_t stall_at;
  uint64_t stall_ns;
};

template <bool FP4, int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc, int k,
                                    uint32_t sfa, uint32_t sfb, bool accumulate) {
  if constexpr (FP4)
    mma_mxf4<CG>(d, da, db, mxf8_idesc_step(idesc, 2 * (k & 1)), sfa, sfb, accumulate);
  else
    mma_mxf8<CG>(d, da, db, mxf8_idesc_step(idesc, k), sfa, sfb, accumulate);
}

template <bool FP4>
__device__ __forceinline__ uint32_t idesc_of(int m, int n) {
  return FP4 ? mxf4_idesc(m, n) : mxf8_idesc(m, n, false, false);
}

// Where scale (row m, column c) lies in a blocked matrix of cols4 padded columns.
__device__ __forceinline__ int64_t scale_at(int64_t m, int64_t c, int64_t cols4) {
  return blocked_offset(m, c, cols4);
}

// Scale byte and multiplier of a block from the bits of its largest magnitude in fp32.
__device__ __forceinline__ void block_scale(uint32_t amax, uint32_t& sbyte, float& mult) {
  mx_scale(amax >> 16, sbyte, mult);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// ---- one tile per cluster ------------------------------------------------------

constexpr int kTileStages = 6;
constexpr int kTileThreads = 192;           // loads, MMA, four epilogue warps
constexpr int kPitch = 132;                 // floats a row of the partial tile

// Sums of eight neighbouring columns over the cluster's partial tiles, in rank order; the
// loads of all CTAs' values are under way before the first is added.
__device__ __forceinline__ void cluster_sum8(const float* part, int split, float (&v)[8]) {
  const uint32_t at = smem_u32(part);
  float4 lo[8], hi[8];
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < split) {
      const uint32_t a = map_to_rank(at, static_cast<uint32_t>(q));
      lo[q] = ld_cluster_f4(a);
      hi[q] = ld_cluster_f4(a + 16);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll
  for (int q = 0; q < 8; ++q)
    if (q < split) {
      v[0] += lo[q].x; v[1] += lo[q].y; v[2] += lo[q].z; v[3] += lo[q].w;
      v[4] += hi[q].x; v[5] += hi[q].y; v[6] += hi[q].z; v[7] += hi[q].w;
    }
}

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]), bf16x2(v[6], v[7]));
}

// Eight values of a 32-block that four neighbouring lanes hold, saved as MX-FP8; `in`: they
// are part of the result.  Every lane of the warp takes part.
__device__ __forceinline__ void save8(const ProductParams& p, int64_t m, int64_t c, const float (&v)[8],
                                      bool in) {
  uint32_t a = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) a = max(a, magnitude(v[j]));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
  a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
  uint32_t sbyte;
  float mult;
  block_scale(a, sbyte, mult);
  if (!in) return;
  uint8_t* q = p.q + m * 2 * p.N + c;
  if (in_span(p.sp_q, q, 8))
    *reinterpret_cast<uint2*>(q) =
        make_uint2(e4m3x4(v[0], v[1], v[2], v[3], mult), e4m3x4(v[4], v[5], v[6], v[7], mult));
  if ((c & 31) == 0) {
    uint8_t* s = p.s + scale_at(m, c >> 5, p.s_cols4);
    if (in_span(p.sp_s, s, 1)) *s = static_cast<uint8_t>(sbyte);
  }
}

// Eight saved values: column c of [gate | up] of row m.
__device__ __forceinline__ void saved8(const ProductParams& p, int64_t m, int64_t c, float (&v)[8]) {
  f32x2 w[4];
  if (p.q) {
    const uint2 q = ld_q8(p.q + m * 2 * p.N + c);
    mx_get_pairs(q, p.s[scale_at(m, c >> 5, p.s_cols4)], w);
  } else {
    get_pairs(__ldg(reinterpret_cast<const uint4*>(p.gu + m * 2 * p.N + c)), w);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) unpair(w[j], v[2 * j], v[2 * j + 1]);
}

// RUNS: the contraction in runs, as in mx_matmul.cu.
template <bool FP4, int EPI, bool RUNS>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ ProductMaps maps, const ProductParams p) {
  using S = Shape<FP4, EPI>;
  static_assert(!RUNS || EPI == kPlain, "16-bit results need no runs");
  static_assert(kBoxRows * kPitch * 4 <= kTileStages * S::kTileStride, "partial tile fits the ring");
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kTileStages], empty[kTileStages], done, stall_bar;
  __shared__ __align__(8) uint64_t ready[2], drained[2];     // RUNS: the places
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int tile = blockIdx.x / p.split;
  // kSwiglu: a tile's columns are half gate, half up.
  const int width = EPI == kSwiglu ? p.cols / 2 : p.cols;
  const int mt = tile % p.m_tiles, n0 = tile / p.m_tiles * width;
  // Stages of this CTA: equal shares, the first ones one longer.
  const int per = p.k_blocks / p.split, more = p.k_blocks % p.split;
  const int kb0 = rank * per + (rank < more ? rank : more);
  const int nkb = per + (rank < more ? 1 : 0);
  const int runs = RUNS ? (nkb + p.run - 1) / p.run : 1;
  auto run_end = [&](int r) { return static_cast<int>(static_cast<int64_t>(nkb) * (r + 1) / runs); };
  constexpr uint32_t kTmemCols = RUNS ? 512 : 256;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTileStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    if (RUNS)
      for (int j = 0; j < 2; ++j) {
        mbar_init(&ready[j], 1);
        mbar_init(&drained[j], 4);            // the epilogue warps
      }
    mbar_init(&done, 1);
    mbar_init(&stall_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.sa);
    prefetch_tmap(&maps.sb);
    if (EPI == kSwiglu) {
      prefetch_tmap(&maps.b2);
      prefetch_tmap(&maps.sb2);
    }
  }
  if (warp == 1) tmem_alloc<1>(&tmem_base, kTmemCols);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_base;
  // Scales: A's, B's (gate's), up's, for either half of a 4-bit stage.
  const uint32_t t_sfa = tmem + kTmemCols / 2, t_sfb = t_sfa + 4 * S::kSf, t_sfu = t_sfb + 4 * S::kSf;
  const int quarter = warp & 3;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  // This lane's row of the runs before the last.
  float sums[RUNS ? kBoxRows : 1] = {};

  if (warp == 0) {
    if (elect_one()) {
      int i = 0, s = 0;
      uint32_t turn = 0;                     // of the ring, mod 2
      for (; i < nkb; ++i) {
        if (kDiagStall && blockIdx.x == 0 && i == p.stall_at) {
          mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
          break;
        }
        if (i >= kTileStages && !mbar_wait(&empty[s], turn ^ 1u, &abort_flag)) break;
        uint8_t* st = ring + s * S::kTileStride;
        uint8_t* sf = st + 2 * kBoxBytes;
        const int kb = kb0 + i, x = kb * kBoxCols, sx = kb * 128 * S::kSf;
        constexpr int kSfTile = S::kSf * kSfBytes;
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(p.load_bytes));
        tma_load_2d(st, &maps.a, x, mt * kBoxRows, &full[s]);
        tma_load_2d(st + kBoxBytes, &maps.b, x, n0, &full[s]);
        tma_load_2d(sf, &maps.sa, sx, mt, &full[s]);
        tma_load_2d(sf + kSfTile, &maps.sb, sx, n0 / kBoxRows, &full[s]);
        if (EPI == kSwiglu) {
          tma_load_2d(st + kBoxBytes + kBoxBytes / 2, &maps.b2, x, n0, &full[s]);
          tma_load_2d(sf + 2 * kSfTile, &maps.sb2, sx, n0 / kBoxRows, &full[s]);
        }
        if (++s == kTileStages) {
          s = 0;
          turn ^= 1u;
        }
      }
      // Gave up: the copies already issued land before the CTA moves on.
      if (i < nkb)
        for (int j = i > kTileStages ? i - kTileStages : 0; j < i; ++j)
          mbar_drain(&full[j % kTileStages], static_cast<uint32_t>((j / kTileStages) & 1));
    }
  } else if (warp == 1) {
    if (elect_one()) {
      const uint32_t idesc = idesc_of<FP4>(128, width);
      // The scales of 32 rows of B take a column of tensor memory: 64 columns read the first
      // or the last two of their rows' four.  (Never an odd one: an MMA of 32 columns whose
      // scales began there ended in a misaligned address.)
      const uint32_t t_sfb_here = t_sfb + (n0 % kBoxRows) / 32;
      const uint32_t t_sfu_here = t_sfu + (n0 % kBoxRows) / 32;
      constexpr uint32_t kUpBox = kBoxBytes / 2 >> 4;
      int s = 0;
      uint32_t turn = 0;
      int run = 0, begin = 0, end = run_end(0);     // this run and its stages
      uint32_t d = tmem;
      for (int i = 0; i < nkb; ++i) {
        if (RUNS && i == end) {
          tcgen05_commit<1>(&ready[run & 1]);
          begin = end;
          end = run_end(++run);
          d = tmem + (run & 1) * kBoxRows;
          if (run >= 2 && !mbar_wait(&drained[run & 1], static_cast<uint32_t>((run >> 1) - 1) & 1u,
                                     &abort_flag))
            break;
        }
        if (!mbar_wait(&full[s], turn, &abort_flag)) break;
        tcgen05_fence_after();
        const uint32_t st = smem_u32(ring + s * S::kTileStride);
        const uint32_t sf = st + 2 * kBoxBytes;
#pragma unroll
        for (int j = 0; j < S::kSf; ++j) {
          tcgen05_cp_scales<1>(t_sfa + 4 * j, scale_desc(sf + j * kSfBytes));
          tcgen05_cp_scales<1>(t_sfb + 4 * j, scale_desc(sf + (S::kSf + j) * kSfBytes));
          if (EPI == kSwiglu)
            tcgen05_cp_scales<1>(t_sfu + 4 * j, scale_desc(sf + (2 * S::kSf + j) * kSfBytes));
        }
        const uint64_t da = operand_desc(st), db = operand_desc(st + kBoxBytes);
        const int mmas = kb0 + i == p.k_blocks - 1 ? p.last_mmas : 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < mmas) {
            const int j = FP4 ? k >> 1 : 0;
            mma<FP4, 1>(d, da + kStepK * k, db + kStepK * k, idesc, k, t_sfa + 4 * j,
                        t_sfb_here + 4 * j, i > begin || k > 0);
            if (EPI == kSwiglu)
              mma<FP4, 1>(d + 64, da + kStepK * k, db + kUpBox + kStepK * k, idesc, k, t_sfa + 4 * j,
                          t_sfu_here + 4 * j, i > begin || k > 0);
          }
        tcgen05_commit<1>(&empty[s]);
        if (++s == kTileStages) {
          s = 0;
          turn ^= 1u;
        }
      }
      tcgen05_commit<1>(&done);
      mbar_drain(&done, 0u, kWaitLimitNs);   // every MMA issued has finished
    }
  } else if (RUNS) {
    for (int run = 0; run < runs - 1; ++run) {
      if (!mbar_wait(&ready[run & 1], static_cast<uint32_t>(run >> 1) & 1u, &abort_flag)) break;
      tcgen05_fence_after();
      const uint32_t at = tmem + lanes + (run & 1) * kBoxRows;
#pragma unroll
      for (int c = 0; c < kBoxRows; c += 16) {
        if (c >= p.cols) break;
        uint32_t v[16];
        tmem_ld_16(at + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) sums[(RUNS ? c : 0) + (RUNS ? j : 0)] += __uint_as_float(v[j]);
      }
      tcgen05_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&drained[run & 1]);
    }
  }
  __syncwarp();
  // All roles meet here; by now this CTA's MMAs and copies are finished.
  __syncthreads();
  tcgen05_fence_after();
  const bool ok = abort_flag == 0;
  const uint32_t last = tmem + lanes + ((runs - 1) & 1) * kBoxRows;
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2 && static_cast<int64_t>(mt) * kBoxRows + quarter * 32 < p.M) {
    const int row = quarter * 32 + lane;
    constexpr int kUnroll = RUNS ? 4 : 1;      // sums are registers: c must be a constant
#pragma unroll kUnroll
    for (int c = 0; c < kBoxRows; c += 32) {
      if (c >= p.cols) break;                  // kSwiglu: gate in columns 0 .., up in 64 ..
      uint32_t v[32];
      tmem_ld_32(last + c, v);
      tmem_ld_wait();
      if constexpr (RUNS)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sums[c + j] + __uint_as_float(v[j]));
      uint4* dst = reinterpret_cast<uint4*>(part + row * kPitch + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dst[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    tcgen05_fence_before();
  }
  cluster_sync();
  // Rows of the tile that this CTA finishes.
  const int rows = kBoxRows / p.split;
  const int64_t m0 = static_cast<int64_t>(mt) * kBoxRows + rank * rows;
  if (ok && m0 < p.M) {
    const int pieces = width >> 3;                       // of eight, a row
    const int shift = 31 - __clz(pieces);
    const int n_rows = static_cast<int>(p.M - m0 < rows ? p.M - m0 : rows);
    const int total = n_rows << shift;
    // Whole warps stay in the loop: four lanes share a block of 32.
    for (int i0 = warp * 32; i0 < total; i0 += kTileThreads) {
      const int i = i0 + lane < total ? i0 + lane : total - 1;
      const int r = i >> shift, c = (i & (pieces - 1)) * 8;
      const int64_t m = m0 + r, n = n0 + c;
      const bool in = i0 + lane < total && n < p.N;
      const float* at = part + (rank * rows + r) * kPitch + c;
      float v[8];
      cluster_sum8(at, p.split, v);
      if constexpr (EPI == kPlain) {
        const bool vec = (p.N & 7) == 0;
        if (in)
          store_out8(p.out, p.out_f32, m * p.N + n, v,
                     vec ? 8 : static_cast<int>(p.N - n < 8 ? p.N - n : 8), vec, p.sp_out);
      } else if constexpr (EPI == kSwiglu) {
        float u[8], h[8];
        cluster_sum8(at + 64, p.split, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) h[j] = gated(v[j], u[j]);
        uint16_t* out = static_cast<uint16_t*>(p.out) + m * p.N + n;
        if (in && in_span(p.sp_out, out, 16)) *reinterpret_cast<uint4*>(out) = pack8(h);
        if (p.q) {
          save8(p, m, n, v, in);
          save8(p, m, p.N + n, u, in);
        }
      } else {
        if (in) {
          float g[8], u[8], dg[8], du[8];
          saved8(p, m, n, g);
          saved8(p, m, p.N + n, u);
#pragma unroll
          for (int j = 0; j < 8; ++j) gated_back(v[j], g[j], u[j], dg[j], du[j]);
          uint16_t* out = static_cast<uint16_t*>(p.out) + m * 2 * p.N + n;
          if (in_span(p.sp_out, out, 16)) *reinterpret_cast<uint4*>(out) = pack8(dg);
          if (in_span(p.sp_out, out + p.N, 16)) *reinterpret_cast<uint4*>(out + p.N) = pack8(du);
        }
      }
    }
  }
  cluster_sync();                             // peers have read this CTA's partial tile
  if (warp == 1) tmem_dealloc<1>(tmem, kTmemCols);
  if (threadIdx.x == 0 && !ok) atomicOr(&g_product_watchdog, 1);
}

// ---- CTA pairs -------------------------------------------------------------------

constexpr int kPairStages = 5;
constexpr int kPairThreads = 320;             // loads, MMA, eight epilogue warps
template <bool FP4, int EPI>
constexpr int kPairSmem = kPairStages * Shape<FP4, EPI>::kPairStride + 8 * kStageOut + 1024;

// Bands of `band` M-tiles, walked along N, M fastest inside a band.
struct Tiles {
  int m_tiles, n_tiles, band;
  __device__ __forceinline__ void at(int t, int& mt, int& nt) const {
    const int per = band * n_tiles;
    const int b = t / per, i = t - b * per;
    const int rows = min(band, m_tiles - b * band);
    nt = i / rows;
    mt = b * band + (i - nt * rows);
  }
};

// A warp's box of 32 rows x 64 bytes in the order of a 64-byte swizzle: sixteen bytes j of
// this lane's row.
__device__ __forceinline__ uint4* box64(uint8_t* box, int lane, int j) {
  return reinterpret_cast<uint4*>(box + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4));
}

// 32 values of [gate | up] of a row, column c on, as they lie in memory.
template <bool SAVED8>
struct Saved;

template <>
struct Saved<true> {
  uint4 w[2];
  uint32_t s;
  __device__ __forceinline__ void load(const ProductParams& p, int64_t m, int64_t c) {
    const uint4* q = reinterpret_cast<const uint4*>(p.q + m * 2 * p.N + c);
    w[0] = __ldg(q);
    w[1] = __ldg(q + 1);
    s = __ldg(p.s + scale_at(m, c >> 5, p.s_cols4));
  }
  // Values 8 j .. 8 j + 7.
  __device__ __forceinline__ void get(int j, f32x2 (&v)[4]) const {
    const uint4& b = w[j >> 1];
    mx_get_pairs((j & 1) ? make_uint2(b.z, b.w) : make_uint2(b.x, b.y), s, v);
  }
};

template <>
struct Saved<false> {
  uint4 w[4];
  __device__ __forceinline__ void load(const ProductParams& p, int64_t m, int64_t c) {
    const uint4* g = reinterpret_cast<const uint4*>(p.gu + m * 2 * p.N + c);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __ldg(g + j);
  }
  __device__ __forceinline__ void get(int j, f32x2 (&v)[4]) const { get_pairs(w[j], v); }
};

// FLAG: kPlain, results in fp32; kSwigluBack, gate and up from 8 bits.
template <bool FP4, int EPI, bool FLAG>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_kernel(const __grid_constant__ ProductMaps maps, const ProductParams p) {
  using S = Shape<FP4, EPI>;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], ready, drained, done,
      stall_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* stage_out = ring + kPairStages * S::kPairStride;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int n_tiles = p.m_tiles * p.n_tiles;
  const Tiles tiles{p.m_tiles, p.n_tiles, p.band};
  constexpr uint32_t kSfaCol = 256, kSfbCol = kSfaCol + 4 * S::kSf;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);                 // in the leader, for both CTAs' loads
      mbar_init(&empty[s], 1);
    }
    mbar_init(&ready, 1);
    mbar_init(&drained, 16);                  // the epilogue warps of both, in the leader
    mbar_init(&done, 1);
    mbar_init(&stall_bar, 1);
    abort_flag = 0;
    issued = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.b);
    prefetch_tmap(&maps.sa);
    prefetch_tmap(&maps.sb);
    if (EPI == kSwiglu) {
      prefetch_tmap(&maps.b2);
      prefetch_tmap(&maps.sb2);
    }
    prefetch_tmap(&maps.out);
  }
  if (warp == 1) tmem_alloc<2>(&tmem_base, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tcgen05_fence_before();
  __syncthreads();
  cluster_sync();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_base;

  if (warp == 0) {
    if (elect_one()) {
      int i = 0;
      bool ok = true;
      for (int t = first; ok && t < n_tiles; t += stride) {
        int mt, nt;
        tiles.at(t, mt, nt);
        const int m = (2 * mt + rank) * kBoxRows;
        // kSwiglu: gate's rows in the leader, up's in its peer.
        const int n = EPI == kSwiglu ? nt * kBoxRows : (2 * nt + rank) * kBoxRows;
        const CUtensorMap* map_b = EPI == kSwiglu && rank ? &maps.b2 : &maps.b;
        for (int kb = 0; kb < p.k_blocks; ++kb, ++i) {
          const int s = i % kPairStages;
          if (kDiagStall && blockIdx.x == 0 && i == p.stall_at) {
            mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
            ok = false;
            break;
          }
          if (i >= kPairStages &&
              !mbar_wait(&empty[s], static_cast<uint32_t>((i / kPairStages - 1) & 1), &abort_flag)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + s * S::kPairStride;
          uint8_t* sf = st + 2 * kBoxBytes;
          const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
          const int x = kb * kBoxCols, sx = kb * 128 * S::kSf;
          constexpr int kSfTile = S::kSf * kSfBytes;
          // The leader alone announces both CTAs' bytes.
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * S::kPairBytes);
          tma_load_2d_pair(st, &maps.a, x, m, bar);
          tma_load_2d_pair(st + kBoxBytes, map_b, x, n, bar);
          tma_load_2d_pair(sf, &maps.sa, sx, 2 * mt + rank, bar);
          if (EPI == kSwiglu) {
            tma_load_2d_pair(sf + kSfTile, &maps.sb, sx, nt, bar);
            tma_load_2d_pair(sf + 2 * kSfTile, &maps.sb2, sx, nt, bar);
          } else {
            tma_load_2d_pair(sf + kSfTile, &maps.sb, sx, 2 * nt, bar);
          }
        }
      }
      issued = i;
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = idesc_of<FP4>(256, 256);
      const uint32_t sfa = tmem + kSfaCol, sfb = tmem + kSfbCol;
      int i = 0, item = 0;
      bool ok = true;
      for (int t = first; ok && t < n_tiles; t += stride) {
        for (int k0 = 0; ok && k0 < p.k_blocks; k0 += p.run, ++item) {
          if (item > 0 && !mbar_wait_cluster(&drained, static_cast<uint32_t>((item - 1) & 1), &abort_flag)) {
            ok = false;
            break;
          }
          tcgen05_fence_after();
          const int k1 = min(k0 + p.run, p.k_blocks);
          for (int kb = k0; kb < k1; ++kb, ++i) {
            const int s = i % kPairStages;
            if (!mbar_wait_cluster(&full[s], static_cast<uint32_t>((i / kPairStages) & 1), &abort_flag)) {
              ok = false;
              break;
            }
            tcgen05_fence_after();
            const uint32_t st = smem_u32(ring + s * S::kPairStride);
            const uint32_t sf = st + 2 * kBoxBytes;
#pragma unroll
            for (int j = 0; j < S::kSf; ++j) {
              auto tile = [&](int row) { return scale_desc(sf + (row * S::kSf + j) * kSfBytes); };
              tcgen05_cp_scales<2>(sfa + 4 * j, tile(0));
              tcgen05_cp_scales<2>(sfb + 8 * j, tile(1));
              tcgen05_cp_scales<2>(sfb + 8 * j + 4, tile(2));
            }
            const uint64_t da = operand_desc(st), db = operand_desc(st + kBoxBytes);
            const int mmas = kb == p.k_blocks - 1 ? p.last_mmas : 4;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < mmas) {
                const int j = FP4 ? k >> 1 : 0;
                mma<FP4, 2>(tmem, da + kStepK * k, db + kStepK * k, idesc, k, sfa + 4 * j,
                            sfb + 8 * j, kb > k0 || k > 0);
              }
            tcgen05_commit<2>(&empty[s]);
          }
          if (ok) tcgen05_commit<2>(&ready);
        }
      }
      tcgen05_commit<2>(&done);
      mbar_drain(&done, 0u, kWaitLimitNs);     // every MMA issued has finished
    }
  } else {
    const int quarter = warp & 3, half = (warp - 2) >> 2;
    uint8_t* so = stage_out + (warp - 2) * kStageOut;
    const uint32_t drained_bar = map_to_rank(smem_u32(&drained), 0);
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    int item = 0;
    bool ok = true;
    for (int t = first; ok && t < n_tiles; t += stride) {
      int mt, nt;
      tiles.at(t, mt, nt);
      const int m = (2 * mt + rank) * kBoxRows + quarter * 32;
      if constexpr (EPI == kPlain) {
        // This lane's row of 128 results, in boxes of 128 bytes: four of fp32, two of
        // bf16 (packed as they are read).
        constexpr bool F32 = FLAG;
        constexpr int kBoxes = F32 ? 4 : 2;
        uint32_t v[kBoxes][32];
        if constexpr (F32) {
#pragma unroll
          for (int x = 0; x < kBoxes; ++x)
#pragma unroll
            for (int j = 0; j < 32; ++j) v[x][j] = 0;
        }
        for (int k0 = 0; k0 < p.k_blocks; k0 += p.run, ++item) {
          if (!mbar_wait(&ready, static_cast<uint32_t>(item & 1), &abort_flag)) {
            ok = false;
            break;
          }
          tcgen05_fence_after();
          const uint32_t at = tmem + lanes + half * 128;
          if constexpr (!F32) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t a[32], b[32];
              tmem_ld_32(at + 64 * x, a);
              tmem_ld_32(at + 64 * x + 32, b);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                v[x][j] = bf16x2(__uint_as_float(a[2 * j]), __uint_as_float(a[2 * j + 1]));
                v[x][16 + j] = bf16x2(__uint_as_float(b[2 * j]), __uint_as_float(b[2 * j + 1]));
              }
            }
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t w[16];
              tmem_ld_16(at + 16 * c, w);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                uint32_t& s = v[(c >> 1) % kBoxes][(c & 1) * 16 + j];
                s = __float_as_uint(__uint_as_float(s) + __uint_as_float(w[j]));
              }
            }
          }
          tcgen05_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(drained_bar);
        }
        if (!ok) break;
        // 32 rows x 128 columns through shared memory, a box at a time, in the
        // swizzled order the tensor map expects.
        const int n = 2 * nt * kBoxRows + half * 128;
        if (m >= p.M || n >= p.N) continue;
        uint8_t* row = so + lane * 128;
#pragma unroll
        for (int x = 0; x < kBoxes; ++x) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[x][4 * j], v[x][4 * j + 1], v[x][4 * j + 2], v[x][4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          const int c = n + x * (128 / kBoxes);
          if (!p.mapped) {
            if (c < p.N) store_box<F32 ? 4 : 2>(so, p.out, m, c, p.M, p.N, lane, p.sp_out);
          } else if (lane == 0) {
            if (c < p.N) tma_store_2d(&maps.out, c, m, so);
            bulk_commit();
          }
        }
      } else {
        const int64_t row = m + lane;
        // kSwiglu: 64 gate columns and their up columns; kSwigluBack: 128 columns of dh.
        uint32_t v[4][32];
        const int n = EPI == kSwiglu ? nt * kBoxRows + half * 64 : 2 * nt * kBoxRows + half * 128;
        // The first block's gate and up are under way before the products are ready.
        Saved<FLAG> g, u;
        const bool in = row < p.M;
        if (EPI == kSwigluBack && in && n < p.N) {
          g.load(p, row, n);
          u.load(p, row, p.N + n);
        }
        if (!mbar_wait(&ready, static_cast<uint32_t>(item++ & 1), &abort_flag)) {
          ok = false;
          break;
        }
        tcgen05_fence_after();
        const uint32_t at = tmem + lanes + half * (EPI == kSwiglu ? 64 : 128);
        constexpr int kNext = EPI == kSwiglu ? 128 : 64;      // where the second 64 columns are
        tmem_ld_32(at, v[0]);
        tmem_ld_32(at + 32, v[1]);
        tmem_ld_32(at + kNext, v[2]);
        tmem_ld_32(at + kNext + 32, v[3]);
        tmem_ld_wait();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(drained_bar);
        if (m >= p.M || n >= p.N) continue;
        if constexpr (EPI == kSwiglu) {
          if (lane == 0) bulk_wait_read<0>();
          __syncwarp();
          uint8_t* dst = so + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float h[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              h[k] = gated(__uint_as_float(v[j >> 2][(j & 3) * 8 + k]),
                           __uint_as_float(v[2 + (j >> 2)][(j & 3) * 8 + k]));
            *reinterpret_cast<uint4*>(dst + ((j ^ (lane & 7)) << 4)) = pack8(h);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&maps.out, n, m, so);
            bulk_commit();
          }
          if (p.q) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              // Block b: gate's two, up's two.
              const int64_t c = n + (b & 1) * 32;
              uint32_t a = 0;
#pragma unroll
              for (int j = 0; j < 32; ++j) a = max(a, v[b][j] & 0x7FFFFFFFu);
              uint32_t sbyte;
              float mult;
              block_scale(a, sbyte, mult);
              auto f = [&](int j) { return __uint_as_float(v[b][j]); };
              auto four = [&](int j) { return e4m3x4(f(j), f(j + 1), f(j + 2), f(j + 3), mult); };
#pragma unroll
              for (int j = 0; j < 2; ++j)
                *box64(so + (b >> 1) * 2048, lane, (b & 1) * 2 + j) =
                    make_uint4(four(16 * j), four(16 * j + 4), four(16 * j + 8), four(16 * j + 12));
              if (in && c < p.N) {
                uint8_t* s = p.s + scale_at(row, ((b >> 1) ? p.N + c : c) >> 5, p.s_cols4);
                if (in_span(p.sp_s, s, 1)) *s = static_cast<uint8_t>(sbyte);
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.gate, n, m, so);
              tma_store_2d(&maps.up, n, m, so + 2048);
              bulk_commit();
            }
          }
        } else {
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int64_t c = n + 32 * b;
            if (c >= p.N) break;
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              f32x2 gv[4], uv[4];
              float dg[8], du[8];
              g.get(j, gv);
              u.get(j, uv);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                float g0, g1, u0, u1;
                unpair(gv[k >> 1], g0, g1);
                unpair(uv[k >> 1], u0, u1);
                gated_back(__uint_as_float(v[b][8 * j + k]), k & 1 ? g1 : g0, k & 1 ? u1 : u0, dg[k],
                           du[k]);
              }
              *box64(so, lane, j) = pack8(dg);
              *box64(so + 2048, lane, j) = pack8(du);
            }
            if (b < 3 && in && c + 32 < p.N) {
              g.load(p, row, c + 32);
              u.load(p, row, p.N + c + 32);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.gate, static_cast<int>(c), m, so);
              tma_store_2d(&maps.up, static_cast<int>(c), m, so + 2048);
              bulk_commit();
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait<0>();
    tcgen05_fence_before();
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();
  // Gave up in either CTA: in the leader, settle the stages that only one CTA
  // loaded, so that what is in flight can be waited for.
  const int peer_abort = ld_cluster_s32(map_to_rank(smem_u32(&abort_flag), rank ^ 1));
  const bool failed = abort_flag != 0 || peer_abort != 0;
  if (failed) {
    if (rank == 0 && threadIdx.x == 0) {
      const int other = ld_cluster_s32(map_to_rank(smem_u32(&issued), 1));
      const int lo = min(issued, other), hi = max(issued, other);
      for (int j = lo; j < hi; ++j) {
        if (issued > other)
          mbar_complete_tx(&full[j % kPairStages], S::kPairBytes);
        else
          mbar_arrive_expect_tx(&full[j % kPairStages], S::kPairBytes);
      }
      for (int j = max(0, hi - kPairStages); j < hi; ++j)
        mbar_drain(&full[j % kPairStages], static_cast<uint32_t>((j / kPairStages) & 1),
                   100000000ull);
    }
    __syncthreads();
  }
  cluster_sync();
  tcgen05_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, 512);
  if (threadIdx.x == 0 && failed) atomicOr(&g_product_watchdog, 1);
}

// ---- launches ----------------------------------------------------------------------

inline cudaLaunchConfig_t cluster_config(cudaLaunchAttribute (&at)[2], int64_t ctas, int threads,
                                         size_t smem, unsigned cluster, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = cluster;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return cfg;
}

template <bool FP4, int EPI, bool FLAG>
int launch_pair_kernel(const ProductMaps& maps, const ProductParams& p, int num_sms,
                       cudaStream_t stream) {
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(pair_kernel<FP4, EPI, FLAG>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                 kPairSmem<FP4, EPI>));
  });
  if (attr != 0) return attr;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  if (tiles > 0x3fffffff) return static_cast<int>(cudaErrorInvalidConfiguration);
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg =
      cluster_config(at, 2 * pairs, kPairThreads, kPairSmem<FP4, EPI>, 2, stream);
  return static_cast<int>(cudaLaunchKernelEx(&cfg, pair_kernel<FP4, EPI, FLAG>, maps, p));
}

template <bool FP4, int EPI, bool RUNS>
int launch_tile_kernel(const ProductMaps& maps, const ProductParams& p, cudaStream_t stream) {
  constexpr int kSmem = kTileStages * Shape<FP4, EPI>::kTileStride + 1024;
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(tile_kernel<FP4, EPI, RUNS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  });
  if (attr != 0) return attr;
  const int64_t ctas = static_cast<int64_t>(p.m_tiles) * p.n_tiles * p.split;
  if (ctas > 0x7fffffff) return static_cast<int>(cudaErrorInvalidConfiguration);
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg =
      cluster_config(at, ctas, kTileThreads, kSmem, static_cast<unsigned>(p.split), stream);
  return static_cast<int>(cudaLaunchKernelEx(&cfg, tile_kernel<FP4, EPI, RUNS>, maps, p));
}

// The tile kernel's tiles: columns of B a tile, and CTAs that share its contraction; the
// quickest as reckoned in ns (tile_shape in mx_matmul.cu has the measurements).
struct TileChoice {
  int cols, split;
};

inline TileChoice choose_tiles(int64_t M, int64_t rows_b, int64_t k_blocks, int num_sms,
                               int least_cols = 64) {
  TileChoice best = {128, 1};
  int64_t least = INT64_MAX;
  for (int cols = 128; cols >= least_cols; cols /= 2) {
    const int64_t tiles = (M + 127) / 128 * ((rows_b + cols - 1) / cols);
    for (int s = 1; s <= 8 && s <= k_blocks; s *= 2) {
      if (s > 1 && tiles * s > (s == 8 ? 96 : s == 4 ? 128 : num_sms)) break;
      const int64_t rounds = (tiles * s + num_sms - 1) / num_sms;
      const int64_t cost = rounds * (500 + (cols == 128 ? 500 : 0) + (k_blocks + s - 1) / s * 220 +
                                     (s > 1 ? 400 + 19 * (M < 128 ? M : 128) * cols / 128 : 0));
      if (cost < least) {
        least = cost;
        best = {cols, s};
      }
    }
  }
  return best;
}

inline ProductParams product_params(int64_t M, int64_t N, int64_t K, bool fp4) {
  ProductParams p = {};
  p.M = M;
  p.N = N;
  const int64_t steps = fp4 ? 256 : 128, mma_steps = fp4 ? 64 : 32;
  p.k_blocks = static_cast<int>((K + steps - 1) / steps);
  p.last_mmas = static_cast<int>((K - (p.k_blocks - 1) * steps + mma_steps - 1) / mma_steps);
  p.run = p.k_blocks;
  p.band = 8;
  p.split = 1;
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  return p;
}

inline int read_product_word(int* out, bool clear) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_product_watchdog, sizeof(int));
  if (e != cudaSuccess) return static_cast<int>(e);
  if (clear && v) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_product_watchdog, &z, sizeof(int));
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  *out = v;
  return 0;
}

}  // namespace
}  // namespace mx
