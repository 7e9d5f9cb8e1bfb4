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
// contraction; each sums and finishes 128 / S of the tile's rows, in rank order.  kSwiglu: 2 S
// CTAs, every other one on gate and on up (both in one CTA, as two MMAs of 64 columns, took
// 12.0 us where one MMA of 128 takes 10.6: 45 MB of weights for one token).
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

template <bool FP4>
struct Shape {
  static constexpr int kSteps = FP4 ? 256 : 128;        // contraction steps of a stage
  static constexpr int kSf = FP4 ? 2 : 1;               // scale tiles of 128 rows in a stage
  // One row tile of A's scales, two of B's.
  static constexpr int kPairBytes = 2 * kBoxBytes + 3 * kSf * kSfBytes;
  static constexpr int kPairStride = (kPairBytes + 1023) / 1024 * 1024;
  static constexpr int kTileBytes = 2 * kBoxBytes + 2 * kSf * kSfBytes;
  static constexpr int kTileStride = (kTileBytes + 1023) / 1024 * 1024;
};

struct ProductParams {
  void* out;
  int64_t M, N;        // N: columns of the results (kSwiglu: of h)
  int k_blocks;        // stages
  int last_mmas;       // of the last stage, 1..4
  int m_tiles, n_tiles;
  int split;           // CTAs of a cluster along the contraction (tile kernel)
  int cluster;         // of the tile kernel: split, or twice that (kSwiglu)
  int out_f32;
  int run;             // stages summed in tensor memory at a time, at most
  int band;            // M-tiles of a band (pair kernel)
  int mapped;          // maps.out describes the result's rows
  int load_bytes;      // of a stage (tile kernel)
  int cols;            // of a tile, 64 or 128 (tile kernel)
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

// Scale byte and multiplier of a block from the bits of its largest magnitude in fp32.
__device__ __forceinline__ void block_scale(uint32_t amax, uint32_t& sbyte, float& mult) {
  mx_scale(amax >> 16, sbyte, mult);
}

__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// ---- one tile per cluster ------------------------------------------------------

constexpr int kTileStages = 6;
// Loads, MMA, and epilogue warps: four, or eight where results are worked on.
template <int EPI>
constexpr int kTileThreads = EPI == kPlain ? 192 : 320;
constexpr int kPitch = 132;                 // floats a row of the partial tile

// Sums of eight neighbouring columns over the partial tiles of the cluster's CTAs first,
// first + STEP .., in rank order; the loads of all values are under way before the first is
// added.
template <int STEP>
__device__ __forceinline__ void cluster_sum8(const float* part, int split, uint32_t first,
                                             float (&v)[8]) {
  if (STEP == 1 && split == 1) {               // this CTA's own
    const float4 a = reinterpret_cast<const float4*>(part)[0], b = reinterpret_cast<const float4*>(part)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    return;
  }
  constexpr int kMost = 8 / STEP;
  const uint32_t at = smem_u32(part);
  float4 lo[kMost], hi[kMost];
#pragma unroll
  for (int q = 0; q < kMost; ++q)
    if (q < split) {
      const uint32_t a = map_to_rank(at, first + STEP * q);
      lo[q] = ld_cluster_f4(a);
      hi[q] = ld_cluster_f4(a + 16);
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = 0.0f;
#pragma unroll
  for (int q = 0; q < kMost; ++q)
    if (q < split) {
      v[0] += lo[q].x; v[1] += lo[q].y; v[2] += lo[q].z; v[3] += lo[q].w;
      v[4] += hi[q].x; v[5] += hi[q].y; v[6] += hi[q].z; v[7] += hi[q].w;
    }
}

__device__ __forceinline__ void store_scale(const ProductParams& p, int64_t m, int64_t c, uint32_t v) {
  uint8_t* s = p.s + blocked_offset(m, c, p.s_cols4);
  if (in_span(p.sp_s, s, 1)) *s = static_cast<uint8_t>(v);
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
  if ((c & 31) == 0) store_scale(p, m, c >> 5, sbyte);
}

// Eight gates and ups of a row, column c on, as they lie in memory.
struct Saved8 {
  uint4 g, u;          // bf16, or e4m3 in the first two words
  uint32_t s;          // both scales
  __device__ __forceinline__ void load(const ProductParams& p, int64_t m, int64_t c) {
    if (p.q) {
      const uint8_t* q = p.q + m * 2 * p.N + c;
      const uint2 a = ld_q8(q), b = ld_q8(q + p.N);
      g.x = a.x;
      g.y = a.y;
      u.x = b.x;
      u.y = b.y;
      s = __ldg(p.s + blocked_offset(m, c >> 5, p.s_cols4)) |
          static_cast<uint32_t>(__ldg(p.s + blocked_offset(m, (p.N + c) >> 5, p.s_cols4))) << 8;
    } else {
      const uint16_t* x = p.gu + m * 2 * p.N + c;
      g = __ldg(reinterpret_cast<const uint4*>(x));
      u = __ldg(reinterpret_cast<const uint4*>(x + p.N));
    }
  }
  // Whether a gate may be low.
  __device__ __forceinline__ bool get(const ProductParams& p, f32x2 (&gv)[4], f32x2 (&uv)[4]) const {
    if (p.q) {
      mx_get_pairs(make_uint2(g.x, g.y), s & 0xFFu, gv);
      mx_get_pairs(make_uint2(u.x, u.y), s >> 8, uv);
      return may_be_low(s & 0xFFu);
    }
    get_pairs(g, gv);
    get_pairs(u, uv);
    return any_low(lowest2(g));
  }
};

// RUNS: the contraction in runs, as in mx_matmul.cu (fp32 results, and saved ones).
template <bool FP4, int EPI, bool RUNS>
__global__ void __launch_bounds__(kTileThreads<EPI>, 1)
    tile_kernel(const __grid_constant__ ProductMaps maps, const ProductParams p) {
  using S = Shape<FP4>;
  static_assert(!RUNS || EPI != kSwigluBack, "16-bit results need no runs");
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
  // kSwiglu: gate in the even CTAs of a cluster, up in the odd ones.
  constexpr int kHalves = EPI == kSwiglu ? 2 : 1;
  const bool up = EPI == kSwiglu && (rank & 1);
  const int share = rank / kHalves;           // of the contraction
  const int tile = blockIdx.x / p.cluster;
  const int mt = tile % p.m_tiles, n0 = tile / p.m_tiles * p.cols;
  // Stages of this CTA: equal shares, the first ones one longer.
  const int per = p.k_blocks / p.split, more = p.k_blocks % p.split;
  const int kb0 = share * per + (share < more ? share : more);
  const int nkb = per + (share < more ? 1 : 0);
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
        mbar_init(&drained[j], kTileThreads<EPI> / 32 - 2);      // the epilogue warps
      }
    mbar_init(&done, 1);
    mbar_init(&stall_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.a);
    prefetch_tmap(&maps.sa);
    prefetch_tmap(up ? &maps.b2 : &maps.b);
    prefetch_tmap(up ? &maps.sb2 : &maps.sb);
  }
  if (warp == 1) tmem_alloc<1>(&tmem_base, kTmemCols);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_base;
  // Scales, A's and B's, for either half of a 4-bit stage.
  const uint32_t t_sfa = tmem + kTmemCols / 2, t_sfb = t_sfa + 4 * S::kSf;
  const int quarter = warp & 3;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  // This lane's row of the runs before the last: an epilogue warp's share of the columns.
  constexpr int kShare = EPI == kPlain ? kBoxRows : kBoxRows / 2;
  const int c0 = EPI == kPlain ? 0 : (warp - 2) / 4 * kShare;
  float sums[RUNS ? kShare : 1] = {};

  if (warp == 0) {
    if (elect_one()) {
      const CUtensorMap *map_b = up ? &maps.b2 : &maps.b, *map_sb = up ? &maps.sb2 : &maps.sb;
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
        tma_load_2d(st + kBoxBytes, map_b, x, n0, &full[s]);
        tma_load_2d(sf, &maps.sa, sx, mt, &full[s]);
        tma_load_2d(sf + kSfTile, map_sb, sx, n0 / kBoxRows, &full[s]);
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
      const uint32_t idesc = idesc_of<FP4>(128, p.cols);
      // The scales of 32 rows of B take a column of tensor memory: a tile of 64 columns reads
      // the first or the last two of its rows' four.  (Never begin at an odd one: an MMA of 32
      // columns that did ended in a misaligned address.)
      const uint32_t t_sfb_here = t_sfb + (n0 % kBoxRows) / 32;
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
        }
        const uint64_t da = operand_desc(st), db = operand_desc(st + kBoxBytes);
        const int mmas = kb0 + i == p.k_blocks - 1 ? p.last_mmas : 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < mmas) {
            const int j = FP4 ? k >> 1 : 0;
            mma<FP4, 1>(d, da + kStepK * k, db + kStepK * k, idesc, k, t_sfa + 4 * j,
                        t_sfb_here + 4 * j, i > begin || k > 0);
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
  } else if (EPI == kSwigluBack) {
    // The tile's gates and ups into L2: whole rows by the warp, 128 bytes a lane.
    const int size = p.q ? 1 : 2;
    const uint8_t* from = p.q ? p.q : reinterpret_cast<const uint8_t*>(p.gu);
    const int64_t left = p.N - n0 < p.cols ? p.N - n0 : p.cols;
    const int lines = static_cast<int>((left * size + 127) / 128);        // of a half row: 1 or 2
    const int64_t m1 = static_cast<int64_t>(mt) * kBoxRows + rank * (kBoxRows / p.split);
    for (int i = threadIdx.x - 64; i < kBoxRows / p.split * 2 * lines; i += kTileThreads<EPI> - 64) {
      const int64_t m = m1 + i / (2 * lines);
      const int k = i % (2 * lines);
      if (m < p.M)
        prefetch_l2(from + (m * 2 * p.N + (k & 1) * p.N + n0) * size + (k >> 1) * 128);
    }
  } else if (RUNS) {
    for (int run = 0; run < runs - 1; ++run) {
      if (!mbar_wait(&ready[run & 1], static_cast<uint32_t>(run >> 1) & 1u, &abort_flag)) break;
      tcgen05_fence_after();
      const uint32_t at = tmem + lanes + (run & 1) * kBoxRows + c0;
#pragma unroll
      for (int c = 0; c < kShare; c += 16) {
        if (c0 + c >= p.cols) break;
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
  // Rows of the tile that this CTA finishes, in pieces of eight columns.
  const int rows = kBoxRows / p.cluster;
  const int64_t m0 = static_cast<int64_t>(mt) * kBoxRows + rank * rows;
  const int pieces = p.cols >> 3, shift = 31 - __clz(pieces);
  const int total = m0 < p.M ? static_cast<int>(p.M - m0 < rows ? p.M - m0 : rows) << shift : 0;
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2 && static_cast<int64_t>(mt) * kBoxRows + quarter * 32 < p.M) {
    const int row = quarter * 32 + lane;
    constexpr int kUnroll = RUNS ? 4 : 1;      // sums are registers: c must be a constant
#pragma unroll kUnroll
    for (int c1 = 0; c1 < kShare; c1 += 32) {
      const int c = c0 + c1;
      if (c >= p.cols) break;
      uint32_t v[32];
      tmem_ld_32(last + c, v);
      tmem_ld_wait();
      if constexpr (RUNS)
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sums[c1 + j] + __uint_as_float(v[j]));
      uint4* dst = reinterpret_cast<uint4*>(part + row * kPitch + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dst[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    tcgen05_fence_before();
  }
  cluster_sync();
  if constexpr (EPI == kSwigluBack) {
    // Two pieces a thread at a time, their gates and ups (asked into L2 while the MMAs went
    // on) a step ahead of the work.
    constexpr int kFew = 2, kStep = kFew * kTileThreads<EPI>;
    struct Few {
      Saved8 w[kFew];
    } next;
    auto load = [&](int i0) {
#pragma unroll
      for (int k = 0; k < kFew; ++k) {
        const int i = i0 + k * kTileThreads<EPI>;
        const int64_t m = m0 + (i >> shift), n = n0 + (i & (pieces - 1)) * 8;
        if (i < total && n < p.N) next.w[k].load(p, m, n);
      }
    };
    load(threadIdx.x);
    if (ok)
      for (int i0 = threadIdx.x; i0 < total; i0 += kStep) {
        const Few now = next;
        load(i0 + kStep);
#pragma unroll
        for (int k = 0; k < kFew; ++k) {
          const int i = i0 + k * kTileThreads<EPI>;
          const int r = i >> shift, c = (i & (pieces - 1)) * 8;
          const int64_t m = m0 + r, n = n0 + c;
          if (i >= total || n >= p.N) continue;
          float v[8];
          cluster_sum8<1>(part + (rank * rows + r) * kPitch + c, p.split, 0, v);
          f32x2 d[4], g[4], u[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = pair(v[2 * j], v[2 * j + 1]);
          const bool low = now.w[k].get(p, g, u);
          uint4 dg, du;
          gated_back8(d, g, u, low, dg, du);
          uint16_t* out = static_cast<uint16_t*>(p.out) + m * 2 * p.N + n;
          if (in_span(p.sp_out, out, 16)) *reinterpret_cast<uint4*>(out) = dg;
          if (in_span(p.sp_out, out + p.N, 16)) *reinterpret_cast<uint4*>(out + p.N) = du;
        }
      }
  } else if (EPI == kPlain && (p.N & 7) != 0) {
    // Rows off the 16-byte boundary: the sums in this CTA's place of its own rows, then a row
    // a warp, neighbouring lanes on neighbouring values (eight values a thread: 1321 x 916 x
    // 5120 12.6 us, 8.5 at 920 columns).
    float* own = part + rank * rows * kPitch;
    const int n_rows = total >> shift;
    const int cols = static_cast<int>(p.N - n0 < p.cols ? p.N - n0 : p.cols);
    if (p.split > 1) {
      if (ok)
        for (int i = threadIdx.x; i < total; i += kTileThreads<EPI>) {
          float* at = own + (i >> shift) * kPitch + (i & (pieces - 1)) * 8;
          float v[8];
          cluster_sum8<kHalves>(at, p.split, 0, v);
          reinterpret_cast<float4*>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
          reinterpret_cast<float4*>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
        }
      __syncthreads();
    }
    auto store_row = [&](int r) {
      const float* at = own + r * kPitch;
      const int64_t to = (m0 + r) * p.N + n0;
      if (p.out_f32) {
        float* o = static_cast<float*>(p.out) + to;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (const int c = lane + 32 * k; c < cols && in_span(p.sp_out, o + c, 4)) o[c] = at[c];
      } else if ((p.N & 1) == 0) {
        uint16_t* o = static_cast<uint16_t*>(p.out) + to;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          if (const int c = 2 * lane + 64 * k; c < cols && in_span(p.sp_out, o + c, 4))
            *reinterpret_cast<uint32_t*>(o + c) = bf16x2(at[c], at[c + 1]);
      } else {
        uint16_t* o = static_cast<uint16_t*>(p.out) + to;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (const int c = lane + 32 * k; c < cols && in_span(p.sp_out, o + c, 2))
            o[c] = static_cast<uint16_t>(bf16x2(at[c], 0.0f));
      }
    };
    if (ok)
#pragma unroll 2
      for (int r = warp; r < n_rows; r += kTileThreads<EPI> / 32) store_row(r);
  } else if (ok) {
    // Whole warps stay in the loop: four lanes share a block of 32.
    for (int i0 = warp * 32; i0 < total; i0 += kTileThreads<EPI>) {
      const int i = i0 + lane < total ? i0 + lane : total - 1;
      const int r = i >> shift, c = (i & (pieces - 1)) * 8;
      const int64_t m = m0 + r, n = n0 + c;
      const bool in = i0 + lane < total && n < p.N;
      const float* at = part + (rank * rows + r) * kPitch + c;
      float v[8];
      cluster_sum8<kHalves>(at, p.split, 0, v);
      if constexpr (EPI == kPlain) {
        if (in) store_out8(p.out, p.out_f32, m * p.N + n, v, 8, true, p.sp_out);
      } else if constexpr (EPI == kSwiglu) {
        float u[8];
        cluster_sum8<kHalves>(at, p.split, 1, u);
        f32x2 g2[4], u2[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          g2[j] = pair(v[2 * j], v[2 * j + 1]);
          u2[j] = pair(u[2 * j], u[2 * j + 1]);
        }
        uint16_t* out = static_cast<uint16_t*>(p.out) + m * p.N + n;
        if (in && in_span(p.sp_out, out, 16)) *reinterpret_cast<uint4*>(out) = gated8(g2, u2);
        if (p.q) {
          save8(p, m, n, v, in);
          save8(p, m, p.N + n, u, in);
        }
      }
    }
  }
  if (EPI == kSwiglu && p.q && rank == 0) {
    // The padding of this tile's saved scales: rows behind the last, columns behind a row.
    const int blocks = static_cast<int>(p.N - n0 < p.cols ? p.N - n0 : p.cols) / 32;
    const int64_t first = static_cast<int64_t>(mt) * kBoxRows;
    const int behind = p.M - first < kBoxRows ? static_cast<int>(kBoxRows - (p.M - first)) : 0;
    for (int i = threadIdx.x; i < behind * 2 * blocks; i += kTileThreads<EPI>) {
      const int r = i / (2 * blocks), b = i % (2 * blocks);
      store_scale(p, p.M + r, n0 / 32 + (b < blocks ? b : static_cast<int>(p.N / 32) + b - blocks), 0);
    }
    const int cols = static_cast<int>(p.s_cols4 - p.N / 16);
    if (n0 + p.cols >= p.N)
      for (int i = threadIdx.x; i < kBoxRows * cols; i += kTileThreads<EPI>)
        store_scale(p, first + i / cols, p.N / 16 + i % cols, 0);
  }
  cluster_sync();                             // peers have read this CTA's partial tile
  if (warp == 1) tmem_dealloc<1>(tmem, kTmemCols);
  if (threadIdx.x == 0 && !ok) atomicOr(&g_product_watchdog, 1);
}

// ---- CTA pairs -------------------------------------------------------------------

// What a pair's epilogue does beside EPI (FLAG): kPlain, results in fp32; kSwiglu, gate and up
// saved; kSwigluBack, gate and up from 8 bits.
//
// Stages of loads, and bytes of an epilogue warp's staging.  A stage counts: 16640 x 8192 x
// 5120 e2m1 takes 199 us with five, 216 with four, 257 with three (six do not fit); h with
// the save in e4m3, its sums in one run, 790 and 860, although with four the warps need not
// wait for the stores.
// Beside five fit 6 KB a warp for kSwiglu: gate's bytes go behind h and only up's wait until
// h has left (13766 x 5344 x 1088 e2m1 with the save 121 us with 4 KB, 114 with 6).
// kSwigluBack does with four, as gates and ups come through shared memory: loads of a row a
// lane touch 32 lines each, and took the load/store units as long as all else (8192 x 8192 x
// 1024 e2m1 135 us with them, 111 without).
template <int EPI>
constexpr int kPairStages = EPI == kSwigluBack ? 4 : 5;
template <int EPI>
constexpr int kWarpStage = EPI == kSwigluBack ? 10 * 1024 : EPI == kSwiglu ? 6 * 1024 : kStageOut;
template <bool FP4, int EPI>
constexpr int kPairSmem = kPairStages<EPI> * Shape<FP4>::kPairStride + 8 * kWarpStage<EPI> + 1024;

// Loads, MMA, eight epilogue warps.  kSwigluBack: two idle warps more, so that the first
// warpgroup can hand registers to the two that hold 128 results and what they need beside
// (168 a thread at launch: 56 x 128 + 224 x 256 are as many).  Of 168 and 224, kSwiglu with
// the save spills 12 words a thread and kSwigluBack from 8 bits 24; no other kernel spills.
template <int EPI>
constexpr int kFirstEpilogueWarp = EPI == kSwigluBack ? 4 : 2;
template <int EPI>
constexpr int kPairThreads = 32 * (kFirstEpilogueWarp<EPI> + 8);
constexpr int kGiven = 56, kTaken = 224;
template <int REGS>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS));
}
template <int REGS>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS));
}

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

// ---- kSwigluBack's gates and ups ---------------------------------------------------
//
// 32 rows of a warp, in blocks of 32 columns, copied into its staging by all lanes (whole
// lines at a time) while the products are computed.  Results leave in boxes of 64 bytes a row
// (of 128: 462 -> 480 us at 16640 x 8192 x 5120 e4m3).
//   8 bits: four blocks of 2 KB at once: gates, then ups, 32 bytes a row, the sixteens of rows
//           4..7 of every eight exchanged (a row a lane is then free of bank conflicts).  The
//           results go out through the places of blocks read and 2 KB behind them.
//   bf16:   two blocks of 4 KB at a time, gates and ups in boxes of 64 bytes a row in the
//           order of a 64-byte swizzle, replaced by dg and du in place.
// What is read or written once is the first to leave L2, where the operands are read again:
// 16640 x 8192 x 5120 e4m3 485 -> 477 us.
__device__ __forceinline__ uint64_t once_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void copy16(uint8_t* smem_dst, const void* g, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(smem_u32(smem_dst)),
               "l"(g), "l"(policy)
               : "memory");
}
__device__ __forceinline__ void tma_store_2d_once(const CUtensorMap* m, int32_t x, int32_t y,
                                                  const void* smem_src, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group.L2::cache_hint [%0, {%1, %2}], [%3], %4;" ::
          "l"(reinterpret_cast<uint64_t>(m)),
      "r"(x), "r"(y), "r"(smem_u32(smem_src)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows m .. m + 31, columns n .. n + 127, of both halves.
__device__ __forceinline__ void copy_saved8(const ProductParams& p, uint8_t* to, int64_t m, int64_t n,
                                            int lane, uint64_t policy) {
  const int c = lane & 7;                    // sixteen bytes of a row's 128
  if (n + 16 * c >= p.N) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = 4 * k + (lane >> 3);
    if (m + r >= p.M) break;
    const uint8_t* q = p.q + (m + r) * 2 * p.N + n + 16 * c;
    uint8_t* dst = to + (c >> 1) * 2048 + r * 32 + (((c ^ (r >> 2)) & 1) << 4);
    copy16(dst, q, policy);
    copy16(dst + 1024, q + p.N, policy);
  }
}

// A row's share of one of those blocks.
struct SavedBlock {
  uint4 g[2], u[2];
  __device__ __forceinline__ void load(const uint8_t* block, int lane) {
    const uint8_t* at = block + lane * 32;
    const int x = ((lane >> 2) & 1) << 4;
    g[0] = *reinterpret_cast<const uint4*>(at + x);
    g[1] = *reinterpret_cast<const uint4*>(at + (x ^ 16));
    u[0] = *reinterpret_cast<const uint4*>(at + 1024 + x);
    u[1] = *reinterpret_cast<const uint4*>(at + 1024 + (x ^ 16));
  }
};

// ... columns c .. c + 31 of bf16.
__device__ __forceinline__ void copy_saved16(const ProductParams& p, uint8_t* to, int64_t m, int64_t c,
                                             int lane, uint64_t policy) {
  const int j = lane & 3;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int r = 8 * k + (lane >> 2);
    if (m + r >= p.M) break;
    const uint16_t* x = p.gu + (m + r) * 2 * p.N + c + 8 * j;
    uint8_t* dst = reinterpret_cast<uint8_t*>(box64(to, r, j));
    copy16(dst, x, policy);
    copy16(dst + 2048, x + p.N, policy);
  }
}

template <bool FP4, int EPI, bool FLAG>
__global__ void __launch_bounds__(kPairThreads<EPI>, 1)
    pair_kernel(const __grid_constant__ ProductMaps maps, const ProductParams p) {
  using S = Shape<FP4>;
  constexpr int kStages = kPairStages<EPI>;
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], empty[kStages], ready, drained, done, stall_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* stage_out = ring + kStages * S::kPairStride;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int n_tiles = p.m_tiles * p.n_tiles;
  const Tiles tiles{p.m_tiles, p.n_tiles, p.band};
  constexpr uint32_t kSfaCol = 256, kSfbCol = kSfaCol + 4 * S::kSf;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
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

  // One branch a warpgroup, so that the compiler sees which registers either has.
  constexpr int kFirst = kFirstEpilogueWarp<EPI>;
  if (warp < kFirst) {
    if (EPI == kSwigluBack) give_registers<kGiven>();
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
            const int s = i % kStages;
            if (kDiagStall && blockIdx.x == 0 && i == p.stall_at) {
              mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
              ok = false;
              break;
            }
            if (i >= kStages &&
                !mbar_wait(&empty[s], static_cast<uint32_t>((i / kStages - 1) & 1), &abort_flag)) {
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
              const int s = i % kStages;
              if (!mbar_wait_cluster(&full[s], static_cast<uint32_t>((i / kStages) & 1), &abort_flag)) {
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
    }
  } else {
    if (EPI == kSwigluBack) take_registers<kTaken>();
    // A quarter of the lanes, and a share of the columns.
    const int quarter = warp & 3, share = (warp - kFirst) >> 2;
    uint8_t* so = stage_out + (warp - kFirst) * kWarpStage<EPI>;
    const uint32_t drained_bar = map_to_rank(smem_u32(&drained), 0);
    const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
    const uint64_t once = once_policy();
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
          const uint32_t at = tmem + lanes + share * 128;
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
        const int n = 2 * nt * kBoxRows + share * 128;
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
        const bool in = row < p.M;
        // kSwiglu: 64 gate columns and their up columns; kSwigluBack: 128 columns of dh.
        uint32_t v[4][32];
        const int n = EPI == kSwiglu ? nt * kBoxRows + share * 64 : 2 * nt * kBoxRows + share * 128;
        uint32_t scales[2] = {};                 // kSwigluBack from 8 bits: of four blocks
        if (lane == 0) bulk_wait_read<0>();      // the last tile's results have left the staging
        __syncwarp();
        if (EPI == kSwigluBack && m < p.M && n < p.N) {
          if constexpr (FLAG) {
            copy_saved8(p, so, m, n, lane, once);
            copies_commit();
            if (in)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (n + 32 * b < p.N) {
                  const int64_t c = n / 32 + b;
                  const uint32_t sg = __ldg(p.s + blocked_offset(row, c, p.s_cols4));
                  const uint32_t su = __ldg(p.s + blocked_offset(row, p.N / 32 + c, p.s_cols4));
                  scales[0] |= sg << (8 * b);
                  scales[1] |= su << (8 * b);
                }
          } else {
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (n + 32 * b < p.N) copy_saved16(p, so + 4096 * b, m, n + 32 * b, lane, once);
              copies_commit();
            }
          }
        }
        const uint32_t at = tmem + lanes + share * (EPI == kSwiglu ? 64 : 128);
        constexpr int kNext = EPI == kSwiglu ? 128 : 64;      // where the second 64 columns are
        if (!mbar_wait(&ready, static_cast<uint32_t>(item++ & 1), &abort_flag)) {
          ok = false;
          break;
        }
        tcgen05_fence_after();
        tmem_ld_32(at, v[0]);
        tmem_ld_32(at + 32, v[1]);
        tmem_ld_32(at + kNext, v[2]);
        tmem_ld_32(at + kNext + 32, v[3]);
        tmem_ld_wait();
        tcgen05_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(drained_bar);
        if constexpr (EPI == kSwiglu && FLAG) {
          // The other runs.
          for (int k0 = p.run; k0 < p.k_blocks; k0 += p.run, ++item) {
            if (!mbar_wait(&ready, static_cast<uint32_t>(item & 1), &abort_flag)) {
              ok = false;
              break;
            }
            tcgen05_fence_after();
#pragma unroll
            for (int b = 0; b < 8; ++b) {
              uint32_t w[16];
              tmem_ld_16(at + (b >> 2) * kNext + 16 * (b & 3), w);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                uint32_t& x = v[b >> 1][(b & 1) * 16 + j];
                x = __float_as_uint(__uint_as_float(x) + __uint_as_float(w[j]));
              }
            }
            tcgen05_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(drained_bar);
          }
          if (!ok) break;
        }
        if constexpr (EPI == kSwiglu && FLAG) {
          // The padding of the saved scales: rows behind the last, columns behind a row.
          const int64_t rows = (p.M + kBoxRows - 1) / kBoxRows * kBoxRows;
          if (row < rows && n < p.N) {
            if (!in)
#pragma unroll
              for (int b = 0; b < 4; ++b)
                if (n + (b & 1) * 32 < p.N)
                  store_scale(p, row, n / 32 + (b & 1) + (b >> 1) * (p.N / 32), 0);
            if (n + 64 >= p.N)
              for (int64_t c = p.N / 16; c < p.s_cols4; ++c) store_scale(p, row, c, 0);
          }
        }
        if (m >= p.M || n >= p.N) continue;
        if constexpr (EPI == kSwiglu) {
          auto value = [&](int b, int j) {
            return pair(__uint_as_float(v[b][2 * j]), __uint_as_float(v[b][2 * j + 1]));
          };
          uint8_t* dst = so + lane * 128;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f32x2 g[4], u[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              g[k] = value(j >> 2, (j & 3) * 4 + k);
              u[k] = value(2 + (j >> 2), (j & 3) * 4 + k);
            }
            *reinterpret_cast<uint4*>(dst + ((j ^ (lane & 7)) << 4)) = gated8(g, u);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&maps.out, n, m, so);
            bulk_commit();
          }
          if constexpr (FLAG) {
            // Gate's bytes behind h, up's in its place when it has left.
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              // Block b: gate's two, up's two.
              if (b == 2) {
                if (lane == 0) bulk_wait_read<0>();
                __syncwarp();
              }
              uint8_t* saved = b < 2 ? so + kStageOut : so;
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
                *box64(saved, lane, (b & 1) * 2 + j) =
                    make_uint4(four(16 * j), four(16 * j + 4), four(16 * j + 8), four(16 * j + 12));
              if (in && c < p.N) store_scale(p, row, ((b >> 1) ? p.N + c : c) >> 5, sbyte);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&maps.gate, n, m, so + kStageOut);
              tma_store_2d(&maps.up, n, m, so);
              bulk_commit();
            }
          }
        } else {
          SavedBlock ahead;
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const int64_t c = n + 32 * b;
            if (c >= p.N) break;
            uint8_t *out_g, *out_u;
            auto dh8 = [&](int j, f32x2 (&d)[4]) {
#pragma unroll
              for (int k = 0; k < 4; ++k)
                d[k] = pair(__uint_as_float(v[b][8 * j + 2 * k]), __uint_as_float(v[b][8 * j + 2 * k + 1]));
            };
            if constexpr (FLAG) {
              // A block ahead in registers, so that two places are free for the results: those
              // of the blocks read, and 2 KB behind them.
              //   block   0          1        2        3
              //   dg, du  behind, 0  1, 2     behind, 3   0, 1
              if (b == 0) {
                copies_wait<0>();
                __syncwarp();
                ahead.load(so, lane);
              }
              const SavedBlock w = ahead;
              if (b < 3) ahead.load(so + 2048 * (b + 1), lane);
              if (lane == 0) bulk_wait_read<1>();
              __syncwarp();
              out_g = so + 2048 * (b & 1 ? (b == 1 ? 1 : 0) : 4);
              out_u = so + 2048 * (b == 0 ? 0 : b == 3 ? 1 : b + 1);
              const uint32_t sg = scales[0] >> (8 * b) & 0xFFu, su = scales[1] >> (8 * b) & 0xFFu;
              auto eight = [&](int j, bool low) {
                f32x2 d[4], gv[4], uv[4];
                dh8(j, d);
                const uint4 &wg = w.g[j >> 1], &wu = w.u[j >> 1];
                mx_get_pairs((j & 1) ? make_uint2(wg.z, wg.w) : make_uint2(wg.x, wg.y), sg, gv);
                mx_get_pairs((j & 1) ? make_uint2(wu.z, wu.w) : make_uint2(wu.x, wu.y), su, uv);
                uint4 dg, du;
                gated_back8(d, gv, uv, low, dg, du);
                *box64(out_g, lane, j) = dg;
                *box64(out_u, lane, j) = du;
              };
              const bool low = may_be_low(sg);
#pragma unroll
              for (int j = 0; j < 4; ++j) eight(j, low);
            } else {
              // Copies of the first two blocks are in flight together, then of the others.
              if (b & 1) copies_wait<0>();
              else copies_wait<1>();
              __syncwarp();
              out_g = so + 4096 * (b & 1);
              out_u = out_g + 2048;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                f32x2 d[4], gv[4], uv[4];
                dh8(j, d);
                const uint4 g = *box64(out_g, lane, j), u = *box64(out_u, lane, j);
                get_pairs(g, gv);
                get_pairs(u, uv);
                uint4 dg, du;
                gated_back8(d, gv, uv, any_low(lowest2(g)), dg, du);
                *box64(out_g, lane, j) = dg;
                *box64(out_u, lane, j) = du;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d_once(&maps.gate, static_cast<int>(c), m, out_g, once);
              tma_store_2d_once(&maps.up, static_cast<int>(c), m, out_u, once);
              bulk_commit();
            }
            if (!FLAG && b == 1) {
              // The next two blocks, as soon as the first two's results have left.
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                if (lane == 0) {
                  if (k == 0) bulk_wait_read<1>();
                  else bulk_wait_read<0>();
                }
                __syncwarp();
                if (c + 32 * (k + 1) < p.N)
                  copy_saved16(p, so + 4096 * k, m, c + 32 * (k + 1), lane, once);
                copies_commit();
              }
            }
          }
        }
      }
    }
    if (EPI == kSwigluBack) copies_wait<0>();
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
          mbar_complete_tx(&full[j % kStages], S::kPairBytes);
        else
          mbar_arrive_expect_tx(&full[j % kStages], S::kPairBytes);
      }
      for (int j = max(0, hi - kStages); j < hi; ++j)
        mbar_drain(&full[j % kStages], static_cast<uint32_t>((j / kStages) & 1),
                   100000000ull);
    }
    __syncthreads();
  }
  cluster_sync();
  tcgen05_fence_after();
  if (warp == 1) tmem_dealloc<2>(tmem, 512);
  if (threadIdx.x == 0 && failed) atomicOr(&g_product_watchdog, 1);
}

// Steps summed in tensor memory at a time, where it matters, at most.  fp32 results: as
// mx_matmul.  Saved ones: fewer, so that about as few of them as of a plain fp32 product's go
// to the other neighbour in e4m3, or whole blocks to the other scale.  e4m3 operands, 5120
// steps: one run is 3e-7 off in the 2-norm, two 1.64e-7, three 1.14e-7, four 9.3e-8, a plain
// fp32 product 1.05e-7.  Of 67 million saved values 98, 221, 379 and 428 are not those of the
// sums in 64 bits at 1024, 2560, 5120 and 8192 steps, of a plain fp32 product's 196, 233, 352
// and 431.  e2m1 operands need it less: products of elements are quarters of whole numbers, so
// that sums under scales near each other fit 24 bits (none of the values differed, in runs of
// 256 to 4096 steps); runs count where a row's scales spread over many powers of two.  A run is
// to outlast the epilogue of the tile before: 16640 x 8192 x 5120 e4m3 takes 797 us in one run,
// 820 to 835 in three, 870 in four; e2m1, at twice the rate, 411 in one, 440 to 450 in two, 497
// in three.
constexpr int kRunSteps = 4096;
template <bool FP4>
constexpr int kSavedRunSteps = FP4 ? 2560 : 1792;

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
    // The warpgroups' shares must be there at launch: one that asked for more would wait.
    cudaFuncAttributes fa;
    if (const cudaError_t e = cudaFuncGetAttributes(&fa, pair_kernel<FP4, EPI, FLAG>))
      return static_cast<int>(e);
    if (EPI == kSwigluBack && fa.numRegs * kPairThreads<EPI> < 128 * kGiven + 256 * kTaken)
      return static_cast<int>(cudaErrorInvalidConfiguration);
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
      cluster_config(at, 2 * pairs, kPairThreads<EPI>, kPairSmem<FP4, EPI>, 2, stream);
  return static_cast<int>(cudaLaunchKernelEx(&cfg, pair_kernel<FP4, EPI, FLAG>, maps, p));
}

template <bool FP4, int EPI, bool RUNS>
int launch_tile_kernel(const ProductMaps& maps, const ProductParams& p, cudaStream_t stream) {
  constexpr int kSmem = kTileStages * Shape<FP4>::kTileStride + 1024;
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(tile_kernel<FP4, EPI, RUNS>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
  });
  if (attr != 0) return attr;
  const int64_t ctas = static_cast<int64_t>(p.m_tiles) * p.n_tiles * p.cluster;
  if (ctas > 0x7fffffff) return static_cast<int>(cudaErrorInvalidConfiguration);
  cudaLaunchAttribute at[2];
  const cudaLaunchConfig_t cfg =
      cluster_config(at, ctas, kTileThreads<EPI>, kSmem, static_cast<unsigned>(p.cluster), stream);
  return static_cast<int>(cudaLaunchKernelEx(&cfg, tile_kernel<FP4, EPI, RUNS>, maps, p));
}

// The tile kernel's tiles: columns, and CTAs that share the contraction; the quickest as
// reckoned in ns (tile_shape in mx_matmul.cu has the measurements).  halves: clusters of twice
// the CTAs, gate and up (kSwiglu).
struct TileChoice {
  int cols, split;
};

inline TileChoice choose_tiles(int64_t M, int64_t N, int64_t k_blocks, int num_sms, int halves) {
  TileChoice best = {128, 1};
  int64_t least = INT64_MAX;
  for (int cols = 128; cols >= 64; cols /= 2) {
    const int64_t tiles = (M + 127) / 128 * ((N + cols - 1) / cols);
    for (int s = 1; s * halves <= 8 && s <= k_blocks; s *= 2) {
      const int cluster = s * halves;
      const int64_t ctas = tiles * cluster;
      if (s > 1 && ctas > (cluster == 8 ? 96 : cluster == 4 ? 128 : num_sms)) break;
      const int64_t rounds = (ctas + num_sms - 1) / num_sms;
      const int64_t cost = rounds * (500 + (cols == 128 ? 500 : 0) + (k_blocks + s - 1) / s * 220 +
                                     (cluster > 1 ? 400 + 19 * (M < 128 ? M : 128) * cols / 128 : 0));
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
  p.split = p.cluster = 1;
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
