// mx_matmul.cu -- the product of two MX-FP8 operands on the block-scaled
// tensor cores of sm_103a:
//
//   C[m][n] = sum_k (qa[m][k] 2^(sa[m][k/32] - 127)) (qb[n][k] 2^(sb[n][k/32] - 127))
//
// qa (M x K) and qb (N x K) are e4m3 with their contraction dimension
// contiguous, sa and sb their e8m0 scales in the 128x4 blocked layout: the
// outputs of the casts as they stand.  tcgen05.mma kind::mxf8f6f4 with
// block_scale multiplies 32 contraction steps at a time, takes one scale per
// row and 32 steps from tensor memory, and accumulates in fp32 in tensor
// memory.  A 128x4 blocked scale tile holds the scales of 128 rows and 128
// contraction steps, in the order in which tcgen05.cp 32x128b.warpx4 lays
// them out in tensor memory, so scales go from global to shared to tensor
// memory without a thread touching them.
//
// Either operand may instead be stored with its rows contiguous (K x M, K x N
// bytes; the scales stay along the contraction): the tensor cores read it
// through an MN-major descriptor.
//
// pair_matmul_kernel: persistent CTA pairs, a 256 x 256 tile of C at a time.
// The pair's two SMs share one MMA (cta_group::2): each loads 128 rows of A and
// 128 of B for every 128 contraction steps and holds 128 rows of the result,
// so a byte of shared memory feeds twice the products that one CTA's tile
// would.  Loads run five stages ahead of the MMAs.  Tensor memory holds a result of
// 256 columns and the scales; the eight epilogue warps of a CTA take a result into
// registers at once, and the next tile's MMAs, which wait for that, run while they
// store it.  (Two results do not fit beside the scales.)  For an fp32 result longer
// sums, in this kernel and the next, are cut into runs of at most 4096 steps that the
// epilogue adds up in registers: the tensor core's accumulator cuts bits off at every
// addition, an error that grows with the run.  Over 16640 steps, in the 2-norm: random
// signs 1.8e-7 (one run 1.2e-6, a plain fp32 product 1.9e-7), one sign 8.8e-7 (9.9e-6,
// 8.2e-7).  A bf16 result does not notice.  16640 x 8192 x 5120 takes 365 us
// (3.8 PFLOP/s); launched again and again 461 us (3.0), where the GPU's power limit
// sets the clock.  The tensor cores are the bound (busy in 78% of all cycles at
// 8192 x 8192 x 4096); the rest goes to a launch's first loads, to the last tiles'
// stores, and to pairs that have no tile left.
//
// Rows of results that no tensor map can describe (no multiple of 16 bytes) leave
// the same shared memory a row at a time, by the warp: 16640 x 8191 x 5120 415 us
// (839 in single tiles, eight values a thread), 2000 x 3001 x 1024 14.0 (30.0; 11.5 at
// 3008).
//
// tile_matmul_kernel: one 128 x 128 (or 64) tile of C per cluster of S CTAs, the
// contraction cut into S equal shares of 128-step blocks; each CTA leaves its
// partial tile in its shared memory, and each then sums 128 / S of the tile's
// rows over the S CTAs in rank order (fixed order: the same bits every time).  The runs
// of long fp32 sums cost 5%: 1536 x 1536 x 16640 37.8 -> 40.1 us, 1024 x 1024 x 65536
// 72.6 -> 76.2.
// 160 x 1024 x 1024 takes 4.9 us, 1 x 8192 x 5120 9.3: latency (loads, the chain of
// a tile's MMAs, the stores), not bandwidth.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx_common.cuh"
#include "mx_kernels.h"
#include "mx_tensor.cuh"

namespace mx {
namespace {

__device__ int g_matmul_watchdog = 0;

}  // namespace

// Rows of an operand's load box in the tile kernel: no more than there are (a box
// past the operand's end is filled with zeros at the price of a load).  What a
// narrower box leaves in shared memory only reaches results that are not stored.
int matmul_box_rows(int64_t rows, bool mn, int tile) {
  return mn || rows >= tile ? tile : static_cast<int>((rows + 7) & ~int64_t{7});
}

namespace {

// The tile kernel's tiles: columns, and CTAs that share a tile's contraction.  Reckoned
// for operands stored by row whatever the order, so that the order does not change
// the sums.
struct TileShape {
  int cols, split;
};

// The quickest as reckoned in ns from what was measured: 220 for 128 contraction
// steps, 500 more for the stores of 128 columns, and for joining (partial sums through
// distributed shared memory, two cluster barriers) 400 and 19 for each row of 128
// results.  160 x 1024 x 1024: 5.7 us in 128 columns, 5.1 in 64, 7.1 in two CTAs;
// 64 x 8192 x 5120: 11.9 in 128 columns and two CTAs, 13.3 in 64; 32 x 32 x 16640: 34
// whole, 8.4 in eight.  Clusters of eight only up to 96 CTAs, of four up to 128: more of
// them do not all find room at once (512 x 512 x 16640, 128 CTAs: 15.8 us in four, 24.5
// in eight; 38 x 2319 x 2112, 148 CTAs in clusters of four: 11.1 us, 76 7.5).
TileShape tile_shape(int64_t M, int64_t N, int64_t k_blocks, int num_sms) {
  TileShape best = {128, 1};
  int64_t least = 500 + k_blocks * 220;
  for (int cols = 128; cols >= 64; cols /= 2) {
    const int64_t tiles = (M + 127) / 128 * ((N + cols - 1) / cols);
    for (int s = 1; s <= 8 && s <= k_blocks; s *= 2) {
      if (tiles * s > (s == 8 ? 96 : s == 4 ? 128 : num_sms)) break;
      const int64_t cost = (cols == 128 ? 500 : 0) + (k_blocks + s - 1) / s * 220 +
                           (s > 1 ? 400 + 19 * (M < 128 ? M : 128) * cols / 128 : 0);
      if (cost < least) {
        least = cost;
        best = {cols, s};
      }
    }
  }
  return best;
}

}  // namespace

// Columns of the tile kernel's tiles (an operand stored by column comes in whole 128).
int matmul_tile_cols(int64_t M, int64_t N, int64_t K, bool b_mn, int num_sms) {
  return b_mn ? 128 : tile_shape(M, N, (K + 127) / 128, num_sms).cols;
}

// Whether a tensor map can describe rows of N results.
bool matmul_mapped(int64_t N, bool out_f32) { return (N * (out_f32 ? 4 : 2)) % 16 == 0; }

namespace {

constexpr int kBK = 128;                    // contraction bytes of one stage
constexpr int kTile = 128;                  // rows of one operand box
constexpr int kBoxBytes = kTile * kBK;      // 16 KB
constexpr int kSfBytes = 512;               // one 128x4 blocked scale tile
constexpr int kStageOut = 4096;             // 32 rows x 128 bytes on their way out
constexpr int kRun = 32;                    // blocks of a run, summed in tensor memory, for fp32

struct MatmulParams {
  void* out;
  int64_t M, N;
  int k_blocks;        // ceil(K / 128)
  int last_steps;      // 32-step MMAs of the last block, 1..4
  int m_tiles, n_tiles;
  int split;           // CTAs of a cluster along the contraction (tile kernel)
  int out_f32;
  int a_mn, b_mn;      // operand stored with its rows contiguous
  int run;             // blocks summed in tensor memory at a time, at most
  int band;            // M-tiles of a band (pair kernel)
  int mapped;          // maps.out describes the result's rows
  int load_bytes;      // of a stage (tile kernel)
  int cols;            // of a tile, 64 or 128 (tile kernel)
  Span sp_out;
  int64_t stall_at;
  uint64_t stall_ns;
};

// ---- one tile per cluster ------------------------------------------------------

// What has more tiles than there are SMs goes to the pairs, so that a CTA has an SM to
// itself and its ring may take most of the shared memory (1024^3: 5.3 us, 6.2 with three
// stages).
constexpr int kTileStages = 6;
constexpr int kTileStageBytes = 2 * kBoxBytes + 2 * kSfBytes;
constexpr int kTileThreads = 192;           // loads, MMA, four epilogue warps
constexpr int kPitch = 132;                 // floats a row of the partial tile
static_assert(kTile * kPitch * 4 <= kTileStages * kTileStageBytes, "partial tile fits the ring");

// Where run r of n blocks' equal runs ends.
__device__ __forceinline__ int run_end(int n, int runs, int r) {
  return static_cast<int>(static_cast<int64_t>(n) * (r + 1) / runs);
}

// RUNS: a CTA's contraction is cut into equal runs of at most p.run blocks, summed in
// two places of tensor memory in turn; the epilogue warps add the runs up in
// registers, a run's place being read while the next one's MMAs go on.
template <bool RUNS>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_matmul_kernel(const __grid_constant__ MatmulMaps maps, const MatmulParams p) {
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
  const int mt = tile % p.m_tiles, n0 = tile / p.m_tiles * p.cols;
  // Blocks of this CTA: equal shares, the first ones one longer.
  const int per = p.k_blocks / p.split, more = p.k_blocks % p.split;
  const int kb0 = rank * per + (rank < more ? rank : more);
  const int nkb = per + (rank < more ? 1 : 0);
  const int runs = RUNS ? (nkb + p.run - 1) / p.run : 1;
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
  }
  if (warp == 1) tmem_alloc<1>(&tmem_base, kTmemCols);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t t_sfa = tmem + kTmemCols / 2, t_sfb = t_sfa + 4;
  const int quarter = warp & 3;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
  // This lane's row of the runs before the last.
  float sums[RUNS ? kTile : 1] = {};

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
        uint8_t* st = ring + s * kTileStageBytes;
        const int kb = kb0 + i;
        mbar_arrive_expect_tx(&full[s], static_cast<uint32_t>(p.load_bytes));
        tma_load_2d(st, &maps.a, p.a_mn ? mt * kTile : kb * kBK, p.a_mn ? kb * kBK : mt * kTile,
                    &full[s]);
        tma_load_2d(st + kBoxBytes, &maps.b, p.b_mn ? n0 : kb * kBK, p.b_mn ? kb * kBK : n0,
                    &full[s]);
        tma_load_2d(st + 2 * kBoxBytes, &maps.sa, kb * 128, mt, &full[s]);
        tma_load_2d(st + 2 * kBoxBytes + kSfBytes, &maps.sb, kb * 128, n0 / kTile, &full[s]);
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
      const uint32_t idesc = mxf8_idesc(128, p.cols, p.a_mn, p.b_mn);
      // The scales of 32 rows of B take a column of tensor memory: a tile of 64 columns
      // reads the first or the last two of its rows' four.
      const uint32_t t_sfb_here = t_sfb + (n0 % kTile) / 32;
      const uint32_t step_a = p.a_mn ? kStepMN : kStepK, step_b = p.b_mn ? kStepMN : kStepK;
      int s = 0;
      uint32_t turn = 0;
      int run = 0, begin = 0, end = run_end(nkb, runs, 0);     // this run and its blocks
      uint32_t d = tmem;
      for (int i = 0; i < nkb; ++i) {
        if (RUNS && i == end) {
          tcgen05_commit<1>(&ready[run & 1]);
          begin = end;
          end = run_end(nkb, runs, ++run);
          d = tmem + (run & 1) * kTile;
          if (run >= 2 && !mbar_wait(&drained[run & 1], static_cast<uint32_t>((run >> 1) - 1) & 1u,
                                     &abort_flag))
            break;
        }
        if (!mbar_wait(&full[s], turn, &abort_flag)) break;
        tcgen05_fence_after();
        const uint32_t st = smem_u32(ring + s * kTileStageBytes);
        tcgen05_cp_scales<1>(t_sfa, scale_desc(st + 2 * kBoxBytes));
        tcgen05_cp_scales<1>(t_sfb, scale_desc(st + 2 * kBoxBytes + kSfBytes));
        const uint64_t da = operand_desc(st), db = operand_desc(st + kBoxBytes);
        const int steps = kb0 + i == p.k_blocks - 1 ? p.last_steps : 4;
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (k < steps)
            mma_mxf8<1>(d, da + step_a * k, db + step_b * k, mxf8_idesc_step(idesc, k), t_sfa,
                        t_sfb_here, i > begin || k > 0);
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
      const uint32_t at = tmem + lanes + (run & 1) * kTile;
#pragma unroll
      for (int c = 0; c < kTile; c += 16) {
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
  // Columns c .. c + 32 of this lane's row: the last run and, RUNS, those before it.
  const uint32_t last = tmem + lanes + ((runs - 1) & 1) * kTile;
  auto get = [&](int c, uint32_t (&v)[32]) {
    tmem_ld_32(last + c, v);
    tmem_ld_wait();
    if constexpr (RUNS)
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(sums[c + j] + __uint_as_float(v[j]));
  };
  constexpr int kUnroll = RUNS ? 4 : 1;      // sums are registers: c must be a constant
  if (p.split == 1) {
    // 32 rows at a time and warp through shared memory, and a tensor map where one
    // can describe the result, 128 bytes of a row a box.
    const int64_t m = static_cast<int64_t>(mt) * kTile + quarter * 32;
    if (warp >= 2 && ok && m < p.M) {
      uint8_t* so = ring + quarter * 4 * kStageOut;
      const int per = p.out_f32 ? 32 : 64;              // columns of a box
#pragma unroll kUnroll
      for (int c = 0; c < kTile; c += 32) {
        if (c >= p.cols || n0 + c >= p.N) break;
        uint32_t v[32];
        get(c, v);
        uint8_t* row = so + c / per * kStageOut + lane * 128;
        if (p.out_f32) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4)) =
                make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
        } else {
          const int j0 = (c >> 3) & 4;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            auto f = [&](int k) { return __uint_as_float(v[8 * j + k]); };
            *reinterpret_cast<uint4*>(row + (((j0 + j) ^ (lane & 7)) << 4)) =
                make_uint4(bf16x2(f(0), f(1)), bf16x2(f(2), f(3)), bf16x2(f(4), f(5)),
                           bf16x2(f(6), f(7)));
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (!p.mapped) {
        for (int c = 0; c < p.cols && n0 + c < p.N; c += per) {
          const uint8_t* box = so + c / per * kStageOut;
          if (p.out_f32) store_box<4>(box, p.out, m, n0 + c, p.M, p.N, lane, p.sp_out);
          else store_box<2>(box, p.out, m, n0 + c, p.M, p.N, lane, p.sp_out);
        }
      } else if (lane == 0) {
        for (int c = 0; c < p.cols && n0 + c < p.N; c += per)
          tma_store_2d(&maps.out, n0 + c, static_cast<int>(m), so + c / per * kStageOut);
        bulk_commit();
        bulk_wait<0>();
      }
      tcgen05_fence_before();
    }
    __syncthreads();
    if (warp == 1) {
      tcgen05_fence_after();
      tmem_dealloc<1>(tmem, kTmemCols);
    }
    if (threadIdx.x == 0 && !ok) atomicOr(&g_matmul_watchdog, 1);
    return;
  }
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2) {
    const int row = quarter * 32 + lane;
#pragma unroll kUnroll
    for (int c = 0; c < kTile; c += 32) {
      if (c >= p.cols) break;
      uint32_t v[32];
      get(c, v);
      uint4* dst = reinterpret_cast<uint4*>(part + row * kPitch + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dst[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
    }
    tcgen05_fence_before();
  }
  cluster_sync();
  // Rows of the tile that this CTA writes, summed over the cluster: the loads of
  // all CTAs' values are under way before the first is added.
  const int rows = kTile / p.split;
  const int64_t m0 = static_cast<int64_t>(mt) * kTile + rank * rows;
  const bool vec = (p.N & 7) == 0;
  if (ok) {
    const int shift = p.cols == 128 ? 4 : 3, pieces = 1 << shift;      // of eight, a row
    for (int i = threadIdx.x; i < rows * pieces; i += kTileThreads) {
      const int r = i >> shift, c = (i & (pieces - 1)) * 8;
      const int64_t m = m0 + r, n = n0 + c;
      if (m >= p.M || n >= p.N) continue;
      const uint32_t at = smem_u32(part + (rank * rows + r) * kPitch + c);
      float4 lo[8], hi[8];
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < p.split) {
          const uint32_t a = map_to_rank(at, static_cast<uint32_t>(q));
          lo[q] = ld_cluster_f4(a);
          hi[q] = ld_cluster_f4(a + 16);
        }
      float v[8] = {};
#pragma unroll
      for (int q = 0; q < 8; ++q)
        if (q < p.split) {
          v[0] += lo[q].x; v[1] += lo[q].y; v[2] += lo[q].z; v[3] += lo[q].w;
          v[4] += hi[q].x; v[5] += hi[q].y; v[6] += hi[q].z; v[7] += hi[q].w;
        }
      store_out8(p.out, p.out_f32, m * p.N + n, v,
                 vec ? 8 : static_cast<int>(p.N - n < 8 ? p.N - n : 8), vec, p.sp_out);
    }
  }
  cluster_sync();                             // peers have read this CTA's partial tile
  if (warp == 1) tmem_dealloc<1>(tmem, kTmemCols);
  if (threadIdx.x == 0 && !ok) atomicOr(&g_matmul_watchdog, 1);
}

// ---- CTA pairs -------------------------------------------------------------------

constexpr int kPairStages = 5;
constexpr int kPairStageBytes = 2 * kBoxBytes + 3 * kSfBytes;
constexpr int kPairStrideBytes = 34 * 1024;   // 1024-byte aligned boxes
constexpr int kPairThreads = 320;             // loads, MMA, eight epilogue warps
constexpr int kPairSmem = kPairStages * kPairStrideBytes + 8 * kStageOut + 1024;
constexpr uint32_t kSfaCol = 256, kSfbCol = 260;

struct Tiles {
  int m_tiles, n_tiles, band;
  // Bands of `band` M-tiles, walked along N, M fastest inside a band.
  __device__ __forceinline__ void at(int t, int& mt, int& nt) const {
    const int per = band * n_tiles;
    const int b = t / per, i = t - b * per;
    const int rows = min(band, m_tiles - b * band);
    nt = i / rows;
    mt = b * band + (i - nt * rows);
  }
};

template <bool F32>
__global__ void __launch_bounds__(kPairThreads, 1)
    pair_matmul_kernel(const __grid_constant__ MatmulMaps maps, const MatmulParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kPairStages], empty[kPairStages], ready, drained, done,
      stall_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag, issued;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* stage_out = ring + kPairStages * kPairStrideBytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int first = blockIdx.x >> 1, stride = gridDim.x >> 1;
  const int n_tiles = p.m_tiles * p.n_tiles;
  const Tiles tiles{p.m_tiles, p.n_tiles, p.band};

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
        const int m = (2 * mt + rank) * kTile, n = (2 * nt + rank) * kTile;
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
          uint8_t* st = ring + s * kPairStrideBytes;
          const uint32_t bar = map_to_rank(smem_u32(&full[s]), 0);
          // The leader alone announces both CTAs' bytes: a remote arrival per
          // stage, with its release over the cluster, took as long as the
          // stage's MMAs twice over (969 us against 428 us at 16640 x 8192 x 5120).
          if (rank == 0) mbar_arrive_expect_tx(&full[s], 2 * kPairStageBytes);
          tma_load_2d_pair(st, &maps.a, p.a_mn ? m : kb * kBK, p.a_mn ? kb * kBK : m, bar);
          tma_load_2d_pair(st + kBoxBytes, &maps.b, p.b_mn ? n : kb * kBK, p.b_mn ? kb * kBK : n,
                           bar);
          tma_load_2d_pair(st + 2 * kBoxBytes, &maps.sa, kb * 128, 2 * mt + rank, bar);
          tma_load_2d_pair(st + 2 * kBoxBytes + kSfBytes, &maps.sb, kb * 128, 2 * nt, bar);
        }
      }
      issued = i;
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      const uint32_t idesc = mxf8_idesc(256, 256, p.a_mn, p.b_mn);
      const uint32_t step_a = p.a_mn ? kStepMN : kStepK, step_b = p.b_mn ? kStepMN : kStepK;
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
            const uint32_t st = smem_u32(ring + s * kPairStrideBytes);
            tcgen05_cp_scales<2>(tmem + kSfaCol, scale_desc(st + 2 * kBoxBytes));
            tcgen05_cp_scales<2>(tmem + kSfbCol, scale_desc(st + 2 * kBoxBytes + kSfBytes));
            tcgen05_cp_scales<2>(tmem + kSfbCol + 4, scale_desc(st + 2 * kBoxBytes + 2 * kSfBytes));
            const uint64_t da = operand_desc(st), db = operand_desc(st + kBoxBytes);
            const int steps = kb == p.k_blocks - 1 ? p.last_steps : 4;
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (k < steps)
                mma_mxf8<2>(tmem, da + step_a * k, db + step_b * k, mxf8_idesc_step(idesc, k),
                            tmem + kSfaCol, tmem + kSfbCol, kb > k0 || k > 0);
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
    // This lane's row of 128 results, in boxes of 128 bytes: four of fp32, two of
    // bf16 (packed as they are read).
    constexpr int kBoxes = F32 ? 4 : 2;
    uint32_t v[kBoxes][32];
    int item = 0;
    bool ok = true;
    for (int t = first; ok && t < n_tiles; t += stride) {
      int mt, nt;
      tiles.at(t, mt, nt);
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
      const int m = (2 * mt + rank) * kTile + quarter * 32;
      const int n = 2 * nt * kTile + half * 128;
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
    }
    if (lane == 0) bulk_wait<0>();
    tcgen05_fence_before();
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();
  // Gave up in either CTA: in the leader, settle the stages that only one CTA
  // loaded (bytes announced for the peer that will not come; the peer's bytes
  // that were not announced), so that what is in flight can be waited for.
  const int peer_abort = ld_cluster_s32(map_to_rank(smem_u32(&abort_flag), rank ^ 1));
  const bool failed = abort_flag != 0 || peer_abort != 0;
  if (failed) {
    if (rank == 0 && threadIdx.x == 0) {
      const int other = ld_cluster_s32(map_to_rank(smem_u32(&issued), 1));
      const int lo = min(issued, other), hi = max(issued, other);
      for (int j = lo; j < hi; ++j) {
        if (issued > other)
          mbar_complete_tx(&full[j % kPairStages], kPairStageBytes);
        else
          mbar_arrive_expect_tx(&full[j % kPairStages], kPairStageBytes);
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
  if (threadIdx.x == 0 && failed) atomicOr(&g_matmul_watchdog, 1);
}

// The pair kernel takes what has enough 256 x 256 tiles to keep the GPU's pairs busy.
bool use_pairs(int64_t M, int64_t N, int num_sms) {
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  return tiles * 4 >= num_sms;
}

}  // namespace

bool matmul_pairs(int64_t M, int64_t N, int num_sms) { return use_pairs(M, N, num_sms); }

template <bool F32>
static int launch_pairs(const MatmulMaps& maps, MatmulParams p, int num_sms, cudaStream_t stream) {
  p.m_tiles = static_cast<int>((p.M + 255) / 256);
  p.n_tiles = static_cast<int>((p.N + 255) / 256);
  // Equal runs: a short last one would leave no time to read the one before.
  const int runs = F32 ? (p.k_blocks + kRun - 1) / kRun : 1;
  p.run = (p.k_blocks + runs - 1) / runs;
  p.band = 8;
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(
        pair_matmul_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPairSmem));
  });
  if (attr != 0) return attr;
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  const int64_t pairs = tiles < num_sms / 2 ? tiles : num_sms / 2;
  if (tiles > 0x3fffffff) return static_cast<int>(cudaErrorInvalidConfiguration);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = 2;
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, pair_matmul_kernel<F32>, maps, p));
}

template <bool RUNS>
static int launch_tiles(const MatmulMaps& maps, const MatmulParams& p, int64_t ctas,
                        cudaStream_t stream) {
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(
        tile_matmul_kernel<RUNS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
        kTileStages * kTileStageBytes + 1024));
  });
  if (attr != 0) return attr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(kTileStages * kTileStageBytes + 1024);
  cfg.stream = stream;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, tile_matmul_kernel<RUNS>, maps, p));
}

int launch_matmul(const MatmulMaps& maps, int64_t M, int64_t N, int64_t K, bool a_mn,
                  bool b_mn, void* out, bool out_f32, int num_sms, cudaStream_t stream) {
  MatmulParams p = {};
  p.a_mn = a_mn;
  p.b_mn = b_mn;
  p.out = out;
  p.M = M;
  p.N = N;
  p.k_blocks = static_cast<int>((K + kBK - 1) / kBK);
  p.last_steps = static_cast<int>((K - static_cast<int64_t>(p.k_blocks - 1) * kBK) / 32);
  p.out_f32 = out_f32;
  p.mapped = matmul_mapped(N, out_f32);
  p.sp_out = make_span(out, static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * (out_f32 ? 4 : 2));
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  if (use_pairs(M, N, num_sms))
    return out_f32 ? launch_pairs<true>(maps, p, num_sms, stream)
                   : launch_pairs<false>(maps, p, num_sms, stream);
  p.m_tiles = static_cast<int>((M + kTile - 1) / kTile);
  const TileShape shape = tile_shape(M, N, p.k_blocks, num_sms);
  p.cols = b_mn ? 128 : shape.cols;
  p.split = shape.split;
  p.n_tiles = static_cast<int>((N + p.cols - 1) / p.cols);
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  p.load_bytes = (matmul_box_rows(M, a_mn, kTile) + matmul_box_rows(N, b_mn, p.cols)) * kBK + 2 * kSfBytes;
  if (tiles * p.split > 0x7fffffff) return static_cast<int>(cudaErrorInvalidConfiguration);
  // The longest of a cluster's shares, in blocks.
  p.run = kRun;
  return out_f32 && (p.k_blocks + p.split - 1) / p.split > kRun
             ? launch_tiles<true>(maps, p, tiles * p.split, stream)
             : launch_tiles<false>(maps, p, tiles * p.split, stream);
}

int out_of_bounds_matmul(bool clear) { return read_out_of_bounds(clear); }

int read_matmul_watchdog(int* out, bool clear) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_matmul_watchdog, sizeof(int));
  if (e != cudaSuccess) return static_cast<int>(e);
  if (clear && v) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_matmul_watchdog, &z, sizeof(int));
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  *out = v;
  return 0;
}

}  // namespace mx
