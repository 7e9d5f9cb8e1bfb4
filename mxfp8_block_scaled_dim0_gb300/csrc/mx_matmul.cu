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
// tile_matmul_kernel: one 128 x 128 tile of C per cluster of S CTAs, the
// contraction cut into S equal runs of 128-step blocks; each CTA leaves its
// partial tile in its shared memory, and each then sums 128 / S of the tile's
// rows over the S CTAs in rank order (fixed order: the same bits every run).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "mx_common.cuh"
#include "mx_kernels.h"
#include "mx_tensor.cuh"

namespace mx {
namespace {

__device__ int g_matmul_watchdog = 0;

constexpr int kBK = 128;                    // contraction bytes of one stage
constexpr int kTile = 128;                  // rows of one operand box
constexpr int kBoxBytes = kTile * kBK;      // 16 KB
constexpr int kSfBytes = 512;               // one 128x4 blocked scale tile

struct MatmulParams {
  void* out;
  int64_t M, N;
  int k_blocks;        // ceil(K / 128)
  int last_steps;      // 32-step MMAs of the last block, 1..4
  int m_tiles, n_tiles;
  int split;           // CTAs of a cluster along the contraction (tile kernel)
  int out_f32;
  Span sp_out;
  int64_t stall_at;
  uint64_t stall_ns;
};

// ---- one tile per cluster ------------------------------------------------------

constexpr int kTileStages = 4;
constexpr int kTileStageBytes = 2 * kBoxBytes + 2 * kSfBytes;
constexpr int kTileThreads = 192;           // loads, MMA, four epilogue warps
constexpr int kPitch = 132;                 // floats a row of the partial tile
constexpr int kTileSmem = kTileStages * kTileStageBytes + 1024;
static_assert(kTile * kPitch * 4 <= kTileStages * kTileStageBytes, "partial tile fits the ring");

__global__ void __launch_bounds__(kTileThreads, 1)
    tile_matmul_kernel(const __grid_constant__ MatmulMaps maps, const MatmulParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kTileStages], empty[kTileStages], done, stall_bar;
  __shared__ uint32_t tmem_base;
  __shared__ int abort_flag;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_rank());
  const int tile = blockIdx.x / p.split;
  const int mt = tile % p.m_tiles, nt = tile / p.m_tiles;
  // Blocks of this CTA: equal runs, the first ones one longer.
  const int per = p.k_blocks / p.split, more = p.k_blocks % p.split;
  const int kb0 = rank * per + (rank < more ? rank : more);
  const int nkb = per + (rank < more ? 1 : 0);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kTileStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
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
  if (warp == 1) tmem_alloc<1>(&tmem_base, 256);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  tcgen05_fence_before();
  __syncthreads();
  tcgen05_fence_after();
  const uint32_t tmem = tmem_base;
  const uint32_t t_sfa = tmem + 128, t_sfb = tmem + 132;

  if (warp == 0) {
    if (lane == 0) {
      int i = 0;
      for (; i < nkb; ++i) {
        const int s = i % kTileStages;
        if (kDiagStall && blockIdx.x == 0 && i == p.stall_at) {
          mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
          break;
        }
        if (i >= kTileStages &&
            !mbar_wait(&empty[s], static_cast<uint32_t>((i / kTileStages - 1) & 1), &abort_flag))
          break;
        uint8_t* st = ring + s * kTileStageBytes;
        const int kb = kb0 + i;
        mbar_arrive_expect_tx(&full[s], kTileStageBytes);
        tma_load_2d(st, &maps.a, kb * kBK, mt * kTile, &full[s]);
        tma_load_2d(st + kBoxBytes, &maps.b, kb * kBK, nt * kTile, &full[s]);
        tma_load_2d(st + 2 * kBoxBytes, &maps.sa, kb * 128, mt, &full[s]);
        tma_load_2d(st + 2 * kBoxBytes + kSfBytes, &maps.sb, kb * 128, nt, &full[s]);
      }
      // Gave up: the copies already issued land before the CTA moves on.
      if (i < nkb)
        for (int j = i > kTileStages ? i - kTileStages : 0; j < i; ++j)
          mbar_drain(&full[j % kTileStages], static_cast<uint32_t>((j / kTileStages) & 1));
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = mxf8_idesc(128, 128);
      for (int i = 0; i < nkb; ++i) {
        const int s = i % kTileStages;
        if (!mbar_wait(&full[s], static_cast<uint32_t>((i / kTileStages) & 1), &abort_flag)) break;
        tcgen05_fence_after();
        const uint32_t st = smem_u32(ring + s * kTileStageBytes);
        tcgen05_cp_scales<1>(t_sfa, scale_desc(st + 2 * kBoxBytes));
        tcgen05_cp_scales<1>(t_sfb, scale_desc(st + 2 * kBoxBytes + kSfBytes));
        const uint64_t da = kmajor_desc(st), db = kmajor_desc(st + kBoxBytes);
        const int steps = kb0 + i == p.k_blocks - 1 ? p.last_steps : 4;
        for (int k = 0; k < steps; ++k)
          mma_mxf8<1>(tmem, da + 2 * k, db + 2 * k, mxf8_idesc_step(idesc, k), t_sfa, t_sfb,
                      i + k > 0);
        tcgen05_commit<1>(&empty[s]);
      }
      tcgen05_commit<1>(&done);
      mbar_drain(&done, 0u, kWaitLimitNs);   // every MMA issued has finished
    }
  }
  __syncwarp();
  // All roles meet here; by now this CTA's MMAs and copies are finished.
  __syncthreads();
  tcgen05_fence_after();
  const bool ok = abort_flag == 0;
  float* part = reinterpret_cast<float*>(ring);
  if (warp >= 2) {
    const int row = (warp & 3) * 32 + lane;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      uint32_t v[32];
      tmem_ld_32(tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + c, v);
      tmem_ld_wait();
      float4* dst = reinterpret_cast<float4*>(part + row * kPitch + c);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        dst[j] = nkb > 0 ? make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                       __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]))
                         : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    tcgen05_fence_before();
  }
  if (p.split > 1)
    cluster_sync();
  else
    __syncthreads();
  // Rows of the tile that this CTA writes, summed over the cluster.
  const int rows = kTile / p.split;
  const int64_t m0 = static_cast<int64_t>(mt) * kTile + rank * rows;
  const int64_t n0 = static_cast<int64_t>(nt) * kTile;
  const bool vec = (p.N & 7) == 0;
  if (ok) {
    for (int i = threadIdx.x; i < rows * 16; i += kTileThreads) {
      const int r = i >> 4, c = (i & 15) * 8;
      const int64_t m = m0 + r, n = n0 + c;
      if (m >= p.M || n >= p.N) continue;
      float v[8] = {};
      const uint32_t at = smem_u32(part + (rank * rows + r) * kPitch + c);
      for (int q = 0; q < p.split; ++q) {
        const uint32_t a = p.split > 1 ? map_to_rank(at, static_cast<uint32_t>(q)) : at;
        const float4 lo = p.split > 1 ? ld_cluster_f4(a) : *reinterpret_cast<const float4*>(part + (rank * rows + r) * kPitch + c);
        const float4 hi = p.split > 1 ? ld_cluster_f4(a + 16) : *reinterpret_cast<const float4*>(part + (rank * rows + r) * kPitch + c + 4);
        v[0] += lo.x; v[1] += lo.y; v[2] += lo.z; v[3] += lo.w;
        v[4] += hi.x; v[5] += hi.y; v[6] += hi.z; v[7] += hi.w;
      }
      store_out8(p.out, p.out_f32, m * p.N + n, v, vec ? 8 : static_cast<int>(p.N - n < 8 ? p.N - n : 8), vec, p.sp_out);
    }
  }
  if (p.split > 1) cluster_sync();            // peers have read this CTA's partial tile
  else __syncthreads();
  if (warp == 1) tmem_dealloc<1>(tmem, 256);
  if (threadIdx.x == 0 && !ok) atomicOr(&g_matmul_watchdog, 1);
}

}  // namespace

int launch_matmul(const MatmulMaps& maps, int64_t M, int64_t N, int64_t K, void* out, bool out_f32,
                  int num_sms, cudaStream_t stream) {
  MatmulParams p = {};
  p.out = out;
  p.M = M;
  p.N = N;
  p.k_blocks = static_cast<int>((K + kBK - 1) / kBK);
  p.last_steps = static_cast<int>((K - static_cast<int64_t>(p.k_blocks - 1) * kBK) / 32);
  p.out_f32 = out_f32;
  p.sp_out = make_span(out, static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * (out_f32 ? 4 : 2));
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  p.m_tiles = static_cast<int>((M + kTile - 1) / kTile);
  p.n_tiles = static_cast<int>((N + kTile - 1) / kTile);
  const int64_t tiles = static_cast<int64_t>(p.m_tiles) * p.n_tiles;
  p.split = 1;
  while (p.split < 8 && tiles * p.split * 2 <= num_sms && p.split * 2 <= p.k_blocks) p.split *= 2;
  if (tiles * p.split > 0x7fffffff) return static_cast<int>(cudaErrorInvalidConfiguration);
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(
        tile_matmul_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem));
  });
  if (attr != 0) return attr;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles * p.split));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kTileSmem;
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
  return static_cast<int>(cudaLaunchKernelEx(&cfg, tile_matmul_kernel, maps, p));
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
