// mx_tensor.cuh -- inline-PTX building blocks of the tensor-core kernels:
// tensor memory, block-scaled MX products, clusters.
#pragma once

#include "mx_common.cuh"

namespace mx {

// One lane of a converged warp.  The compiler knows that the branch it guards
// runs in one thread and keeps the operands of the tensor instructions there in
// uniform registers; with `lane == 0` the MMA thread of mx_matmul.cu was bound
// by its own instructions (256 x 256 x 128 a 560 ns stage, 370 ns with this).
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// ---- clusters ----------------------------------------------------------------

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}

// Address in CTA `rank`'s shared memory of what `addr` is in this CTA's.
__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// Arrival on a barrier of another CTA of the cluster (`bar` from map_to_rank).  It
// orders tensor memory, with the tcgen05 fences around it, not shared memory of
// the cluster: no release at cluster scope, which waits for the thread's stores.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// Counts `bytes` that no copy will bring as if they had arrived.
__device__ __forceinline__ void mbar_complete_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// mbar_wait for a barrier on which another CTA of the cluster arrives.
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity,
                                                  volatile int* abort_flag) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait_cluster(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      return false;
    }
  }
}

__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// Tile load of a CTA pair: into this CTA's shared memory, completing on the
// barrier `bar` (a cluster address) of either CTA of the pair.
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* m, int32_t x,
                                                 int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}

// ---- tensor memory -------------------------------------------------------------

// A whole warp allocates / frees `cols` columns (a power of two, 32..512) of
// tensor memory in each CTA of the group; the kernels that use it take more
// than half of an SM's shared memory, so one CTA per SM holds any.
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* smem_dst, uint32_t cols) {
  if (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(smem_dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     smem_u32(smem_dst)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
}

template <int CG>
__device__ __forceinline__ void tmem_dealloc(uint32_t addr, uint32_t cols) {
  if (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}

__device__ __forceinline__ void tcgen05_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tcgen05_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 32 columns of this warp's 32 lanes: v[j] = column j of lane `lane`.
__device__ __forceinline__ void tmem_ld_32(uint32_t addr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_16(uint32_t addr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(addr)
      : "memory");
}

__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// ---- descriptors ---------------------------------------------------------------

// Shared-memory matrix descriptor of an operand box of 128 x 128 bytes: rows of
// 128 bytes, 128-byte swizzle, groups of eight rows 1024 bytes apart; the rows
// run along the operand's rows (K-major) or along the contraction (MN-major).
// `addr` is 1024-byte aligned; the k-th 32-step slice starts 32 k bytes later
// (K-major) or 32 k rows later (MN-major): kStepK and kStepMN in the
// descriptor's units of 16 bytes.
constexpr uint32_t kStepK = 32 >> 4, kStepMN = 32 * 128 >> 4;
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (uint64_t{1024 >> 4} << 32) |
         (uint64_t{1} << 46) | (uint64_t{2} << 61);
}

// ... of a 512-byte scale tile: 32 rows of 16 bytes, no swizzle, groups of
// eight rows 128 bytes apart.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (uint64_t{128 >> 4} << 32) |
         (uint64_t{1} << 46);
}

// Instruction descriptor of a kind::mxf8f6f4 product of shape m x n: both
// operands e4m3, each K-major or MN-major, scales ue8m0.
__device__ __forceinline__ uint32_t mxf8_idesc(int m, int n, bool a_mn, bool b_mn) {
  return (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n >> 3) << 17) |
         (1u << 23) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The same with byte `k` of each 32-bit scale word (the k-th of four 32-step
// slices) selected for both operands.
__device__ __forceinline__ uint32_t mxf8_idesc_step(uint32_t idesc, int k) {
  return idesc | (static_cast<uint32_t>(k) << 4) | (static_cast<uint32_t>(k) << 29);
}

// ... of a kind::mxf4 product: both operands e2m1, K-major, scales ue8m0.
__device__ __forceinline__ uint32_t mxf4_idesc(int m, int n) {
  return (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// ---- block-scaled products -------------------------------------------------------

// 512-byte scale tile -> four tensor-memory columns, repeated for the four
// groups of 32 lanes.  Ordered with the MMAs of the issuing thread.
template <int CG>
__device__ __forceinline__ void tcgen05_cp_scales(uint32_t taddr, uint64_t desc) {
  if (CG == 1)
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
                 : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_mxf8(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// The same for 4-bit operands: 64 contraction steps (32 bytes a row), two scales a row and
// 64 steps.
template <int CG>
__device__ __forceinline__ void mma_mxf4(uint32_t d, uint64_t da, uint64_t db, uint32_t idesc,
                                         uint32_t sfa, uint32_t sfb, bool accumulate) {
  const uint32_t acc = accumulate ? 1u : 0u;
  if (CG == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X "
        "[%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d),
        "l"(da), "l"(db), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// One arrival on `bar` once every tensor operation issued so far by this
// thread has finished; with CG == 2, on the barrier at this address in both
// CTAs of the pair.
template <int CG>
__device__ __forceinline__ void tcgen05_commit(uint64_t* bar) {
  if (CG == 1)
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                     smem_u32(bar))
                 : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// ---- output ------------------------------------------------------------------

// `n` (1..8) fp32 values to elements at.. of a bf16 or fp32 matrix; `vec`: the
// address is 16-byte aligned and n is 8.
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ void store_out8(void* out, int f32, int64_t at, const float (&v)[8],
                                           int n, bool vec, const Span& sp) {
  if (f32) {
    float* o = static_cast<float*>(out) + at;
    if (!in_span(sp, o, 4 * n)) return;
    if (vec) {
      reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
      reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) o[j] = v[j];
    }
  } else {
    uint16_t* o = static_cast<uint16_t*>(out) + at;
    if (!in_span(sp, o, 2 * n)) return;
    const uint32_t w[4] = {bf16x2(v[0], v[1]), bf16x2(v[2], v[3]), bf16x2(v[4], v[5]),
                           bf16x2(v[6], v[7])};
    if (vec) {
      *reinterpret_cast<uint4*>(o) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j < n) o[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
}

// A warp's box of 32 rows x 128 bytes of results (ITEM bytes each), in the swizzled
// order that a tensor map expects, to rows of N at (m, n) of `out`, whose rows no map
// can describe: a row at a time, in words where rows begin on a word.
template <int ITEM>
__device__ __forceinline__ void store_box(const uint8_t* box, void* out, int64_t m, int64_t n,
                                          int64_t M, int64_t N, int lane, const Span& sp) {
  const int rows = static_cast<int>(M - m < 32 ? M - m : 32);
  const int cols = static_cast<int>(N - n < 128 / ITEM ? N - n : 128 / ITEM);
  uint8_t* at = static_cast<uint8_t*>(out) + (m * N + n) * ITEM;
  const int64_t pitch = N * ITEM;
  if (ITEM == 4 || (N & 1) == 0) {
    constexpr int kPer = 4 / ITEM;
    const bool in = lane * kPer < cols;
#pragma unroll 8
    for (int r = 0; r < rows; ++r, at += pitch) {
      const uint32_t v = *reinterpret_cast<const uint32_t*>(box + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                                            (lane & 3) * 4);
      if (in && in_span(sp, at + 4 * lane, 4)) *reinterpret_cast<uint32_t*>(at + 4 * lane) = v;
    }
  } else {
#pragma unroll 4
    for (int r = 0; r < rows; ++r, at += pitch)
#pragma unroll
      for (int e = lane; e < 64; e += 32) {
        const uint16_t v = *reinterpret_cast<const uint16_t*>(box + r * 128 + (((e >> 3) ^ (r & 7)) << 4) +
                                                              (e & 7) * 2);
        if (e < cols && in_span(sp, at + 2 * e, 2)) *reinterpret_cast<uint16_t*>(at + 2 * e) = v;
      }
  }
}

}  // namespace mx
