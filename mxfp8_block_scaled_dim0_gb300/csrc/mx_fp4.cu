// mx_fp4.cu -- MX-FP4 casts of bf16 matrices and the way back: e2m1 elements (0, 0.5, 1,
// 1.5, 2, 3, 4, 6 and a sign), two to a byte, the first in the low half, blocks of 32 with
// an e8m0 scale, scales in the 128x4 blocked layout.
//
//   E = biased exponent of the block's largest |x|;  s = max(E - 2, 0)
//   q = e2m1(x 2^(127 - s)), nearest even, saturated to +-6
//
// rows_kernel (dim0 of few rows): a thread takes eight values of a row, four threads share a block;
// nothing but the 16-byte loads and 4-byte stores of whole warps goes to memory.
// tile_kernel (one direction, or both in one read): 128 x 128 tiles by TMA into two stages,
// three CTAs an SM; blocks along columns are read from shared memory as pairs of columns
// (free of bank conflicts under the 128-byte swizzle), and their bytes leave through a
// staging tile by a TMA store.  A tile gives one 512-byte scale tile a direction.
// dequant_tile_kernel: 128 x 128 tiles too, in four stages and out through two staging tiles,
// two CTAs an SM; dequant_kernel: eight values a thread, four of these under way at once.
// All are bound by memory: 16640 x 5120 both directions 40.3 us (0.96 of the copy bandwidth),
// dim1 33.6 (0.95), dim0 33.5 (0.95), dequantisation 36.3 (0.88), 8192 x 5120 17.3 (0.90).
#include <cuda_runtime.h>

#include "mx_common.cuh"
#include "mx_kernels.h"
#include "mx_rows.cuh"

namespace mx {
namespace {

__device__ int g_fp4_watchdog = 0;

// ---- the rule ----------------------------------------------------------------------

// Scale byte and multiplier from a block's largest magnitude (bf16 bits): as mx_scale, with
// the exponent of e2m1's largest power of two.  Inf or NaN: byte 0xFF and a NaN multiplier,
// which the conversion below writes as 6.
__device__ __forceinline__ void mx4_scale(uint32_t amax_bits, uint32_t& sbyte, float& mult) {
  const int E = static_cast<int>(amax_bits >> 7);
  const int s = E > 2 ? E - 2 : 0;
  sbyte = E == 255 ? 0xFFu : static_cast<uint32_t>(s);
  mult = __uint_as_float(E == 255 ? 0x7FC00000u : static_cast<uint32_t>(254 - s) << 23);
}

// Eight floats -> eight e2m1 codes, the first in the lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}

// Eight bf16 values times m as codes.
__device__ __forceinline__ uint32_t cast8(const uint4& w, float m) {
  f32x2 v[4];
  get_pairs(w, v);
  const f32x2 m2 = pair(m, m);
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) unpair(mul2(v[j], m2), f[2 * j], f[2 * j + 1]);
  return e2m1x8(f);
}

__device__ __forceinline__ uint32_t amax8(const uint4& w) {
  const uint32_t m = absmax2(absmax2(w.x, w.y), absmax2(w.z, w.w));
  return max(mag_lo(m), mag_hi(m));
}

// ---- rows --------------------------------------------------------------------------

constexpr int kRowThreads = 256;
constexpr int kAtOnce = 4;                   // pieces of a warp under way

// A warp's pieces of 32 chunks of eight values: of one row, or of several short ones.  Walked
// in steps of the whole grid without a division.
struct Pieces {
  int cpr;             // chunks of a row
  int rows;            // rows of a piece
  int per_row;         // pieces of a row
  int64_t groups;      // pieces' rows
};

struct Walk {
  int64_t g, dg;
  int piece, dpiece, per_row;
  __device__ __forceinline__ Walk(const Pieces& p, int64_t warp, int64_t warps) : per_row(p.per_row) {
    g = warp / per_row;
    piece = static_cast<int>(warp - g * per_row);
    dg = warps / per_row;
    dpiece = static_cast<int>(warps - dg * per_row);
  }
  __device__ __forceinline__ void next() {
    g += dg;
    piece += dpiece;
    if (piece >= per_row) {
      piece -= per_row;
      ++g;
    }
  }
};

struct RowsParams {
  const uint16_t* x;
  uint8_t* q;
  uint8_t* s;
  int64_t M, K;
  Pieces pieces;
  int c, c4;           // scales of a row, and padded to four
  Span sp_q, sp_s;
};

__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowsParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kRowThreads;
  const int row_in = p.pieces.rows > 1 ? lane / p.pieces.cpr : 0;
  const int chunk_in = lane - row_in * p.pieces.cpr;
  Walk at(p.pieces, thread >> 5, threads >> 5);
  while (at.g < p.pieces.groups) {
    int64_t row[kAtOnce];
    int chunk[kAtOnce];
    uint4 w[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      row[k] = at.g * p.pieces.rows + row_in;
      chunk[k] = at.piece * 32 + chunk_in;
      const bool in = row_in < p.pieces.rows && row[k] < p.M && chunk[k] < p.pieces.cpr;
      if (!in) row[k] = -1;
      Piece<8> v;
      v.zero();
      if (in) v.load(p.x + row[k] * p.K + 8 * chunk[k]);
      w[k] = v.w;
      at.next();
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      uint32_t a = amax8(w[k]);
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
      a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
      uint32_t sbyte;
      float mult;
      mx4_scale(a, sbyte, mult);
      if (row[k] < 0) continue;
      uint8_t* q = p.q + (row[k] * p.K >> 1) + 4 * chunk[k];
      if (in_span(p.sp_q, q, 4)) *reinterpret_cast<uint32_t*>(q) = cast8(w[k], mult);
      if ((chunk[k] & 3) == 0) {
        uint8_t* s = p.s + blocked_offset(row[k], chunk[k] >> 2, p.c4);
        if (in_span(p.sp_s, s, 1)) *s = static_cast<uint8_t>(sbyte);
      }
    }
  }
  // The scales' padding: words of the rows behind the last, bytes behind the last column.
  const int64_t m4 = (p.M + 127) / 128 * 128, words = p.c4 / 4;
  for (int64_t i = thread; i < (m4 - p.M) * words; i += threads) {
    const int64_t r = i / words, c = i - r * words;
    uint8_t* s = p.s + blocked_offset(p.M + r, 4 * c, p.c4);
    if (in_span(p.sp_s, s, 4)) *reinterpret_cast<uint32_t*>(s) = 0;
  }
  if (p.c < p.c4)
    for (int64_t r = thread; r < p.M; r += threads)
      for (int c = p.c; c < p.c4; ++c) {
        uint8_t* s = p.s + blocked_offset(r, c, p.c4);
        if (in_span(p.sp_s, s, 1)) *s = 0;
      }
}

struct DequantParams {
  const uint8_t* q;
  const uint8_t* s;
  uint16_t* out;
  int64_t R, C;
  Pieces pieces;
  int c4;
  Span sp_out;
};

// Eight codes times 2^(s - 127) as bf16.  A code's three magnitude bits, at the top of an
// fp32's mantissa and the end of its exponent, are its value times 2^-126.  One rounding, at
// the end: the products with 2^126 and 2^(s - 127) are exact.
__device__ __forceinline__ uint4 dequant8(uint32_t codes, uint32_t sbyte) {
  const float m = scale_mult(sbyte);
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float v[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t code = codes >> (8 * j + 4 * k);
      const float f = __uint_as_float((code & 7u) << 22 | (code & 8u) << 28);
      v[k] = mul_rn(mul_rn(f, 0x1p126f), m);
    }
    o[j] = pack_bf16(v[0], v[1]);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

__global__ void __launch_bounds__(kRowThreads) dequant_kernel(const DequantParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int64_t thread = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kRowThreads;
  const int row_in = p.pieces.rows > 1 ? lane / p.pieces.cpr : 0;
  const int chunk_in = lane - row_in * p.pieces.cpr;
  Walk at(p.pieces, thread >> 5, threads >> 5);
  while (at.g < p.pieces.groups) {
    uint16_t* out[kAtOnce];
    uint32_t codes[kAtOnce], s[kAtOnce];
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k) {
      const int64_t row = at.g * p.pieces.rows + row_in;
      const int chunk = at.piece * 32 + chunk_in;
      const bool in = row_in < p.pieces.rows && row < p.R && chunk < p.pieces.cpr;
      out[k] = in ? p.out + row * p.C + 8 * chunk : nullptr;
      if (in) {
        codes[k] = __ldg(reinterpret_cast<const uint32_t*>(p.q + (row * p.C >> 1) + 4 * chunk));
        s[k] = __ldg(p.s + blocked_offset(row, chunk >> 2, p.c4));
      }
      at.next();
    }
#pragma unroll
    for (int k = 0; k < kAtOnce; ++k)
      if (out[k] && in_span(p.sp_out, out[k], 16))
        *reinterpret_cast<uint4*>(out[k]) = dequant8(codes[k], s[k]);
  }
}

// ---- dequantisation by tiles ---------------------------------------------------------

constexpr int kDqThreads = 256;
constexpr int kDqIn = 128 * 64;                  // 128 rows x 128 codes
constexpr int kDqScales = 512;
constexpr int kDqStage = 9 * 1024;               // codes and scales
constexpr int kDqStages = 4;
constexpr int kDqOut = 2 * 128 * 128;            // two boxes of 64 columns
constexpr int kDqCtas = 2;
constexpr int kDqSmem = kDqStages * kDqStage + 2 * kDqOut + 1024;

struct DqTileParams {
  const uint8_t* s;
  int64_t C, tiles_c, tiles;
  int64_t stall_at;
  uint64_t stall_ns;
};

__global__ void __launch_bounds__(kDqThreads, kDqCtas)
    dequant_tile_kernel(const __grid_constant__ DequantFp4Maps maps, const DqTileParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kDqStages], stall_bar;
  __shared__ int abort_flag;
  uint8_t* out = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* ring = out + 2 * kDqOut;
  const int tid = threadIdx.x;
  if (tid == 0) {
    for (int s = 0; s < kDqStages; ++s) mbar_init(&full[s], 1);
    mbar_init(&stall_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.q);
    prefetch_tmap(&maps.out);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  int64_t issued = 0;
  auto load = [&](int64_t i) {
    const int64_t t = blockIdx.x + i * gridDim.x;
    if (t >= p.tiles || i > issued) return;
    if (kDiagStall && blockIdx.x == 0 && i == p.stall_at) {
      mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
      return;
    }
    const int s = static_cast<int>(i % kDqStages);
    const int64_t tr = t / p.tiles_c, tc = t - tr * p.tiles_c;
    mbar_arrive_expect_tx(&full[s], kDqIn + kDqScales);
    tma_load_2d(ring + s * kDqStage, &maps.q, static_cast<int>(tc * 64), static_cast<int>(tr * 128),
                &full[s]);
    bulk_load(ring + s * kDqStage + kDqIn, p.s + t * kDqScales, kDqScales, &full[s]);
    ++issued;
  };
  if (tid == 0)
    for (int i = 0; i < kDqStages; ++i) load(i);
  int64_t i = 0;
  bool failed = false;
  for (int64_t t = blockIdx.x; t < p.tiles; t += gridDim.x, ++i) {
    const int s = static_cast<int>(i % kDqStages);
    const int64_t tr = t / p.tiles_c, tc = t - tr * p.tiles_c;
    const uint8_t* in = ring + s * kDqStage;
    const uint8_t* sf = in + kDqIn;
    uint8_t* o = out + (i & 1) * kDqOut;
    if (tid == 0) bulk_wait_read<1>();           // this half of the staging is free
    const bool ok = mbar_wait(&full[s], static_cast<uint32_t>((i / kDqStages) & 1), &abort_flag);
    if (__syncthreads_or(!ok)) {
      failed = true;
      break;
    }
    // Sixteen lanes a row, eight codes each.
    const int c = tid & 15;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = (tid >> 4) + 16 * k;
      const uint32_t codes = *reinterpret_cast<const uint32_t*>(in + r * 64 + c * 4);
      const uint4 v = dequant8(codes, sf[blocked_in_tile(r, c >> 2)]);
      *reinterpret_cast<uint4*>(o + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v;
    }
    fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      tma_store_2d(&maps.out, static_cast<int>(tc * 128), static_cast<int>(tr * 128), o);
      // A half wholly past the last column is not stored.
      if (tc * 128 + 64 < p.C)
        tma_store_2d(&maps.out, static_cast<int>(tc * 128 + 64), static_cast<int>(tr * 128), o + 16384);
      bulk_commit();
      load(i + kDqStages);
    }
  }
  if (tid == 0) {
    if (failed) {
      for (int64_t j = i; j < issued; ++j)
        mbar_drain(&full[j % kDqStages], static_cast<uint32_t>((j / kDqStages) & 1));
      atomicOr(&g_fp4_watchdog, 1);
    }
    bulk_wait<0>();
  }
}

int launch_dequant_tiles(const DequantFp4Maps& maps, const DqTileParams& p, int num_sms,
                         cudaStream_t stream) {
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(
        dequant_tile_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDqSmem));
  });
  if (attr != 0) return attr;
  const int64_t most = static_cast<int64_t>(num_sms) * kDqCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(p.tiles < most ? p.tiles : most));
  cfg.blockDim = dim3(kDqThreads);
  cfg.dynamicSmemBytes = kDqSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, dequant_tile_kernel, maps, p));
}

Pieces pieces_of(int64_t rows, int64_t cols) {
  Pieces p;
  p.cpr = static_cast<int>(cols / 8);
  p.rows = p.cpr < 32 ? 32 / p.cpr : 1;
  p.per_row = (p.cpr + 31) / 32;
  p.groups = (rows + p.rows - 1) / p.rows;
  return p;
}

template <typename P>
int launch_rows(void (*kernel)(P), const P& p, int64_t extra, int num_sms, cudaStream_t stream) {
  const int64_t warps = (p.pieces.groups * p.pieces.per_row + kAtOnce - 1) / kAtOnce;
  const int64_t tasks = warps * 32 > extra ? warps * 32 : extra;
  int64_t ctas = (tasks + kRowThreads - 1) / kRowThreads;
  // A CTA for every piece as long as there are SMs without one.
  const int64_t single = (p.pieces.groups * p.pieces.per_row * 32 + kRowThreads - 1) / kRowThreads;
  const int64_t few = single < num_sms ? single : num_sms;
  if (ctas < few) ctas = few;
  if (ctas > int64_t{8} * num_sms) ctas = int64_t{8} * num_sms;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(ctas));
  cfg.blockDim = dim3(kRowThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p));
}

// ---- tiles -------------------------------------------------------------------------

constexpr int kTile = 128;
constexpr int kHalfBytes = 64 * 2 * kTile;      // 64 columns of a tile
constexpr int kInBytes = 2 * kHalfBytes;
constexpr int kStages = 2;
constexpr int kQ1Bytes = kTile * kTile / 2;
constexpr int kSfTile = 512;
constexpr int kTileThreads = 256;
constexpr int kTileCtas = 3;                     // of an SM
constexpr int kTileSmem = kStages * kInBytes + kQ1Bytes + 2 * kSfTile + 1024;

struct TileParams {
  uint8_t* q0;
  uint8_t* s0;
  uint8_t* s1;
  int64_t M, K;
  int64_t tiles_m, tiles_k;
  Span sp_q0, sp_s0, sp_s1;
  int64_t stall_at;
  uint64_t stall_ns;
};

template <bool DIM0, bool DIM1>
__global__ void __launch_bounds__(kTileThreads, kTileCtas)
    tile_kernel(const __grid_constant__ CastFp4Maps maps, const TileParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kStages], stall_bar;
  __shared__ int abort_flag;
  uint8_t* ring = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  uint8_t* q1 = ring + kStages * kInBytes;
  uint8_t* sf0 = q1 + kQ1Bytes;
  uint8_t* sf1 = sf0 + kSfTile;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t tiles = p.tiles_m * p.tiles_k;
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    mbar_init(&stall_bar, 1);
    abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&maps.x);
    if (DIM1) prefetch_tmap(&maps.q1);
    // While earlier grids finish, ask L2 for the first tiles (a hint: nothing is read).
    for (int64_t i = 0; i < kStages; ++i) {
      const int64_t t = blockIdx.x + i * gridDim.x;
      if (t >= tiles) break;
      const int m = static_cast<int>(t / p.tiles_k * kTile), k = static_cast<int>(t % p.tiles_k * kTile);
      tma_prefetch_2d(&maps.x, k, m);
      tma_prefetch_2d(&maps.x, k + 64, m);
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __syncthreads();
  // Tile number `i` of this CTA into its stage.
  int64_t issued = 0;
  auto load = [&](int64_t i) {
    const int64_t t = blockIdx.x + i * gridDim.x;
    if (t >= tiles || i > issued) return;        // (none behind one that did not come)
    if (kDiagStall && blockIdx.x == 0 && i == p.stall_at) {
      mbar_wait(&stall_bar, 0u, &abort_flag, p.stall_ns);
      return;
    }
    const int s = static_cast<int>(i % kStages);
    const int m = static_cast<int>(t / p.tiles_k * kTile), k = static_cast<int>(t % p.tiles_k * kTile);
    mbar_arrive_expect_tx(&full[s], kInBytes);
    // A half wholly past the last column is zeros.
    tma_load_2d(ring + s * kInBytes, &maps.x, k, m, &full[s]);
    tma_load_2d(ring + s * kInBytes + kHalfBytes, &maps.x, k + 64, m, &full[s]);
    ++issued;
  };
  if (tid == 0)
    for (int i = 0; i < kStages; ++i) load(i);
  int64_t i = 0;
  bool failed = false;
  for (int64_t t = blockIdx.x; t < tiles; t += gridDim.x, ++i) {
    const int s = static_cast<int>(i % kStages);
    const int64_t tm = t / p.tiles_k, tk = t - tm * p.tiles_k;
    const uint8_t* in = ring + s * kInBytes;
    if (DIM1 && tid == 0) bulk_wait_read<0>();   // the staging tile is free
    const bool ok = mbar_wait(&full[s], static_cast<uint32_t>((i / kStages) & 1), &abort_flag);
    if (__syncthreads_or(!ok)) {
      failed = true;
      break;
    }
    if (DIM1) {
      // Blocks along columns: 32 rows of two columns a thread.
      const int b = warp >> 1, half = warp & 1;
      const uint8_t* src = in + half * kHalfBytes + b * 32 * 128 + (lane & 3) * 4;
      uint32_t w[32];
#pragma unroll
      for (int r = 0; r < 32; ++r)
        w[r] = *reinterpret_cast<const uint32_t*>(src + r * 128 + (((lane >> 2) ^ (r & 7)) << 4));
      uint32_t a = 0;
#pragma unroll
      for (int r = 0; r < 32; r += 4)
        a = absmax2(a, absmax2(absmax2(w[r], w[r + 1]), absmax2(w[r + 2], w[r + 3])));
      uint32_t s_lo, s_hi;
      float m_lo, m_hi;
      mx4_scale(mag_lo(a), s_lo, m_lo);
      mx4_scale(mag_hi(a), s_hi, m_hi);
      uint32_t lo[4], hi[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float f[8], g[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          f[k] = mul_rn(bf_lo(w[8 * j + k]), m_lo);
          g[k] = mul_rn(bf_hi(w[8 * j + k]), m_hi);
        }
        lo[j] = e2m1x8(f);
        hi[j] = e2m1x8(g);
      }
      // Rows 2 lane and 2 lane + 1 of this half, in the order of a 64-byte swizzle; every
      // other four lanes begin with the second, so that eight lanes fill 128 bytes.
      const int row = half * 64 + 2 * lane;
      uint8_t* dst = q1 + row * 64 + ((b ^ (lane & 3)) << 4);
      const uint4 first = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      const uint4 second = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      const bool swap = lane & 4;
      *reinterpret_cast<uint4*>(dst + (swap ? 64 : 0)) = swap ? second : first;
      *reinterpret_cast<uint4*>(dst + (swap ? 0 : 64)) = swap ? first : second;
      sf1[blocked_in_tile(row, b)] = static_cast<uint8_t>(s_lo);
      sf1[blocked_in_tile(row + 1, b)] = static_cast<uint8_t>(s_hi);
    }
    if (DIM0) {
      // Blocks along rows: half a block a thread, four rows a warp at a time.  The lanes of
      // the right half read their two chunks in the other order: no bank conflicts.
      const int half = (lane >> 2) & 1, piece = lane & 3;
      const int64_t col = tk * kTile + (lane & 7) * 16;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = warp * 16 + k * 4 + (lane >> 3);
        const uint8_t* src = in + half * kHalfBytes + r * 128;
        const uint4 a = *reinterpret_cast<const uint4*>(src + (((2 * piece + half) ^ (r & 7)) << 4));
        const uint4 c = *reinterpret_cast<const uint4*>(src + (((2 * piece + 1 - half) ^ (r & 7)) << 4));
        uint32_t m = max(amax8(a), amax8(c));
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        uint32_t sbyte;
        float mult;
        mx4_scale(m, sbyte, mult);
        const uint32_t x = cast8(a, mult), y = cast8(c, mult);
        if ((lane & 1) == 0) sf0[blocked_in_tile(r, (lane & 7) >> 1)] = static_cast<uint8_t>(sbyte);
        const int64_t row = tm * kTile + r;
        uint8_t* q = p.q0 + ((row * p.K + col) >> 1);
        if (row < p.M && col < p.K && in_span(p.sp_q0, q, 8))
          *reinterpret_cast<uint2*>(q) = half ? make_uint2(y, x) : make_uint2(x, y);
      }
    }
    if (DIM1) fence_proxy_async_smem();
    __syncthreads();
    if (tid == 0) {
      if (DIM1) {
        tma_store_2d(&maps.q1, static_cast<int>(tm * (kTile / 2)), static_cast<int>(tk * kTile), q1);
        bulk_commit();
      }
      load(i + kStages);
    } else if (DIM1 && tid >= 32 && tid < 64) {
      uint8_t* dst = p.s1 + (tk * p.tiles_m + tm) * kSfTile + lane * 16;
      if (in_span(p.sp_s1, dst, 16))
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(sf1 + lane * 16);
    } else if (DIM0 && tid >= 64 && tid < 96) {
      uint8_t* dst = p.s0 + (tm * p.tiles_k + tk) * kSfTile + lane * 16;
      if (in_span(p.sp_s0, dst, 16))
        *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(sf0 + lane * 16);
    }
  }
  if (tid == 0) {
    if (failed) {
      // The copies already issued land before the CTA ends.
      for (int64_t j = i; j < issued; ++j)
        mbar_drain(&full[j % kStages], static_cast<uint32_t>((j / kStages) & 1));
      atomicOr(&g_fp4_watchdog, 1);
    }
    if (DIM1) bulk_wait<0>();
  }
}

template <bool DIM0, bool DIM1>
int launch_tiles(const CastFp4Maps& maps, const TileParams& p, int num_sms, cudaStream_t stream) {
  static DeviceCache attr_cache;
  const int attr = attr_cache.get([] {
    return static_cast<int>(cudaFuncSetAttribute(
        tile_kernel<DIM0, DIM1>, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem));
  });
  if (attr != 0) return attr;
  const int64_t tiles = p.tiles_m * p.tiles_k, most = static_cast<int64_t>(num_sms) * kTileCtas;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles < most ? tiles : most));
  cfg.blockDim = dim3(kTileThreads);
  cfg.dynamicSmemBytes = kTileSmem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, tile_kernel<DIM0, DIM1>, maps, p));
}

}  // namespace

// Rows alone: tiles as soon as there is one for every SM (16640 x 5120 45.2 us in rows, 33.5 in
// tiles, 512 x 5120 4.0 and 3.2; 128 x 5120, 40 tiles, 1.9 and 2.0).
bool cast_fp4_tiles(int64_t M, int64_t K, int num_sms) {
  return (M + 127) / 128 * ((K + 127) / 128) >= num_sms;
}

// Tiles as soon as there is one for every SM and none is half empty (16640 x 5120 46.9 us in
// rows, 36.3 in tiles, 512 x 5120 3.9 and 3.6; 128 x 5120 1.8 and 2.9, 100000 x 64 5.5 and 6.2).
bool dequant_fp4_tiles(int64_t R, int64_t C, int num_sms) {
  return cast_fp4_tiles(R, C, num_sms) && C > 64;
}

int launch_cast_fp4(const CastFp4Maps* maps, const void* x, int64_t M, int64_t K, void* q0, void* s0,
                    void* s1, int num_sms, cudaStream_t stream) {
  const uint64_t values = static_cast<uint64_t>(M) * static_cast<uint64_t>(K);
  const int64_t m4 = (M + 127) / 128 * 128, k4 = (K + 127) / 128 * 128;
  const int64_t c = K / 32, c4 = (c + 3) / 4 * 4;
  if (!s1 && !cast_fp4_tiles(M, K, num_sms)) {
    RowsParams p = {static_cast<const uint16_t*>(x), static_cast<uint8_t*>(q0),
                    static_cast<uint8_t*>(s0), M, K, pieces_of(M, K), static_cast<int>(c),
                    static_cast<int>(c4), make_span(q0, values / 2),
                    make_span(s0, static_cast<uint64_t>(m4 * c4))};
    return launch_rows(rows_kernel, p, (m4 - M) * (c4 / 4), num_sms, stream);
  }
  TileParams p = {};
  p.q0 = static_cast<uint8_t*>(q0);
  p.s0 = static_cast<uint8_t*>(s0);
  p.s1 = static_cast<uint8_t*>(s1);
  p.M = M;
  p.K = K;
  p.tiles_m = m4 / 128;
  p.tiles_k = k4 / 128;
  p.sp_q0 = make_span(q0, values / 2);
  p.sp_s0 = make_span(s0, static_cast<uint64_t>(m4 * c4));
  p.sp_s1 = make_span(s1, static_cast<uint64_t>(k4 * ((M / 32 + 3) / 4 * 4)));
  const Stall stall = take_stall();
  p.stall_at = stall.at;
  p.stall_ns = stall.ns;
  if (!s1) return launch_tiles<true, false>(*maps, p, num_sms, stream);
  return q0 ? launch_tiles<true, true>(*maps, p, num_sms, stream)
            : launch_tiles<false, true>(*maps, p, num_sms, stream);
}

int launch_dequant_fp4(const DequantFp4Maps* maps, const void* q, int64_t R, int64_t C, const void* s_blk, void* out, int num_sms,
                       cudaStream_t stream) {
  if (dequant_fp4_tiles(R, C, num_sms)) {
    const int64_t tiles_c = (C + 127) / 128, tiles = (R + 127) / 128 * tiles_c;
    const Stall stall = take_stall();
    const DqTileParams t = {static_cast<const uint8_t*>(s_blk), C, tiles_c, tiles, stall.at, stall.ns};
    return launch_dequant_tiles(*maps, t, num_sms, stream);
  }
  DequantParams p = {static_cast<const uint8_t*>(q), static_cast<const uint8_t*>(s_blk),
                     static_cast<uint16_t*>(out), R, C, pieces_of(R, C),
                     static_cast<int>((C / 32 + 3) / 4 * 4),
                     make_span(out, 2 * static_cast<uint64_t>(R) * static_cast<uint64_t>(C))};
  return launch_rows(dequant_kernel, p, 0, num_sms, stream);
}

int out_of_bounds_fp4(bool clear) { return read_out_of_bounds(clear); }

int read_fp4_watchdog(int* out, bool clear) {
  int v = 0;
  cudaError_t e = cudaMemcpyFromSymbol(&v, g_fp4_watchdog, sizeof(int));
  if (e != cudaSuccess) return static_cast<int>(e);
  if (clear && v) {
    const int z = 0;
    e = cudaMemcpyToSymbol(g_fp4_watchdog, &z, sizeof(int));
    if (e != cudaSuccess) return static_cast<int>(e);
  }
  *out = v;
  return 0;
}

}  // namespace mx
