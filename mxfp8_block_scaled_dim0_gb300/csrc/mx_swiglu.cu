// mx_swiglu.cu -- gated SiLU of bf16 rows [gate | up], forward and backward,
// with its input saved as MX-FP8 for the backward pass.
//
//   h  = g sg u,  sg = 1 / (1 + exp(-g))
//   dg = dh u sg (1 + g (1 - sg)),  du = dh g sg
//
// A warp works on 32 pieces of a row's gate half and the same pieces of its up
// half (256 columns where the width is a multiple of 8).  Every byte is read
// and written once, which is what bounds the kernels: 16640 x 8192, forward 123 us
// (6.7 TB/s), with the save 171 us (6.4), backward from 8 bits 168.5 us (6.5), from
// bf16 206 us (6.6).  The exponential and the division go through the fast
// hardware functions, whose error (a few units of 2^-22) is far below the
// bf16 rounding of the results.
#include <cuda_runtime.h>

#include "mx_gate.cuh"
#include "mx_kernels.h"
#include "mx_rows.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;
// Tiles of an SM from which swiglu_tiles_kernel is taken: 16640 x 8192 (55 tiles an
// SM) 171 us against 185, 8192 x 4096 (13) 46.3 against 46.0, 4096^2 (7) 24.3
// against 19.1 with a row at a time.
constexpr int kManyTiles = 20;
constexpr int kOdd = 4;                // pieces of a lane, rows that are no multiple of 8

struct SwigluParams {
  const uint16_t* gu;
  const uint16_t* dh;
  uint16_t* out;        // h, or the gradient of gu
  uint8_t* q;
  uint8_t* s;
  int64_t M, rows;      // rows: M, or M padded to 128 where scales are written
  int F, runs;          // runs: warps' pieces of a row
  int s_cols4;          // scales of a row, padded to four
  Span sp_out, sp_q, sp_s;
};

// A warp's place: row r, piece `run` of the row, walked in steps of the whole
// grid without a division.  Rows in 32 bits (M < 2^31), so that an address is one
// wide multiplication.
struct Place {
  uint32_t r, dr;
  int run, drun, runs;
  __device__ __forceinline__ Place(uint32_t warp, uint32_t warps, int runs_) : runs(runs_) {
    r = warp / runs;
    run = static_cast<int>(warp - r * runs);
    dr = warps / runs;
    drun = static_cast<int>(warps - dr * runs);
  }
  __device__ __forceinline__ void next() {
    r += dr;
    run += drun;
    if (run >= runs) {
      run -= runs;
      ++r;
    }
  }
};

// blockIdx.x, read so that the compiler does not keep what it made of it the first time.
__device__ __forceinline__ uint32_t again() {
  uint32_t b;
  asm volatile("mov.u32 %0, %%ctaid.x;" : "=r"(b));
  return b;
}

__device__ __forceinline__ int64_t wide(uint32_t r, int n) {
  return static_cast<int64_t>(static_cast<uint64_t>(r) * static_cast<uint32_t>(n));
}

// Bytes of a row of scales: where row r of the blocked layout begins, and block
// `b` of a row.
__device__ __forceinline__ int64_t scale_row(uint32_t r, int cols4) {
  return wide(r >> 7, cols4 * 128) + (r & 31) * 16 + (r >> 5 & 3) * 4;
}
__device__ __forceinline__ int scale_block(int b) { return (b >> 2) * 512 + (b & 3); }

// Gate and up value e of row r.
template <bool SAVE>
__device__ __forceinline__ float2 gate_and_up(const SwigluParams& p, uint32_t r, int e) {
  auto value = [&](int at) {
    if constexpr (SAVE) {
      float lo, hi;
      e4m3x2_get(p.q[wide(r, 2 * p.F) + at], lo, hi);
      return lo * scale_mult(p.s[scale_row(r, p.s_cols4) + scale_block(at >> 5)]);
    } else {
      return __uint_as_float(static_cast<uint32_t>(p.gu[wide(r, 2 * p.F) + at]) << 16);
    }
  };
  return make_float2(value(e), value(e + p.F));
}

__device__ __forceinline__ uint16_t to_bf16(float v) {
  return static_cast<uint16_t>(pack_bf16(v, 0.0f));
}

// Low gates are worked on apart from the pieces, from their inputs in memory, a value
// at a time.
//
// Forward, at the kernel's end, by threads that have met one: in the loop even a
// branch that is not taken costs 1024 x 4096 0.4 of 3.8 us and 8000 x 8191 5 of 84.
// The n values from column c of row r:
__device__ __forceinline__ void low_gates(const SwigluParams& p, uint32_t r, int c, int n) {
#pragma unroll 1
  for (int k = c; k < c + n; ++k) {
    const float2 x = gate_and_up<false>(p, r, k);
    uint16_t* h = p.out + wide(r, p.F) + k;
    if (x.x < kLow && in_span(p.sp_out, h, 2)) *h = to_bf16(low_gated(x.x, x.y));
  }
}

__device__ __forceinline__ void low_gates8(const SwigluParams& p, uint32_t r, int c) {
  Piece<8> g;
  g.load(p.gu + wide(r, 2 * p.F) + c);
  if (any_low(lowest2(g.w))) low_gates(p, r, c, 8);
}

// In place of what the pieces' arithmetic made of them, before it is stored: forward by
// rows with the save, where the block's scale tells (4096 x 4096 19.8 us; at the end,
// which takes registers through the loop, 20.2, without low gates 19.1), ...
__device__ __forceinline__ void low_gates_in(const SwigluParams& p, uint32_t r, int c, uint4& h) {
  uint32_t w[4] = {h.x, h.y, h.z, h.w};
  uint16_t* v = reinterpret_cast<uint16_t*>(w);
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    const float2 x = gate_and_up<false>(p, r, c + k);
    if (x.x < kLow) v[k] = to_bf16(low_gated(x.x, x.y));
  }
  h = make_uint4(w[0], w[1], w[2], w[3]);
}

// ... and backward, whose result may lie where gu does.  (Both ways in registers: 57
// and not 48.)
template <bool SAVE>
__device__ __forceinline__ void low_gates_back(const SwigluParams& p, uint32_t r, int c, uint4& dg,
                                               uint4& du) {
  uint32_t w[8] = {dg.x, dg.y, dg.z, dg.w, du.x, du.y, du.z, du.w};
  uint16_t* v = reinterpret_cast<uint16_t*>(w);
#pragma unroll 1
  for (int k = 0; k < 8; ++k) {
    const float2 x = gate_and_up<SAVE>(p, r, c + k);
    if (!(x.x < kLow)) continue;
    float a, b;
    gated_back(__uint_as_float(static_cast<uint32_t>(p.dh[wide(r, p.F) + c + k]) << 16), x.x, x.y, a, b);
    v[k] = to_bf16(a);
    v[8 + k] = to_bf16(b);
  }
  dg = make_uint4(w[0], w[1], w[2], w[3]);
  du = make_uint4(w[4], w[5], w[6], w[7]);
}

// Rows whose halves are a multiple of 8 values: pieces of eight, as pairs.  The
// next piece's loads are issued before this one is worked on, without a condition
// (past the matrix its last row, past the row its first piece: not used), for
// loads under one are waited for where it ends.  16640 x 8192 with the save: 189 us
// with two pieces' loads and no prefetch, 182 us so, 215 us with two pieces of
// prefetch (98 registers).
template <bool SAVE>
__global__ void __launch_bounds__(kThreads, SAVE ? 0 : 6) swiglu_rows8_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  Place at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), p.runs);
  const uint32_t M = static_cast<uint32_t>(p.M);
  uint32_t lowest = 0;                         // of this thread's gates, without the save
  Piece<8> next_g, next_u;
  auto fetch = [&]() {
    const int c = (at.run * 32 + lane) * 8;
    const uint16_t* x = p.gu + wide(min(at.r, M - 1), 2 * p.F) + (c < p.F ? c : 0);
    next_g.load(x);
    next_u.load(x + p.F);
  };
  fetch();
  const uint32_t rows = static_cast<uint32_t>(p.rows);
  const bool whole = p.F % 128 == 0;           // the up half's scales begin a tile
  while (at.r < rows) {
    const uint32_t r = at.r;
    const int c = (at.run * 32 + lane) * 8;
    Piece<8> pg = next_g, pu = next_u;
    at.next();
    fetch();
    const bool live = r < M && c < p.F;
    bool low = false;
    f32x2 g[4], u[4];
    if constexpr (SAVE) {
      if (!live) {
        pg.zero();
        pu.zero();
      }
    }
    get_pairs(pg.w, g);
    get_pairs(pu.w, u);
    if constexpr (SAVE) {
      uint32_t sg, su;
      const uint2 qg = mx_cast_pairs(pg.w, g, sg);
      const uint2 qu = mx_cast_pairs(pu.w, u, su);
      low = may_be_low(sg);
      uint8_t* q = p.q + wide(r, 2 * p.F) + c;
      if (live && in_span(p.sp_q, q, 8) && in_span(p.sp_q, q + p.F, 8)) {
        *reinterpret_cast<uint2*>(q) = qg;
        *reinterpret_cast<uint2*>(q + p.F) = qu;
      }
      // One lane of a block's four writes its byte.  Rows past the matrix are zero
      // and give 0, the padding of the blocked layout.
      uint8_t* s = p.s + scale_row(r, p.s_cols4);
      if (c < p.F && (lane & 3) == 0) {
        uint8_t* a = s + scale_block(c >> 5);
        uint8_t* b = whole ? a + (p.F >> 7) * 512 : s + scale_block((c + p.F) >> 5);
        if (in_span(p.sp_s, a, 1)) *a = static_cast<uint8_t>(sg);
        if (in_span(p.sp_s, b, 1)) *b = static_cast<uint8_t>(su);
      }
      // Columns of scales past the row: zero.
      if (!whole && c == 0)
        for (int j = p.F / 16; j < p.s_cols4; ++j)
          if (in_span(p.sp_s, s + scale_block(j), 1)) s[scale_block(j)] = 0;
    }
    if (!live) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) g[j] = mul2(mul2(g[j], sigmoid2(g[j])), u[j]);
    if (!SAVE) lowest = __vmaxu2(lowest, lowest2(pg.w));
    uint16_t* h = p.out + wide(r, p.F) + c;
    uint4 w = pack_pairs(g);
    if (SAVE && low) low_gates_in(p, r, c, w);
    if (in_span(p.sp_out, h, 16)) *reinterpret_cast<uint4*>(h) = w;
  }
  if (!SAVE && any_low(lowest))
    for (at = Place(again() * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), p.runs);
         at.r < M; at.next()) {
      const int c = (at.run * 32 + lane) * 8;
      if (c < p.F) low_gates8(p, at.r, c);
    }
}

// The forward pass with the save on many rows whose halves are whole 128x4 scale
// tiles: a CTA works on 128 rows x 128 columns of either half at a time, gathers
// their 2 x 512 bytes of scales in shared memory and writes each tile at once.  (A
// row at a time leaves them in bytes all over the tiles, which cost 12 of 183 us
// at 16640 x 8192 though the bytes are 1 in 130.)  Loads ahead as above.
__global__ void __launch_bounds__(kThreads) swiglu_tiles_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ __align__(16) uint8_t scales[2][2][512];   // two tiles in turn, g and u
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kSteps = 128 / (kThreads / 16);         // 16 lanes a row
  const uint32_t M = static_cast<uint32_t>(p.M);
  // The place is a tile: r its 128 rows, run its 128 columns.
  Place at(blockIdx.x, gridDim.x, p.runs);
  uint32_t largest = 0;                        // scale of this thread's gates
  const uint32_t tiles = static_cast<uint32_t>(p.rows) >> 7;
  const int row0 = warp * 2 * kSteps + (lane >> 4), col = (lane & 15) * 8;
  Piece<8> next_g, next_u;
  auto fetch = [&](const Place& a, int step) {
    const uint16_t* x = p.gu + wide(min(a.r * 128 + row0 + 2 * step, M - 1), 2 * p.F) + a.run * 128 + col;
    next_g.load(x);
    next_u.load(x + p.F);
  };
  if (at.r < tiles) fetch(at, 0);
  for (int turn = 0; at.r < tiles; turn ^= 1) {
    const Place here = at;
    at.next();
#pragma unroll 1
    for (int step = 0; step < kSteps; ++step) {
      Piece<8> pg = next_g, pu = next_u;
      const bool more = step + 1 < kSteps;
      fetch(more || at.r >= tiles ? here : at, more ? step + 1 : 0);
      const int row = row0 + 2 * step;
      const uint32_t r = here.r * 128 + row;
      const bool live = r < M;
      if (!live) {
        pg.zero();
        pu.zero();
      }
      f32x2 g[4], u[4];
      get_pairs(pg.w, g);
      get_pairs(pu.w, u);
      uint32_t sg, su;
      const uint2 qg = mx_cast_pairs(pg.w, g, sg);
      const uint2 qu = mx_cast_pairs(pu.w, u, su);
      if ((lane & 3) == 0) {
        const int k = blocked_in_tile(row, (lane & 15) >> 2);
        scales[turn][0][k] = static_cast<uint8_t>(sg);
        scales[turn][1][k] = static_cast<uint8_t>(su);
      }
      if (!live) continue;
      const int c = here.run * 128 + col;
      uint8_t* q = p.q + wide(r, 2 * p.F) + c;
      if (in_span(p.sp_q, q, 8) && in_span(p.sp_q, q + p.F, 8)) {
        *reinterpret_cast<uint2*>(q) = qg;
        *reinterpret_cast<uint2*>(q + p.F) = qu;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) g[j] = mul2(mul2(g[j], sigmoid2(g[j])), u[j]);
      largest = max(largest, sg);
      uint16_t* h = p.out + wide(r, p.F) + c;
      if (in_span(p.sp_out, h, 16)) *reinterpret_cast<uint4*>(h) = pack_pairs(g);
    }
    // One barrier a tile: these bytes are written again two tiles on.
    __syncthreads();
    if (threadIdx.x < 64) {
      const int half = threadIdx.x >> 5;
      uint8_t* s = p.s + wide(here.r, p.s_cols4 * 128) + (here.run + half * (p.F >> 7)) * 512 + lane * 16;
      if (in_span(p.sp_s, s, 16))
        *reinterpret_cast<uint4*>(s) = *reinterpret_cast<const uint4*>(&scales[turn][half][lane * 16]);
    }
  }
  if (may_be_low(largest))
    for (at = Place(again(), gridDim.x, p.runs); at.r < tiles; at.next())
#pragma unroll 1
      for (int step = 0; step < kSteps; ++step) {
        const uint32_t r = at.r * 128 + row0 + 2 * step;
        if (r < M) low_gates8(p, r, at.run * 128 + col);
      }
}

// Loads ahead as in swiglu_rows8_kernel.
template <bool SAVE>
__global__ void __launch_bounds__(kThreads) swiglu_back_rows8_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  Place at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), p.runs);
  const uint32_t M = static_cast<uint32_t>(p.M);
  const f32x2 one = pair(1.0f, 1.0f), minus = pair(-1.0f, -1.0f);
  Piece<8> next_d, next_g, next_u;
  uint2 next_qg, next_qu;
  uint32_t next_sg, next_su;
  auto fetch = [&]() {
    const uint32_t r = min(at.r, M - 1);
    int c = (at.run * 32 + lane) * 8;
    c = c < p.F ? c : 0;
    next_d.load(p.dh + wide(r, p.F) + c);
    if constexpr (SAVE) {
      const uint8_t* q = p.q + wide(r, 2 * p.F) + c;
      next_qg = ld_q8(q);
      next_qu = ld_q8(q + p.F);
      const uint8_t* s = p.s + scale_row(r, p.s_cols4);
      asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(next_sg) : "l"(s + scale_block(c >> 5)));
      asm volatile("ld.global.nc.u8 %0, [%1];" : "=r"(next_su) : "l"(s + scale_block((c + p.F) >> 5)));
    } else {
      const uint16_t* x = p.gu + wide(r, 2 * p.F) + c;
      next_g.load(x);
      next_u.load(x + p.F);
    }
  };
  fetch();
  while (at.r < M) {
    const uint32_t r = at.r;
    const int c = (at.run * 32 + lane) * 8;
    f32x2 d[4], g[4], u[4];
    get_pairs(next_d.w, d);
    const bool low = SAVE ? may_be_low(next_sg) : any_low(lowest2(next_g.w));
    if constexpr (SAVE) {
      mx_get_pairs(next_qg, next_sg, g);
      mx_get_pairs(next_qu, next_su, u);
    } else {
      get_pairs(next_g.w, g);
      get_pairs(next_u.w, u);
    }
    at.next();
    fetch();
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 s = sigmoid2(g[j]);
      const f32x2 a = mul2(g[j], s);
      const f32x2 t = fma2(a, fma2(s, minus, one), s);    // s (1 + g (1 - s))
      u[j] = mul2(mul2(d[j], u[j]), t);
      g[j] = mul2(d[j], a);
    }
    if (c >= p.F) continue;
    uint4 dg = pack_pairs(u), du = pack_pairs(g);
    if (low) low_gates_back<SAVE>(p, r, c, dg, du);
    uint16_t* o = p.out + wide(r, 2 * p.F) + c;
    if (in_span(p.sp_out, o, 16) && in_span(p.sp_out, o + p.F, 16)) {
      *reinterpret_cast<uint4*>(o) = dg;
      *reinterpret_cast<uint4*>(o + p.F) = du;
    }
  }
}

// Other widths, in pieces of two values or one.
template <int VEC>
__global__ void __launch_bounds__(kThreads) swiglu_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  Place at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), p.runs);
  const uint32_t M = static_cast<uint32_t>(p.M);
  float lowest = 0.0f;                         // of this thread's gates
  for (; at.r < M; at.next()) {
    const uint16_t* x = p.gu + wide(at.r, 2 * p.F);
    uint16_t* out = p.out + wide(at.r, p.F);
    Piece<VEC> pg[kOdd], pu[kOdd];
    const int c0 = (at.run * 32 * kOdd + lane) * VEC;
#pragma unroll
    for (int i = 0; i < kOdd; ++i) {
      const int c = c0 + i * 32 * VEC;
      if (c >= p.F) continue;
      pg[i].load(x + c);
      pu[i].load(x + p.F + c);
    }
#pragma unroll
    for (int i = 0; i < kOdd; ++i) {
      const int c = c0 + i * 32 * VEC;
      if (c >= p.F) continue;
      float g[VEC], u[VEC], h[VEC];
      pg[i].get(g);
      pu[i].get(u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) h[j] = g[j] * sigmoid(g[j]) * u[j];
      lowest = fminf(fminf(lowest, g[0]), g[VEC - 1]);
      store_bf16<VEC>(out + c, h, p.sp_out);
    }
  }
  if (lowest < kLow)
    for (at = Place(again() * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), p.runs);
         at.r < M; at.next())
#pragma unroll 1
      for (int i = 0; i < kOdd; ++i) {
        const int c = (at.run * 32 * kOdd + lane + i * 32) * VEC;
        if (c < p.F) low_gates(p, at.r, c, VEC);
      }
}

template <int VEC>
__global__ void __launch_bounds__(kThreads) swiglu_back_kernel(const SwigluParams p) {
  asm volatile("griddepcontrol.launch_dependents;");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  Place at(blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5), gridDim.x * (kThreads / 32), p.runs);
  const uint32_t M = static_cast<uint32_t>(p.M);
  for (; at.r < M; at.next()) {
    const uint16_t* x = p.gu + wide(at.r, 2 * p.F);
    const uint16_t* dh = p.dh + wide(at.r, p.F);
    uint16_t* out = p.out + wide(at.r, 2 * p.F);
    Piece<VEC> pd[kOdd], pg[kOdd], pu[kOdd];
    const int c0 = (at.run * 32 * kOdd + lane) * VEC;
#pragma unroll
    for (int i = 0; i < kOdd; ++i) {
      const int c = c0 + i * 32 * VEC;
      if (c >= p.F) continue;
      pd[i].load(dh + c);
      pg[i].load(x + c);
      pu[i].load(x + p.F + c);
    }
#pragma unroll
    for (int i = 0; i < kOdd; ++i) {
      const int c = c0 + i * 32 * VEC;
      if (c >= p.F) continue;
      float g[VEC], u[VEC], d[VEC], dg[VEC], du[VEC];
      pd[i].get(d);
      pg[i].get(g);
      pu[i].get(u);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float s = sigmoid(g[j]);
        const float a = g[j] * s;
        du[j] = d[j] * a;
        dg[j] = d[j] * u[j] * (s + a * (1.0f - s));
      }
      if (fminf(g[0], g[VEC - 1]) < kLow)
#pragma unroll
        for (int j = 0; j < VEC; ++j) gated_back(d[j], g[j], u[j], dg[j], du[j]);
      store_bf16<VEC>(out + c, dg, p.sp_out);
      store_bf16<VEC>(out + p.F + c, du, p.sp_out);
    }
  }
}

// `tasks`: warps' pieces of work.
template <typename K>
int run(K kernel, const SwigluParams& p, int64_t tasks, int num_sms, cudaStream_t stream) {
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, kThreads, 0) != cudaSuccess ||
      per < 1)
    per = 1;
  const int64_t want = (tasks + kThreads / 32 - 1) / (kThreads / 32);
  const int64_t most = static_cast<int64_t>(num_sms) * per;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, kernel, p));
}

SwigluParams params(const SwigluArgs& a, int vec, bool padded) {
  SwigluParams p = {};
  p.gu = static_cast<const uint16_t*>(a.gu);
  p.dh = static_cast<const uint16_t*>(a.dh);
  p.out = static_cast<uint16_t*>(a.out);
  p.q = static_cast<uint8_t*>(a.q);
  p.s = static_cast<uint8_t*>(a.s);
  p.M = a.M;
  p.rows = padded ? (a.M + 127) / 128 * 128 : a.M;
  p.F = static_cast<int>(a.F);
  const int64_t run = vec == 8 ? 256 : 32 * kOdd * vec;
  p.runs = static_cast<int>((a.F + run - 1) / run);
  p.s_cols4 = static_cast<int>((a.F / 16 + 3) / 4 * 4);
  const uint64_t n = static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.F);
  p.sp_out = make_span(a.out, a.dh ? 4 * n : 2 * n);
  p.sp_q = make_span(a.q, 2 * n);
  p.sp_s = make_span(a.s, static_cast<uint64_t>((a.M + 127) / 128 * 128) * p.s_cols4);
  return p;
}

int vec_of(int64_t F) { return F % 8 == 0 ? 8 : F % 2 == 0 ? 2 : 1; }

}  // namespace

int launch_swiglu(const SwigluArgs& a, int num_sms, cudaStream_t stream) {
  const int v = vec_of(a.F);
  SwigluParams p = params(a, v, a.q != nullptr);
  if (a.q && a.F % 128 == 0 && p.rows / 128 * (a.F / 128) >= kManyTiles * num_sms) {
    p.runs = static_cast<int>(a.F / 128);
    return run(swiglu_tiles_kernel, p, p.rows / 128 * p.runs * (kThreads / 32), num_sms, stream);
  }
  if (a.q) return run(swiglu_rows8_kernel<true>, p, p.rows * p.runs, num_sms, stream);
  if (v == 8) return run(swiglu_rows8_kernel<false>, p, p.rows * p.runs, num_sms, stream);
  if (v == 2) return run(swiglu_kernel<2>, p, p.rows * p.runs, num_sms, stream);
  return run(swiglu_kernel<1>, p, p.rows * p.runs, num_sms, stream);
}

int launch_swiglu_backward(const SwigluArgs& a, int num_sms, cudaStream_t stream) {
  const int v = vec_of(a.F);
  const SwigluParams p = params(a, v, false);
  if (a.q) return run(swiglu_back_rows8_kernel<true>, p, p.rows * p.runs, num_sms, stream);
  if (v == 8) return run(swiglu_back_rows8_kernel<false>, p, p.rows * p.runs, num_sms, stream);
  if (v == 2) return run(swiglu_back_kernel<2>, p, p.rows * p.runs, num_sms, stream);
  return run(swiglu_back_kernel<1>, p, p.rows * p.runs, num_sms, stream);
}

int out_of_bounds_swiglu(bool clear) { return read_out_of_bounds(clear); }

}  // namespace mx
