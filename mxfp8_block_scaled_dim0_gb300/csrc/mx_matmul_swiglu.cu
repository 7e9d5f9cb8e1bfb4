// mx_matmul_swiglu.cu -- products of MX operands joined with the gated SiLU: the two
// projections, the activation and their product of a gated feed-forward layer in one kernel,
// and the gradient of the projections' results from that of the layer's output.
//
// The kernels are those of mx_product.cuh, for operands of 8 and of 4 bits.  Gate and up in one
// launch read X once and store neither; 16640 x 8192 x 5120 e4m3 with the save takes 820 us
// (the product of that size alone, to bf16, 769; its gated SiLU with the save 171), the
// backward 470 (product 390, gated SiLU backward 169).  Those are a few calls after a pause:
// repeated without one, the power limit makes them 950 and 525.  The tensor cores are the bound
// (busy in 68% of all cycles at 4096 x 4096 x 4096 with the save), the backward shares the
// memory with 817 MB of saved values and results.  In e2m1 the epilogue outlasts short
// contractions: 367 us without the save, 440 with it, 280 backward, and 76, 114 at 13766 x 5344
// x 1088.  One token, 1 x 8192 x 5120: e2m1 10.6 us for 45 MB of weights, e4m3 16.9 for 87.
#include "mx_product.cuh"

namespace mx {
namespace {

template <bool FP4>
int launch_forward(const ProductMaps& maps, ProductParams& p, int num_sms,
                   cudaStream_t stream) {
  // Saved sums go in runs.
  constexpr int kRun = kSavedRunSteps<FP4> / Shape<FP4>::kSteps;
  if (product_pairs(p.M, 2 * p.N, num_sms)) {
    p.m_tiles = static_cast<int>((p.M + 255) / 256);
    p.n_tiles = static_cast<int>((p.N + 127) / 128);
    if (p.q) {
      const int runs = (p.k_blocks + kRun - 1) / kRun;
      p.run = (p.k_blocks + runs - 1) / runs;
    }
    return p.q ? launch_pair_kernel<FP4, kSwiglu, true>(maps, p, num_sms, stream)
               : launch_pair_kernel<FP4, kSwiglu, false>(maps, p, num_sms, stream);
  }
  const TileChoice t = choose_tiles(p.M, p.N, p.k_blocks, num_sms, 2);
  p.cols = t.cols;
  p.split = t.split;
  p.cluster = 2 * t.split;
  p.m_tiles = static_cast<int>((p.M + 127) / 128);
  p.n_tiles = static_cast<int>((p.N + t.cols - 1) / t.cols);
  p.load_bytes = (matmul_box_rows(p.M, false, 128) + matmul_box_rows(p.N, false, t.cols)) * kBoxCols +
                 2 * Shape<FP4>::kSf * kSfBytes;
  p.run = kRun;
  return p.q && (p.k_blocks + p.split - 1) / p.split > kRun
             ? launch_tile_kernel<FP4, kSwiglu, true>(maps, p, stream)
             : launch_tile_kernel<FP4, kSwiglu, false>(maps, p, stream);
}

template <bool FP4>
int launch_backward(const ProductMaps& maps, ProductParams& p, int num_sms, cudaStream_t stream) {
  if (product_pairs(p.M, p.N, num_sms)) {
    p.m_tiles = static_cast<int>((p.M + 255) / 256);
    p.n_tiles = static_cast<int>((p.N + 255) / 256);
    return p.q ? launch_pair_kernel<FP4, kSwigluBack, true>(maps, p, num_sms, stream)
               : launch_pair_kernel<FP4, kSwigluBack, false>(maps, p, num_sms, stream);
  }
  const TileChoice t = choose_tiles(p.M, p.N, p.k_blocks, num_sms, 1);
  p.cols = t.cols;
  p.split = p.cluster = t.split;
  p.m_tiles = static_cast<int>((p.M + 127) / 128);
  p.n_tiles = static_cast<int>((p.N + t.cols - 1) / t.cols);
  p.load_bytes = (matmul_box_rows(p.M, false, 128) + matmul_box_rows(p.N, false, t.cols)) * kBoxCols +
                 2 * Shape<FP4>::kSf * kSfBytes;
  return launch_tile_kernel<FP4, kSwigluBack, false>(maps, p, stream);
}

ProductParams params_of(const MatmulSwigluArgs& a) {
  ProductParams p = product_params(a.M, a.F, a.K, a.fp4);
  const uint64_t values = static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.F);
  p.out = a.out;
  p.q = static_cast<uint8_t*>(a.q);
  p.s = static_cast<uint8_t*>(a.s);
  p.gu = static_cast<const uint16_t*>(a.gu);
  p.s_cols4 = (2 * a.F / 32 + 3) / 4 * 4;
  p.sp_q = make_span(a.q, 2 * values);
  p.sp_s = make_span(a.s, static_cast<uint64_t>((a.M + 127) / 128 * 128 * p.s_cols4));
  return p;
}

}  // namespace

int matmul_swiglu_tile_cols(int64_t M, int64_t F, int64_t K, bool fp4, bool backward, int num_sms) {
  return choose_tiles(M, F, (K + (fp4 ? 255 : 127)) / (fp4 ? 256 : 128), num_sms, backward ? 1 : 2).cols;
}

int launch_matmul_swiglu(const ProductMaps& maps, const MatmulSwigluArgs& a, int num_sms,
                         cudaStream_t stream) {
  ProductParams p = params_of(a);
  p.sp_out = make_span(a.out, static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.F) * 2);
  return a.fp4 ? launch_forward<true>(maps, p, num_sms, stream)
               : launch_forward<false>(maps, p, num_sms, stream);
}

int launch_matmul_swiglu_backward(const ProductMaps& maps, const MatmulSwigluArgs& a, int num_sms,
                                  cudaStream_t stream) {
  ProductParams p = params_of(a);
  p.sp_out = make_span(a.out, static_cast<uint64_t>(a.M) * static_cast<uint64_t>(a.F) * 4);
  return a.fp4 ? launch_backward<true>(maps, p, num_sms, stream)
               : launch_backward<false>(maps, p, num_sms, stream);
}

int out_of_bounds_matmul_swiglu(bool clear) { return read_out_of_bounds(clear); }
int read_matmul_swiglu_watchdog(int* out, bool clear) { return read_product_word(out, clear); }

}  // namespace mx
