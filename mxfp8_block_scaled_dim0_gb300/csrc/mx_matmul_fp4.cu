// mx_matmul_fp4.cu -- the product of two MX-FP4 operands (e2m1, blocks of 32, e8m0 scales):
// the kernels of mx_product.cuh with results in bf16 or fp32.  16640 x 8192 x 5120 to bf16 takes
// 199 us (7.0 PFLOP/s; repeated without a pause 214, at the power limit), bound by how long
// the operands' loads are under way (3.0 GB from L2, 15 TB/s, is not its bandwidth, but four and
// three stages of loads ahead instead of five take 216 and 257); 8192 x 5120 x 16640 to fp32
// 218; 1 x 8192 x 5120 7.1 (22 MB, 3.1 TB/s): a CTA on 128 of 152 SMs.
#include "mx_product.cuh"

namespace mx {

// The pair kernel's 256 rows cost a few tokens' product their loads (128 rows of zeros in
// either CTA): single tiles load only the rows that there are.  5120 4-bit steps, pairs and
// tiles: 1 x 16384 17.3 and 10.3 us, 1 x 65536 53.6 and 39.1; 64 x 16384 13.3 and 12.2, but
// 64 x 65536, more than a round of tiles, 37.7 and 46.8.
bool product_pairs(int64_t M, int64_t N, int num_sms) {
  if (!matmul_pairs(M, N, num_sms)) return false;
  return M > 128 || (M > 32 && (N + 127) / 128 > num_sms);
}

int launch_matmul_fp4(const ProductMaps& maps, int64_t M, int64_t N, int64_t K, void* out,
                      bool out_f32, int num_sms, cudaStream_t stream) {
  ProductParams p = product_params(M, N, K, true);
  p.out = out;
  p.out_f32 = out_f32;
  p.mapped = matmul_mapped(N, out_f32);
  p.sp_out = make_span(out, static_cast<uint64_t>(M) * static_cast<uint64_t>(N) * (out_f32 ? 4 : 2));
  // Longer fp32 sums go in runs.
  constexpr int kRun = kRunSteps / Shape<true>::kSteps;
  if (product_pairs(M, N, num_sms)) {
    p.m_tiles = static_cast<int>((M + 255) / 256);
    p.n_tiles = static_cast<int>((N + 255) / 256);
    if (!out_f32) return launch_pair_kernel<true, kPlain, false>(maps, p, num_sms, stream);
    const int runs = (p.k_blocks + kRun - 1) / kRun;
    p.run = (p.k_blocks + runs - 1) / runs;
    return launch_pair_kernel<true, kPlain, true>(maps, p, num_sms, stream);
  }
  const TileChoice t = choose_tiles(M, N, p.k_blocks, num_sms, 1);
  p.cols = t.cols;
  p.split = p.cluster = t.split;
  p.m_tiles = static_cast<int>((M + 127) / 128);
  p.n_tiles = static_cast<int>((N + t.cols - 1) / t.cols);
  p.load_bytes = (matmul_box_rows(M, false, 128) + matmul_box_rows(N, false, t.cols)) * kBoxCols +
                 2 * Shape<true>::kSf * kSfBytes;
  p.run = kRun;
  return out_f32 && (p.k_blocks + p.split - 1) / p.split > kRun
             ? launch_tile_kernel<true, kPlain, true>(maps, p, stream)
             : launch_tile_kernel<true, kPlain, false>(maps, p, stream);
}

int matmul_fp4_tile_cols(int64_t M, int64_t N, int64_t K, int num_sms) {
  return choose_tiles(M, N, (K + 255) / 256, num_sms, 1).cols;
}

int out_of_bounds_matmul_fp4(bool clear) { return read_out_of_bounds(clear); }
int read_matmul_fp4_watchdog(int* out, bool clear) { return read_product_word(out, clear); }

}  // namespace mx
