/*
 * mxfp8_cast.h -- C ABI of libmxfp8_cast.so: MX-FP8 (e4m3 elements, e8m0
 * block scales, blocks of 32) and MX-FP4 (e2m1 elements) quantisation of bf16
 * matrices on sm_103a, and the operators that work on such values: products of two
 * MX operands, alone or joined with the gated SiLU, layer norm and gated SiLU whose
 * inputs are saved for the backward pass in MX-FP8.
 *
 * Conventions for every entry point below
 *   - All data pointers are DEVICE pointers of the calling thread's current
 *     CUDA device (or managed memory), allocated and owned by the caller; the
 *     library allocates no device memory and keeps no pointer after the call
 *     returns.  Each pointer's memory type and device are checked on the
 *     host (MX_ERR_DEVICE), so a host pointer or another device's pointer is
 *     refused before any kernel sees it.  `stream` must belong to the same
 *     device.
 *   - Every pointer must be 16-byte aligned (int32 / int64 offset arrays:
 *     4- / 8-byte aligned), tensors are dense row-major with no padding.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Work is
 *     enqueued asynchronously; no call synchronises the device or reads
 *     device memory on the host.  Results are valid once the stream has
 *     executed the work.
 *   - Return value: MX_OK, or a negative MX_ERR_* code.  Argument errors are
 *     detected on the host before anything is enqueued (outputs untouched).
 *     MX_ERR_CUDA means a CUDA call failed; mx_last_cuda_error() has its code.
 *   - Calls that share an output buffer and run concurrently on the GPU race.
 *     Inputs and outputs of one call must not overlap.
 *   - Entry points may be called from several host threads at once: the only
 *     host state is a per-thread cache of TMA descriptors and per-device
 *     launch attributes set once.
 *
 * The rule, per 32-element block (OCP Microscaling Formats v1.0 conversion
 * with E4M3 elements and an E8M0 scale):
 *   amax  = max |x_i|
 *   scale byte s = clamp(floor(log2 amax) - 8, -127, 127) + 127; amax = 0
 *                  gives s = 0; a block holding Inf or NaN gives s = 0xFF
 *   q_i   = e4m3(x_i * 2^(127 - s)), round to nearest even, saturated to
 *           +-448 (e4m3 NaN for every element of an Inf/NaN block)
 * Directions (pytorch/ao PR #1869 "triton kernel to cast to mx across dim0
 * and dim1", summary):
 *   dim0: blocks along each row of X (M x K)    -> q0 (M x K) bytes
 *   dim1: blocks along each column of X         -> q1 (K x M) bytes, the
 *         row-major copy of X^T (X's column-major copy); q1[k][m] encodes
 *         X[m][k]
 * Blocked scale layout (the 128x4 layout of block-scaled GEMM scale factors;
 * 128x4 is the granularity named in pytorch/ao PR #3416 "[mxfp8 moe training]
 * parallelize along col blocks in scale blocked format kernel for groups
 * along K"): a scale matrix S (R x C) is padded with zeros to
 * ceil(R/128)*128 x ceil(C/4)*4, cut into 128x4 tiles stored one after
 * another in row-major tile order (512 bytes each), and S[r][c] sits at byte
 * (r%32)*16 + ((r%128)/32)*4 + c%4 of its tile.  Its size is
 * mx_blocked_bytes(R, C).
 */
#ifndef MXFP8_CAST_H
#define MXFP8_CAST_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  MX_OK = 0,
  MX_ERR_NULL = -1,    /* a required pointer is NULL */
  MX_ERR_SHAPE = -2,   /* a size is zero, negative, too large or not a multiple of 32 */
  MX_ERR_ALIGN = -3,   /* a pointer is not suitably aligned */
  MX_ERR_CUDA = -4,    /* a CUDA call failed (see mx_last_cuda_error) */
  MX_ERR_GROUPS = -5,  /* invalid group count, or (device status) invalid offsets */
  MX_ERR_DEVICE = -6,  /* a pointer is not device memory of the current device */
  MX_ERR_TYPE = -7     /* a type or order argument has none of its values */
};

/* Element types of arguments that may have either. */
enum {
  MX_BF16 = 0,
  MX_F32 = 1
};

/* Element formats of operands that may have either: e4m3, a byte an element, or e2m1,
 * two to a byte. */
enum {
  MX_E4M3 = 0,
  MX_E2M1 = 1
};

/* Storage orders of mx_matmul's operands. */
enum {
  MX_A_BY_COLUMN = 1,  /* qa is stored K x M */
  MX_B_BY_COLUMN = 2   /* qb is stored K x N */
};

/* Fused dim0 + dim1 cast with both scale sets in blocked layout; one read of
 * X.  Defined by pytorch/ao PR #1869 "triton kernel to cast to mx across dim0
 * and dim1" (summary: read 32x32 tiles once, write the row-major and
 * column-major casts and their scales from each tile; future work: outer
 * tile 128, swizzled scales, coalesced writes).
 *   x       bf16 (M x K), row-major                      [in]
 *   M, K    M % 32 == 0, K % 32 == 0, 32 <= M, K <= 2^31 - 256
 *   q0      M x K bytes, e4m3, dim0                      [out]
 *   s0_blk  mx_blocked_bytes(M, K/32) bytes, e8m0        [out]
 *   q1      K x M bytes, e4m3, dim1                      [out]
 *   s1_blk  mx_blocked_bytes(K, M/32) bytes, e8m0        [out]
 * Padding bytes of the blocked buffers are written as zero. */
int mx_cast_dim0_dim1(const void* x, int64_t M, int64_t K, void* q0, void* s0_blk, void* q1,
                      void* s1_blk, void* stream);

/* mx_cast_dim0_dim1 for callers that must not allocate device memory, with
 * its one piece of scratch in device memory reserved when the library is
 * loaded.  The pages have no counterpart: this is an entry point of this
 * library only.
 *
 * Who needs it: a process whose device memory is handed out by a caching
 * allocator that reserved it up front (a training or serving framework),
 * where an allocation from outside the pool can fail for lack of memory or
 * fragment it; and code that must not risk the device-wide synchronisation
 * an allocation can bring.  None of the entry points here allocate; this one
 * also keeps no per-stream state on the host: its scratch is one fixed
 * array instead of mx_cast_dim0_dim1's counter per stream.
 *
 * Arguments, layouts, output and errors as mx_cast_dim0_dim1, byte for byte.
 * The scratch is 256 bytes (64 words) of device memory, held by every GPU
 * that loads the library until the process exits; a call needs one word
 * (its tile-claim counter, for launches of 32 rounds of tiles or more), and
 * a call that would need more than 64 words is refused with MX_ERR_SHAPE.
 * The first call on a device looks up the array's device address (with that
 * device current); make that first call before any stream capture.  Each call
 * clears the word it uses on the stream before its kernel.  All calls share
 * the array: calls whose kernels overlap on the GPU (different streams, no
 * ordering between them) race on it and give wrong output; order them on one
 * stream or with events. */
int mx_cast_dim0_dim1_noalloc(const void* x, int64_t M, int64_t K, void* q0, void* s0_blk,
                              void* q1, void* s1_blk, void* stream);

/* dim1 cast only (the column-major copy and its blocked scales), as split out
 * of the fused kernel in the same pull request's follow-up (dim1 logic in its
 * own kernel).  Arguments as in mx_cast_dim0_dim1. */
int mx_cast_dim1(const void* x, int64_t M, int64_t K, void* q1, void* s1_blk, void* stream);

/* dim0 cast only (the row-major copy and its blocked scales): the dim0 half of
 * the fused kernel of pytorch/ao PR #1869 (summary), for callers that need
 * only the K-block copy (a forward-pass operand).
 *   x       bf16 (M x K), row-major                      [in]
 *   M, K    M >= 1 (any; dim0 blocks run along K), K % 32 == 0, K >= 32,
 *           M, K <= 2^31 - 256
 *   q0      M x K bytes, e4m3                            [out]
 *   s0_blk  mx_blocked_bytes(M, K/32) bytes, e8m0        [out]
 * Padding bytes of the blocked buffer are written as zero. */
int mx_cast_dim0(const void* x, int64_t M, int64_t K, void* q0, void* s0_blk, void* stream);

/* Standalone conversion of a plain scale matrix to the blocked layout, the
 * operation of the scale-blocking kernels in pytorch/ao PR #3416 (Changes
 * list) and PR #2990 (perf analysis, scale swizzle kernels).
 *   s    R x C bytes, row-major, any alignment           [in]
 *   R, C >= 1, R <= 65535 * 128
 *   out  mx_blocked_bytes(R, C) bytes, 16-byte aligned   [out] */
int mx_scales_to_blocked(const void* s, int64_t R, int64_t C, void* out, void* stream);

/* Fused dim0 + dim1 cast of MoE activations with groups along M (pytorch/ao
 * PR #2990 "[mxfp8 moe training] add compile support": groups of rows given
 * by offsets; scale buffers sized by the bound rows + groups * 128 so that no
 * device-to-host read is needed).
 *   x            bf16 (M x K)                                   [in]
 *   M, K         M >= 1, K % 32 == 0, M, K <= 2^31 - 256
 *   offs         G int32 cumulative group ends (group g = rows
 *                [offs[g-1], offs[g]), offs[-1] = 0; offs[G-1] == M;
 *                empty groups allowed), device memory           [in]
 *   G            >= 1 (else MX_ERR_GROUPS)
 *   q0           M x K bytes: the ungrouped dim0 cast           [out]
 *   s0_blk       mx_grouped_m_scale_bytes(M, K, G, 0) bytes: group g's scale
 *                rows in blocked layout on their own, starting at row
 *                s0_row_offs[g] (byte s0_row_offs[g] * ceil4(K/32)) [out]
 *   s0_row_offs  G + 1 int64: sum over h < g of ceil(m_h/128)*128 [out]
 *   q1           K x M bytes: group g is the dim1 cast of its own rows
 *                (blocks of 32 start at the group's first row; the last
 *                block may be partial and counts missing rows as zero),
 *                in columns [offs[g-1], offs[g])                [out]
 *   s1_blk       mx_grouped_m_scale_bytes(M, K, G, 1) bytes: group g's
 *                (K x ceil(m_g/32)) scales in blocked layout on their own at
 *                byte ceil128(K) * s1_col_offs[g]                [out]
 *   s1_col_offs  G + 1 int64: sum over h < g of ceil(m_h/128)*4 [out]
 *   status       one int32, device memory: 0, or MX_ERR_GROUPS if the offsets
 *                are invalid (then nothing else is written)     [out]
 * Every byte of both scale buffers is written (padding zero). */
int mx_cast_grouped_m(const void* x, int64_t M, int64_t K, const int32_t* offs, int32_t G,
                      void* q0, void* s0_blk, int64_t* s0_row_offs, void* q1, void* s1_blk,
                      int64_t* s1_col_offs, int32_t* status, void* stream);

/* dim1 cast of 3D expert weights (pytorch/ao PR #2990, perf analysis: cast
 * the (E, N, K) weights as the reshaped 2D matrix (E*N, K) with the dim1
 * kernel, scales per expert).
 *   w       bf16 (E, N, K)                                       [in]
 *   E >= 1, N % 32 == 0, K % 32 == 0, E*N and K <= 2^31 - 256
 *   q1      K x (E*N) bytes: the dim1 cast of the (E*N, K) matrix;
 *           expert e owns columns [e*N, (e+1)*N)                  [out]
 *   s1_blk  mx_3d_scale_bytes(E, N, K) bytes: expert e's (K x N/32)
 *           scales in blocked layout at byte e * mx_blocked_bytes(K, N/32)
 *                                                                 [out] */
int mx_cast_3d_dim1(const void* w, int64_t E, int64_t N, int64_t K, void* q1, void* s1_blk,
                    void* stream);

/* dim0 cast of 3D expert weights: blocks of 32 along K, the direction the
 * forward pass reads the weights in.  The pages cast 3D weights only along N
 * with the dim1 kernel through the reshape to (E*N, K) (pytorch/ao PR #2990,
 * perf analysis); this applies the same reshape to the dim0 cast of PR #1869
 * and blocks each expert's scales on their own, like the dim1 variant.
 *   w       bf16 (E, N, K)                                       [in]
 *   E >= 1, N >= 1 (any), K % 32 == 0, K >= 32, E*N and K <= 2^31 - 256
 *   q0      E x N x K bytes: the dim0 cast of the (E*N, K) matrix [out]
 *   s0_blk  mx_3d_dim0_scale_bytes(E, N, K) bytes: expert e's (N x K/32)
 *           scales in blocked layout at byte e * mx_blocked_bytes(N, K/32);
 *           padding zero                                          [out] */
int mx_cast_3d_dim0(const void* w, int64_t E, int64_t N, int64_t K, void* q0, void* s0_blk,
                    void* stream);

/* Both directions of 3D expert weights in one read: mx_cast_3d_dim0's q0 and
 * s0_blk and mx_cast_3d_dim1's q1 and s1_blk (N % 32 == 0 required, as for
 * mx_cast_3d_dim1).  Buffer sizes as in those two calls. */
int mx_cast_3d_dim0_dim1(const void* w, int64_t E, int64_t N, int64_t K, void* q0, void* s0_blk,
                         void* q1, void* s1_blk, void* stream);

/* MX dequantisation to bf16.  The pages define no dequantisation kernel; the
 * value of an MX element is its scale times its element value (OCP
 * Microscaling Formats v1.0, MX block definition), here rounded once to bf16
 * (nearest even; subnormals kept; magnitudes rounding to 2^128 or more give
 * infinity; a NaN scale (0xFF) or NaN element gives NaN).  Applied to
 * (q0, s0_blk) of a cast it gives X back up to the cast's rounding; applied
 * to (q1, s1_blk), with R = K and C = M, it gives X^T.
 *   q       R x C bytes, e4m3, blocks of 32 along rows      [in]
 *   R, C    R >= 1, C % 32 == 0, C >= 32, R, C <= 2^31 - 256
 *   s_blk   mx_blocked_bytes(R, C/32) bytes, e8m0           [in]
 *   out     R x C bf16                                      [out] */
int mx_dequant_blocked(const void* q, int64_t R, int64_t C, const void* s_blk, void* out,
                       void* stream);

/* Tensorwise fp8: one dynamic scale for the whole tensor, the conversion of
 * pytorch/ao PR #1445 "[float8nocompile] Triton kernels for conversion to
 * float8 dtypes" (local amaxes in parallel, a global amax, then the
 * conversion, each block of which computes the scale itself).  Not an MX
 * format: the contrast case with a non-power-of-two scale.
 *   amax  = max |x|, written to *amax (fp32; NaN if x holds a NaN)
 *   scale = fp32 nearest to 448 / amax, written to *scale; amax = 0 gives
 *           1, a quotient beyond the largest finite fp32 gives that value
 *   q     = e4m3(fp32(x * scale)), nearest even, saturated to +-448
 *   x      n bf16 values, any shape, dense                    [in]
 *   n      >= 1, <= 2^40
 *   q      n bytes, e4m3                                      [out]
 *   scale  one fp32, device memory                            [out]
 *   amax   one fp32, device memory; also the call's reduction
 *          target (cleared, then reduced into)                [out]
 * Enqueues a 4-byte memset and two kernels. */
int mx_cast_tensorwise(const void* x, int64_t n, void* q, float* scale, float* amax,
                       void* stream);

/* Rowwise fp8: one scale per row, quantize_fp8_rowwise of the "FP8 linear
 * triton with row-wise scaling" gist.
 *   scale_r = bf16 nearest to max_j |x_rj| / 448 (bf16, the input's dtype)
 *   q_rj    = e4m3(fp32(x_rj / scale_r)), nearest even, saturated to +-448;
 *             a row whose scale is 0 (all zero, or amax below about 2^-125)
 *             gives signed zeros rather than the formula's 0/0
 *   x       bf16 (M x K)                                      [in]
 *   M, K    M >= 1, K >= 8, K % 8 == 0, M, K <= 2^31 - 256
 *   q       M x K bytes, e4m3                                 [out]
 *   scale   M bf16 values                                     [out] */
int mx_cast_rowwise(const void* x, int64_t M, int64_t K, void* q, void* scale, void* stream);

/* Product of two MX operands, accumulated in fp32 on the tensor cores:
 *   out[m][n] = sum_k A[m][k] B[n][k],  A[m][k] = qa[m][k] 2^(sa[m][k/32] - 127)
 * and B likewise, rounded once to the output type.  The pages name the
 * block-scaled GEMM as the reader of the casts' outputs (pytorch/ao PR #3416,
 * Changes list: the blocked format for grouped GEMM) and leave it to libraries;
 * here it closes the loop.  A linear layer y = x W^T (x T x K, W N x K) is
 *   forward          (q0, s0) of x    with (q0, s0) of W    -> y  (T x N)
 *   input gradient   (q0, s0) of dy   with (q1, s1) of W    -> dx (T x K)
 *   weight gradient  (q1, s1) of dy   with (q1, s1) of x    -> dW (N x K)
 * so that (q1, s1) of x, half the size of x, is all that the layer saves for
 * its backward pass.
 *   qa      M x K bytes, e4m3, blocks of 32 along rows      [in]
 *   sa_blk  mx_blocked_bytes(M, K/32) bytes, e8m0           [in]
 *   qb      N x K bytes, e4m3                               [in]
 *   sb_blk  mx_blocked_bytes(N, K/32) bytes, e8m0           [in]
 *   M, N    >= 1 (any); K % 32 == 0, K >= 32; all <= 2^31 - 256
 *   orders  0, or MX_A_BY_COLUMN, MX_B_BY_COLUMN or both: that operand's bytes
 *           are stored transposed (K x M, K x N; M, N then a multiple of 16),
 *           its scales as always by row and 32 contraction steps
 *   out     M x N values of out_type (MX_BF16 or MX_F32)    [out]
 * A NaN scale (0xFF) or element makes the results that use it NaN; sums
 * beyond the output type's range give infinity, sums below 2^-126 may come out as
 * zero.  Sums run in the tensor core's accumulator, which cuts bits off where
 * fp32 would round; for an fp32 output over 4096 steps at most, and those are added
 * up in fp32 (2.3e-7 of the 2-norm after 131072 steps, 1.4e-6 where all terms have
 * one sign, at any size of the output).
 * A call gives the same bits every time.  The sizes choose where a sum is cut, so a
 * row's last bits may be others in a batch of another M; at one M they do not depend
 * on what the other rows hold. */
int mx_matmul(const void* qa, const void* sa_blk, const void* qb, const void* sb_blk, int64_t M,
              int64_t N, int64_t K, int32_t orders, void* out, int32_t out_type, void* stream);

/* Layer norm of bf16 rows, with its input saved in 8 bits for the backward
 * pass.  The pages have no counterpart: the casts' formats put to use for what
 * a training step keeps.
 *   mean = (1/D) sum x, rstd = (eps + (1/D) sum (x - mean)^2)^(-1/2)
 *   y    = (x - mean) rstd w + b, rounded once to bf16
 *   x       bf16 (M x D)                                        [in]
 *   w, b    D values of w_type (MX_BF16 or MX_F32); b may be NULL (no bias)
 *                                                               [in]
 *   M, D    M >= 1, 1 <= D <= 16384; with a saved input D % 32 == 0
 *   eps     >= 0
 *   y       bf16 (M x D)                                        [out]
 *   mean, rstd  M floats each (4-byte aligned)                  [out]
 *   q0, s0_blk  both NULL, or x saved: mx_cast_dim0's outputs for x, byte for
 *           byte (M x D bytes; mx_blocked_bytes(M, D/32) bytes) [out]
 * A row that holds Inf or NaN gives NaN. */
int mx_layer_norm(const void* x, const void* w, const void* b, int32_t w_type, int64_t M, int64_t D,
                  float eps, void* y, float* mean, float* rstd, void* q0, void* s0_blk,
                  void* stream);

/* Its backward pass, from x itself or from the saved input (x is then what
 * (q0, s0_blk) stand for, mean and rstd still those of the forward pass; bytes of
 * s0_blk that belong to no block reach no result):
 *   xh = (x - mean) rstd, g = dy w
 *   dx = rstd (g - (1/D) sum g - xh (1/D) sum g xh), rounded once to bf16
 *   dw = sum over rows of dy xh, db = sum over rows of dy, summed in fp32 in a
 *        fixed order, rounded once to w_type
 *   dy      bf16 (M x D)                                        [in]
 *   x       bf16 (M x D), or NULL with q0, s0_blk given         [in]
 *   w       D values of w_type                                  [in]
 *   dx      bf16 (M x D)                                        [out]
 *   dw, db  D values of w_type; db may be NULL                  [out]
 *   work    mx_layer_norm_backward_work_bytes(M, D) bytes of scratch, 16-byte
 *           aligned; calls that overlap on the GPU need their own
 * Other arguments and limits as mx_layer_norm. */
int mx_layer_norm_backward(const void* dy, const void* x, const void* q0, const void* s0_blk,
                           const void* w, int32_t w_type, const float* mean, const float* rstd,
                           int64_t M, int64_t D, void* dx, void* dw, void* db, void* work,
                           void* stream);

/* Gated SiLU of bf16 rows [g | u], with its input saved in 8 bits.  The pages
 * have no counterpart (see mx_layer_norm).
 *   h = g u / (1 + exp(-g)), rounded once to bf16
 *   gu      bf16 (M x 2F): g in columns [0, F), u in [F, 2F)    [in]
 *   M, F    M >= 1, 1 <= F <= 2^24; with a saved input F % 32 == 0
 *   h       bf16 (M x F)                                        [out]
 *   q0, s0_blk  both NULL, or gu saved: mx_cast_dim0's outputs for gu, byte
 *           for byte                                            [out] */
int mx_swiglu(const void* gu, int64_t M, int64_t F, void* h, void* q0, void* s0_blk, void* stream);

/* Its backward pass, from gu itself or from the saved input:
 *   sg = 1 / (1 + exp(-g)), dg = dh u sg (1 + g (1 - sg)), du = dh g sg
 *   dh      bf16 (M x F)                                        [in]
 *   gu      bf16 (M x 2F), or NULL with q0, s0_blk given        [in]
 *   dgu     bf16 (M x 2F): dg | du                              [out] */
int mx_swiglu_backward(const void* dh, const void* gu, const void* q0, const void* s0_blk,
                       int64_t M, int64_t F, void* dgu, void* stream);

/* MX-FP4 casts: the casts above with e2m1 elements (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign),
 * a quarter of bf16's bytes.  The pages have no counterpart;
 * OCP Microscaling Formats v1.0 defines the format, its blocks of 32 and its e8m0 scales.
 *   scale byte s = clamp(floor(log2 amax) - 2, -127, 127) + 127; amax = 0 gives s = 0;
 *                  a block holding Inf or NaN gives s = 0xFF
 *   q_i          = e2m1(x_i * 2^(127 - s)), round to nearest even, saturated to +-6 (6 for
 *                  every element of an Inf/NaN block, whose value is its scale's NaN)
 * Two elements share a byte, the first in the low four bits.  Directions, blocked scales
 * and padding as for mx_cast_dim0, mx_cast_dim1 and mx_cast_dim0_dim1:
 *   x       bf16 (M x K), row-major                      [in]
 *   q0      M x K/2 bytes                                [out]
 *   s0_blk  mx_blocked_bytes(M, K/32) bytes, e8m0        [out]
 *   q1      K x M/2 bytes: q1[k][m/2] holds X[m][k] and X[m+1][k]  [out]
 *   s1_blk  mx_blocked_bytes(K, M/32) bytes, e8m0        [out]
 *   M, K    K % 32 == 0; M % 32 == 0, or for dim0 alone any M >= 1; <= 2^31 - 256 */
int mx_cast_fp4_dim0(const void* x, int64_t M, int64_t K, void* q0, void* s0_blk, void* stream);
int mx_cast_fp4_dim1(const void* x, int64_t M, int64_t K, void* q1, void* s1_blk, void* stream);
int mx_cast_fp4_dim0_dim1(const void* x, int64_t M, int64_t K, void* q0, void* s0_blk, void* q1,
                          void* s1_blk, void* stream);

/* MX-FP4 dequantisation to bf16, as mx_dequant_blocked: e2m1 times 2^(s - 127), rounded once
 * (exact but for magnitudes of 2^128 or more, which give infinity; scale 0xFF gives NaN).
 *   q       R x C/2 bytes                                [in]
 *   R, C    R >= 1, C % 32 == 0, C >= 32, R, C <= 2^31 - 256
 *   s_blk   mx_blocked_bytes(R, C/32) bytes, e8m0        [in]
 *   out     R x C bf16                                   [out] */
int mx_dequant_fp4(const void* q, int64_t R, int64_t C, const void* s_blk, void* out, void* stream);

/* Product of two MX-FP4 operands, as mx_matmul at twice its rate:
 *   out[m][n] = sum_k A[m][k] B[n][k]
 * The three products of a linear layer take the same casts as there; both operands are
 * stored by row.
 *   qa      M x K/2 bytes, e2m1, blocks of 32 along rows    [in]
 *   sa_blk  mx_blocked_bytes(M, K/32) bytes, e8m0           [in]
 *   qb      N x K/2 bytes, e2m1                             [in]
 *   sb_blk  mx_blocked_bytes(N, K/32) bytes, e8m0           [in]
 *   M, N    >= 1 (any); K % 64 == 0 (the tensor cores take 64 steps at a time), K >= 64;
 *           all <= 2^31 - 256
 *   out     M x N values of out_type (MX_BF16 or MX_F32)    [out]
 * Sums, their dependence on the sizes, NaN scales and ranges as mx_matmul. */
int mx_matmul_fp4(const void* qa, const void* sa_blk, const void* qb, const void* sb_blk, int64_t M,
                  int64_t N, int64_t K, void* out, int32_t out_type, void* stream);

/* The first half of a gated feed-forward layer in one kernel: both projections of MX
 * operands, the activation and the product.
 *   g = X Wg^T, u = X Wu^T, summed in fp32
 *   h = g u / (1 + exp(-g)), from the sums, rounded once to bf16
 * g and u do not reach memory unless they are saved for the backward pass, in 8 bits: the
 * layout of mx_swiglu's save, (M x 2F) rows [g | u], each value rounded once from its sum.
 * Sums as mx_matmul's for bf16; where they are saved, over at most 1792 steps (MX_E2M1:
 * 2560) in the tensor core's accumulator, and those in fp32.  So over more steps than that
 * h with the save and h without it may differ in the last bits, as may a row's results in
 * batches of another M.
 * The pages have no counterpart (see mx_layer_norm).
 *   qx      M x K elements of `format`, blocks of 32 along rows (mx_cast_dim0 or
 *           mx_cast_fp4_dim0 of X)                          [in]
 *   sx_blk  mx_blocked_bytes(M, K/32) bytes, e8m0           [in]
 *   qg, qu  F x K elements of `format` each: Wg, Wu         [in]
 *   sg_blk, su_blk  mx_blocked_bytes(F, K/32) bytes each    [in]
 *           (with F % 128 == 0 the two halves of a cast of [Wg; Wu], bytes and scales, are
 *           these operands)
 *   M, F, K M >= 1; F % 32 == 0, 32 <= F <= 2^24; K % 32 == 0 (MX_E2M1: 64), K >= 32 (64);
 *           M, K <= 2^31 - 256
 *   format  MX_E4M3 or MX_E2M1, of all operands
 *   h       bf16 (M x F)                                    [out]
 *   q0, s0_blk  both NULL, or [g | u] saved: M x 2F bytes, e4m3, and
 *           mx_blocked_bytes(M, 2F/32) bytes                [out] */
int mx_matmul_swiglu(const void* qx, const void* sx_blk, const void* qg, const void* sg_blk,
                     const void* qu, const void* su_blk, int64_t M, int64_t F, int64_t K,
                     int32_t format, void* h, void* q0, void* s0_blk, void* stream);

/* Its backward pass, through the layer's second projection y = h W2^T: from the gradient of
 * y to that of [g | u], in one kernel; the gradient of h does not reach memory.
 *   dh = dY W2, summed in fp32
 *   sg = 1 / (1 + exp(-g)), dg = dh u sg (1 + g (1 - sg)), du = dh g sg, rounded once to bf16
 *   qdy     M x K elements of `format`, blocks along rows (the dim0 cast of dY)  [in]
 *   sdy_blk mx_blocked_bytes(M, K/32) bytes, e8m0           [in]
 *   qw      F x K elements of `format`: W2 transposed (the dim1 cast of W2, K x F)  [in]
 *   sw_blk  mx_blocked_bytes(F, K/32) bytes, e8m0           [in]
 *   gu      bf16 (M x 2F), or NULL with q0, s0_blk given    [in]
 *   dgu     bf16 (M x 2F): dg | du                          [out]
 * Sizes and format as mx_matmul_swiglu.  The weights' gradients are products of the casts of
 * dY and dgu (mx_matmul, mx_matmul_fp4). */
int mx_matmul_swiglu_backward(const void* qdy, const void* sdy_blk, const void* qw,
                              const void* sw_blk, int64_t M, int64_t F, int64_t K, int32_t format,
                              const void* gu, const void* q0, const void* s0_blk, void* dgu,
                              void* stream);

/* Size helpers (host only, no CUDA calls).  Return -1 for invalid sizes. */
int64_t mx_blocked_bytes(int64_t R, int64_t C);
/* dim 0: (M + 128*G) * ceil4(K/32); dim 1: ceil128(K) * (ceil(M/32) + 4*G). */
int64_t mx_grouped_m_scale_bytes(int64_t M, int64_t K, int32_t G, int32_t dim);
/* E * mx_blocked_bytes(K, N/32): dim1 scales of 3D weights. */
int64_t mx_3d_scale_bytes(int64_t E, int64_t N, int64_t K);
/* E * mx_blocked_bytes(N, K/32): dim0 scales of 3D weights. */
int64_t mx_3d_dim0_scale_bytes(int64_t E, int64_t N, int64_t K);

/* Scratch of mx_layer_norm_backward: partial sums of dw and db. */
int64_t mx_layer_norm_backward_work_bytes(int64_t M, int64_t D);

/* Text for an MX_* code (static storage). */
const char* mx_strerror(int code);

/* cudaError_t value of the last failed CUDA call made by this thread. */
int mx_last_cuda_error(void);

/* Device watchdog: every wait inside the kernels is bounded.  A CTA that
 * gives up stops all its roles, lets the copies it has in flight land, and
 * sets a device word (one per kernel file).  Returns the words OR-ed (0 or 1)
 * after synchronising the current device, clearing them if `clear` is
 * non-zero, or MX_ERR_CUDA. */
int mx_watchdog(int clear);

/* Bounds-checked builds (compiled with -DMX_DEBUG_BOUNDS): the number of
 * global stores the kernels refused because they would have left their
 * output buffer (each is skipped and counted, never trapped), cleared if
 * `clear` is non-zero.  The stand-in for a device memory checker.  Returns -1
 * in a release build (no checks compiled in), MX_ERR_CUDA if the count could
 * not be read.  Synchronises the current device. */
int mx_bounds_check(int clear);

/* Diagnostic for bounds-checked builds: one thread tries a 4-byte store just
 * past an 8-byte span over `buf16` (16 bytes of device memory owned by the
 * caller, 16-byte aligned); the check refuses it, leaves bytes 8..11
 * untouched and adds one to the count read by mx_bounds_check().  Returns
 * MX_OK, MX_ERR_NULL / MX_ERR_ALIGN / MX_ERR_DEVICE / MX_ERR_CUDA, or -1 in
 * a release build (nothing is launched). */
int mx_selftest_bounds(void* buf16, void* stream);

/* Diagnostic: enqueue one warp that waits, with a limit of `wait_ns`
 * nanoseconds (1e3 .. 1e10), on a barrier that nothing completes.  The wait
 * gives up, sets the watchdog word read by mx_watchdog() and the kernel
 * returns normally: the failure path of the bounded waits, exercised without
 * any fault.  Returns MX_OK, MX_ERR_SHAPE or MX_ERR_CUDA. */
int mx_selftest_watchdog(int64_t wait_ns, void* stream);

/* Diagnostic of checked builds (compiled with -DMX_DEBUG_BOUNDS, as
 * libmxfp8_cast_bounds.so): arm a stall for the calling thread's next launch
 * of a kernel whose waits are bounded (the cast kernels of mx_cast_dim0_dim1,
 * mx_cast_dim0, mx_cast_dim1, mx_cast_grouped_m and the 3D casts; the
 * bulk-staged kernel of mx_cast_rowwise, used for K <= 24576; the tiled
 * kernel of mx_dequant_blocked, used for C >= 1024; the kernels of mx_matmul,
 * mx_matmul_fp4, mx_matmul_swiglu, mx_matmul_swiglu_backward, mx_cast_fp4_dim1,
 * mx_cast_fp4_dim0_dim1, the tiled ones of mx_cast_fp4_dim0 and mx_dequant_fp4 (used
 * where there is a tile of 128 x 128 for every SM), mx_layer_norm and the first of
 * mx_layer_norm_backward).  In that launch the thread of CTA 0 that issues its loads waits, at its `at`-th tile (rowwise:
 * step; products: block of 128 contraction bytes; layer norm: row of its first
 * group), on a barrier that nothing completes, for at most `wait_ns` nanoseconds
 * (1e3 .. 1e10).  The wait gives up, the CTA stops every role, lets the
 * copies it has in flight land, sets the word read by mx_watchdog(), and the
 * kernel returns normally: the abort path of a real cast, exercised without
 * any fault.  That launch's outputs are incomplete.  Without a kernel to take
 * it the stall stays armed; a launch consumes it.  Returns MX_OK,
 * MX_ERR_SHAPE (at < 0 or wait_ns out of range), or -1 in a release build,
 * whose kernels carry no stall hook (nothing is armed). */
int mx_selftest_arm_stall(int64_t at, int64_t wait_ns);

#ifdef __cplusplus
}
#endif

#endif /* MXFP8_CAST_H */
