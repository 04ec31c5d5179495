/*
 * moe_fp8_block.h -- FP8 operators with a scale for each block of 128: the
 * quantisation of activations, products of such rows with FP8 weights (dense,
 * and grouped by expert), the gated feed-forward block (both projections,
 * SwiGLU and the quantisation of its rows), its backward pass, and the
 * gradient of the weights.
 *
 * The conventions of moe_fp4.h hold: device pointers unless a comment says
 * (host), every call only enqueues on `stream`, all checks run before anything
 * is enqueued, nothing is allocated, freed or synchronised, so every call can
 * be captured in a HIP graph; the same inputs give the same bits.  Tensors are
 * row-major and contiguous unless a stride is given; outputs overlap nothing.
 * The device that `stream` belongs to has to be current.
 *
 * Formats: e4m3fn codes (largest value 448, 0x7F and 0xFF NaN), one a byte.
 * Rows: one fp32 scale for 128 consecutive elements; the scales of M rows of K
 * elements are held block by block, s[K/128][M], so that neighbouring rows'
 * scales of a block are neighbours.  Weights [N, K]: one fp32 scale for each
 * block of 128 x 128, s[ceil(N/128)][K/128]; a last block may have fewer rows.
 * A value is code * scale.
 */
#ifndef MOE_FP8_BLOCK_H
#define MOE_FP8_BLOCK_H

#include "moe_mx4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Quantisation of rows.  For each block of 128 elements of a row:
 * a = max(max|v|, 2^-110); scale = a / 448; each code is v * (448 / a) rounded
 * to e4m3, nearest, ties to even, at most 448, sign kept; division and product
 * each one fp32 operation.  A block that holds a NaN or an infinity gets a NaN
 * scale and zero codes.
 *   x [M, K] of x_type (bf16, fp16 or fp32), rows ldx elements apart,
 *     ldx >= K, 16-byte aligned as is every row; K % 128 == 0, K <= 2^20,
 *     M < 2^31 - 256
 *   q [M, K] (out, 8-byte aligned), s [K/128, M] (out)
 */
moe_status_t moe_quant_fp8_block(const void* x, int32_t x_type, int32_t M, int32_t K, int64_t ldx, uint8_t* q,
                                 float* s, hipStream_t stream);

/*
 * The values of such rows: code * scale, one fp32 product, rounded to nearest
 * even in bf16 and fp16.
 *   q [M, K] (8-byte aligned), s [K/128, M]; out [M, K] of out_type (16-byte
 *   aligned); M and K as above
 */
moe_status_t moe_dequant_fp8_block(const uint8_t* q, const float* s, int32_t M, int32_t K, void* out,
                                   int32_t out_type, hipStream_t stream);

/*
 * Weights of the products: E matrices [N, K] (E = 1 for a dense projection),
 * brought into the kernels' tile order once.
 *   moe_fp8_block_prepack: wq [E, N, K] (16-byte aligned), ws [E, ceil(N/128),
 *     K/128] fp32.  uq, us: null for a plain product; with them wq/ws are the
 *     gate projection's and uq/us the up projection's (the form that
 *     moe_fp8_block_glu_forward takes).
 *   moe_fp8_block_prepack_t: the same bytes transposed, for the backward pass.
 *     wq [E, K, N], ws [E, K/128, N/128]: product with W^T.  With uq, us of the
 *     same shape K is the two matrices' K together: [wq; uq] [E, K/2 + K/2, N],
 *     so that one product of rows [dg, du] is dg W1 + du W3.  N % 128 == 0,
 *     K % 256 == 0 with uq.
 *   packed >= moe_fp8_block_packed_bytes(E, N, K, glu) bytes, 256-byte aligned;
 *     the caller keeps it alive and unmodified while desc (host) is in use, the
 *     inputs may go once the stream has passed this call
 *   1 <= E <= 1024, N % 32 == 0, K % 128 == 0, N and K at most 2^20
 */
#define MOE_FP8_BLOCK_LAYOUT_VERSION 1u

typedef struct moe_fp8_block_weights {
  int32_t E, N, K;
  int32_t glu; /* 1: gate and up */
  uint32_t layout_version;
  const void* packed; /* device */
  size_t packed_bytes;
} moe_fp8_block_weights_t;

size_t moe_fp8_block_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t glu);
moe_status_t moe_fp8_block_prepack(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us, int32_t E,
                                   int32_t N, int32_t K, void* packed, size_t packed_bytes,
                                   moe_fp8_block_weights_t* desc /*(host)*/, hipStream_t stream);
moe_status_t moe_fp8_block_prepack_t(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us,
                                     int32_t E, int32_t N, int32_t K, void* packed, size_t packed_bytes,
                                     moe_fp8_block_weights_t* desc /*(host)*/, hipStream_t stream);

/*
 * Dense product: y[t, n] = sum_k x[t, k] W[n, k].  The products of a block of
 * 128 are summed in the matrix cores, the blocks' sums times both scales by
 * fp32 fused multiply-adds; rounded once to y_type (bf16, or fp32 as it is).
 * For bf16 (and for rows that are quantised) they are summed in the FP8 matrix
 * cores, which add eight neighbouring products with 14 bits below the largest of
 * them: 2^-13 of that for each at most, 1.5e-5 of a block's sum of ordinary values.
 * For fp32 the codes go through the bf16 cores, where every product is exact, at
 * half the rate.
 *   w plain, E == 1; xq [T, K] (16-byte aligned), xs [K/128, T]
 *   y [T, N] (16-byte aligned); T * K <= 2^32 - 4096
 *   flags: MOE_FLAG_FORCE_DECODE streams the weights for every 16 or 32 tokens,
 *   MOE_FLAG_FORCE_PREFILL takes the tiled product; both compute the same
 *   function, by default the sizes decide.
 */
moe_status_t moe_fp8_block_dense_forward(const moe_fp8_block_weights_t* w /*(host)*/, const uint8_t* xq,
                                         const float* xs, int32_t T, void* y, int32_t y_type, uint32_t flags,
                                         hipStream_t stream);

/*
 * Product grouped by expert: for each expert e and each row s of y with
 * offsets[e] <= s < offsets[e+1], y[s] = W[e] x[r(s)], r(s) = rows[s] /
 * row_div, or s where rows is null.  With the sorted_pair of moe_sort_permute
 * and row_div = k, r(s) is the pair's token.
 *   w plain; xq [X, K] (16-byte aligned), xs [K/128, X]
 *   offsets [E+1] int32, not decreasing; groups may be empty.  Rows of y in
 *     front of offsets[0] and from offsets[E] on are left as they were.
 *   rows [P] int32 or null.  What the two arrays hold is not checked, but
 *     offsets past P and rows past X are read as the last row's, never beyond.
 *   y [P, N] of y_type (16-byte aligned), rows in expert order
 *   workspace >= moe_fp8_block_grouped_workspace_size(P, E, N, K) bytes,
 *     256-byte aligned; contents ignored on entry.  Calls (or captured graphs)
 *     that may overlap need one each.
 *   flags as above; by default P, E and N decide, not the groups' sizes (which
 *   are on the device): where a few groups hold most of few rows,
 *   MOE_FLAG_FORCE_PREFILL is faster.  X * K <= 2^32 - 4096, P < 2^31 - 256
 */
size_t moe_fp8_block_grouped_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K);
moe_status_t moe_fp8_block_grouped_forward(const moe_fp8_block_weights_t* w /*(host)*/, const uint8_t* xq,
                                           const float* xs, int32_t X, const int32_t* offsets, const int32_t* rows,
                                           int32_t row_div, int32_t P, void* y, int32_t y_type, void* workspace,
                                           size_t workspace_bytes, uint32_t flags, hipStream_t stream);

/*
 * Gated feed-forward block up to its down projection, grouped as above:
 * g = W1[e] x[r(s)], u = W3[e] x[r(s)], h = g / (1 + e^-g) * u in fp32, and
 * the rows of h quantised as by moe_quant_fp8_block (of the fp32 values).
 * SiLU takes the hardware's exponential and reciprocal: h is within
 * (|g| + 8) 2^-22 of its size; below g = -87, where silu(g) < 2^-118, it may be 0.
 *   w gate and up, N % 128 == 0
 *   offsets, rows null: one group of P rows (E == 1), row s reads x[s]
 *   q [P, N] (out, 8-byte aligned), s [N/128, P] (out)
 *   gate, up [P, N] bf16 bits (out, 16-byte aligned): g and u for the backward
 *     pass, or both null
 *   Rows outside [offsets[0], offsets[E]) are left as they were in all outputs.
 *   workspace >= moe_fp8_block_glu_workspace_size(P, E, N, K, flags) bytes,
 *     256-byte aligned, as above.  The size serves this call and the backward one,
 *     for P rows and for any fewer of them, under the same flags.
 */
size_t moe_fp8_block_glu_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K, uint32_t flags);
moe_status_t moe_fp8_block_glu_forward(const moe_fp8_block_weights_t* w /*(host)*/, const uint8_t* xq,
                                       const float* xs, int32_t X, const int32_t* offsets, const int32_t* rows,
                                       int32_t row_div, int32_t P, uint8_t* q, float* s, uint16_t* gate, uint16_t* up,
                                       void* workspace, size_t workspace_bytes, uint32_t flags, hipStream_t stream);

/*
 * Backward of h = silu(g) u behind the backward of the down projection, grouped
 * as above: dh[s] = W2[e]^T dO[r(s)], sig = 1 / (1 + e^-g),
 *   dg = dh u sig (1 + g (1 - sig)),  du = dh g sig
 * in fp32 (sig from the hardware's exponential and reciprocal; 0 below g = -87.3,
 * where |g| sig < 2^-118), quantised in blocks of 128 of each.  [dg, du] are the
 * rows of the input gradient's product (moe_fp8_block_prepack_t of both
 * projections) and of the weight gradient.
 *   w plain, from moe_fp8_block_prepack_t of W2 [E, K, N]: N the block's inner
 *     width, N % 128 == 0
 *   yq [X, K], ys [K/128, X]: the rows dO
 *   gate, up [P, N] bf16 bits (16-byte aligned) as moe_fp8_block_glu_forward wrote them
 *   q [P, 2 N] (out, 8-byte aligned): dg, then du; s [2 N/128, P] (out)
 *   the rest as for moe_fp8_block_glu_forward
 */
moe_status_t moe_fp8_block_glu_backward(const moe_fp8_block_weights_t* w /*(host)*/, const uint8_t* yq,
                                        const float* ys, int32_t X, const int32_t* offsets, const int32_t* rows,
                                        int32_t row_div, int32_t P, const uint16_t* gate, const uint16_t* up,
                                        uint8_t* q, float* s, void* workspace, size_t workspace_bytes,
                                        uint32_t flags, hipStream_t stream);

/*
 * Gradient of the weights: dw[e, n, k] = sum over the rows s of group e of
 * dy[s, n] x[r(s), k], both rows quantised.  Their scales vary along this sum,
 * so it runs in the fp16 matrix cores: x's codes are exact there; the product of
 * a row's two scales, relative to the largest such product of the group's rows, and
 * dy's code times it are rounded to fp16: 2^-10 of each product together, or, where a
 * row's product of scales is less than 2^-18 of the largest one, 2^-29 of what that
 * would make.
 * Sums in fp32, rounded once to dw_type (bf16, or fp32 as it is).  A group without
 * rows gets zeros.
 *   yq [P, N], ys [N/128, P]; xq [X, K], xs [K/128, X]; codes 16-byte aligned
 *   offsets null, then rows too: one group of P rows (E == 1); else as above
 *   dw [E, N, K] (out, 16-byte aligned); N % 128 == 0, K % 128 == 0
 *   workspace >= moe_fp8_block_weight_grad_workspace_size(P, E, N, K) bytes,
 *     256-byte aligned, as above
 */
size_t moe_fp8_block_weight_grad_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K);
moe_status_t moe_fp8_block_weight_grad(const uint8_t* yq, const float* ys, const uint8_t* xq, const float* xs,
                                       int32_t X, const int32_t* offsets, const int32_t* rows, int32_t row_div,
                                       int32_t P, int32_t E, int32_t N, int32_t K, void* dw, int32_t dw_type,
                                       void* workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_FP8_BLOCK_H */
