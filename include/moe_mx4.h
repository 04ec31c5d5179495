/*
 * moe_mx4.h -- the operators around the FP4 routed-expert layer of moe_fp4.h:
 * MXFP4 quantisation and the reading back of microscaled rows, products of
 * MXFP4 rows with MXFP4 weights (dense, and grouped by expert), and the norms
 * before and after a block with its gate, residual and quantisation.
 *
 * The conventions of moe_fp4.h hold: device pointers unless a comment says
 * (host), every call only enqueues on `stream`, all checks run before anything
 * is enqueued, nothing is allocated, freed or synchronised, so every call can
 * be captured in a HIP graph; the same inputs give the same bits.  Tensors are
 * row-major and contiguous unless a stride is given.  The device that `stream`
 * belongs to has to be current.
 *
 * MXFP4: e2m1 codes (0, .5, 1, 1.5, 2, 3, 4, 6 and their negatives), two per
 * byte along K, the EVEN element in the LOW nibble, with one E8M0 scale code
 * c = 2^(c-127) for 32 consecutive elements of a row; 255 is NaN, and every
 * value of such a block reads as NaN.
 */
#ifndef MOE_MX4_H
#define MOE_MX4_H

#include "moe_fp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of the arguments that leave a choice. */
#define MOE_TYPE_BF16 0
#define MOE_TYPE_FP16 1
#define MOE_TYPE_FP32 2

/* Microscaled formats: what moe_dequant_mx reads and the norms write. */
#define MOE_QUANT_NONE 0
#define MOE_QUANT_MXFP8 1 /* e4m3fn, as moe_quant_act_mxfp8 */
#define MOE_QUANT_MXFP4 2

/*
 * MXFP4 quantisation.  For each row and each block of 32 elements:
 * X = floor(log2(max|v|)) - 2 (2 = largest e2m1 exponent), kept in
 * [-127, 127], X = -127 for a block of zeros; scale code X + 127; each code is
 * v * 2^-X rounded to e2m1, nearest, ties to the even code, at most 6, sign
 * kept.  A block that holds a NaN or an infinity gets scale code 255 and zero
 * codes.
 *   x [M, K] of x_type (bf16, fp16 or fp32), rows ldx elements apart,
 *     ldx >= K, 16-byte aligned as is every row; K % 32 == 0
 *   q [M, K/2] (out, 4-byte aligned), s [M, K/32] (out)
 */
moe_status_t moe_quant_mxfp4(const void* x, int32_t x_type, int32_t M, int32_t K, int64_t ldx, uint8_t* q,
                             uint8_t* s, hipStream_t stream);

/*
 * The values of microscaled rows: code * 2^(c-127), exact in fp32 (infinite
 * past its range), rounded to nearest even in bf16 and fp16.
 *   format MOE_QUANT_MXFP4: q [M, K/2] (4-byte aligned); MOE_QUANT_MXFP8:
 *     q [M, K] (8-byte aligned); s [M, K/32]; K % 32 == 0
 *   out [M, K] of out_type (16-byte aligned)
 */
moe_status_t moe_dequant_mx(const uint8_t* q, const uint8_t* s, int32_t format, int32_t M, int32_t K, void* out,
                            int32_t out_type, hipStream_t stream);

/*
 * Weights of the MXFP4 products: E matrices [N, K] (E = 1 for a dense
 * projection), brought into the kernels' tile order once.
 *   wq [E, N, K/2] (16-byte aligned), ws [E, N, K/32]
 *   uq, us: null for a plain product.  With the SwiGLU form wq/ws are the gate
 *     projection's and uq/us the up projection's, of the same shape, and the
 *     products return silu(gate) * up [., N].
 *   packed >= moe_mxfp4_packed_bytes(E, N, K, glu) bytes, 256-byte aligned;
 *     the caller keeps it alive and unmodified while desc (host) is in use,
 *     the inputs may go once the stream has passed this call
 *   1 <= E <= 1024, N % 32 == 0, K % 128 == 0, N and K at most 2^20
 */
#define MOE_MXFP4_LAYOUT_VERSION 1u

typedef struct moe_mxfp4_weights {
  int32_t E, N, K;
  int32_t glu; /* 1: the SwiGLU form */
  uint32_t layout_version;
  const void* packed; /* device */
  size_t packed_bytes;
} moe_mxfp4_weights_t;

size_t moe_mxfp4_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t glu);
moe_status_t moe_mxfp4_prepack(const uint8_t* wq, const uint8_t* ws, const uint8_t* uq, const uint8_t* us, int32_t E,
                               int32_t N, int32_t K, void* packed, size_t packed_bytes,
                               moe_mxfp4_weights_t* desc /*(host)*/, hipStream_t stream);

/*
 * Dense product: y[t, n] = sum_k x[t, k] W[n, k] (or its SwiGLU form), both
 * operands MXFP4, accumulated in fp32 in the matrix cores and rounded once to
 * y_type (bf16, or fp32 as it is).  SiLU takes the hardware's exponential and
 * reciprocal: with a gate sum g, fp32 outputs are within (|g| + 8) 2^-22 of
 * their size of silu(g) * up; below g = -87, where silu(g) < 2^-118, they may
 * be 0.
 *   xq [T, K/2] (16-byte aligned), xs [T, K/32] (4-byte aligned)
 *   y [T, N] (16-byte aligned); T * K <= 2^33 - 8192
 *   flags: MOE_FLAG_FORCE_DECODE streams the weights for every 32 tokens,
 *   MOE_FLAG_FORCE_PREFILL takes the tiled product; both compute the same
 *   function, by default the sizes decide.
 */
moe_status_t moe_mxfp4_dense_forward(const moe_mxfp4_weights_t* w /*(host), E == 1*/, const uint8_t* xq,
                                     const uint8_t* xs, int32_t T, void* y, int32_t y_type, uint32_t flags,
                                     hipStream_t stream);

/*
 * Product grouped by expert: for each expert e and each row s of y with
 * offsets[e] <= s < offsets[e+1], y[s] = W[e] x[r(s)] (or its SwiGLU form),
 * r(s) = rows[s] / row_div, or s where rows is null.  With the sorted_pair of
 * moe_sort_permute and row_div = k, r(s) is the pair's token.
 *   xq [X, K/2] (16-byte aligned), xs [X, K/32] (4-byte aligned)
 *   offsets [E+1] int32, not decreasing; groups may be empty.  Rows of y in
 *     front of offsets[0] and from offsets[E] on are left as they were.
 *   rows [P] int32 or null.  What the two arrays hold is not checked, but
 *     offsets past P and rows past X are read as the last row's, never beyond.
 *   y [P, N] of y_type (16-byte aligned), rows in expert order
 *   workspace >= moe_mxfp4_grouped_workspace_size(P, E, N, K, glu) bytes,
 *     256-byte aligned; contents ignored on entry.  Calls (or captured graphs)
 *     that may overlap need one each.
 *   flags as above; by default P, E and N decide, not the groups' sizes (which
 *   are on the device): where a few groups hold most of few rows,
 *   MOE_FLAG_FORCE_PREFILL is faster.  X * K <= 2^33 - 8192, P < 2^31 - 256
 */
size_t moe_mxfp4_grouped_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K, int32_t glu);
moe_status_t moe_mxfp4_grouped_forward(const moe_mxfp4_weights_t* w /*(host)*/, const uint8_t* xq, const uint8_t* xs,
                                       int32_t X, const int32_t* offsets, const int32_t* rows, int32_t row_div,
                                       int32_t P, void* y, int32_t y_type, void* workspace, size_t workspace_bytes,
                                       uint32_t flags, hipStream_t stream);

/*
 * Norm before a block: z = bf16((x r) w), r = 1 / sqrt(mean(x^2) + eps), with
 * the mean square in 64 bits and r, x r and (x r) w each rounded to fp32, and
 * the microscaled rows of z that the block's products read.
 *   x [T, H] of x_type (bf16 or fp32); w [H] of w_type (bf16 or fp32)
 *   z [T, H] bf16 bits (out), or null where only the codes are wanted
 *   quant: MOE_QUANT_NONE (q, s null), MOE_QUANT_MXFP8: q [T, H], the bytes of
 *     moe_quant_act_mxfp8(z); MOE_QUANT_MXFP4: q [T, H/2], the bytes of
 *     moe_quant_mxfp4(z); s [T, H/32].  A block with a NaN or an infinity gets
 *     scale code 255 in both.
 *   1 <= H <= 16384, H % 8 == 0 (H % 32 == 0 with quant); eps >= 0; all
 *   pointers but s 16-byte aligned
 */
moe_status_t moe_norm_before(const void* x, int32_t x_type, const void* w, int32_t w_type, int32_t T, int32_t H,
                             float eps, uint16_t* z, uint8_t* q, uint8_t* s, int32_t quant, hipStream_t stream);

/*
 * Norm after a block, its gate, the residual, and the norm before the next:
 *   b = y, or (y r(y)) w_post where w_post is given; b = b g where a gate is;
 *   out = beta residual + alpha b, rounded to the residual's type;
 *   where w_next is given z, q, s = moe_norm_before(out, w_next).
 * Every step one fp32 operation, in this order.
 *   y [T, H] of y_type (bf16 or fp32); residual, out [T, H] of residual_type
 *     (bf16 or fp32); out may be residual itself, nothing else may overlap
 *   w_post, w_next [H] of w_type, or null; z, q, s, quant as above (null and
 *     MOE_QUANT_NONE without w_next; with it z or q at least)
 *   gate fp32 or null: g[t, h] = gate[t gate_t + h gate_h], gate_h 0 or 1
 *     (one for each token: gate_h = 0; for each channel: gate_t = 0)
 */
moe_status_t moe_norm_after(const void* y, int32_t y_type, const void* residual, int32_t residual_type,
                            const void* w_post, const void* w_next, int32_t w_type, const float* gate,
                            int64_t gate_t, int64_t gate_h, float alpha, float beta, float eps, int32_t T, int32_t H,
                            void* out, uint16_t* z, uint8_t* q, uint8_t* s, int32_t quant, hipStream_t stream);

/*
 * The layer between its norms:
 *   z = moe_norm_before(x, w_pre); y = moe_fp4_layer_forward_full(z);
 *   out = moe_norm_after(y, x, w_post, gate, alpha, beta)
 * with the bits of that chain (for finite z).  Above 16 tokens the norm writes
 * the experts' MXFP8 rows itself.
 *   x, out [T, H] of x_type (bf16 or fp32); out may be x itself
 *   the other arguments as for those calls
 *   workspace >= moe_fp4_block_workspace_size(...) bytes, 256-byte aligned
 */
typedef struct moe_block_norms {
  const void* w_pre;  /* [H] */
  const void* w_post; /* [H], or null: no norm behind the layer */
  int32_t w_type;     /* of both */
  const float* gate;  /* or null */
  int64_t gate_t, gate_h;
  float alpha, beta, eps;
} moe_block_norms_t;

size_t moe_fp4_block_workspace_size(int32_t T, int32_t E, int32_t k, int32_t H, int32_t I, int32_t n_shared,
                                    uint32_t flags);
moe_status_t moe_fp4_block_forward(const moe_fp4_weights_t* w /*(host)*/, int32_t n_shared, const uint16_t* router_w,
                                   const moe_block_norms_t* norms /*(host)*/, const void* x, int32_t x_type, int32_t T,
                                   int32_t k, void* out, void* workspace, size_t workspace_bytes, uint32_t flags,
                                   hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MX4_H */
