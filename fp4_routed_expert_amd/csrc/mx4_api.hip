// C ABI of the MXFP4 operators and the norms (declared in include/moe_mx4.h):
// host-side argument checks and path selection.  Every check runs before any
// launch, so a failing call enqueues nothing and touches no output.
#include <math.h>

#include "api.h"
#include "mx4.h"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

bool known_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_FP16 || t == MOE_TYPE_FP32; }
bool norm_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_FP32; }

constexpr int kMaxMx4E = 1024;
// A tile past the last row still counts in 32 bits; the streaming product's passes step by next_pass.
constexpr int kMaxMx4P = INT32_MAX - 256;
constexpr int kMaxNormH = 16384;

// A grid of one workgroup of 256 threads per 1024 groups of eight elements has
// to stay below 2^32 threads.
bool too_many(int32_t M, int32_t K) { return (int64_t)M * K / 8192 >= ((int64_t)1 << 24) - 1; }

moe_status_t check_enk(int32_t E, int32_t N, int32_t K, int32_t glu) {
  if (E < 1 || N < 1 || K < 1 || (glu != 0 && glu != 1)) return MOE_ERR_INVALID_ARGUMENT;
  if (E > kMaxMx4E || N % 32 != 0 || K % 128 != 0 || N > (1 << 20) || K > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  // packing runs a grid of up to 2^20 x 65535 workgroups of 4 KiB
  if (Mx4Layout(E, N, K, glu).s_off / 4096 > (size_t)65535 << 20) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_mx4_weights(const moe_mxfp4_weights_t* w) {
  if (!w || !w->packed || w->layout_version != MOE_MXFP4_LAYOUT_VERSION) return MOE_ERR_INVALID_ARGUMENT;
  moe_status_t st = check_enk(w->E, w->N, w->K, w->glu);
  if (st != MOE_OK) return st;
  if (!aligned(w->packed, 256) || w->packed_bytes < Mx4Layout(w->E, w->N, w->K, w->glu != 0).total)
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// The tiled product addresses activation rows by 32-bit byte offsets.
bool rows_too_large(int32_t X, int32_t K) { return (int64_t)X * K / 2 > ((int64_t)1 << 32) - 4096; }

// 0: stream the weights, 1: tiled, -1: bad flags.  By default the weights are
// streamed while the groups average at most 16 rows (measured with 64 and 256
// experts: at 12 rows streaming is 3-17 % faster, at 24 rows 5-24 % slower), or
// while streaming makes at most 1024 passes of 32 rows over a weight tile, four
// per CU: the tiled product has few tiles then.  Dense, us, streaming against
// tiled: K 4096, N 1536, 333 rows (528 passes) 12 and 16, 1024 rows (1536) 20
// and 16; K 16384, N 7168, 128 rows (896) 63 and 70, 256 rows (1792) 119 and
// 70; K 1536, N 4096, 256 rows (1024) 8.2 and 9.7, 512 rows (2048) 12 and 10.
// Grouped, where the tiled product lists its tiles first, up to 1280 (a group's
// last pass counted half): 16 experts, K 2048, N 512, 2000 rows (1120) 12 and
// 21; 4 experts, K 2048, N 4096, 256 rows (1280) 11 and 15; 8 experts, K 16384,
// N 2048, 400 rows (1024) 70 and 59, K 4096, N 4096, 512 rows (2560) 47 and 30.
// The averages do not see skew, which only the device knows: streaming walks a
// group's rows 32 at a time, by one workgroup per tile pair once the groups' tiles
// fill the CUs.  64 experts, K 4096, N 1536, 1024 rows, even / Zipf (largest group
// 305) / all in one group: streaming 49 / 111 / 183, tiled 43 / 42 / 20; SwiGLU 83 /
// 137 / 259 and 84 / 82 / 22.  A caller that knows its routing to be skewed forces
// the tiled product.
constexpr int64_t kStreamRows = 16, kStreamPasses = 1024, kStreamGroupedPasses = 1280;
int choose_path(int64_t P, const Mx4Layout& L, bool grouped, uint32_t flags) {
  const bool fd = flags & MOE_FLAG_FORCE_DECODE, fp = flags & MOE_FLAG_FORCE_PREFILL;
  if ((flags & ~(MOE_FLAG_FORCE_DECODE | MOE_FLAG_FORCE_PREFILL)) != 0 || (fd && fp)) return -1;
  if (fd) return 0;
  if (fp) return 1;
  const int64_t passes = grouped ? P / 32 + (L.E + 1) / 2 : (P + 31) / 32;
  return P <= kStreamRows * L.E || passes * L.NT <= (grouped ? kStreamGroupedPasses : kStreamPasses) ? 0 : 1;
}

moe_status_t run_product(const Mx4Args& a, const Mx4Layout& L, int path, int32_t y_type, void* ws, hipStream_t stream) {
  const bool f32 = y_type == MOE_TYPE_FP32;
  return hip_status(path == 0 ? launch_mx4_stream(a, L, f32, stream) : launch_mx4_tiled(a, L, f32, ws, stream));
}

}  // namespace

moe_status_t moe::check_norm_before(const void* x, int32_t x_type, const void* w, int32_t w_type, int32_t T, int32_t H,
                                    float eps, const uint16_t* z, const uint8_t* q, const uint8_t* s, int32_t quant) {
  if (T < 0 || H < 1 || !(eps >= 0.0f) || isinf(eps)) return MOE_ERR_INVALID_ARGUMENT;
  if (!norm_type(x_type) || !norm_type(w_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (quant != MOE_QUANT_NONE && quant != MOE_QUANT_MXFP8 && quant != MOE_QUANT_MXFP4) return MOE_ERR_INVALID_ARGUMENT;
  if (H > kMaxNormH || H % 8 != 0 || (quant != MOE_QUANT_NONE && H % 32 != 0)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w || (quant == MOE_QUANT_NONE ? (!z || q || s) : (!q || !s))) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(z, 16) || !aligned(q, 16)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status_t moe::check_norm_after(const void* y, int32_t y_type, const void* residual, int32_t residual_type,
                                   const void* w_post, const void* w_next, int32_t w_type, const float* gate,
                                   int64_t gate_t, int64_t gate_h, float eps, int32_t T, int32_t H, const void* out,
                                   const uint16_t* z, const uint8_t* q, const uint8_t* s, int32_t quant) {
  if (T < 0 || H < 1 || !(eps >= 0.0f) || isinf(eps)) return MOE_ERR_INVALID_ARGUMENT;
  if (!norm_type(y_type) || !norm_type(residual_type) || !norm_type(w_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (quant != MOE_QUANT_NONE && quant != MOE_QUANT_MXFP8 && quant != MOE_QUANT_MXFP4) return MOE_ERR_INVALID_ARGUMENT;
  if (gate && (gate_t < 0 || gate_h < 0 || gate_h > 1)) return MOE_ERR_INVALID_ARGUMENT;
  if (H > kMaxNormH || H % 8 != 0 || (quant != MOE_QUANT_NONE && H % 32 != 0)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!y || !residual || !out) return MOE_ERR_INVALID_ARGUMENT;
  if (w_next ? (quant == MOE_QUANT_NONE ? (!z || q || s) : (!q || !s)) : (z || q || s || quant != MOE_QUANT_NONE))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(w_post, 16) || !aligned(w_next, 16) ||
      !aligned(gate, 4) || !aligned(z, 16) || !aligned(q, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

extern "C" {

moe_status_t moe_quant_mxfp4(const void* x, int32_t x_type, int32_t M, int32_t K, int64_t ldx, uint8_t* q, uint8_t* s,
                             hipStream_t stream) {
  if (M < 0 || K < 1 || ldx < K || !known_type(x_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 32 != 0 || too_many(M, K)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !q || !s || !aligned(x, 16) || !aligned(q, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (M > 1 && ldx % (x_type == MOE_TYPE_FP32 ? 4 : 8) != 0) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_mx4_quant(x, (ElemType)x_type, M, K, M == 1 ? K : (long)ldx, q, s, stream));
}

moe_status_t moe_dequant_mx(const uint8_t* q, const uint8_t* s, int32_t format, int32_t M, int32_t K, void* out,
                            int32_t out_type, hipStream_t stream) {
  if (M < 0 || K < 1 || !known_type(out_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (format != MOE_QUANT_MXFP8 && format != MOE_QUANT_MXFP4) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 32 != 0 || too_many(M, K)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  const bool fp4 = format == MOE_QUANT_MXFP4;
  if (!q || !s || !out || !aligned(q, fp4 ? 4 : 8) || !aligned(out, 16)) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_mx_dequant(q, s, fp4, M, K, out, (ElemType)out_type, stream));
}

size_t moe_mxfp4_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t glu) {
  if (check_enk(E, N, K, glu) != MOE_OK) return 0;
  return Mx4Layout(E, N, K, glu != 0).total;
}

moe_status_t moe_mxfp4_prepack(const uint8_t* wq, const uint8_t* ws, const uint8_t* uq, const uint8_t* us, int32_t E,
                               int32_t N, int32_t K, void* packed, size_t packed_bytes, moe_mxfp4_weights_t* desc,
                               hipStream_t stream) {
  const int32_t glu = uq != nullptr;
  moe_status_t st = check_enk(E, N, K, glu);
  if (st != MOE_OK) return st;
  if (!wq || !ws || (uq == nullptr) != (us == nullptr) || !packed || !desc) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(wq, 16) || !aligned(uq, 16) || !aligned(packed, 256)) return MOE_ERR_INVALID_ARGUMENT;
  const Mx4Layout L(E, N, K, glu != 0);
  if (packed_bytes < L.total) return MOE_ERR_INVALID_ARGUMENT;
  st = hip_status(launch_mx4_pack(wq, ws, uq, us, L, static_cast<uint8_t*>(packed), stream));
  if (st != MOE_OK) return st;
  desc->E = E;
  desc->N = N;
  desc->K = K;
  desc->glu = glu;
  desc->layout_version = MOE_MXFP4_LAYOUT_VERSION;
  desc->packed = packed;
  desc->packed_bytes = packed_bytes;
  return MOE_OK;
}

moe_status_t moe_mxfp4_dense_forward(const moe_mxfp4_weights_t* w, const uint8_t* xq, const uint8_t* xs, int32_t T,
                                     void* y, int32_t y_type, uint32_t flags, hipStream_t stream) {
  moe_status_t st = check_mx4_weights(w);
  if (st != MOE_OK) return st;
  if (w->E != 1 || T < 0 || !norm_type(y_type)) return MOE_ERR_INVALID_ARGUMENT;
  const Mx4Layout L(1, w->N, w->K, w->glu != 0);
  const int path = choose_path(T, L, false, flags);
  if (path < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (rows_too_large(T, w->K)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!xq || !xs || !y || !aligned(xq, 16) || !aligned(xs, 4) || !aligned(y, 16)) return MOE_ERR_INVALID_ARGUMENT;
  const Mx4Args a{static_cast<const uint8_t*>(w->packed), xq, xs, T, nullptr, nullptr, 1, T, y};
  return run_product(a, L, path, y_type, nullptr, stream);
}

size_t moe_mxfp4_grouped_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K, int32_t glu) {
  if (P < 0 || P > kMaxMx4P || check_enk(E, N, K, glu) != MOE_OK) return 0;
  return PackedLayout::align256(mx4_tiled_ws_bytes(P, E, K));
}

moe_status_t moe_mxfp4_grouped_forward(const moe_mxfp4_weights_t* w, const uint8_t* xq, const uint8_t* xs, int32_t X,
                                       const int32_t* offsets, const int32_t* rows, int32_t row_div, int32_t P,
                                       void* y, int32_t y_type, void* workspace, size_t workspace_bytes,
                                       uint32_t flags, hipStream_t stream) {
  moe_status_t st = check_mx4_weights(w);
  if (st != MOE_OK) return st;
  if (P < 0 || X < 0 || row_div < 1 || !norm_type(y_type)) return MOE_ERR_INVALID_ARGUMENT;
  const Mx4Layout L(w->E, w->N, w->K, w->glu != 0);
  const int path = choose_path(P, L, true, flags);
  if (path < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (rows_too_large(X, w->K) || P > kMaxMx4P) return MOE_ERR_UNSUPPORTED;
  if (P == 0) return MOE_OK;
  if (X < 1 || (!rows && X < P)) return MOE_ERR_INVALID_ARGUMENT;
  if (!xq || !xs || !offsets || !y) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(y, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  const size_t need = PackedLayout::align256(mx4_tiled_ws_bytes(P, w->E, w->K));
  if (!workspace || workspace_bytes < need) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
  const Mx4Args a{static_cast<const uint8_t*>(w->packed), xq, xs, X, offsets, rows, row_div, P, y};
  return run_product(a, L, path, y_type, workspace, stream);
}

moe_status_t moe_norm_before(const void* x, int32_t x_type, const void* w, int32_t w_type, int32_t T, int32_t H,
                             float eps, uint16_t* z, uint8_t* q, uint8_t* s, int32_t quant, hipStream_t stream) {
  moe_status_t st = check_norm_before(x, x_type, w, w_type, T, H, eps, z, q, s, quant);
  if (st != MOE_OK || T == 0) return st;
  NormArgs a{};
  a.y = x;
  a.w_next = w;
  a.eps = eps;
  a.z = z;
  a.q = q;
  a.s = s;
  a.quant = quant;
  a.y_type = (ElemType)x_type;
  a.w_type = (ElemType)w_type;
  a.T = T;
  a.H = H;
  return hip_status(launch_norm(a, stream));
}

moe_status_t moe_norm_after(const void* y, int32_t y_type, const void* residual, int32_t residual_type,
                            const void* w_post, const void* w_next, int32_t w_type, const float* gate, int64_t gate_t,
                            int64_t gate_h, float alpha, float beta, float eps, int32_t T, int32_t H, void* out,
                            uint16_t* z, uint8_t* q, uint8_t* s, int32_t quant, hipStream_t stream) {
  moe_status_t st = check_norm_after(y, y_type, residual, residual_type, w_post, w_next, w_type, gate, gate_t, gate_h,
                                     eps, T, H, out, z, q, s, quant);
  if (st != MOE_OK || T == 0) return st;
  NormArgs a{};
  a.y = y;
  a.res = residual;
  a.w_post = w_post;
  a.gate = gate;
  a.gate_t = gate_t;
  a.gate_h = gate_h;
  a.alpha = alpha;
  a.beta = beta;
  a.eps = eps;
  a.out = out;
  a.w_next = w_next;
  a.z = z;
  a.q = q;
  a.s = s;
  a.quant = quant;
  a.y_type = (ElemType)y_type;
  a.res_type = (ElemType)residual_type;
  a.w_type = (ElemType)w_type;
  a.T = T;
  a.H = H;
  return hip_status(launch_norm(a, stream));
}

}  // extern "C"
