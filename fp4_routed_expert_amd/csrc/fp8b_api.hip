// C ABI of the FP8 operators with block scales (declared in
// include/moe_fp8_block.h): host-side argument checks and path selection.  Every
// check runs before any launch, so a failing call enqueues nothing and touches no
// output.
#include "api.h"
#include "fp8b.h"

using namespace moe;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }
bool known_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_FP16 || t == MOE_TYPE_FP32; }
bool sum_type(int32_t t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_FP32; }

constexpr int kMaxE = 1024;
// A tile past the last row still counts in 32 bits; the streaming product's passes step by next_pass.
constexpr int kMaxP = INT32_MAX - 256;

// (one workgroup per 16 rows and 4 blocks)
bool too_many(int32_t M, int32_t K) { return M > kMaxP || K > (1 << 20); }

moe_status_t check_enk(int32_t E, int32_t N, int32_t K, int32_t glu) {
  if (E < 1 || N < 1 || K < 1 || (glu != 0 && glu != 1)) return MOE_ERR_INVALID_ARGUMENT;
  if (E > kMaxE || N % 32 != 0 || K % 128 != 0 || N > (1 << 20) || K > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  // packing runs one thread per 16 bytes and per scale, the latter in one launch dimension
  if (Fp8bLayout(E, N, K, glu).s_off > (size_t)1 << 42) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status_t check_weights(const moe_fp8_block_weights_t* w, int32_t glu) {
  if (!w || !w->packed || w->layout_version != MOE_FP8_BLOCK_LAYOUT_VERSION || w->glu != glu)
    return MOE_ERR_INVALID_ARGUMENT;
  const moe_status_t st = check_enk(w->E, w->N, w->K, w->glu);
  if (st != MOE_OK) return st;
  if (!aligned(w->packed, 256) || w->packed_bytes < Fp8bLayout(w->E, w->N, w->K, glu != 0).total)
    return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

// The tiled product addresses activation rows by 32-bit byte offsets.
bool rows_too_large(int32_t X, int32_t K) { return (int64_t)X * K > ((int64_t)1 << 32) - 4096; }

// The rows up to which a call streams the weights by default (figures: us,
// streaming against tiled).
// - While the groups average at most 12 rows.  64 experts, SwiGLU K 4096 N 1536, 6 rows
//   119 and 142, 12 rows 145 and 146, 24 rows 181 and 148; 256 experts, K 7168 N 2048, 8
//   rows 1202 and 1277, 16 rows 1830 and 1320.  The backward call 6 rows: evenly routed
//   it gains up to 12 (64 experts, K 4096 N 2048, 6 rows 84 and 100, 8 rows 88 and 102, 12
//   rows 103 and 102; 256 experts, K 7168 N 2048, 7 rows 579 and 638, 12 rows 663 and 645),
//   but skewed by Zipf's law it loses more (8 rows on average 96 and 78, 12 rows 128 and
//   78; 256 experts, 7 rows 425 and 209, 12 rows 718 and 244).
// - While streaming makes at most 2048 passes of 32 rows over a weight tile, eight per
//   CU: the tiled product has few items then.  Dense: K 4096 N 1536, 512 rows (1536
//   passes) 20 and 27, 768 rows (2304) 30 and 27; K 16384 N 7168, 128 rows (1792) 80 and
//   120, 160 rows (2240) 125 and 116; K 7168 N 2048, 512 rows (2048) 38 and 43; K 512 N
//   7168, 128 rows (1792) 6.8 and 9.0, 160 rows (2240) 9.0 and 9.0.
// - Grouped, where the tiled product lists its tiles first, up to 2400 (a group's last
//   pass counted half): 8 experts, K 512 N 512, 2272 rows (2400) 7.7 and 11.8; 30 experts,
//   K 1024 N 1024, 704 rows (2368) 9.0 and 13.3, 992 rows (2944) 14.8 and 14.2; 16
//   experts, K 2048 N 512, 2144 rows (2400) 21.0 and 19.6; 8 experts, K 4096 N 4096, 160
//   rows (2304) 24 and 34, 320 rows (3584) 49 and 36.  Off by 10 % or more: 4 experts,
//   K 7168 N 2048, 512 rows (2304) 59 and 46; 8 experts, K 4096 N 4096, 224 rows (2816)
//   27 and 34; 8 and 64 experts, K 512, 2976 passes 10 and 12, 9 and 11.
// - Where the sums stay in fp32 the tiled product is half as fast.  Dense, up to four
//   rounds of the CUs of 64-row passes over a pair of tiles: K 4096 N 1536, 1344 rows (1008
//   passes) 49 and 53, 1440 rows (1104) 60 and 53; K 16384 N 4096, 512 rows (1024) 171 and
//   186, 544 rows (1152) 199 and 187; K 2048 N 2048, 1024 rows (1024) 24 and 30.  Half a
//   round more for short K, whose workgroups overlap: K 1024 N 4096, 576 rows (1152) 16 and
//   19; K 2048 N 7168, 288 rows (1120) 28 and 31, 352 rows (1344) 34 and 31; K 3584 N 7168,
//   288 rows (1120) 48 and 47.  Or at most 3584 passes of 32 rows, where half of a last
//   one of 64 would be empty: K 4096, N 36864, 32 rows (2304) 36 and 40, N 11264, 160 rows
//   (3520) 49 and 53, N 18432, 96 rows (3456) 50 and 52, N 48000, 32 rows (3000) 44 and
//   43.  (Off by 10 % or more: K 4096 N 57344, 32 rows (3584) 51 and 46; K 256 N 1024,
//   2432 rows (1216) 9.0 and 10.4; K 1024 N 4096, 608 rows (1280) 17.5 and 19.3.)
// - Grouped in fp32 up to 3000 passes of 32 rows, for short K 3584: 4 experts, K 7168 N
//   2048, 672 rows (2944) 89 and 88, 832 rows (3584) 111 and 89; 16 experts, K 2048 N 512,
//   2720 rows (2976) 32 and 33, 3328 rows (3584) 39 and 33; 8 experts, K 512 N 512, 3456
//   rows (3584) 9.4 and 16.3; 30 experts, K 1024 N 1024, 1312 rows (3584) 17 and 21.  (Evenly
//   routed short K gains up to 4200 passes, 10 and 16.5, 18 and 22; skewed it would not.)
// The averages do not see skew, which only the device knows: streaming walks a
// group's rows 16 or 32 at a time, by one workgroup per tile pair once the groups'
// tiles fill the CUs (64 experts, K 1536 N 4096, 512 rows in one of them: 58 and 18).  A
// caller that knows its routing to be skewed forces the tiled product.
int64_t streamed_rows(const Fp8bLayout& L, Fp8bOut out, bool grouped) {
  const bool fp32 = out == Fp8bOut::kFp32;
  int64_t few;
  if (grouped) {  // P / 32 + (E + 1) / 2 passes, times NT
    const int64_t most = !fp32 ? 2400 : L.K < 2048 ? 3584 : 3000;
    few = 32 * (most / L.NT - (L.E + 1) / 2) + 31;
  } else if (fp32) {
    const int64_t wide = 64 * ((L.K <= 2048 ? 1152 : 1024) / (L.NT / 2)), narrow = 32 * (3584 / L.NT);
    few = wide > narrow ? wide : narrow;
  } else {
    few = 32 * (2048 / L.NT);
  }
  const int64_t rows = (out == Fp8bOut::kGluGrad ? 6 : 12) * (int64_t)L.E;
  return few > rows ? few : rows;
}

// 0: stream the weights, 1: tiled, -1: bad flags.
int choose_path(int64_t P, const Fp8bLayout& L, Fp8bOut out, bool grouped, uint32_t flags) {
  const bool fd = flags & MOE_FLAG_FORCE_DECODE, fp = flags & MOE_FLAG_FORCE_PREFILL;
  if ((flags & ~(MOE_FLAG_FORCE_DECODE | MOE_FLAG_FORCE_PREFILL)) != 0 || (fd && fp)) return -1;
  if (fd) return 0;
  if (fp) return 1;
  return P <= streamed_rows(L, out, grouped) ? 0 : 1;
}

size_t tiled_bytes(int32_t P, int32_t E) { return PackedLayout::align256(fp8b_tiled_ws_bytes(P, E)); }

// Workspace of the calls whose rows are quantised: where the weights are streamed, fp32 rows.
size_t rows_bytes(int64_t P, const Fp8bLayout& L, int path) {
  return path == 0 ? PackedLayout::align256((size_t)P * L.N * 4) : tiled_bytes((int32_t)P, L.E);
}

// The same for P rows or fewer.  (Few rows that are streamed need more than many that are not, and a program keeps
// one workspace for both: 250 experts, N 2048, flags 0, 3000 rows 25 MB, 3001 rows by themselves 18 KB.)
size_t rows_bytes_up_to(int64_t P, const Fp8bLayout& L, Fp8bOut out, uint32_t flags) {
  const int path = choose_path(P, L, out, true, flags);
  const size_t own = rows_bytes(P, L, path);
  if (path == 0 || flags != 0) return own;
  const size_t streamed = rows_bytes(streamed_rows(L, out, true), L, 0);
  return own > streamed ? own : streamed;
}

// One size for the forward and the backward call, which may take different paths (twice the tiles with gate and up).
size_t glu_bytes(int32_t P, int32_t E, int32_t N, int32_t K, uint32_t flags) {
  const Fp8bLayout one(E, N, K, false), two(E, N, K, true);
  if (choose_path(P, one, Fp8bOut::kGluGrad, true, flags) < 0) return 0;
  const size_t a = rows_bytes_up_to(P, one, Fp8bOut::kGluGrad, flags), b = rows_bytes_up_to(P, two, Fp8bOut::kGlu, flags);
  return a > b ? a : b;
}

// What the grouped calls share: rows and offsets.
moe_status_t check_rows(int32_t X, const int32_t* offsets, const int32_t* rows, int32_t P, int32_t E) {
  if (X < 1 || (!rows && X < P)) return MOE_ERR_INVALID_ARGUMENT;
  if (!offsets && (E != 1 || rows)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(offsets, 4) || !aligned(rows, 4)) return MOE_ERR_INVALID_ARGUMENT;
  return MOE_OK;
}

moe_status_t run(const Fp8bArgs& a, const Fp8bLayout& L, int path, Fp8bOut out, void* ws, hipStream_t stream) {
  return hip_status(path == 0 ? launch_fp8b_stream(a, L, out, static_cast<float*>(ws), stream)
                              : launch_fp8b_tiled(a, L, out, ws, stream));
}

moe_status_t prepack(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us, int32_t E, int32_t N,
                     int32_t K, bool transposed, void* packed, size_t packed_bytes, moe_fp8_block_weights_t* desc,
                     hipStream_t stream) {
  const int32_t glu = uq != nullptr && !transposed;
  moe_status_t st = check_enk(E, N, K, glu);
  if (st != MOE_OK) return st;
  if (transposed && (N % 128 != 0 || (uq && K % 256 != 0))) return MOE_ERR_UNSUPPORTED;
  if (!wq || !ws || (uq == nullptr) != (us == nullptr) || !packed || !desc) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(wq, 16) || !aligned(uq, 16) || !aligned(ws, 4) || !aligned(us, 4) || !aligned(packed, 256))
    return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bLayout L(E, N, K, glu != 0);
  if (packed_bytes < L.total) return MOE_ERR_INVALID_ARGUMENT;
  st = hip_status(launch_fp8b_pack(wq, ws, uq, us, L, transposed, static_cast<uint8_t*>(packed), stream));
  if (st != MOE_OK) return st;
  desc->E = E;
  desc->N = N;
  desc->K = K;
  desc->glu = glu;
  desc->layout_version = MOE_FP8_BLOCK_LAYOUT_VERSION;
  desc->packed = packed;
  desc->packed_bytes = packed_bytes;
  return MOE_OK;
}

// moe_fp8_block_glu_forward and moe_fp8_block_glu_backward
moe_status_t gated(const moe_fp8_block_weights_t* w, Fp8bOut out, const uint8_t* xq, const float* xs, int32_t X,
                   const int32_t* offsets, const int32_t* rows, int32_t row_div, int32_t P, uint8_t* q, float* s,
                   uint16_t* gate, uint16_t* up, void* workspace, size_t workspace_bytes, uint32_t flags,
                   hipStream_t stream) {
  const bool grad = out == Fp8bOut::kGluGrad;
  moe_status_t st = check_weights(w, grad ? 0 : 1);
  if (st != MOE_OK) return st;
  if (P < 0 || X < 0 || row_div < 1) return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bLayout L(w->E, w->N, w->K, w->glu != 0);
  const int path = choose_path(P, L, out, true, flags);
  if (path < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (w->N % 128 != 0 || rows_too_large(X, w->K) || P > kMaxP) return MOE_ERR_UNSUPPORTED;
  if (P == 0) return MOE_OK;
  st = check_rows(X, offsets, rows, P, w->E);
  if (st != MOE_OK) return st;
  if (!xq || !xs || !q || !s || (gate == nullptr) != (up == nullptr) || (grad && !gate)) return MOE_ERR_INVALID_ARGUMENT;
  if (!aligned(xq, 16) || !aligned(xs, 4) || !aligned(q, 8) || !aligned(s, 4) || !aligned(gate, 16) || !aligned(up, 16))
    return MOE_ERR_INVALID_ARGUMENT;
  if (!workspace || workspace_bytes < rows_bytes(P, L, path)) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bArgs a{static_cast<const uint8_t*>(w->packed), xq, xs, X, offsets, rows, row_div, P, nullptr, q, s, gate, up};
  return run(a, L, path, out, workspace, stream);
}

}  // namespace

extern "C" {

moe_status_t moe_quant_fp8_block(const void* x, int32_t x_type, int32_t M, int32_t K, int64_t ldx, uint8_t* q, float* s,
                                 hipStream_t stream) {
  if (M < 0 || K < 1 || ldx < K || !known_type(x_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 128 != 0 || too_many(M, K)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !q || !s || !aligned(x, 16) || !aligned(q, 8) || !aligned(s, 4)) return MOE_ERR_INVALID_ARGUMENT;
  if (M > 1 && ldx % (x_type == MOE_TYPE_FP32 ? 4 : 8) != 0) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_fp8b_quant(x, (ElemType)x_type, M, K, M == 1 ? K : (long)ldx, q, s, stream));
}

moe_status_t moe_dequant_fp8_block(const uint8_t* q, const float* s, int32_t M, int32_t K, void* out, int32_t out_type,
                                   hipStream_t stream) {
  if (M < 0 || K < 1 || !known_type(out_type)) return MOE_ERR_INVALID_ARGUMENT;
  if (K % 128 != 0 || too_many(M, K)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!q || !s || !out || !aligned(q, 8) || !aligned(s, 4) || !aligned(out, 16)) return MOE_ERR_INVALID_ARGUMENT;
  return hip_status(launch_fp8b_dequant(q, s, M, K, out, (ElemType)out_type, stream));
}

size_t moe_fp8_block_packed_bytes(int32_t E, int32_t N, int32_t K, int32_t glu) {
  if (check_enk(E, N, K, glu) != MOE_OK) return 0;
  return Fp8bLayout(E, N, K, glu != 0).total;
}

moe_status_t moe_fp8_block_prepack(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us, int32_t E,
                                   int32_t N, int32_t K, void* packed, size_t packed_bytes,
                                   moe_fp8_block_weights_t* desc, hipStream_t stream) {
  return prepack(wq, ws, uq, us, E, N, K, false, packed, packed_bytes, desc, stream);
}

moe_status_t moe_fp8_block_prepack_t(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us, int32_t E,
                                     int32_t N, int32_t K, void* packed, size_t packed_bytes,
                                     moe_fp8_block_weights_t* desc, hipStream_t stream) {
  return prepack(wq, ws, uq, us, E, N, K, true, packed, packed_bytes, desc, stream);
}

moe_status_t moe_fp8_block_dense_forward(const moe_fp8_block_weights_t* w, const uint8_t* xq, const float* xs, int32_t T,
                                         void* y, int32_t y_type, uint32_t flags, hipStream_t stream) {
  moe_status_t st = check_weights(w, 0);
  if (st != MOE_OK) return st;
  if (w->E != 1 || T < 0 || !sum_type(y_type)) return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bLayout L(1, w->N, w->K, false);
  const Fp8bOut out = y_type == MOE_TYPE_FP32 ? Fp8bOut::kFp32 : Fp8bOut::kBf16;
  const int path = choose_path(T, L, out, false, flags);
  if (path < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (rows_too_large(T, w->K) || T > kMaxP) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!xq || !xs || !y || !aligned(xq, 16) || !aligned(xs, 4) || !aligned(y, 16)) return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bArgs a{static_cast<const uint8_t*>(w->packed), xq, xs, T, nullptr, nullptr, 1, T, y, nullptr, nullptr,
                   nullptr, nullptr};
  return run(a, L, path, out, nullptr, stream);
}

size_t moe_fp8_block_grouped_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K) {
  if (P < 0 || P > kMaxP || check_enk(E, N, K, 0) != MOE_OK) return 0;
  return tiled_bytes(P, E);
}

moe_status_t moe_fp8_block_grouped_forward(const moe_fp8_block_weights_t* w, const uint8_t* xq, const float* xs,
                                           int32_t X, const int32_t* offsets, const int32_t* rows, int32_t row_div,
                                           int32_t P, void* y, int32_t y_type, void* workspace, size_t workspace_bytes,
                                           uint32_t flags, hipStream_t stream) {
  moe_status_t st = check_weights(w, 0);
  if (st != MOE_OK) return st;
  if (P < 0 || X < 0 || row_div < 1 || !sum_type(y_type)) return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bLayout L(w->E, w->N, w->K, false);
  const Fp8bOut out = y_type == MOE_TYPE_FP32 ? Fp8bOut::kFp32 : Fp8bOut::kBf16;
  const int path = choose_path(P, L, out, true, flags);
  if (path < 0) return MOE_ERR_INVALID_ARGUMENT;
  if (rows_too_large(X, w->K) || P > kMaxP) return MOE_ERR_UNSUPPORTED;
  if (P == 0) return MOE_OK;
  if (!offsets) return MOE_ERR_INVALID_ARGUMENT;
  st = check_rows(X, offsets, rows, P, w->E);
  if (st != MOE_OK) return st;
  if (!xq || !xs || !y || !aligned(xq, 16) || !aligned(xs, 4) || !aligned(y, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (!workspace || workspace_bytes < tiled_bytes(P, w->E)) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
  const Fp8bArgs a{static_cast<const uint8_t*>(w->packed), xq, xs, X, offsets, rows, row_div, P, y, nullptr, nullptr,
                   nullptr, nullptr};
  return run(a, L, path, out, workspace, stream);
}

size_t moe_fp8_block_glu_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K, uint32_t flags) {
  if (P < 0 || P > kMaxP || check_enk(E, N, K, 0) != MOE_OK) return 0;
  return glu_bytes(P, E, N, K, flags);
}

moe_status_t moe_fp8_block_glu_forward(const moe_fp8_block_weights_t* w, const uint8_t* xq, const float* xs, int32_t X,
                                       const int32_t* offsets, const int32_t* rows, int32_t row_div, int32_t P,
                                       uint8_t* q, float* s, uint16_t* gate, uint16_t* up, void* workspace,
                                       size_t workspace_bytes, uint32_t flags, hipStream_t stream) {
  return gated(w, Fp8bOut::kGlu, xq, xs, X, offsets, rows, row_div, P, q, s, gate, up, workspace, workspace_bytes, flags,
               stream);
}

moe_status_t moe_fp8_block_glu_backward(const moe_fp8_block_weights_t* w, const uint8_t* yq, const float* ys, int32_t X,
                                        const int32_t* offsets, const int32_t* rows, int32_t row_div, int32_t P,
                                        const uint16_t* gate, const uint16_t* up, uint8_t* q, float* s, void* workspace,
                                        size_t workspace_bytes, uint32_t flags, hipStream_t stream) {
  return gated(w, Fp8bOut::kGluGrad, yq, ys, X, offsets, rows, row_div, P, q, s, const_cast<uint16_t*>(gate),
               const_cast<uint16_t*>(up), workspace, workspace_bytes, flags, stream);
}

size_t moe_fp8_block_weight_grad_workspace_size(int32_t P, int32_t E, int32_t N, int32_t K) {
  if (P < 0 || P > kMaxP || check_enk(E, N, K, 0) != MOE_OK || N % 128 != 0) return 0;
  return PackedLayout::align256(fp8b_grad_ws_bytes(P, E, N, K));
}

moe_status_t moe_fp8_block_weight_grad(const uint8_t* yq, const float* ys, const uint8_t* xq, const float* xs, int32_t X,
                                       const int32_t* offsets, const int32_t* rows, int32_t row_div, int32_t P,
                                       int32_t E, int32_t N, int32_t K, void* dw, int32_t dw_type, void* workspace,
                                       size_t workspace_bytes, hipStream_t stream) {
  moe_status_t st = check_enk(E, N, K, 0);
  if (st != MOE_OK) return st;
  if (P < 0 || X < 0 || row_div < 1 || !sum_type(dw_type)) return MOE_ERR_INVALID_ARGUMENT;
  // one workgroup of 512 threads per 256 x 256 outputs (a last tile may be half of one), in multiples of eight:
  // below 2^32 threads
  const int64_t tiles = (int64_t)((N + 255) / 256) * ((K + 255) / 256);
  if (N % 128 != 0 || P > kMaxP || tiles > (1 << 23) - 8) return MOE_ERR_UNSUPPORTED;
  if (!dw || !aligned(dw, 16)) return MOE_ERR_INVALID_ARGUMENT;
  if (P > 0) {
    st = check_rows(X, offsets, rows, P, E);
    if (st != MOE_OK) return st;
    if (!yq || !ys || !xq || !xs || !aligned(yq, 16) || !aligned(xq, 16) || !aligned(ys, 4) || !aligned(xs, 4))
      return MOE_ERR_INVALID_ARGUMENT;
  }
  const size_t need = PackedLayout::align256(fp8b_grad_ws_bytes(P, E, N, K));
  if (P > 0 && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARGUMENT;
  // without rows nothing is read: dw is zeros
  const Fp8bGradArgs a{yq, ys, xq, xs, X, P > 0 ? offsets : nullptr, rows, row_div, P, E, N, K, dw};
  return hip_status(launch_fp8b_grad(a, dw_type == MOE_TYPE_FP32, workspace, stream));
}

}  // extern "C"
