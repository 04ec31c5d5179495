// FP8 operators with a scale for each block of 128: the packed layout of their
// weights, the device helpers that their kernels share, and the launchers that
// fp8b_api.hip calls.
#pragma once

#include "common.h"
#include "mx4.h"

namespace moe {

// ------------------------------------------------------------ packed weights
// One tile is an operand of v_mfma_f32_16x16x128_f8f6f4: 16 weight rows x 128 K
// (one scale block of K), 2 KiB.  Lane l = 16 g + r holds row r's K [16 g, +16)
// in the first KiB and [64 + 16 g, +16) in the second, so that a lane's share of
// an activation row is two 16-byte pieces of its 128 bytes.  (Which K a lane
// holds is free as long as both operands agree.)  A tile's K-steps are
// consecutive.
//
// Weights are the A operand: a lane ends with four consecutive weight rows
// 4 g + v of one token.  Tiles come in pairs whose rows interleave so that a
// lane's two tiles are eight neighbouring output columns: row i of tile t of a
// pair of 32 columns is column 8 (i / 4) + 4 t + i % 4.  With gate and up, tiles
// alternate gate, up; the two gate tiles of a group of four interleave in that
// way, and the two up tiles.
//
// Scales: [expert][row block][K-step] fp32, a row block being 128 weight rows;
// with gate and up row blocks alternate gate, up.
struct Fp8bLayout {
  int E, N, K, J;  // J = K / 128
  int NT, NB;      // tiles and row blocks of an expert
  bool glu;
  size_t s_off, total;
  __host__ __device__ Fp8bLayout(int E_, int N_, int K_, bool glu_)
      : E(E_), N(N_), K(K_), J(K_ / 128), NT(N_ / 16 * (glu_ ? 2 : 1)), NB((N_ + 127) / 128 * (glu_ ? 2 : 1)), glu(glu_) {
    s_off = (size_t)E * NT * J * 2048;
    total = PackedLayout::align256(s_off + (size_t)E * NB * J * 4);
  }
  __host__ __device__ size_t tile_off(int e, int nt) const { return ((size_t)e * NT + nt) * J * 2048; }
  // output column of row i of tile nt
  __host__ __device__ int column(int nt, int i) const {
    const int p = glu ? nt >> 1 : nt;
    return 32 * (p >> 1) + 8 * (i >> 2) + 4 * (p & 1) + (i & 3);
  }
};

// D = A B of one block of 128: A 16 weight rows, B 16 tokens, unscaled e4m3.
// Lane l's element v is weight row 4 (l / 16) + v of token l % 16.  The FP8 matrix
// cores add the products of eight neighbouring elements with about 14 bits below
// the largest (measured: 2^16 + 2^2 is 2^16), so that a sum of a block of normal
// values is off by 1.5e-5 of its size: nothing beside a rounding to bf16 or e4m3,
// too much for results that stay in fp32.
__device__ __forceinline__ v4f mfma_block(v8i w, v8i x) {
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, v4f{0.f, 0.f, 0.f, 0.f}, 0, 0, 0, 0, 0, 0);
}

__device__ __forceinline__ v8i cat_pieces(v4u lo, v4u hi) {
  return v8i{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
}

// The same sum with every product exact, for those: the codes as bf16 values
// (exact), four MFMAs of 32 K each, at half the rate.
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
struct Wide {
  v4u k[4];
};
__device__ __forceinline__ Wide widen(v8i c) {
  Wide w;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    w.k[i >> 1][2 * (i & 1)] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, false));
    w.k[i >> 1][2 * (i & 1) + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[i], 1.0f, true));
  }
  return w;
}
__device__ __forceinline__ v4f mfma_wide(const Wide& w, const Wide& x) {
  v4f d = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, w.k[i]), __builtin_bit_cast(v8bf, x.k[i]), d, 0, 0, 0);
  return d;
}

// ------------------------------------------------------------- quantisation
// Scale of a block whose largest magnitude has the bits `top` (NaN and infinity
// order above every number), and what its values are multiplied by.
struct BlockScale {
  float scale, mul;
};
__device__ __forceinline__ BlockScale block_scale(uint32_t top) {
  const bool bad = top >= 0x7F800000u;
  const float a = fmaxf(bad ? 1.0f : __uint_as_float(top), 0x1p-110f);
  return {bad ? __uint_as_float(0x7FC00000u) : a / 448.0f, 448.0f / a};
}
// Four codes; zero where the block holds a NaN or an infinity.
__device__ __forceinline__ uint32_t block_codes(float a, float b, float c, float d, const BlockScale& k) {
  const uint32_t w = f32x4_to_e4m3(a * k.mul, b * k.mul, c * k.mul, d * k.mul);
  return k.scale != k.scale ? 0u : w;
}
__device__ __forceinline__ uint32_t magnitude_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Maximum over lanes l, l^16, l^32, l^48, of bit patterns.
__device__ __forceinline__ uint32_t max_lanes_xor16_32_u32(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}
// Maximum over each row of 16 lanes.
__device__ __forceinline__ uint32_t row16_max_u32(uint32_t v) {
  v = quad_max_u32(v);
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));
}

// Backward of silu(g) u for the gradient dh: dg and du.  sig = 1 / (1 + e^-g) as
// in glu_out (mx4.h); 1 - sig keeps its precision near 1 as e^-g sig.  Below g =
// -87.3 sig is 0, as |g| e^g < 2^-118 is: a sig that stays at 2^-126 would be
// multiplied by gates of any size.
__device__ __forceinline__ void glu_grad(float dh, float g, float u, float& dg, float& du) {
  const float t = __builtin_amdgcn_exp2f(fminf(g * -1.44269504f, 126.0f));  // e^-g
  const float sig = t < 0x1p126f ? __builtin_amdgcn_rcpf(1.0f + t) : 0.0f;
  du = dh * (g * sig);
  dg = dh * u * (sig * (1.0f + g * (t * sig)));
}

// ---------------------------------------------------------------- launchers
hipError_t launch_fp8b_quant(const void* x, ElemType type, long M, int K, long ldx, uint8_t* q, float* s,
                             hipStream_t st);
hipError_t launch_fp8b_dequant(const uint8_t* q, const float* s, long M, int K, void* out, ElemType type,
                               hipStream_t st);
// transposed: wq (and uq) are [E, K, N]; uq then follows wq along K
hipError_t launch_fp8b_pack(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us,
                            const Fp8bLayout& L, bool transposed, uint8_t* packed, hipStream_t st);

// What becomes of a product's sums.
enum class Fp8bOut : int { kBf16, kFp32, kGlu, kGluGrad };

// A product's activations and outputs.  offsets == nullptr: one group of P rows.
// rows == nullptr: row s reads x row s, else row rows[s] / div.
struct Fp8bArgs {
  const uint8_t* packed;
  const uint8_t* xq;
  const float* xs;
  int X;  // rows of x
  const int32_t* offsets;
  const int32_t* rows;
  int div;
  int P;  // rows of the outputs
  void* y;         // kBf16, kFp32: the sums
  uint8_t* q;      // kGlu, kGluGrad: codes and scales
  float* s;
  uint16_t* gate;  // kGlu: written, or null; kGluGrad: read
  uint16_t* up;
};
// ws: fp32 rows [P, N] of kGlu and kGluGrad
hipError_t launch_fp8b_stream(const Fp8bArgs& a, const Fp8bLayout& L, Fp8bOut out, float* ws, hipStream_t st);
size_t fp8b_tiled_ws_bytes(long P, int E);
hipError_t launch_fp8b_tiled(const Fp8bArgs& a, const Fp8bLayout& L, Fp8bOut out, void* ws, hipStream_t st);
// Quantisation of fp32 rows h [P, N] (kGlu), or of glu_grad(h, gate, up) (kGluGrad), rows offsets[0] to offsets[E].
hipError_t launch_fp8b_rows(const float* h, const Fp8bArgs& a, int E, int N, Fp8bOut out, hipStream_t st);

struct Fp8bGradArgs {
  const uint8_t* yq;
  const float* ys;
  const uint8_t* xq;
  const float* xs;
  int X;
  const int32_t* offsets;
  const int32_t* rows;
  int div;
  int P, E, N, K;
  void* dw;
};
// The x row of entry p of `rows`: past the last one (negative entries too) the last.
__device__ __forceinline__ int entry_row(const int32_t* rows, int p, int div, int X) {
  return (int)min((uint32_t)rows[p] / (uint32_t)div, (uint32_t)(X - 1));
}
size_t fp8b_grad_ws_bytes(long P, int E, int N, int K);
hipError_t launch_fp8b_grad(const Fp8bGradArgs& a, bool fp32_out, void* ws, hipStream_t st);

}  // namespace moe
