// MXFP4 operators: the packed layout of their weights, the device helpers
// that their kernels share, and the launchers that mx4_api.hip calls.
#pragma once

#include "common.h"

namespace moe {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef float v16f __attribute__((ext_vector_type(16)));

// Element types of the C ABI (moe_mx4.h).
enum class ElemType : int { kBf16 = 0, kFp16 = 1, kFp32 = 2 };

// ------------------------------------------------------------ packed weights
// One tile is the B operand of two v_mfma_scale_f32_32x32x64_f8f6f4: 32 weight
// rows x 128 K, 2 KiB.  Lane l = 32 g + n of K-half s (s = 0, 1) holds 16
// consecutive bytes: row n's K block 2 g + s of the step (a block is the 32
// elements of one scale), so that a lane's two blocks are neighbours: a token
// row's 64 bytes of a step are read as two 16-byte pieces at 32 g, and its
// two scale bytes as one 16-bit word.  (Which K a lane holds is free as long
// as both operands agree.)  A tile's K-steps are consecutive; an odd number of
// them is followed by one of zeros.
//
// Columns: tiles come in groups of four, which one wave of the tiled kernel
// multiplies.  The f tiles of a group (f = 4, fewer in the last) interleave
// their columns: row n of tile t is output column 128 group + f n + t, so
// that a lane ends with f neighbouring outputs of a token.  With the SwiGLU
// form the tiles alternate gate, up, gate, up; the two pairs of a group
// interleave their 32 columns in the same way.
//
// Scales: per group of four tiles and pair of K-steps 1 KiB,
// [lane][step][tile][2]: a lane's bytes are the scales of its blocks of K-halves
// 0 and 1, so that one 128-bit read serves four tiles for two steps.  Tiles
// that the last group lacks leave their bytes unused.
struct Mx4Layout {
  int E, N, K, J, D;  // J = K / 128 K-steps, D pairs of them
  int NT, NG;         // 32-row tiles of an expert, groups of four
  bool glu;
  size_t s_off, total;
  __host__ __device__ Mx4Layout(int E_, int N_, int K_, bool glu_)
      : E(E_), N(N_), K(K_), J(K_ / 128), D((J + 1) / 2), NT(N_ / 32 * (glu_ ? 2 : 1)), NG((NT + 3) / 4), glu(glu_) {
    s_off = (size_t)E * NT * D * 4096;
    total = PackedLayout::align256(s_off + (size_t)E * NG * D * 1024);
  }
  __host__ __device__ size_t tile_off(int e, int nt) const { return ((size_t)e * NT + nt) * D * 4096; }
  // scales of group q; the next pair of K-steps is 1024 further
  __host__ __device__ size_t scale_off(int e, int q) const { return s_off + ((size_t)e * NG + q) * D * 1024; }
  // output column of row n of tile nt
  __host__ __device__ int column(int nt, int n) const {
    if (glu) {
      const int p = nt >> 1, u = p >> 1, left = N / 32 - 2 * u, f = left < 2 ? left : 2;
      return 64 * u + f * n + (p & 1);
    }
    const int q = nt >> 2, left = NT - 4 * q, f = left < 4 ? left : 4;
    return 128 * q + f * n + (nt & 3);
  }
};

// One MFMA of 32 token rows x 32 weight rows x 64 K, both operands e2m1 (A:
// lane l = 32 g + r holds token r's K block g; B likewise; D: lane l's element
// v is token 8 (v / 4) + 4 (l / 32) + v % 4 of weight row l % 32), each lane's
// scale byte kA of sa and kB of sb.
template <int kA, int kB>
__device__ __forceinline__ v16f mfma_fp4(v4u a, v4u b, v16f c, uint32_t sa, uint32_t sb) {
  const v4i ai = __builtin_bit_cast(v4i, a), bi = __builtin_bit_cast(v4i, b);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
      __builtin_shufflevector(ai, ai, 0, 1, 2, 3, -1, -1, -1, -1),
      __builtin_shufflevector(bi, bi, 0, 1, 2, 3, -1, -1, -1, -1), c, 4, 4, kA, (int)sa, kB, (int)sb);
}

// SiLU(g) u.  The exponential comes straight from the exp2 instruction, whose
// results below 2^-126 are 0 here, as 1 + them is 1 anyway; SiLU first, so that
// a product g u past fp32's range does not meet a sigmoid of zero.  Its argument
// is rounded to 2^-24 of its size (|g| 2^-24 of the result), it and the
// reciprocal are good to an ulp: under (|g| + 8) 2^-22 in all, which bf16 does not
// see for any gate that is not closed.  Below g = -87 the reciprocal of 1 + 2^126
// and more is 0.
__device__ __forceinline__ float glu_out(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f)) * u;
}

// ------------------------------------------------------------------- MXFP4
// Maximum over each quad of 4 lanes (as quad_max, on bit patterns: the bits of
// magnitudes order as the magnitudes do, infinity and then NaN above them).
__device__ __forceinline__ uint32_t quad_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));
}

// Eight elements of a block whose largest magnitude has the bits amax: their
// codes (element i in nibble i) and the block's scale code.  Where the scale
// would be below 2^-127 it stays there; the product v 2^-X is exact unless it
// is too small to round to anything but zero.  v_cvt_scalef32_pk_fp4_f32
// rounds to the nearest code, ties to even, and keeps at 6 what is above.
__device__ __forceinline__ void mx4_block8(const float (&v)[8], uint32_t amax, uint32_t& code, uint32_t& scale) {
  const uint32_t ef = amax >> 23;           // biased exponent; 255: NaN or infinity
  const uint32_t c = ef < 2 ? 0 : ef - 2;   // X + 127
  const float mul = __uint_as_float((254u - min(c, 253u)) << 23);  // 2^-X
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0] * mul, v[1] * mul, 1.0f, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2] * mul, v[3] * mul, 1.0f, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4] * mul, v[5] * mul, 1.0f, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6] * mul, v[7] * mul, 1.0f, 3);
  code = ef == 255 ? 0 : w;
  scale = ef == 255 ? 255 : c;
}

// The pass behind the one at row m0 in a workgroup's walk over rows of a group,
// end where there is none (m0 + stride may not fit in 32 bits then).
__host__ __device__ __forceinline__ int next_pass(int m0, int stride, int end) {
  return end - m0 > stride ? m0 + stride : end;
}

// ---------------------------------------------------------------- launchers
hipError_t launch_mx4_quant(const void* x, ElemType type, long M, int K, long ldx, uint8_t* q, uint8_t* s,
                            hipStream_t st);
hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* s, bool fp4, long M, int K, void* out,
                             ElemType type, hipStream_t st);
// wq/ws: plain weights, or the gate's with uq/us the up projection's (SwiGLU form)
hipError_t launch_mx4_pack(const uint8_t* wq, const uint8_t* ws, const uint8_t* uq, const uint8_t* us,
                           const Mx4Layout& L, uint8_t* packed, hipStream_t st);

// A product's activations and output.  offsets == nullptr: one group of P rows
// (the dense product).  rows == nullptr: sorted row s reads x row s, else row
// rows[s] / div.
struct Mx4Args {
  const uint8_t* packed;
  const uint8_t* xq;
  const uint8_t* xs;
  int X;  // rows of x
  const int32_t* offsets;
  const int32_t* rows;
  int div;
  int P;  // rows of y
  void* y;
};
hipError_t launch_mx4_stream(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, hipStream_t st);
// (no workspace without offsets)
size_t mx4_tiled_ws_bytes(long P, int E, int K);
hipError_t launch_mx4_tiled(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, void* ws, hipStream_t st);

// The norms' rows: what is read, what is written (null: not wanted).
struct NormArgs {
  const void* y;         // branch (or the norm's input) [T, H]
  const void* res;       // residual, bf16 or fp32; null: no residual (norm_before)
  const void* w_post;    // post-norm weight [H]; null: the branch is taken as it is
  const float* gate;     // null, or gate[t * gate_t + h * gate_h]
  long gate_t, gate_h;
  float alpha, beta, eps;
  void* out;             // residual's type
  const void* w_next;    // weight of the norm that follows; null: none
  uint16_t* z;           // bf16 rows of that norm
  uint8_t* q;            // their codes
  uint8_t* s;            // and scales
  int quant;             // 0 none, 1 MXFP8, 2 MXFP4
  ElemType y_type, res_type, w_type;
  int T, H;
};
hipError_t launch_norm(const NormArgs& a, hipStream_t st);

}  // namespace moe
