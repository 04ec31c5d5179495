// RMS norms before and after a block, with the block's gate, the residual and
// the quantisation of what the next product reads, in one pass over the rows.
//
//   before:  z = bf16((x r) w),  r = 1 / sqrt(mean(x^2) + eps)
//   after:   b = y, or (y r(y)) w_post;  b = b gate;
//            out = beta res + alpha b, rounded to the residual's type;
//            z = bf16((out r(out)) w_next) of the stored out
//   and the MXFP8 or MXFP4 codes of z.
//
// The sum of squares is taken in 64 bits (the squares of bf16 are exact even
// in 32) and r rounded once to fp32; every later operation is one fp32
// operation in the order written above, none contracted.  So z, and with it
// each code next to a rounding border, does not depend on how a row is split
// over lanes.  The double-precision work is two instructions per element, far
// under the time that the row's bytes take.
//
// Bound by HBM for many rows and by latency for few.  A row stays in
// registers from its first load to the last store: a workgroup owns a row,
// each thread kC groups of eight columns.  Measured: after, H 7168, fp32 branch
// and bf16 residual, MXFP4 rows: 4604 rows 74 us (4.7 TB/s); MXFP8 rows,
// 16384 rows 249 us (5.2 TB/s); before, bf16 rows and MXFP8: 8 rows of 4096 4.5 us,
// 4604 of 7168 40 us (4.1 TB/s), 16384 126 us (4.7 TB/s).
#include "mx4.h"

#pragma clang fp contract(off)

namespace moe {
namespace {

// Eight neighbouring elements of a row, converted to fp32 (exact).
__device__ __forceinline__ void row_load8(const void* p, ElemType type, size_t i, float (&v)[8]) {
  if (type == ElemType::kFp32) {
    const v4f* q = reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
    const v4f a = __builtin_nontemporal_load(q), b = __builtin_nontemporal_load(q + 1);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = a[k], v[4 + k] = b[k];
  } else {
    const v4u w = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(p) + i));
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// The same for weights and gates, which every row reads again.
__device__ __forceinline__ void vec_load8(const void* p, ElemType type, int i, float (&v)[8]) {
  if (type == ElemType::kFp32) {
    const v4f* q = reinterpret_cast<const v4f*>(static_cast<const float*>(p) + i);
    const v4f a = q[0], b = q[1];
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = a[k], v[4 + k] = b[k];
  } else {
    const v4u w = *reinterpret_cast<const v4u*>(static_cast<const uint16_t*>(p) + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[2 * k] = __uint_as_float(w[k] << 16), v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void row_store8(void* p, ElemType type, size_t i, const float (&v)[8]) {
  if (type == ElemType::kFp32) {
    v4f* q = reinterpret_cast<v4f*>(static_cast<float*>(p) + i);
    q[0] = v4f{v[0], v[1], v[2], v[3]};
    q[1] = v4f{v[4], v[5], v[6], v[7]};
  } else {
    v4u w;
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = f32x2_to_bf16(v[2 * k], v[2 * k + 1]);
    *reinterpret_cast<v4u*>(static_cast<uint16_t*>(p) + i) = w;
  }
}

__device__ __forceinline__ double sum_squares(const float (&v)[8]) {
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 8; ++k) s = fma((double)v[k], (double)v[k], s);
  return s;
}

// Sum over the workgroup, in a fixed order; every thread gets it.
template <int NW>
__device__ __forceinline__ double block_sum(double s, double (&part)[NW]) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d, 64);
  if (NW == 1) return s;
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = s;
  __syncthreads();
  s = part[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) s += part[w];
  return s;
}

__device__ __forceinline__ float inv_rms(double ss, int H, float eps) {
  return (float)(1.0 / sqrt(ss / (double)H + (double)eps));
}

// Gate and residual of eight elements of the branch b (normed or not); b
// becomes what the residual's type holds.
__device__ __forceinline__ void join_residual(const NormArgs& a, size_t t, int h, const float (&res)[8], float (&b)[8]) {
  if (a.gate) {
    const float* gp = a.gate + t * a.gate_t;
    if (a.gate_h == 0) {
      const float gv = gp[0];
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = b[k] * gv;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) b[k] = b[k] * gp[h + k];
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    b[k] = res[k] * a.beta + b[k] * a.alpha;
    if (a.res_type != ElemType::kFp32) b[k] = __uint_as_float((uint32_t)f32_to_bf16(b[k]) << 16);
  }
}

// Codes of eight elements z (bf16 values); the four lanes of a block call it
// together.  live: false on lanes past the row.
__device__ __forceinline__ void store_codes(const NormArgs& a, size_t i, const float (&z)[8], bool live) {
  uint32_t amax = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) amax = max(amax, __float_as_uint(z[k]) & 0x7FFFFFFFu);
  amax = quad_max_u32(live ? amax : 0u);
  if (a.quant == 2) {
    uint32_t code, scale;
    mx4_block8(z, amax, code, scale);
    if (live) {
      *reinterpret_cast<uint32_t*>(a.q + i / 2) = code;
      if ((i & 31) == 0) a.s[i / 32] = (uint8_t)scale;
    }
  } else {
    // the rule of the MXFP8 activation quantiser; a block with a NaN or an
    // infinity gets the NaN scale
    float mul;
    const uint32_t scale = mx_scale_from_amax(__uint_as_float(min(amax, 0x7F7FFFFFu)), &mul);
    const uint32_t lo = f32x4_to_e4m3(z[0] * mul, z[1] * mul, z[2] * mul, z[3] * mul);
    const uint32_t hi = f32x4_to_e4m3(z[4] * mul, z[5] * mul, z[6] * mul, z[7] * mul);
    const bool bad = amax >= 0x7F800000u;
    if (live) {
      *reinterpret_cast<uint2*>(a.q + i) = bad ? make_uint2(0, 0) : make_uint2(lo, hi);
      if ((i & 31) == 0) a.s[i / 32] = bad ? 255 : (uint8_t)scale;
    }
  }
}

// z of eight elements v of the normed row, stored and quantised.
__device__ __forceinline__ void finish8(const NormArgs& a, size_t row, int h, const float (&v)[8], float r, bool live) {
  float w[8], z[8];
  vec_load8(a.w_next, a.w_type, live ? h : 0, w);
#pragma unroll
  for (int k = 0; k < 8; ++k) z[k] = v[k] * r * w[k];
  v4u p;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    p[k] = f32x2_to_bf16(z[2 * k], z[2 * k + 1]);
    z[2 * k] = __uint_as_float(p[k] << 16);
    z[2 * k + 1] = __uint_as_float(p[k] & 0xFFFF0000u);
  }
  if (a.z && live) *reinterpret_cast<v4u*>(a.z + row + h) = p;
  if (a.quant) store_codes(a, row + h, z, live);
}

// One row per workgroup of NW waves, kC groups of eight columns per thread
// (H <= 512 NW kC, H % 8 == 0).  A launch dimension holds fewer than 2^32
// threads, so more rows than kRowsX run in y too.
constexpr unsigned kRowsX = 1 << 16;
template <int NW, int kC>
__global__ __launch_bounds__(64 * NW) void norm_kernel(NormArgs a) {
  __shared__ double part[2][NW];
  const int H = a.H;
  const size_t t = blockIdx.y * kRowsX + blockIdx.x, row = t * H;
  if (t >= (size_t)a.T) return;
  float v[kC][8];
  const bool after = a.res != nullptr;
  float res[kC][8];
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int h = 8 * (c * 64 * NW + (int)threadIdx.x);
    if (h < H) {
      row_load8(a.y, a.y_type, row + h, v[c]);
      if (after) row_load8(a.res, a.res_type, row + h, res[c]);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[c][k] = 0.0f;
    }
  }
  if (after) {
    if (a.w_post) {
      double ss = 0.0;
#pragma unroll
      for (int c = 0; c < kC; ++c) ss += sum_squares(v[c]);
      const float r = inv_rms(block_sum<NW>(ss, part[0]), H, a.eps);
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        const int h = 8 * (c * 64 * NW + (int)threadIdx.x);
        if (h < H) {
          float w[8];
          vec_load8(a.w_post, a.w_type, h, w);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[c][k] = v[c][k] * r * w[k];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < kC; ++c) {
      const int h = 8 * (c * 64 * NW + (int)threadIdx.x);
      if (h < H) {
        join_residual(a, t, h, res[c], v[c]);
        row_store8(a.out, a.res_type, row + h, v[c]);
      }
    }
  }
  if (!a.w_next) return;
  double ss = 0.0;
#pragma unroll
  for (int c = 0; c < kC; ++c) ss += sum_squares(v[c]);
  const float r = inv_rms(block_sum<NW>(ss, part[1]), H, a.eps);
#pragma unroll
  for (int c = 0; c < kC; ++c) {
    const int h = 8 * (c * 64 * NW + (int)threadIdx.x);
    finish8(a, row, h, v[c], r, h < H);
  }
}

template <int NW, int kC>
void norm_as(const NormArgs& a, hipStream_t st) {
  const unsigned T = (unsigned)a.T;
  const dim3 grid(T < kRowsX ? T : kRowsX, (T + kRowsX - 1) / kRowsX);
  hipLaunchKernelGGL((norm_kernel<NW, kC>), grid, dim3(64 * NW), 0, st, a);
}

}  // namespace

hipError_t launch_norm(const NormArgs& a, hipStream_t st) {
  const int groups = (a.H + 7) / 8;
  if (groups <= 64)
    norm_as<1, 1>(a, st);
  else if (groups <= 256)
    norm_as<4, 1>(a, st);
  else if (groups <= 512)
    norm_as<4, 2>(a, st);
  else if (groups <= 1024)
    norm_as<4, 4>(a, st);
  else
    norm_as<8, 4>(a, st);
  return hipGetLastError();
}

}  // namespace moe
