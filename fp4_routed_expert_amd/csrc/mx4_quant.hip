// MXFP4 quantisation (e2m1 codes, one E8M0 scale per 32 elements of a row)
// and the reading back of MXFP4 and MXFP8 rows.
//
// quantisation, for each block of 32: X = floor(log2 max|v|) - 2 (2 = the
// largest e2m1 exponent), kept in [-127, 127]; the scale code is X + 127 and
// each code is v 2^-X rounded to {0, .5, 1, 1.5, 2, 3, 4, 6}, nearest, ties to
// the even code, at most 6, sign kept.  A block that holds a NaN or an
// infinity gets the scale code 255 (NaN) and zero codes.
//
// Bound by HBM: 2 (or 4) bytes in and 17/32 out per element.  A thread takes
// eight elements (one or two 128-bit loads); four neighbouring lanes hold one
// block and join their maxima with two lane swaps, so that loads and stores of
// a wave are contiguous without a trip through LDS.  Four groups per thread keep
// 64 bytes in flight each.  Measured: 98304 x 4096 bf16 in 158 us (6.5 TB/s of
// reads and writes), read back in 166 us (6.2 TB/s); 8 x 4096 in 2.4 us, a
// launch.  Rows that are further apart cost a division per group: 162 us with 4104
// elements from row to row, 164 with 8192.
#include "mx4.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kGroups = 4;  // groups of eight elements per thread, all loads in flight together

template <ElemType kT>
struct Eight {
  v4u r[kT == ElemType::kFp32 ? 2 : 1];
};

template <ElemType kT>
__device__ __forceinline__ void load8(Eight<kT>& e, const uint8_t* p) {
  e.r[0] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p));
  if constexpr (kT == ElemType::kFp32) e.r[1] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(p + 16));
}

template <ElemType kT>
__device__ __forceinline__ void values8(const Eight<kT>& e, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (kT == ElemType::kFp32) {
      v[i] = __uint_as_float(e.r[i >> 2][i & 3]);
    } else {
      const uint32_t w = e.r[0][i >> 1] >> (16 * (i & 1));
      if constexpr (kT == ElemType::kBf16)
        v[i] = __uint_as_float(w << 16);
      else
        v[i] = (float)__builtin_bit_cast(_Float16, (uint16_t)w);
    }
  }
}

// Row and column (in groups of eight) of flat group i; contiguous rows need no
// division.
template <ElemType kT, bool kStrided>
__global__ __launch_bounds__(kThreads) void quant_kernel(const uint8_t* __restrict__ x, long n8, int K8, long ld_bytes,
                                                         uint32_t* __restrict__ q, uint8_t* __restrict__ s) {
  constexpr int kBytes = kT == ElemType::kFp32 ? 32 : 16;
  const long i0 = (long)blockIdx.x * (kThreads * kGroups) + threadIdx.x;
  Eight<kT> e[kGroups];
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    // groups past the end read the last one again (n8 is a multiple of four,
    // so a block is all inside or all outside) and are not stored
    const long i = min(i0 + (long)u * kThreads, n8 - 1);
    load8<kT>(e[u], kStrided ? x + (i / K8) * ld_bytes + (i % K8) * kBytes : x + i * kBytes);
  }
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const long i = i0 + (long)u * kThreads;
    float v[8];
    values8<kT>(e[u], v);
    uint32_t amax = 0;
#pragma unroll
    for (int c = 0; c < 8; ++c) amax = max(amax, __float_as_uint(v[c]) & 0x7FFFFFFFu);
    uint32_t code, scale;
    mx4_block8(v, quad_max_u32(amax), code, scale);
    if (i < n8) {
      __builtin_nontemporal_store(code, q + i);
      if ((i & 3) == 0) s[i >> 2] = (uint8_t)scale;
    }
  }
}

// 2^(c - 127) of a scale code, NaN for 255.
__device__ __forceinline__ float e8m0(uint32_t c) {
  return __uint_as_float(c == 0 ? 0x00400000u : c == 255 ? 0x7FC00000u : c << 23);
}

template <bool kFp4, ElemType kT>
__global__ __launch_bounds__(kThreads) void dequant_kernel(const uint8_t* __restrict__ q, const uint8_t* __restrict__ s,
                                                           long n8, uint8_t* __restrict__ out) {
  const long i0 = (long)blockIdx.x * (kThreads * kGroups) + threadIdx.x;
  uint32_t lo[kGroups], hi[kGroups], c[kGroups];
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const long i = min(i0 + (long)u * kThreads, n8 - 1);
    if constexpr (kFp4) {
      lo[u] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(q) + i);
      hi[u] = 0;
    } else {
      const uint64_t w = __builtin_nontemporal_load(reinterpret_cast<const uint64_t*>(q) + i);
      lo[u] = (uint32_t)w;
      hi[u] = (uint32_t)(w >> 32);
    }
    c[u] = s[i >> 2];
  }
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    const long i = i0 + (long)u * kThreads;
    const float m = e8m0(c[u]);
    float v[8];
    if constexpr (kFp4) {
      v2f p;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[u], 1.0f, 0);
      v[0] = p.x, v[1] = p.y;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[u], 1.0f, 1);
      v[2] = p.x, v[3] = p.y;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[u], 1.0f, 2);
      v[4] = p.x, v[5] = p.y;
      p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(lo[u], 1.0f, 3);
      v[6] = p.x, v[7] = p.y;
    } else {
      v2f p;
      p = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo[u], false);
      v[0] = p.x, v[1] = p.y;
      p = __builtin_amdgcn_cvt_pk_f32_fp8((int)lo[u], true);
      v[2] = p.x, v[3] = p.y;
      p = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi[u], false);
      v[4] = p.x, v[5] = p.y;
      p = __builtin_amdgcn_cvt_pk_f32_fp8((int)hi[u], true);
      v[6] = p.x, v[7] = p.y;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] *= m;  // exact in fp32, or past its range (infinity)
    if (i >= n8) continue;
    if constexpr (kT == ElemType::kFp32) {
      v4f* o = reinterpret_cast<v4f*>(out + i * 32);
      __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, o);
      __builtin_nontemporal_store(v4f{v[4], v[5], v[6], v[7]}, o + 1);
    } else {
      v4u w;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if constexpr (kT == ElemType::kBf16) {
          w[k] = f32x2_to_bf16(v[2 * k], v[2 * k + 1]);
        } else {
          w[k] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * k]) |
                 (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * k + 1]) << 16;
        }
      }
      __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(out + i * 16));
    }
  }
}

dim3 grid_of(long n8) { return dim3((unsigned)((n8 + kThreads * kGroups - 1) / (kThreads * kGroups))); }

template <ElemType kT>
void quant_as(const void* x, long n8, int K, long ldx, uint8_t* q, uint8_t* s, hipStream_t st) {
  const uint8_t* p = static_cast<const uint8_t*>(x);
  const long ld_bytes = ldx * (kT == ElemType::kFp32 ? 4 : 2);
  uint32_t* q32 = reinterpret_cast<uint32_t*>(q);
  if (ldx == K)
    hipLaunchKernelGGL((quant_kernel<kT, false>), grid_of(n8), dim3(kThreads), 0, st, p, n8, K / 8, ld_bytes, q32, s);
  else
    hipLaunchKernelGGL((quant_kernel<kT, true>), grid_of(n8), dim3(kThreads), 0, st, p, n8, K / 8, ld_bytes, q32, s);
}

template <bool kFp4>
void dequant_as(const uint8_t* q, const uint8_t* s, long n8, void* out, ElemType type, hipStream_t st) {
  uint8_t* o = static_cast<uint8_t*>(out);
  switch (type) {
    case ElemType::kBf16:
      hipLaunchKernelGGL((dequant_kernel<kFp4, ElemType::kBf16>), grid_of(n8), dim3(kThreads), 0, st, q, s, n8, o);
      break;
    case ElemType::kFp16:
      hipLaunchKernelGGL((dequant_kernel<kFp4, ElemType::kFp16>), grid_of(n8), dim3(kThreads), 0, st, q, s, n8, o);
      break;
    case ElemType::kFp32:
      hipLaunchKernelGGL((dequant_kernel<kFp4, ElemType::kFp32>), grid_of(n8), dim3(kThreads), 0, st, q, s, n8, o);
      break;
  }
}

}  // namespace

hipError_t launch_mx4_quant(const void* x, ElemType type, long M, int K, long ldx, uint8_t* q, uint8_t* s,
                            hipStream_t st) {
  const long n8 = M * (long)K / 8;
  switch (type) {
    case ElemType::kBf16: quant_as<ElemType::kBf16>(x, n8, K, ldx, q, s, st); break;
    case ElemType::kFp16: quant_as<ElemType::kFp16>(x, n8, K, ldx, q, s, st); break;
    case ElemType::kFp32: quant_as<ElemType::kFp32>(x, n8, K, ldx, q, s, st); break;
  }
  return hipGetLastError();
}

hipError_t launch_mx_dequant(const uint8_t* q, const uint8_t* s, bool fp4, long M, int K, void* out, ElemType type,
                             hipStream_t st) {
  const long n8 = M * (long)K / 8;
  if (fp4)
    dequant_as<true>(q, s, n8, out, type, st);
  else
    dequant_as<false>(q, s, n8, out, type, st);
  return hipGetLastError();
}

}  // namespace moe
