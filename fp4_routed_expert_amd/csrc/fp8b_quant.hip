// FP8 quantisation of rows with one fp32 scale per 128 elements, the reading
// back of such rows, and the packing of FP8 weights with block scales.
//
// quantisation, for each block of 128: a = max(max|v|, 2^-110), scale = a / 448,
// code = e4m3(v (448 / a)), nearest, ties to even.  The floor keeps 448 / a and
// the scale normal numbers.  A block with a NaN or an infinity gets a NaN scale.
//
// Bound by HBM: 2 (or 4) bytes in and 1 + 1/32 out per element.  Sixteen lanes
// take a block, eight elements each (one or two 128-bit loads), and join their
// maxima by lane swaps; a workgroup takes 16 rows, so that the scales of a block,
// held side by side for neighbouring rows, leave as runs of 64 bytes.  16384 x 7168
// bf16: 60 us, 5.9 TB/s; read back 53 us, 6.7 TB/s (a copy of 1 GiB: 5.15); 8 x 7168: 3.2
// and 2.6 us.
#include "fp8b.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;   // rows of a workgroup
constexpr int kBlocks = 4;  // blocks of a row that a thread takes, all loads in flight together

// First row of a workgroup.  A launch dimension holds fewer than 2^32 threads, so the
// rows run in x and z.
__device__ __forceinline__ long first_row() { return ((long)blockIdx.z * gridDim.x + blockIdx.x) * kRows; }

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

// Quantises the eight values of this lane's share of a block and stores them;
// the block's first lane stores its scale.  All lanes of the 16 take part.
__device__ __forceinline__ void put8(const float (&v)[8], uint8_t* q, float* s, bool live) {
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, magnitude_bits(v[i]));
  const BlockScale k = block_scale(row16_max_u32(top));
  if (!live) return;
  *reinterpret_cast<uint2*>(q) =
      make_uint2(block_codes(v[0], v[1], v[2], v[3], k), block_codes(v[4], v[5], v[6], v[7], k));
  if ((threadIdx.x & 15) == 0) *s = k.scale;
}

template <ElemType kT>
__global__ __launch_bounds__(kThreads) void quant_kernel(const uint8_t* __restrict__ x, long M, int J, long ld_bytes,
                                                         uint8_t* __restrict__ q, float* __restrict__ s) {
  constexpr int kBytes = kT == ElemType::kFp32 ? 32 : 16;
  const long row = first_row() + (threadIdx.x >> 4);
  const int j0 = (int)blockIdx.y * kBlocks, lane = threadIdx.x & 15;
  const bool live = row < M;
  const uint8_t* src = x + (live ? row : M - 1) * ld_bytes + lane * kBytes;
  Eight<kT> e[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (j0 + b < J) load8<kT>(e[b], src + (size_t)(j0 + b) * (16 * kBytes));
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (j0 + b < J) {
      float v[8];
      values8<kT>(e[b], v);
      put8(v, q + (row * J + j0 + b) * 128 + 8 * lane, s + (long)(j0 + b) * M + row, live);
    }
}

// Rows offsets[0] to offsets[E] of h [P, N] fp32 (kGrad: the gradient dh, turned
// into dg and du first, blocks of N / 128 each).
template <bool kGrad>
__global__ __launch_bounds__(kThreads) void rows_kernel(const float* __restrict__ h, Fp8bArgs a, int E, int N) {
  const int lane = threadIdx.x & 15;
  long row = first_row() + (threadIdx.x >> 4);
  const int j = (int)blockIdx.y, J = N / 128;
  int begin = 0, end = a.P;
  if (a.offsets) {
    begin = min(max(a.offsets[0], 0), a.P);
    end = min(max(a.offsets[E], begin), a.P);
  }
  const bool live = row >= begin && row < end;
  if (!live) row = 0;  // lanes of 16 go together, so that no block mixes rows
  const size_t at = (size_t)row * N + (size_t)j * 128 + 8 * lane;
  float v[8];
  {
    const v4f lo = *reinterpret_cast<const v4f*>(h + at), hi = *reinterpret_cast<const v4f*>(h + at + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lo[i], v[4 + i] = hi[i];
  }
  if constexpr (!kGrad) {
    put8(v, a.q + at, a.s + (size_t)j * a.P + row, live);
  } else {
    Eight<ElemType::kBf16> eg, eu;
    eg.r[0] = *reinterpret_cast<const v4u*>(a.gate + at);
    eu.r[0] = *reinterpret_cast<const v4u*>(a.up + at);
    float g[8], u[8], dg[8], du[8];
    values8(eg, g);
    values8(eu, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) glu_grad(v[i], g[i], u[i], dg[i], du[i]);
    uint8_t* q = a.q + (size_t)row * (2 * (size_t)N) + (size_t)j * 128 + 8 * lane;
    put8(dg, q, a.s + (size_t)j * a.P + row, live);
    put8(du, q + N, a.s + (size_t)(J + j) * a.P + row, live);
  }
}

template <ElemType kT>
__global__ __launch_bounds__(kThreads) void dequant_kernel(const uint8_t* __restrict__ q, const float* __restrict__ s,
                                                           long M, int J, uint8_t* __restrict__ out) {
  constexpr int kBytes = kT == ElemType::kFp32 ? 32 : 16;
  const long row = first_row() + (threadIdx.x >> 4);
  const int j0 = (int)blockIdx.y * kBlocks, lane = threadIdx.x & 15;
  if (row >= M) return;
  uint2 c[kBlocks];
  float k[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (j0 + b < J) {
      c[b] = *reinterpret_cast<const uint2*>(q + (row * J + j0 + b) * 128 + 8 * lane);
      k[b] = s[(long)(j0 + b) * M + row];
    }
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
    if (j0 + b < J) {
      const v2f p[4] = {__builtin_amdgcn_cvt_pk_f32_fp8((int)c[b].x, false),
                        __builtin_amdgcn_cvt_pk_f32_fp8((int)c[b].x, true),
                        __builtin_amdgcn_cvt_pk_f32_fp8((int)c[b].y, false),
                        __builtin_amdgcn_cvt_pk_f32_fp8((int)c[b].y, true)};
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[i] = p[i >> 1][i & 1] * k[b];
        // (kept apart from the conversion to fp16, which the compiler would join to one rounding)
        if constexpr (kT == ElemType::kFp16) asm volatile("" : "+v"(v[i]));
      }
      uint8_t* o = out + (size_t)((row * J + j0 + b) * 16 + lane) * kBytes;
      if constexpr (kT == ElemType::kFp32) {
        __builtin_nontemporal_store(v4f{v[0], v[1], v[2], v[3]}, reinterpret_cast<v4f*>(o));
        __builtin_nontemporal_store(v4f{v[4], v[5], v[6], v[7]}, reinterpret_cast<v4f*>(o + 16));
      } else {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (kT == ElemType::kBf16)
            w[i] = f32x2_to_bf16(v[2 * i], v[2 * i + 1]);
          else
            w[i] = (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i]) |
                   (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v[2 * i + 1]) << 16;
        }
        __builtin_nontemporal_store(w, reinterpret_cast<v4u*>(o));
      }
    }
}

// ------------------------------------------------------------------- packing
// One workgroup per 4 KiB (two K-steps of a tile, or its last one), one thread
// per 16 bytes.  A launch dimension holds fewer than 2^32 threads, so larger
// weights run in y too.
constexpr size_t kPackX = 1 << 20;
__global__ __launch_bounds__(kThreads) void pack_kernel(const uint8_t* __restrict__ wq, const uint8_t* __restrict__ uq,
                                                        Fp8bLayout L, uint8_t* __restrict__ packed) {
  const size_t pieces = (size_t)L.E * L.NT * L.J * 128;
  const size_t i = (blockIdx.y * kPackX + blockIdx.x) * kThreads + threadIdx.x;
  if (i >= pieces) return;
  const int lane = (int)(i & 63), half = (int)(i >> 6) & 1;
  const size_t t = i >> 7;  // (expert, tile, K-step)
  const int j = (int)(t % L.J);
  const size_t et = t / L.J;
  const int nt = (int)(et % L.NT), e = (int)(et / L.NT);
  const int row = L.column(nt, lane & 15), k = 128 * j + 64 * half + 16 * (lane >> 4);
  const uint8_t* w = L.glu && (nt & 1) ? uq : wq;
  *reinterpret_cast<v4u*>(packed + i * 16) = *reinterpret_cast<const v4u*>(w + ((size_t)e * L.N + row) * L.K + k);
}

// Transposed: the source rows run along N.  A workgroup takes eight tiles (128
// columns) x one K-step through LDS: 128 source rows of 128 bytes.
__global__ __launch_bounds__(kThreads) void pack_t_kernel(const uint8_t* __restrict__ wq,
                                                          const uint8_t* __restrict__ uq, Fp8bLayout L,
                                                          uint8_t* __restrict__ packed) {
  __shared__ uint8_t lds[128][128 + 4];  // [k][column], padded: columns are read across rows
  const size_t i = blockIdx.y * kPackX + blockIdx.x;
  const int nbs = L.N / 128, j = (int)(i % L.J);
  const size_t en = i / L.J;
  const int nb = (int)(en % nbs), e = (int)(en / nbs);
  if (e >= L.E) return;  // uniform: before any barrier
  // source rows of the K-step
  const int K1 = uq ? L.K / 2 : L.K;
  const bool second = 128 * j >= K1;
  const uint8_t* src = (second ? uq : wq) + ((size_t)e * K1 + 128 * j - (second ? K1 : 0)) * L.N + 128 * (size_t)nb;
  for (int u = threadIdx.x; u < 128 * 32; u += kThreads) {
    const int k = u >> 5, c = 4 * (u & 31);
    *reinterpret_cast<uint32_t*>(&lds[k][c]) = *reinterpret_cast<const uint32_t*>(src + (size_t)k * L.N + c);
  }
  __syncthreads();
  for (int u = threadIdx.x; u < 8 * 128; u += kThreads) {  // 16-byte pieces: tile, half, lane
    const int t = u >> 7, half = (u >> 6) & 1, lane = u & 63;
    const int nt = 8 * nb + t, c = L.column(nt, lane & 15) - 128 * nb, k0 = 64 * half + 16 * (lane >> 4);
    v4u w;
#pragma unroll
    for (int d = 0; d < 4; ++d)
      w[d] = (uint32_t)lds[k0 + 4 * d][c] | (uint32_t)lds[k0 + 4 * d + 1][c] << 8 |
             (uint32_t)lds[k0 + 4 * d + 2][c] << 16 | (uint32_t)lds[k0 + 4 * d + 3][c] << 24;
    *reinterpret_cast<v4u*>(packed + L.tile_off(e, nt) + (size_t)j * 2048 + 1024 * half + 16 * lane) = w;
  }
}

__global__ __launch_bounds__(kThreads) void pack_scales_kernel(const float* __restrict__ ws,
                                                               const float* __restrict__ us, Fp8bLayout L,
                                                               bool transposed, float* __restrict__ out) {
  const size_t i = (size_t)blockIdx.x * kThreads + threadIdx.x;
  if (i >= (size_t)L.E * L.NB * L.J) return;
  const int j = (int)(i % L.J);
  const size_t eb = i / L.J;
  const int b = (int)(eb % L.NB);
  const size_t e = eb / L.NB;
  if (transposed) {
    const int J1 = us ? L.J / 2 : L.J;
    out[i] = (j >= J1 ? us : ws)[(e * J1 + (j >= J1 ? j - J1 : j)) * L.NB + b];
  } else {
    const int nb = L.glu ? L.NB / 2 : L.NB;
    out[i] = (L.glu && (b & 1) ? us : ws)[(e * nb + (L.glu ? b >> 1 : b)) * L.J + j];
  }
}

dim3 rows_grid(long M, int by) {
  constexpr long kX = 1 << 20;
  const long n = (M + kRows - 1) / kRows;
  return dim3((unsigned)(n < kX ? n : kX), (unsigned)by, (unsigned)((n + kX - 1) / kX));
}
dim3 pack_grid(size_t n) { return dim3((unsigned)(n < kPackX ? n : kPackX), (unsigned)((n + kPackX - 1) / kPackX)); }

}  // namespace

hipError_t launch_fp8b_quant(const void* x, ElemType type, long M, int K, long ldx, uint8_t* q, float* s,
                             hipStream_t st) {
  const int J = K / 128;
  const dim3 grid = rows_grid(M, (J + kBlocks - 1) / kBlocks);
  const uint8_t* p = static_cast<const uint8_t*>(x);
  if (type == ElemType::kFp32)
    hipLaunchKernelGGL(quant_kernel<ElemType::kFp32>, grid, dim3(kThreads), 0, st, p, M, J, 4 * ldx, q, s);
  else if (type == ElemType::kFp16)
    hipLaunchKernelGGL(quant_kernel<ElemType::kFp16>, grid, dim3(kThreads), 0, st, p, M, J, 2 * ldx, q, s);
  else
    hipLaunchKernelGGL(quant_kernel<ElemType::kBf16>, grid, dim3(kThreads), 0, st, p, M, J, 2 * ldx, q, s);
  return hipGetLastError();
}

hipError_t launch_fp8b_dequant(const uint8_t* q, const float* s, long M, int K, void* out, ElemType type,
                               hipStream_t st) {
  const int J = K / 128;
  const dim3 grid = rows_grid(M, (J + kBlocks - 1) / kBlocks);
  uint8_t* o = static_cast<uint8_t*>(out);
  if (type == ElemType::kFp32)
    hipLaunchKernelGGL(dequant_kernel<ElemType::kFp32>, grid, dim3(kThreads), 0, st, q, s, M, J, o);
  else if (type == ElemType::kFp16)
    hipLaunchKernelGGL(dequant_kernel<ElemType::kFp16>, grid, dim3(kThreads), 0, st, q, s, M, J, o);
  else
    hipLaunchKernelGGL(dequant_kernel<ElemType::kBf16>, grid, dim3(kThreads), 0, st, q, s, M, J, o);
  return hipGetLastError();
}

hipError_t launch_fp8b_rows(const float* h, const Fp8bArgs& a, int E, int N, Fp8bOut out, hipStream_t st) {
  const dim3 grid = rows_grid(a.P, N / 128);
  if (out == Fp8bOut::kGluGrad)
    hipLaunchKernelGGL(rows_kernel<true>, grid, dim3(kThreads), 0, st, h, a, E, N);
  else
    hipLaunchKernelGGL(rows_kernel<false>, grid, dim3(kThreads), 0, st, h, a, E, N);
  return hipGetLastError();
}

hipError_t launch_fp8b_pack(const uint8_t* wq, const float* ws, const uint8_t* uq, const float* us,
                            const Fp8bLayout& L, bool transposed, uint8_t* packed, hipStream_t st) {
  if (transposed)
    hipLaunchKernelGGL(pack_t_kernel, pack_grid((size_t)L.E * (L.N / 128) * L.J), dim3(kThreads), 0, st, wq, uq, L,
                       packed);
  else
    hipLaunchKernelGGL(pack_kernel, pack_grid(((size_t)L.E * L.NT * L.J + 1) / 2), dim3(kThreads), 0, st, wq, uq, L,
                       packed);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const size_t scales = (size_t)L.E * L.NB * L.J;
  hipLaunchKernelGGL(pack_scales_kernel, dim3((unsigned)((scales + kThreads - 1) / kThreads)), dim3(kThreads), 0, st,
                     ws, us, L, transposed, reinterpret_cast<float*>(packed + L.s_off));
  return hipGetLastError();
}

}  // namespace moe
