// MXFP4 x MXFP4 products for few rows: y[s, n] = sum_k x[r(s), k] W[e, n, k]
// with both operands e2m1 and one E8M0 scale per 32 along K, fp32 accumulation
// in the scaled MFMA, rounded once to bf16 (or stored as fp32); with the
// SwiGLU form h[s, i] = silu(sum x W1[e, i]) (sum x W3[e, i]).  Also the
// packing of the weights (layout in mx4.h).
//
// Weight streaming, bound by HBM: a workgroup owns two neighbouring weight
// tiles (64 rows, or a gate/up pair) of one expert and up to 32 of its token
// rows at a time; its waves take the K-steps in turn, so that at any moment
// they read neighbouring 2 KiB blocks of each tile, kB steps in flight per
// wave, and their sums are joined through LDS in wave order (the same inputs
// give the same bits).  32 x 32 x 64 MFMAs waste rows when there are few
// tokens, but a 2 KiB tile step costs 64 clocks of one SIMD's matrix unit
// while its share of HBM takes three times that.  Measured: K 2048, N 7168, 256
// experts, 512 rows: 265 us, 6.5 TB/s; SwiGLU, K 4096, N 1536, 64 experts, 48
// rows: 42 us, 5.4 TB/s; dense K 16384, N 7168, 8 rows: 15.2 us, 4.1 TB/s (14.6 and
// 15.1 us a call back to back on one weight and on eight in turn, 0.5 GB).
#include "mx4.h"

namespace moe {
namespace {

// ------------------------------------------------------------------- packing
// One thread per 16 bytes of a tile: piece i of the packed weights.  A launch
// dimension holds fewer than 2^32 threads, so larger weights run in y too.
constexpr size_t kPackX = 1 << 20;
__global__ __launch_bounds__(256) void pack_kernel(const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws,
                                                   const uint8_t* __restrict__ uq, const uint8_t* __restrict__ us,
                                                   Mx4Layout L, uint8_t* __restrict__ packed) {
  const size_t i = (blockIdx.y * kPackX + blockIdx.x) * 256 + threadIdx.x;
  const size_t n = (size_t)L.E * L.NT * L.D * 256;
  if (i >= n) return;
  const int lane = (int)(i & 63), s = (int)(i >> 6) & 1;
  size_t t = i >> 7;
  const int j = (int)(t % (2 * L.D));
  t /= 2 * L.D;
  const int nt = (int)(t % L.NT), e = (int)(t / L.NT);
  const int g = lane >> 5, col = L.column(nt, lane & 31);
  const bool up = L.glu && (nt & 1);
  const size_t row = (size_t)e * L.N + col;
  const int blk = 4 * j + 2 * g + s;
  uint4 codes = make_uint4(0, 0, 0, 0);
  uint8_t scale = 0;
  if (j < L.J) {
    codes = *reinterpret_cast<const uint4*>((up ? uq : wq) + row * (L.K / 2) + 16 * (size_t)blk);
    scale = (up ? us : ws)[row * (L.K / 32) + blk];
  }
  *reinterpret_cast<uint4*>(packed + L.tile_off(e, nt) + (size_t)j * 2048 + 1024 * s + 16 * lane) = codes;
  packed[L.scale_off(e, nt >> 2) + (size_t)(j >> 1) * 1024 + 16 * lane + 8 * (j & 1) + 2 * (nt & 3) + s] = scale;
}

// -------------------------------------------------------------------- stream
constexpr int kRows = 32;  // token rows of one pass

template <int NT>
struct Step {
  v4u w[NT][2], x[2];
  uint32_t sw, sx;
};

// wt[t] / st: this lane's bytes of tile t and of both tiles' scales at K-step 0
template <int NT>
__device__ __forceinline__ void load_step(Step<NT>& p, const uint8_t* const (&wt)[NT], const uint8_t* st,
                                          const uint8_t* xrow, const uint8_t* xscale, int j) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // weights are read once: non-temporal loads leave the caches to the rows
    const uint8_t* w = wt[t] + (size_t)j * 2048;
    p.w[t][0] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(w));
    p.w[t][1] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(w + 1024));
  }
  const uint8_t* sc = st + (size_t)(j >> 1) * 1024 + 8 * (j & 1);
  p.sw = NT == 2 ? *reinterpret_cast<const uint32_t*>(sc) : *reinterpret_cast<const uint16_t*>(sc);
  p.x[0] = *reinterpret_cast<const v4u*>(xrow + (size_t)j * 64);
  p.x[1] = *reinterpret_cast<const v4u*>(xrow + (size_t)j * 64 + 16);
  p.sx = *reinterpret_cast<const uint16_t*>(xscale + (size_t)j * 4);
}

// sw holds tile t's scale bytes at 2 t (NT = 1: at 0)
template <int NT>
__device__ __forceinline__ void multiply(const Step<NT>& p, v16f (&acc)[NT]) {
  acc[0] = mfma_fp4<0, 0>(p.x[0], p.w[0][0], acc[0], p.sx, p.sw);
  if constexpr (NT == 2) acc[1] = mfma_fp4<0, 2>(p.x[0], p.w[1][0], acc[1], p.sx, p.sw);
  acc[0] = mfma_fp4<1, 1>(p.x[1], p.w[0][1], acc[0], p.sx, p.sw);
  if constexpr (NT == 2) acc[1] = mfma_fp4<1, 3>(p.x[1], p.w[1][1], acc[1], p.sx, p.sw);
}

template <int NW, int NT, int kB, bool kGlu, bool kF32>
__global__ __launch_bounds__(64 * NW) void stream_kernel(Mx4Args a, Mx4Layout L) {
  static_assert(NT == 2 || (NT == 1 && !kGlu), "a gate tile with its up tile");
  __shared__ v4f red[NW][NT * 4][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n = lane & 31, g = lane >> 5;
  const int nt0 = blockIdx.x * NT;
  const int J = L.J;
  int e, begin, end, stride;
  if (a.offsets) {
    // offsets come from device memory: kept inside the rows of y whatever they hold
    e = blockIdx.y;
    begin = min(max(a.offsets[e], 0), a.P);
    end = min(max(a.offsets[e + 1], begin), a.P);
    if ((int)blockIdx.z >= (end - begin + kRows - 1) / kRows) return;  // uniform: before any barrier
    begin += blockIdx.z * kRows;
    stride = kRows * gridDim.z;
  } else {
    e = 0;
    begin = blockIdx.y * kRows;
    end = a.P;
    stride = kRows * gridDim.y;
  }
  const uint8_t* wt[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t)  // a last tile without a partner is read twice, stored once
    wt[t] = a.packed + L.tile_off(e, min(nt0 + t, L.NT - 1)) + 16 * lane;
  const uint8_t* st = a.packed + L.scale_off(e, nt0 >> 2) + 16 * lane + 2 * (nt0 & 3);
  const int nsteps = J > wave ? (J - wave + NW - 1) / NW : 0;
  for (int m0 = begin; m0 < end; m0 = next_pass(m0, stride, end)) {
    const int rows = min(kRows, end - m0);
    int xr = m0 + min(n, rows - 1);
    if (a.rows) xr = (int)((unsigned)a.rows[xr] / (unsigned)a.div);
    xr = min(xr, a.X - 1);
    xr = max(xr, 0);
    const uint8_t* xrow = a.xq + (size_t)xr * (L.K / 2) + 32 * g;
    const uint8_t* xscale = a.xs + (size_t)xr * (L.K / 32) + 2 * g;
    v16f acc[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[t][v] = 0.0f;
    Step<NT> p[kB];
    int u = 0;
    for (; u + kB <= nsteps; u += kB) {
#pragma unroll
      for (int b = 0; b < kB; ++b) load_step<NT>(p[b], wt, st, xrow, xscale, wave + NW * (u + b));
#pragma unroll
      for (int b = 0; b < kB; ++b) multiply<NT>(p[b], acc);
    }
    for (; u < nsteps; ++u) {
      load_step<NT>(p[0], wt, st, xrow, xscale, wave + NW * u);
      multiply<NT>(p[0], acc);
    }
    // element v of a lane is token 8 (v / 4) + 4 g + v % 4: only the groups of
    // eight tokens that exist are joined
    const int nb = (rows + 7) / 8;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (b < nb) red[wave][4 * t + b][lane] = v4f{acc[t][4 * b], acc[t][4 * b + 1], acc[t][4 * b + 2], acc[t][4 * b + 3]};
    __syncthreads();
    constexpr int kOut = kGlu ? 1 : NT;  // outputs per (token group, lane)
    for (int i = wave; i < kOut * nb; i += NW) {
      const int t = kGlu ? 0 : i / nb, b = kGlu ? i : i % nb;
      v4f s = red[0][4 * t + b][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) s += red[w][4 * t + b][lane];
      if constexpr (kGlu) {
        v4f up = red[0][4 + b][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) up += red[w][4 + b][lane];
#pragma unroll
        for (int v = 0; v < 4; ++v) s[v] = glu_out(s[v], up[v]);
      }
      if (nt0 + t >= L.NT) continue;
      const int col = L.column(nt0 + t, n);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int m = 8 * b + 4 * g + v;
        if (m >= rows) continue;
        const size_t o = (size_t)(m0 + m) * L.N + col;
        if constexpr (kF32)
          static_cast<float*>(a.y)[o] = s[v];
        else
          static_cast<uint16_t*>(a.y)[o] = f32_to_bf16(s[v]);
      }
    }
    __syncthreads();  // the sums are read before the next pass writes them
  }
}

// Passes of 32 rows of one group that run side by side: one where the groups'
// tiles alone fill the CUs, more where there are few (E 1, SwiGLU, K 4096, N
// 1536, 256 rows: 12 us against 52 with one; 500 rows: 17 against 82).
int passes_at_once(int P, const Mx4Layout& L) {
  return min(max(1536 / (int)min((long)L.E * L.NT, 1536l), 1), max((P + kRows - 1) / kRows, 1));
}

template <int NW, int NT, int kB, bool kGlu>
void stream_as(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, hipStream_t st) {
  const dim3 grid((unsigned)((L.NT + NT - 1) / NT), a.offsets ? (unsigned)L.E : (unsigned)min((a.P + kRows - 1) / kRows, 65535),
                  a.offsets ? (unsigned)passes_at_once(a.P, L) : 1u);
  if (fp32_out)
    hipLaunchKernelGGL((stream_kernel<NW, NT, kB, kGlu, true>), grid, dim3(64 * NW), 0, st, a, L);
  else
    hipLaunchKernelGGL((stream_kernel<NW, NT, kB, kGlu, false>), grid, dim3(64 * NW), 0, st, a, L);
}

}  // namespace

hipError_t launch_mx4_pack(const uint8_t* wq, const uint8_t* ws, const uint8_t* uq, const uint8_t* us,
                           const Mx4Layout& L, uint8_t* packed, hipStream_t st) {
  const size_t n = (size_t)L.E * L.NT * L.D;  // workgroups
  const dim3 grid((unsigned)(n < kPackX ? n : kPackX), (unsigned)((n + kPackX - 1) / kPackX));
  hipLaunchKernelGGL(pack_kernel, grid, dim3(256), 0, st, wq, ws, uq, us, L, packed);
  return hipGetLastError();
}

// What a launch's workgroups look like, by how many there are and how much a
// wave of them has to do (us; dense products, weights not in any cache):
// - While single tiles are at most one workgroup per CU: one tile each, so that
//   more CUs read weights.  K 2048, N 7168, 32 rows (224 tiles): 6.0 against
//   6.9 with pairs; 64 rows (448 passes): 8.6 against 7.0; K 7168, N 2048, 128
//   rows (256): 11.5 against 14.6; 256 rows (512): 20 against 14.7.  Sixteen
//   waves where each has two K-steps or more and at most 16 rows to join: K
//   16384, N 7168, 8 rows 16.2 against 17.9 with eight; 32 rows 25.5 against 23.3.
// - Otherwise pairs, by eight waves where K is long or the pairs too are at most
//   one per CU, else by four, whose sums take less LDS and joining: K 7168, N
//   2048, 256 rows (256 pairs): 14.7 with eight, 16.5 with four; 256 experts, K
//   2048, N 7168, 512 rows: 307 and 262; 16 experts, K 16384, N 2048, 128 rows:
//   50.6 and 55.2.
// The counts are against the 256 CUs that these were measured on; a device with
// fewer gets the same results.
hipError_t launch_mx4_stream(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, hipStream_t st) {
  constexpr long kCUs = 256;
  const long passes = (a.P + kRows - 1) / kRows;
  const long groups = a.offsets ? min((long)L.E * passes_at_once(a.P, L), L.E + passes - 1) : passes;
  const bool wide = L.J >= 64 || groups * ((L.NT + 1) / 2) <= kCUs;
  if (L.glu) {
    if (wide)
      stream_as<8, 2, 2, true>(a, L, fp32_out, st);
    else
      stream_as<4, 2, 2, true>(a, L, fp32_out, st);
  } else if (groups * L.NT <= kCUs) {
    if (L.J >= 32 && a.P <= 16 * groups)
      stream_as<16, 1, 2, false>(a, L, fp32_out, st);
    else
      stream_as<8, 1, 2, false>(a, L, fp32_out, st);
  } else {
    if (wide)
      stream_as<8, 2, 2, false>(a, L, fp32_out, st);
    else
      stream_as<4, 2, 2, false>(a, L, fp32_out, st);
  }
  return hipGetLastError();
}

}  // namespace moe
