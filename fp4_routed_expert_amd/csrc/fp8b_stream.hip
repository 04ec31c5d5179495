// FP8 products with block scales of 128 for few rows: y[s, n] = sum over blocks
// b of sx[b, r] sw[n / 128, b] (sum_{k in b} xq[r, k] wq[e, n, k]).  One MFMA
// (K = 128) is one block's sum (four with exact products where the result is fp32 for
// the caller); the two scales meet it in one fp32 multiply-add per element, since they
// are no powers of two.
//
// Weight streaming, bound by HBM: a workgroup owns two neighbouring weight
// tiles (32 columns, or 16 columns of gate and up) of one expert, or one tile
// where there are few, and 16 or 32 of its token rows at a time; its waves take
// the K-steps in turn, so that at any moment they read neighbouring 2 KiB blocks
// of each tile, kB steps in flight per wave, and their sums are joined through
// LDS in wave order (the same inputs give the same bits).  8 rows, K 16384, N 7168:
// 19.3 us, 6.1 TB/s; SwiGLU, 64 experts, K 4096, N 1536, 48 rows: 66 us, 6.5 TB/s.
#include "fp8b.h"

namespace moe {
namespace {

template <int NT, int TT>
struct Step {
  v4u w[NT][2], x[TT][2];
  float sw[NT], sx[TT];
};

// What one pass reads: this lane's bytes of each tile and token row at K-step 0.
template <int NT, int TT>
struct Source {
  const uint8_t* w[NT];
  const float* sw[NT];  // uniform
  const uint8_t* x[TT];
  const float* sx[TT];
  long X;  // floats from a block's row scales to the next one's
};

template <int NT, int TT>
__device__ __forceinline__ void load_step(Step<NT, TT>& p, const Source<NT, TT>& s, int j) {
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    // weights are read once: non-temporal loads leave the caches to the rows
    const uint8_t* w = s.w[t] + (size_t)j * 2048;
    p.w[t][0] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(w));
    p.w[t][1] = __builtin_nontemporal_load(reinterpret_cast<const v4u*>(w + 1024));
    p.sw[t] = s.sw[t][j];
  }
#pragma unroll
  for (int i = 0; i < TT; ++i) {
    p.x[i][0] = *reinterpret_cast<const v4u*>(s.x[i] + (size_t)j * 128);
    p.x[i][1] = *reinterpret_cast<const v4u*>(s.x[i] + (size_t)j * 128 + 64);
    p.sx[i] = s.sx[i][(size_t)j * s.X];
  }
}

template <int NT, int TT, bool kExact>
__device__ __forceinline__ void multiply(const Step<NT, TT>& p, v4f (&acc)[NT][TT]) {
  v4f d[NT][TT];
  if constexpr (kExact) {
    Wide x[TT];
#pragma unroll
    for (int i = 0; i < TT; ++i) x[i] = widen(cat_pieces(p.x[i][0], p.x[i][1]));
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const Wide w = widen(cat_pieces(p.w[t][0], p.w[t][1]));
#pragma unroll
      for (int i = 0; i < TT; ++i) d[t][i] = mfma_wide(w, x[i]);
    }
  } else {
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < TT; ++i)
        d[t][i] = mfma_block(cat_pieces(p.w[t][0], p.w[t][1]), cat_pieces(p.x[i][0], p.x[i][1]));
  }
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      const float k = p.sx[i] * p.sw[t];
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[t][i][v] = fmaf(d[t][i][v], k, acc[t][i][v]);
    }
}

// kOut: kBf16 and kFp32 write a.y; kGlu writes h to a.y as fp32 rows, and gate
// and up where they are wanted; kGluGrad writes dh to a.y as fp32 rows, summed as what
// is quantised behind it is (with exact products 64 experts of 6 rows, K 4096, N 2048,
// take 100 us instead of 86).
template <int NW, int NT, int TT, int kB, Fp8bOut kOut>
__global__ __launch_bounds__(64 * NW) void stream_kernel(Fp8bArgs a, Fp8bLayout L) {
  constexpr bool kGlu = kOut == Fp8bOut::kGlu, kExact = kOut == Fp8bOut::kFp32;
  static_assert(NT == 2 || (NT == 1 && !kGlu), "a gate tile with its up tile");
  constexpr int kRows = 16 * TT;
  __shared__ v4f red[NW][NT * TT][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, g = lane >> 4;
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
  Source<NT, TT> src;
  src.X = a.X;
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    src.w[t] = a.packed + L.tile_off(e, nt0 + t) + 16 * lane;
    // row block: of the pair's 16 columns with gate and up, else of the tile's pair
    const int b = kGlu ? 2 * (nt0 >> 4) + t : (nt0 + t) >> 3;
    src.sw[t] = reinterpret_cast<const float*>(a.packed + L.s_off) + ((size_t)e * L.NB + b) * J;
  }
  const int nsteps = J > wave ? (J - wave + NW - 1) / NW : 0;
  for (int m0 = begin; m0 < end; m0 = next_pass(m0, stride, end)) {
    const int rows = min(kRows, end - m0);
#pragma unroll
    for (int i = 0; i < TT; ++i) {
      int xr = m0 + min(16 * i + r, rows - 1);
      if (a.rows) xr = entry_row(a.rows, xr, a.div, a.X);
      src.x[i] = a.xq + (size_t)xr * L.K + 16 * g;
      src.sx[i] = a.xs + xr;
    }
    v4f acc[NT][TT];
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < TT; ++i) acc[t][i] = v4f{0.f, 0.f, 0.f, 0.f};
    Step<NT, TT> p[kB];
    int u = 0;
    for (; u + kB <= nsteps; u += kB) {
#pragma unroll
      for (int b = 0; b < kB; ++b) load_step(p[b], src, wave + NW * (u + b));
#pragma unroll
      for (int b = 0; b < kB; ++b) multiply<NT, TT, kExact>(p[b], acc);
    }
    for (; u < nsteps; ++u) {
      load_step(p[0], src, wave + NW * u);
      multiply<NT, TT, kExact>(p[0], acc);
    }
    const int nb = (rows + 15) / 16;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int i = 0; i < TT; ++i)
        if (i < nb) red[wave][NT * i + t][lane] = acc[t][i];
    __syncthreads();
    constexpr int kEach = kGlu ? 1 : NT;  // outputs of a token tile
    for (int o = wave; o < kEach * nb; o += NW) {
      const int i = o / kEach, t = o % kEach;
      v4f s = red[0][NT * i + t][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) s += red[w][NT * i + t][lane];
      v4f up{};
      if constexpr (kGlu) {
        up = red[0][NT * i + 1][lane];
#pragma unroll
        for (int w = 1; w < NW; ++w) up += red[w][NT * i + 1][lane];
      }
      const int m = 16 * i + r;
      if (m >= rows) continue;
      const size_t at = (size_t)(m0 + m) * L.N + L.column(nt0 + t, 4 * g);
      if constexpr (kGlu) {
        if (a.gate) {
          *reinterpret_cast<uint2*>(a.gate + at) = make_uint2(f32x2_to_bf16(s[0], s[1]), f32x2_to_bf16(s[2], s[3]));
          *reinterpret_cast<uint2*>(a.up + at) = make_uint2(f32x2_to_bf16(up[0], up[1]), f32x2_to_bf16(up[2], up[3]));
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) s[v] = glu_out(s[v], up[v]);
      }
      if constexpr (kOut == Fp8bOut::kBf16)
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) =
            make_uint2(f32x2_to_bf16(s[0], s[1]), f32x2_to_bf16(s[2], s[3]));
      else
        *reinterpret_cast<v4f*>(static_cast<float*>(a.y) + at) = s;
    }
    __syncthreads();  // the sums are read before the next pass writes them
  }
}

// Passes over one group's rows that run side by side: one where the groups'
// tiles alone fill the CUs, more where there are few.
int passes_at_once(int P, const Fp8bLayout& L, int rows) {
  return min(max(1536 / (int)min((long)L.E * L.NT, 1536l), 1), max((P + rows - 1) / rows, 1));
}

template <int NW, int NT, int TT, int kB, Fp8bOut kOut>
void stream_as(const Fp8bArgs& a, const Fp8bLayout& L, hipStream_t st) {
  constexpr int kRows = 16 * TT;
  const dim3 grid((unsigned)(L.NT / NT), a.offsets ? (unsigned)L.E : (unsigned)min((a.P + kRows - 1) / kRows, 65535),
                  a.offsets ? (unsigned)passes_at_once(a.P, L, kRows) : 1u);
  hipLaunchKernelGGL((stream_kernel<NW, NT, TT, kB, kOut>), grid, dim3(64 * NW), 0, st, a, L);
}

// What a launch's workgroups look like, by the rows of a group on average and by
// how many tiles there are (us; weights not in any cache):
// - Up to 16 rows, tiles at most one per CU: one tile each, by 16 waves.  K 4096, N
//   1536, 8 rows (96 tiles): 5.1 against 6.2 with pairs by four waves; K 7168, N
//   2048 (128 tiles): 7.0 and 9.2.
// - Up to 16 rows, more tiles: pairs, by four waves with four K-steps each in
//   flight.  K 16384, N 7168, 8 rows (448 tiles): 19.7 against 23.8 with single tiles
//   by 16 waves, 21.5 with pairs by eight; SwiGLU, 64 experts, K 4096, N 1536, 48
//   rows: 63.8 and, by 16 waves, 81.  Pairs of gate and up are one per CU: 16 waves.
// - More rows: two token tiles to a pass over a pair, by eight waves.  K 16384, N
//   7168, 32 rows: 27 against 30 with four waves; K 7168, N 2048, 256 rows: 23 and 23.
//   With exact products (whose operands take more registers) and more pairs than
//   CUs by four: K 4096, N 1536, 333 rows 18 against 21.
// - Four token tiles to a pass, of one group, where that saves enough rounds of
//   workgroups on the CUs: such a pass takes 1.5-1.7 times as long.  (Rounds of two
//   and of four tiles, us: K 4096, N 4096, 64 rows, 1 and 1, 8.6 and 12.9; 128 rows, 2 and
//   1, 14.4 and 12.9; 192 rows, 3 and 2, 20.3 and 23.4; K 16384, N 7168, 64 rows, 2 and 1,
//   51 and 42; 128 rows, 4 and 2, 100 and 80; in fp32 56 and 46, 108 and 87.)  Below K
//   4096 the rounds of small workgroups overlap, so one round only: K 2048, N 2048, 160
//   rows, 2 and 1, 8.3 and 7.9; N 7168, 256 rows, 7 and 4, 26.0 and 27.6.
// The counts are against the 256 CUs that these were measured on; a device with
// fewer gets the same results.
template <Fp8bOut kOut>
void stream_for(const Fp8bArgs& a, const Fp8bLayout& L, hipStream_t st) {
  constexpr bool kGlu = kOut == Fp8bOut::kGlu;
  constexpr long kCUs = 256;
  const long groups = a.offsets ? min((long)L.E, (long)a.P) : 1;
  if (a.P > 16 * groups) {
    const long passes = a.offsets ? groups : (a.P + 31) / 32;
    if constexpr (!kGlu) {
      const long wide = (a.P + 63) / 64;
      auto rounds = [&](long passes) { return (passes * (L.NT / 2) + kCUs - 1) / kCUs; };
      if (!a.offsets && 17 * rounds(wide) < 10 * rounds(passes) && (L.J >= 32 || rounds(wide) == 1)) {
        stream_as<8, 2, 4, 2, kOut>(a, L, st);
        return;
      }
    }
    if (kOut == Fp8bOut::kFp32 && passes * L.NT > 2 * kCUs)
      stream_as<4, 2, 2, 2, kOut>(a, L, st);
    else
      stream_as<8, 2, 2, 2, kOut>(a, L, st);
  } else if (groups * L.NT > (kGlu ? 2 : 1) * kCUs) {
    stream_as<4, 2, 1, 4, kOut>(a, L, st);
  } else {
    stream_as<16, kGlu ? 2 : 1, 1, 2, kOut>(a, L, st);
  }
}

}  // namespace

hipError_t launch_fp8b_stream(const Fp8bArgs& args, const Fp8bLayout& L, Fp8bOut out, float* ws, hipStream_t st) {
  Fp8bArgs a = args;
  if (out == Fp8bOut::kBf16) {
    stream_for<Fp8bOut::kBf16>(a, L, st);
    return hipGetLastError();
  }
  if (out == Fp8bOut::kFp32) {
    stream_for<Fp8bOut::kFp32>(a, L, st);
    return hipGetLastError();
  }
  // A block of 128 outputs is spread over several workgroups here, so the rows
  // go through memory as fp32 and are quantised by a second launch.
  a.y = ws;
  if (out == Fp8bOut::kGlu)
    stream_for<Fp8bOut::kGlu>(a, L, st);
  else
    stream_for<Fp8bOut::kGluGrad>(a, L, st);
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_fp8b_rows(ws, args, L.E, L.N, out, st);
}

}  // namespace moe
