// Gradient of the weights from FP8 rows with block scales of 128:
// dw[e, n, k] = sum over the rows s of group e of dy[s, n] x[r(s), k].
//
// The sum runs over rows, along which both scales vary, so the products are made
// in the bf16 matrix cores.  x's codes are exact in bf16; dy's codes are
// multiplied by both scales and rounded once (by at most 2^-8 of each product),
// for each of the tile's two blocks of k.
//
// A workgroup makes 256 x 256 outputs of one expert, eight waves of 64 x 128 by
// v_mfma_f32_32x32x16_bf16, in steps of 32 rows.  The matrix cores want eight
// neighbouring rows of one column in a lane: a thread reads four bytes of eight
// rows each, and the conversion of pairs of rows to bf16 is the transposition.
// Waves 0-3 convert dy, waves 4-7 x.  LDS holds [eight rows][column c of four]
// [group of four columns], 16 bytes each, so that writes and reads run along
// neighbouring addresses; a lane ends with four neighbouring outputs.
//
// Where the tiles are fewer than the CUs, the rows are split; the parts' sums go
// through memory in fp32 and are added in the order of the rows.
#include "fp8b.h"
#include "tiled.h"

namespace moe {
namespace {

constexpr int kTile = 256;
constexpr int kStepRows = 32;
constexpr int kPanel = kTile * kStepRows * 2;  // bytes of one operand's step
constexpr int kBuf = 3 * kPanel;               // dy for each block of k, x

struct GradLaunch {
  Fp8bGradArgs a;
  int ntn, ntk;     // tiles of an expert
  int parts;        // row ranges of each group
  float* partial;   // their sums, where there are several
};

__device__ __forceinline__ v16f mfma_bf16(v4u a, v4u b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
}

constexpr int kRing = 3;    // steps whose rows and scales are in registers or on their way
constexpr int kPanel8 = 8;  // k tiles of a panel

template <bool kF32, bool kGather>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void grad_kernel(GradLaunch g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[2 * kBuf];
  __shared__ __attribute__((aligned(16))) float scl[2][4][kStepRows];  // dy's scale x x's: [n block][k block]
  const Fp8bGradArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroup b runs on XCD b % 8, which takes a contiguous eighth of an expert's
  // tiles, in panels of eight k tiles: a compact block that shares its rows in L2.
  const int tiles = g.ntn * g.ntk, per = (tiles + 7) / 8, tile = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (tile >= tiles) return;  // uniform: before any barrier
  const int panel = tile / (g.ntn * kPanel8), rest = tile - panel * (g.ntn * kPanel8);
  const int wide = min(kPanel8, g.ntk - panel * kPanel8);
  const int tn = rest / wide, tk = panel * kPanel8 + rest % wide, e = (int)blockIdx.y, part = (int)blockIdx.z;
  int begin = 0, end = a.P;
  if (a.offsets) {
    begin = min(max(a.offsets[e], 0), a.P);
    end = min(max(a.offsets[e + 1], begin), a.P);
  }
  if (g.parts > 1) {  // whole steps to each part
    const int steps = (end - begin + kStepRows - 1) / kStepRows, each = (steps + g.parts - 1) / g.parts;
    const int first = begin + (int)min((long)part * each * kStepRows, (long)(end - begin));
    end = (int)min((long)first + (long)each * kStepRows, (long)end);
    begin = first;
  }
  const int steps = (end - begin + kStepRows - 1) / kStepRows;
  auto row_of = [&](int step, int r) { return (int)min((long)begin + (long)kStepRows * step + r, (long)end - 1); };

  // Conversion: this thread's four columns of rows 8 o .. 8 o + 7 of a step.  The
  // loads of a step go out kRing steps before its conversion, the row indices that
  // they need kRing steps before that.
  const bool is_x = wave >= 4;
  const int o = wave & 3;
  const int width = is_x ? a.K : a.N;
  const int col = min(kTile * (is_x ? tk : tn) + 4 * lane, width - 4);  // columns past the last: not stored
  const uint8_t* codes = (is_x ? a.xq : a.yq) + col;
  uint32_t raw[kRing][8];
  int entry[kRing];  // lanes 0 .. 7: x rows of the step's rows 8 o + lane
  auto load_entries = [&](int step, int slot) {
    if constexpr (kGather)
      if (is_x) entry[slot] = entry_row(a.rows, row_of(step, 8 * o + (lane & 7)), a.div, a.X);
  };
  auto load_codes = [&](int step, int slot) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      int s = row_of(step, 8 * o + i);
      if constexpr (kGather)
        if (is_x) s = __builtin_amdgcn_readlane(entry[slot], i);
      raw[slot][i] = *reinterpret_cast<const uint32_t*>(codes + (size_t)s * width);
    }
  };
  // scales: threads 0 .. 127, one product each
  const int sn = (tid >> 6) & 1, sk = (tid >> 5) & 1, sr = tid & 31;
  const int nb = min(2 * tn + sn, a.N / 128 - 1), kb = min(2 * tk + sk, a.K / 128 - 1);
  const float* ys = a.ys + (size_t)nb * a.P;
  const float* xs = a.xs + (size_t)kb * a.X;
  float fy[kRing], fx[kRing];
  int fentry[kRing];
  auto load_scale_entries = [&](int step, int slot) {
    if constexpr (kGather)
      if (wave < 2) fentry[slot] = entry_row(a.rows, row_of(step, sr), a.div, a.X);
  };
  auto load_scales = [&](int step, int slot) {
    if (wave < 2) {
      const int s = row_of(step, sr);
      fy[slot] = ys[s];
      fx[slot] = xs[kGather ? fentry[slot] : s];
    }
  };
  auto put_scales = [&](int step, int slot) {
    if (wave < 2) scl[step & 1][2 * sn + sk][sr] = begin + kStepRows * (long)step + sr < end ? fy[slot] * fx[slot] : 0.0f;
  };
  auto convert = [&](int step, int slot) {
    uint8_t* buf = lds + (step & 1) * kBuf;
    float v[8][4];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const v2f lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[slot][i], false);
      const v2f hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)raw[slot][i], true);
      v[i][0] = lo[0], v[i][1] = lo[1], v[i][2] = hi[0], v[i][3] = hi[1];
    }
    auto put = [&](uint8_t* panel, const float (&k)[8], bool scaled) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        v4u w;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          w[i] = scaled ? f32x2_to_bf16(v[2 * i][c] * k[2 * i], v[2 * i + 1][c] * k[2 * i + 1])
                        : f32x2_to_bf16(v[2 * i][c], v[2 * i + 1][c]);
        *reinterpret_cast<v4u*>(panel + (o * kTile + c * 64 + lane) * 16) = w;
      }
    };
    if (is_x) {
      const float none[8] = {};
      put(buf + 2 * kPanel, none, false);
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const float* p = &scl[step & 1][2 * (lane >> 5) + b][8 * o];
        const v4f k0 = *reinterpret_cast<const v4f*>(p), k1 = *reinterpret_cast<const v4f*>(p + 4);
        const float k[8] = {k0[0], k0[1], k0[2], k0[3], k1[0], k1[1], k1[2], k1[3]};
        put(buf + b * kPanel, k, true);
      }
    }
  };

  // products: n rows 4 q + c for q of half wn % 2, c = 2 (wn / 2) + {0, 1}; k columns of block wk
  const int wn = wave >> 1, wk = wave & 1, r = lane & 31, h = lane >> 5;
  v16f acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;
  // Step j: its products from one buffer while step j + 1 is converted into the
  // other; put_scales(j + 2), which the next step's conversion reads.  Loads past
  // the last step read its rows again.
  auto iterate = [&](int j, int slot) {  // slot: (j + 1) % kRing
    const uint8_t* buf = lds + (j & 1) * kBuf;
    const uint8_t* pa = buf + wk * kPanel + (size_t)(128 * (wn >> 1) + 32 * (wn & 1) + r) * 16;
    const uint8_t* pb = buf + 2 * kPanel + (size_t)(32 * wk + r) * 16;
    convert(j + 1, slot);
    load_codes(j + 1 + kRing, slot);
    load_entries(j + 1 + 2 * kRing, slot);
#pragma unroll
    for (int u = 0; u < 2; ++u) {  // 16 rows
      const size_t at = (size_t)((2 * u + h) * kTile) * 16;
      v4u fa[2], fb[4];
#pragma unroll
      for (int i = 0; i < 2; ++i) fa[i] = *reinterpret_cast<const v4u*>(pa + at + 64 * 16 * i);
#pragma unroll
      for (int c = 0; c < 4; ++c) fb[c] = *reinterpret_cast<const v4u*>(pb + at + 64 * 16 * c);
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[i][c] = mfma_bf16(fa[i], fb[c], acc[i][c]);
    }
    const int next = (slot + 1) % kRing;
    put_scales(j + 2, next);
    load_scales(j + 2 + kRing, next);
    load_scale_entries(j + 2 + 2 * kRing, next);
    // (not __syncthreads, which would wait for the loads of the steps to come)
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  if (steps > 0) {
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
      load_entries(q, q);
      load_scale_entries(q, q);
    }
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
      load_codes(q, q);
      load_scales(q, q);
      load_entries(kRing + q, q);
      load_scale_entries(kRing + q, q);
    }
    put_scales(0, 0);
    put_scales(1, 1);
    load_scales(kRing, 0);
    load_scales(kRing + 1, 1);
    load_scale_entries(2 * kRing, 0);
    load_scale_entries(2 * kRing + 1, 1);
    __syncthreads();
    convert(0, 0);
    load_codes(kRing, 0);
    load_entries(2 * kRing, 0);
    __syncthreads();
    // (the last step converts one that does not exist, whose scales are zeros)
    int j = 0;
    for (; j + kRing <= steps; j += kRing) {
      iterate(j, 1);
      iterate(j + 1, 2);
      iterate(j + 2, 0);
    }
    if (j < steps) iterate(j, 1);
    if (j + 1 < steps) iterate(j + 1, 2);
  }

  // element v of a lane: row q = 32 (wn % 2) + 8 (v / 4) + 4 h + v % 4, its four columns in the four tiles
  const int k0 = kTile * tk + 128 * wk + 4 * r;
  if (k0 >= a.K) return;
  const size_t plane = (size_t)a.N * a.K;
  float* sums = g.parts > 1 ? g.partial + ((size_t)part * a.E + e) * plane : static_cast<float*>(a.dw) + (size_t)e * plane;
  uint16_t* half = static_cast<uint16_t*>(a.dw) + (size_t)e * plane;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int v = 0; v < 16; ++v) {
      const int n = kTile * tn + 4 * (32 * (wn & 1) + 8 * (v >> 2) + 4 * h + (v & 3)) + 2 * (wn >> 1) + i;
      if (n >= a.N) continue;
      const size_t at = (size_t)n * a.K + k0;
      const v4f s = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
      if (kF32 || g.parts > 1)
        __builtin_nontemporal_store(s, reinterpret_cast<global<v4f>*>((uintptr_t)(sums + at)));
      else
        __builtin_nontemporal_store(v2u{f32x2_to_bf16(s[0], s[1]), f32x2_to_bf16(s[2], s[3])},
                                    reinterpret_cast<global<v2u>*>((uintptr_t)(half + at)));
    }
}

// The parts' sums, in the order of the rows.
template <bool kF32>
__global__ __launch_bounds__(256) void join_kernel(const float* __restrict__ partial, int parts, size_t n4,
                                                   void* __restrict__ dw) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= n4) return;
  const v4f* p = reinterpret_cast<const v4f*>(partial) + i;
  v4f s = *p;
  for (int k = 1; k < parts; ++k) s += p[k * n4];
  if constexpr (kF32)
    static_cast<v4f*>(dw)[i] = s;
  else
    static_cast<v2u*>(dw)[i] = v2u{f32x2_to_bf16(s[0], s[1]), f32x2_to_bf16(s[2], s[3])};
}

// Row ranges of each group: as many as there are idle CUs for, each of 256 rows
// and more on average.
int row_parts(long P, int E, int N, int K) {
  const long tiles = (long)E * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
  return (int)max(min((long)256 / tiles, P / E / 256), 1l);
}

}  // namespace

size_t fp8b_grad_ws_bytes(long P, int E, int N, int K) {
  const int parts = row_parts(P, E, N, K);
  return parts > 1 ? 4 * (size_t)parts * E * N * K : 0;
}

hipError_t launch_fp8b_grad(const Fp8bGradArgs& a, bool fp32_out, void* ws, hipStream_t st) {
  const int parts = row_parts(a.P, a.E, a.N, a.K);
  const GradLaunch g{a, (a.N + kTile - 1) / kTile, (a.K + kTile - 1) / kTile, parts, static_cast<float*>(ws)};
  const dim3 grid((unsigned)((g.ntn * g.ntk + 7) / 8 * 8), (unsigned)a.E, (unsigned)parts);
  if (fp32_out) {
    if (a.rows)
      hipLaunchKernelGGL((grad_kernel<true, true>), grid, dim3(512), 0, st, g);
    else
      hipLaunchKernelGGL((grad_kernel<true, false>), grid, dim3(512), 0, st, g);
  } else {
    if (a.rows)
      hipLaunchKernelGGL((grad_kernel<false, true>), grid, dim3(512), 0, st, g);
    else
      hipLaunchKernelGGL((grad_kernel<false, false>), grid, dim3(512), 0, st, g);
  }
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || parts == 1) return e;
  const size_t n4 = (size_t)a.E * a.N * a.K / 4;
  const dim3 join((unsigned)((n4 + 255) / 256));
  if (fp32_out)
    hipLaunchKernelGGL(join_kernel<true>, join, dim3(256), 0, st, g.partial, parts, n4, a.dw);
  else
    hipLaunchKernelGGL(join_kernel<false>, join, dim3(256), 0, st, g.partial, parts, n4, a.dw);
  return hipGetLastError();
}

}  // namespace moe
