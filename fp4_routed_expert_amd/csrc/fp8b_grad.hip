// Gradient of the weights from FP8 rows with block scales of 128:
// dw[e, n, k] = sum over the rows s of group e of dy[s, n] x[r(s), k].
//
// The sum runs over rows, along which both scales vary, so the products are made
// in the fp16 matrix cores (the rate of bf16, three bits more).  x's codes are
// exact in fp16; dy's codes are multiplied by both scales, once for each of the
// tile's two blocks of k.  The scales' products are divided first by a power of two
// that brings the largest of the group's rows to [2^4, 2^6), so that the range of
// fp16 costs nothing: a product's two roundings, of the scale and of the product, are
// 2^-10 of it, and for rows whose scales are 2^-20 of the largest and less 2^-31 of
// that.  The sums are fp32.
//
// A workgroup makes 256 x 256 outputs of one expert, eight waves of 64 x 128 by
// v_mfma_f32_32x32x16_f16, in steps of 32 rows.  The matrix cores want eight
// neighbouring rows of one column in a lane: a thread reads four bytes of eight
// rows each, converts them to pairs of columns and swaps halves to pairs of rows.
// Waves 0-3 convert dy, waves 4-7 x, each between its MFMAs; a SIMD has one of
// either.  LDS holds [eight rows][column c of four][group of four columns], 16 bytes
// each, so that writes and reads run along neighbouring addresses; a lane ends with
// four neighbouring outputs.
//
// Where the tiles are fewer than the CUs, the rows are split; the parts' sums go
// through memory in fp32 and are added in the order of the rows.
#include <type_traits>

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

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v16f mfma_f16(v4u a, v4u b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) * __builtin_bit_cast(v2h, b));
}

constexpr int kRing = 3;    // steps whose rows and scales are in registers or on their way, and steps in LDS
constexpr int kPanel8 = 8;  // k tiles of a panel

template <bool kF32, bool kGather>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void grad_kernel(GradLaunch g) {
  __shared__ __attribute__((aligned(16))) uint8_t lds[kRing * kBuf];
  __shared__ __attribute__((aligned(16))) _Float16 scl[2][4][kStepRows];  // the scales' products: [n block][k block]
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
  // row r of a step, past the group its last one
  auto row_of = [&](int step, int r) { return (int)min((uint32_t)begin + (uint32_t)(kStepRows * step + r), (uint32_t)(end - 1)); };

  // The largest scales of the group's rows in the tile's blocks, as powers of two:
  // y_exp and x_exp with scale < 2^exp.
  const int nb0 = min(2 * tn, a.N / 128 - 1), nb1 = min(2 * tn + 1, a.N / 128 - 1);
  const int kb0 = min(2 * tk, a.K / 128 - 1), kb1 = min(2 * tk + 1, a.K / 128 - 1);
  auto x_row = [&](int s) { return kGather ? entry_row(a.rows, s, a.div, a.X) : s; };
  int y_exp[2], x_exp[2];
  {
    const float* p[4] = {a.ys + (size_t)nb0 * a.P, a.ys + (size_t)nb1 * a.P, a.xs + (size_t)kb0 * a.X,
                         a.xs + (size_t)kb1 * a.X};
    float top[4] = {0.f, 0.f, 0.f, 0.f};
    for (int s = begin + tid; s < end; s += 512) {
      const int x = x_row(s);
#pragma unroll
      for (int i = 0; i < 4; ++i) top[i] = fmaxf(top[i], fabsf(p[i][i < 2 ? s : x]));
    }
    __shared__ float tops[8][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float m = max_lanes_xor16_32(row16_max(top[i]));
      if (lane == 0) tops[wave][i] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float m = 0.0f;
#pragma unroll
      for (int w = 0; w < 8; ++w) m = fmaxf(m, tops[w][i]);
      const int exp = (int)wave_u32((uint32_t)__builtin_amdgcn_frexp_expf(m));
      (i < 2 ? y_exp[i & 1] : x_exp[i & 1]) = exp;
    }
  }
  constexpr int kUp = 6;  // the scales' products are brought below 2^kUp, times 448 below 2^15

  // products: n rows 4 q + c for q of half wn % 2 (block wn % 2), c = 2 (wn / 2) + {0, 1}; k columns of block wk
  const int wn = wave >> 1, wk = wave & 1, r = lane & 31, h = lane >> 5;
  v16f acc[2][4];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  // The loop of a wave that converts x (kIsX) or dy: four columns a thread of rows
  // 8 o .. 8 o + 7 of a step.  The loads of a step go out kRing steps before its
  // conversion, the row indices that they need kRing steps before that.
  auto run = [&](auto is_x) {
    constexpr bool kIsX = decltype(is_x)::value, kIndexed = kIsX && kGather;
    const int o = wave & 3;
    const int width = kIsX ? a.K : a.N;
    const uint32_t col = (uint32_t)min(kTile * (kIsX ? tk : tn) + 4 * lane, width - 4);  // columns past the last: not stored
    const uint8_t* codes = kIsX ? a.xq : a.yq;  // (uniform: a row's address is made by the scalar unit)
    uint32_t raw[kRing][8];
    int entry[kRing];  // lanes 0 .. 7: x rows of the step's rows 8 o + lane
    auto load_entries = [&](int step, int slot) {
      if constexpr (kIndexed) entry[slot] = x_row(row_of(step, 8 * o + (lane & 7)));
    };
    auto load_codes = [&](int step, int slot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int s = kIndexed ? __builtin_amdgcn_readlane(entry[slot], i) : row_of(step, 8 * o + i);
        raw[slot][i] = *reinterpret_cast<const uint32_t*>(wave_ptr(codes + (size_t)s * (size_t)width) + col);
      }
    };
    // scales: a dy wave one k block and n block each (two waves an n block), for 32 rows; its lanes' upper half idles
    const int sn = o >> 1, sk = o & 1, sr = lane & 31;
    const float* ys = a.ys + (size_t)(sn ? nb1 : nb0) * a.P;
    const float* xs = a.xs + (size_t)(sk ? kb1 : kb0) * a.X;
    const int up_y = -y_exp[sn], up_x = kUp - x_exp[sk];
    float fy[kRing], fx[kRing];
    int fentry[kRing];
    auto load_scale_entries = [&](int step, int slot) {
      if constexpr (!kIsX && kGather) fentry[slot] = x_row(row_of(step, sr));
    };
    auto load_scales = [&](int step, int slot) {
      if constexpr (!kIsX) {
        const int s = row_of(step, sr);
        fy[slot] = ys[s];
        fx[slot] = xs[kGather ? fentry[slot] : s];
      }
    };
    auto put_scales = [&](int step, int slot) {
      if constexpr (!kIsX) {
        const float k = __builtin_amdgcn_ldexpf(fy[slot], up_y) * __builtin_amdgcn_ldexpf(fx[slot], up_x);
        scl[step & 1][2 * sn + sk][sr] = (_Float16)((uint32_t)begin + (uint32_t)(kStepRows * step + sr) < (uint32_t)end ? k : 0.0f);
      }
    };
    // a step's conversion in pieces: two rows to fp16; the scales; each column
    uint32_t v[8][2], k[2][4];
    auto rows_to_half = [&](int m, int slot) {
#pragma unroll
      for (int i = 2 * m; i < 2 * m + 2; ++i) {
        v[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)raw[slot][i], 1.0f, false));
        v[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)raw[slot][i], 1.0f, true));
      }
    };
    auto get_scales = [&](int step) {
      if constexpr (!kIsX) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const v4u t = *reinterpret_cast<const v4u*>(&scl[step & 1][2 * (lane >> 5) + b][8 * o]);
          k[b][0] = t.x, k[b][1] = t.y, k[b][2] = t.z, k[b][3] = t.w;
        }
      }
    };
    auto put_column = [&](int slot, int c) {
      uint8_t* to = lds + slot * kBuf + (kIsX ? 2 * kPanel : 0) + (o * kTile + c * 64 + lane) * 16;
      v4u w;
#pragma unroll
      for (int i = 0; i < 4; ++i)  // halves c % 2 of rows 2 i and 2 i + 1
        w[i] = __builtin_amdgcn_perm(v[2 * i + 1][c >> 1], v[2 * i][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
      if constexpr (kIsX) {
        *reinterpret_cast<v4u*>(to) = w;
      } else {
#pragma unroll
        for (int b = 0; b < 2; ++b)
          *reinterpret_cast<v4u*>(to + b * kPanel) =
              v4u{mul_pair(w[0], k[b][0]), mul_pair(w[1], k[b][1]), mul_pair(w[2], k[b][2]), mul_pair(w[3], k[b][3])};
      }
    };
    // fragments of 16 rows u of the step in a buffer
    v4u fa[2], fb[4];
    const uint8_t* pa = lds + wk * kPanel + (h * kTile + 128 * (wn >> 1) + 32 * (wn & 1) + r) * 16;
    const uint8_t* pb = lds + 2 * kPanel + (h * kTile + 32 * wk + r) * 16;
    auto read_a = [&](int slot, int u, int i) {
      fa[i] = *reinterpret_cast<const v4u*>(pa + slot * kBuf + (2 * u * kTile + 64 * i) * 16);
    };
    auto read_b = [&](int slot, int u, int c) {
      fb[c] = *reinterpret_cast<const v4u*>(pb + slot * kBuf + (2 * u * kTile + 64 * c) * 16);
    };
    // Step j, j % kRing = slot: its products, while step j + 2 is converted into the
    // buffer of step j - 1 and the scales of step j + 3 go to LDS; a fragment's
    // registers take its successor's (at the end the next step's, which the last
    // barrier has published) behind their last use.  Loads past the last step read
    // its rows again.
    auto iterate = [&](int j, int slot) {
      const int next = (slot + 1) % kRing, to = (slot + 2) % kRing;
#pragma unroll
      for (int m = 0; m < 16; ++m) {
        const int u = m >> 3, i = (m >> 2) & 1, c = m & 3;
        acc[i][c] = mfma_f16(fa[i], fb[c], acc[i][c]);
        if (c == 3) read_a(u ? next : slot, 1 - u, i);
        if (i == 1) read_b(u ? next : slot, 1 - u, c);
        if (m < 4) rows_to_half(m, to);
        if (m == 2) get_scales(j + 2);
        if (m == 4) {
          load_codes(j + 2 + kRing, to);
          load_entries(j + 2 + 2 * kRing, to);
        }
        if (m >= 5 && m % 3 == 2) put_column(to, (m - 5) / 3);
        __builtin_amdgcn_sched_barrier(0);
      }
      put_scales(j + 3, slot);
      load_scales(j + 3 + kRing, slot);
      load_scale_entries(j + 3 + 2 * kRing, slot);
      // (not __syncthreads, which would wait for the loads of the steps to come)
      asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    };
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
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      get_scales(q);
#pragma unroll
      for (int m = 0; m < 4; ++m) rows_to_half(m, q);
#pragma unroll
      for (int c = 0; c < 4; ++c) put_column(q, c);
      load_codes(kRing + q, q);
      load_entries(2 * kRing + q, q);
    }
    __syncthreads();
    put_scales(2, 2);
#pragma unroll
    for (int q = 0; q < kRing; ++q) {
      load_scales(kRing + q, q);
      load_scale_entries(2 * kRing + q, q);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) read_a(0, 0, i);
#pragma unroll
    for (int c = 0; c < 4; ++c) read_b(0, 0, c);
    __syncthreads();
    // (the last steps convert ones that do not exist, whose scales are zeros)
    int j = 0;
    for (; j + kRing <= steps; j += kRing) {
      iterate(j, 0);
      iterate(j + 1, 1);
      iterate(j + 2, 2);
    }
    if (j < steps) iterate(j, 0);
    if (j + 1 < steps) iterate(j + 1, 1);
  };
  if (steps > 0) {
    if (wave >= 4)
      run(std::true_type{});
    else
      run(std::false_type{});
  }
  const int down = (wn & 1 ? y_exp[1] : y_exp[0]) + (wk ? x_exp[1] : x_exp[0]) - kUp;

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
      const v4f s = {__builtin_amdgcn_ldexpf(acc[i][0][v], down), __builtin_amdgcn_ldexpf(acc[i][1][v], down),
                     __builtin_amdgcn_ldexpf(acc[i][2][v], down), __builtin_amdgcn_ldexpf(acc[i][3][v], down)};
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
