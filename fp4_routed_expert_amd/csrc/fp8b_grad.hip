// Gradient of the weights from FP8 rows with block scales of 128:
// dw[e, n, k] = sum over the rows s of group e of dy[s, n] x[r(s), k].
//
// The sum runs over rows, along which both scales vary, so the products are made
// in the fp16 matrix cores (the rate of bf16, three bits more).  x's codes are
// exact in fp16; dy's codes are multiplied by both scales.  The scales' products are
// divided first by a power of two that brings the largest of the group's rows to [2^4,
// 2^6), so that the range of fp16 costs little: a row's two roundings, of the
// scales' product and of the code times it, are 2^-10 of it, and where its scales'
// product is less than 2^-18 of the largest row's 2^-29 of what that would make.  (The
// largest product of a row, not that of the largest dy and the largest x scale: an
// outlier of each in different rows would cost the others their bits.)  The sums are
// fp32.
//
// A workgroup makes 256 x 256 outputs of one expert, eight waves of 64 x 128 by
// v_mfma_f32_32x32x16_f16, in steps of 32 rows.  The matrix cores want eight
// neighbouring rows of one column in a lane.  The codes go to LDS by LDS-DMA as they
// are, four steps of them; transposing LDS reads bring eight rows of a column to each
// lane, which converts them itself.  (A column of dy is converted by two waves, one of
// x by four.  Converted once, by one wave each, and handed on through LDS in fp16, the
// LDS port was the limit: 16384 rows, 4096 x 7168, 923 us, now 797; four waves of 128 x
// 128, which convert less but leave a SIMD with one wave, 860.)
//
// Bound by what two waves per SIMD issue (the matrix cores are busy 58 % of the time,
// 66 % of the rounds that 448 tiles take on 256 CUs) and by the power limit: 1.85 GHz.
// 16384 rows, 4096 x 7168: 1.2 PFLOP/s; 64 experts of 432 rows, 4096 x 1536: 437 us,
// 0.8 PFLOP/s, where a tile's start and its stores count.
//
// Where the tiles are fewer than the CUs, the rows are split; the parts' sums go
// through memory in fp32 and are added in the order of the rows.
#include <type_traits>
#include <utility>

#include "fp8b.h"
#include "tiled.h"

namespace moe {
namespace {

constexpr int kTile = 256;
constexpr int kStepRows = 32;
constexpr int kCodes = kTile * kStepRows;  // bytes of one operand's step
constexpr int kRing = 4;                   // steps in LDS
constexpr int kPanelTiles = 8;             // k tiles of a panel of the walk
// LDS: the steps' codes (dy, x), their scales (dy's blocks 0 and 1, x's; 32 rows each,
// twice), two steps' products of them, row indices of twice as many steps
constexpr int kOffScale = kRing * 2 * kCodes, kOffProd = kOffScale + kRing * 1024;
constexpr int kOffIdx = kOffProd + 2 * 256, kOffTop = kOffIdx + 2 * kRing * 256;
constexpr int kOut = 16 * 1024;  // of a wave, at the end: 64 rows of 128 outputs in bf16, or 32 in fp32
constexpr int kLds = 8 * kOut;
static_assert(kOffTop + 128 <= kLds && kLds <= 160 * 1024, "LDS");

struct GradLaunch {
  Fp8bGradArgs a;
  const int32_t* xrows;  // x row of each row of dy, or null: the same row
  int ntn, ntk;          // tiles of an expert
  int parts;             // row ranges of each group
  float* partial;        // their sums, where there are several
};

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef int v2i __attribute__((ext_vector_type(2)));

__device__ __forceinline__ v16f mfma_f16(v4u a, v4u b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) * __builtin_bit_cast(v2h, b));
}

// Each lane of 16 gives the address of eight neighbouring bytes, the lanes 2 i and 2 i
// + 1 those of row i, and gets its column's byte of the eight rows.
__device__ __forceinline__ v2i lds_columns(uint32_t addr) {
  return __builtin_amdgcn_ds_read_tr8_b64_v2i32(reinterpret_cast<__attribute__((address_space(3))) v2i*>((uintptr_t)addr));
}
// Eight codes as fp16.
__device__ __forceinline__ v4u to_half(v2i c) {
  v4u w;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[2 * i] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, false));
    w[2 * i + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[i], 1.0f, true));
  }
  return w;
}

// x row of each row of dy
__global__ __launch_bounds__(1024) void entries_kernel(Fp8bGradArgs a, int32_t* __restrict__ xrows) {
  const int p = (int)(blockIdx.x * 1024 + threadIdx.x);
  if (p < a.P) xrows[p] = entry_row(a.rows, p, a.div, a.X);
}

// LDS-DMA of 16 bytes for each lane from an address of its own.
__device__ __forceinline__ void dma16_lanes(const uint8_t* p, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, off"
      :
      : "v"(p), "s"(wave_u32(lds))
      : "memory");
}

// f(0), f(1), ... with constants, so that what it indexes is in registers from the start.
template <class F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

constexpr int kUp = 6;  // the scales' products are brought below 2^kUp, times 448 below 2^15

// A scale's exponent: |v| < 2^exponent.  (What is below 2^-126, zeros too, counts as
// 2^-126: fp16's normal numbers reach 2^-18 below the largest row.  A NaN or an
// infinity shows in the outputs whatever they are divided by.)
__device__ __forceinline__ int scale_exponent(float v) { return (int)((__float_as_uint(v) >> 23) & 255u) - 126; }
// Maximum over a wave.
__device__ __forceinline__ int wave_max_i32(int v) { return (int)(max_lanes_xor16_32_u32(row16_max_u32((uint32_t)v + 512u)) - 512u); }

// What the loop is given.
struct GradCtx {
  uint32_t lds0;
  int lane, wave;
  int begin, end, steps;  // rows of the group (or its part), and their steps
  const uint8_t* codes;   // of what this wave moves: dy or x
  int width, tile;        // its columns, and the tile's place among them
  const float* scales;    // of the blocks that a dy wave moves
  const int32_t* xrows;
  int up_y, up_x;         // powers of two for a dy wave's scales, whose products come to 2^kUp less
};

// The loop of a wave; it moves rows 8 o .. 8 o + 7 of every step of x (kIsX) or dy.
template <bool kIsX, bool kGather>
__device__ __forceinline__ void run_rows(const GradCtx& g, v16f (&acc)[4][2]) {
  const uint32_t lds0 = g.lds0;
  const int lane = g.lane, wave = g.wave, begin = g.begin, steps = g.steps, width = g.width;
  const int wn = wave >> 1, wk = wave & 1, h = lane >> 5;
  const int o = wave & 3;
  const uint8_t* base = g.codes;
  const uint32_t last = (uint32_t)(g.end - 1);
  auto row_at = [&](int step, int r) { return min((uint32_t)begin + (uint32_t)(kStepRows * step + r), last); };
  auto entry = [&](int step, int r) {  // of the index ring
    return (uint32_t)lds_i32(lds0 + kOffIdx + 256u * (uint32_t)(step & (2 * kRing - 1)) + 4u * (uint32_t)r);
  };
  // A row's piece p of 16 bytes lies at p ^ 2 (row % 8), so that eight rows' pieces of
  // neighbouring columns are in different banks.  (Columns past the last one read the
  // last 16: not stored.)
  uint32_t piece[2];
#pragma unroll
  for (int t = 0; t < 2; ++t)
    piece[t] = (uint32_t)min(kTile * g.tile + 16 * ((lane & 15) ^ (2 * (4 * t + (lane >> 4)))), width - 16);
  // Loads of a step: codes, scales (dy wave o those of dy's block o, or of x's block o -
  // 2) and, much further ahead, row indices.  A lane's offsets from the step's first
  // row change only where the rows end.
  uint32_t code_off[2], scale_off, entry_off;
  auto first_of = [&](int step) { return wave_u32(min((uint32_t)begin + (uint32_t)(kStepRows * step), last)); };
  auto word_of = [&](int step) { return 4u * min((uint32_t)(lane & 31), last - first_of(step)); };
  auto set_offsets = [&](int codes, int scales, int entries) {  // of these steps
#pragma unroll
    for (int t = 0; t < 2; ++t)
      code_off[t] = min((uint32_t)(8 * o + 4 * t + (lane >> 4)), last - first_of(codes)) * (uint32_t)width + piece[t];
    scale_off = word_of(scales);
    entry_off = word_of(entries);
  };
  auto load_codes = [&](int step, int slot, int t) {
    const uint32_t to = lds0 + (uint32_t)((2 * slot + (kIsX ? 1 : 0)) * kCodes + 2048 * o + 1024 * t);
    if constexpr (kIsX && kGather)
      dma16_lanes(base + (size_t)entry(step, 8 * o + 4 * t + (lane >> 4)) * (size_t)width + piece[t], to);
    else
      dma16(base + (size_t)first_of(step) * (size_t)width, code_off[t], to);
  };
  auto load_scales = [&](int step, int slot) {
    if constexpr (!kIsX) {
      const uint32_t to = lds0 + (uint32_t)(kOffScale + 1024 * slot + 256 * o);
      if (kGather && o >= 2)
        dma4_lanes(reinterpret_cast<const uint8_t*>(g.scales + entry(step, lane & 31)), to);
      else
        dma4(reinterpret_cast<const uint8_t*>(g.scales + first_of(step)), scale_off, to);
    }
  };
  auto load_entries = [&](int step) {
    if constexpr (kIsX && kGather)
      dma4(reinterpret_cast<const uint8_t*>(g.xrows + first_of(step)), entry_off,
           lds0 + (uint32_t)(kOffIdx + 256 * (step & (2 * kRing - 1))));
  };
  constexpr int kLoads = kIsX ? (kGather ? 3 : 2) : 3;  // of a step
  // products of the scales, one of the four pairs of blocks a dy wave, for 32 rows (the upper lanes repeat them)
  float fy, fx;
  const uint32_t scales_at = lds0 + (uint32_t)(kOffScale + 256 * (o >> 1) + 4 * (lane & 31));
  const uint32_t x_scales_at = lds0 + (uint32_t)(kOffScale + 512 + 256 * (o & 1) + 4 * (lane & 31));
  const uint32_t product_at = lds0 + (uint32_t)(kOffProd + 64 * o + 2 * (lane & 31));
  auto get_scales = [&](int slot) {
    if constexpr (!kIsX) {
      fy = __int_as_float(lds_i32(scales_at + 1024u * slot));
      fx = __int_as_float(lds_i32(x_scales_at + 1024u * slot));
    }
  };
  auto put_products = [&](int step, int slot) {
    if constexpr (!kIsX) {
      float k = __builtin_amdgcn_ldexpf(fy, g.up_y) * __builtin_amdgcn_ldexpf(fx, g.up_x) * (float)(1 << kUp);
      if (step >= steps - 1)  // rows past the last one
        k = (uint32_t)begin + (uint32_t)(kStepRows * step + (lane & 31)) <= last ? k : 0.0f;
      *reinterpret_cast<__attribute__((address_space(3))) _Float16*>((uintptr_t)(product_at + 256u * (slot & 1))) = (_Float16)k;
    }
  };
  // A wave's 64 columns of dy (f = 4, 5) and 128 of x (f < 4), for 16 rows u of a step:
  // lane l holds eight rows 8 (l / 32) of column l % 32 of 32.
  v2i raw[6];
  v4u half[2][6], k;
  uint32_t at[6];
#pragma unroll
  for (int f = 0; f < 6; ++f) {
    const int p = (f < 4 ? 8 * wk + 2 * f : 4 * wn + 2 * (f - 4)) + ((lane >> 4) & 1), r = (lane & 15) >> 1;
    at[f] = opaque(lds0 + (uint32_t)((f < 4 ? kCodes : 0) + 256 * (8 * h + r) + 16 * (p ^ (2 * r)) + 8 * (lane & 1)));
  }
  const uint32_t my_products = opaque(lds0 + (uint32_t)(kOffProd + 64 * (2 * (wn >> 1) + wk) + 16 * h));
  auto get_codes = [&](int slot, int u, int f) { raw[f] = lds_columns(at[f] + (uint32_t)(slot * 2 * kCodes + 4096 * u)); };
  auto get_products = [&](int slot, int u) { k = lds_v4(my_products + (uint32_t)(256 * (slot & 1) + 32 * u)); };
  auto convert = [&](int u, int f) __attribute__((always_inline)) {
    v4u w = to_half(raw[f]);
    if (f >= 4) w = v4u{mul_pair(w[0], k[0]), mul_pair(w[1], k[1]), mul_pair(w[2], k[2]), mul_pair(w[3], k[3])};
    half[u][f] = w;
  };
  // the first steps' codes, scales and (by plain loads) indices
  if constexpr (kGather)
    *reinterpret_cast<__attribute__((address_space(3))) int*>((uintptr_t)(lds0 + (uint32_t)(kOffIdx + 256 * wave) + 4u * (uint32_t)lane)) =
        g.xrows[row_at(wave, lane & 31)];
  __syncthreads();
  each([&](auto q_) {
    constexpr int q = decltype(q_)::value;
    set_offsets(q, q, q);
    load_codes(q, q, 0);
    load_codes(q, q, 1);
    load_scales(q, q);
  }, std::make_integer_sequence<int, kRing>{});
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    get_scales(q);
    put_products(q, q);
  }
  __syncthreads();
  set_offsets(kRing, kRing, kRing);
  load_scales(kRing, 0);
  get_products(0, 0);
#pragma unroll
  for (int f = 0; f < 6; ++f) {
    get_codes(0, 0, f);
    convert(0, f);
    get_codes(0, 1, f);
  }
  get_products(0, 1);
  // Step j, in place j % kRing: under the products of 16 rows the next 16 rows' codes
  // are converted, and those behind them read.  The barrier publishes step j + 1, its
  // scales' products and the scales of step j + 2, and frees step j's place, whose
  // codes are in registers.  (Loads past the last step read its last row again; a step
  // past the last has products of zero.)  What a wave issues counts: an instruction
  // takes it eight clocks, an MFMA 32, and a SIMD has two waves, so that the places are
  // constants and the loads' offsets are kept (836 us without, now 797).
  int j = 0;
  auto step = [&](auto place) __attribute__((always_inline)) {
    constexpr int p = decltype(place)::value, next = (p + 1) % kRing, after = (p + 2) % kRing;
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((kRing - 2) * kLoads) : "memory");
    if (j + (kGather ? 2 * kRing : kRing + 1) >= steps - 1)  // the rows end in these loads
      set_offsets(j + kRing, j + kRing + 1, j + 2 * kRing);
    each([&](auto m_) __attribute__((always_inline)) {
      constexpr int m = decltype(m_)::value, u = m >> 3, q = m & 7, c = q >> 1, i = q & 1;
      acc[c][i] = mfma_f16(half[u][c], half[u][4 + i], acc[c][i]);
      if constexpr (q < 6) {
        convert(u ^ 1, q);
        get_codes(next, u, q);
      }
      if (q == 6) get_products(next, u);
      if (m == 0) get_scales(after);
      if (m == 6) load_codes(j + kRing, p, 0);
      if (m == 7) load_codes(j + kRing, p, 1);
      if (m == 14) load_scales(j + kRing + 1, next);
      if (m == 15) load_entries(j + 2 * kRing);
      if (m == 10) put_products(j + 2, after);
      if (i == 1) __builtin_amdgcn_sched_barrier(0);
    }, std::make_integer_sequence<int, 16>{});
    return ++j < steps;
  };
  static_assert(kRing == 4, "places of the loop");
  while (step(std::integral_constant<int, 0>{}) && step(std::integral_constant<int, 1>{}) &&
         step(std::integral_constant<int, 2>{}) && step(std::integral_constant<int, 3>{})) {
  }
  wait_vmcnt<0>();  // the loads past the last step land before the LDS is given back
}

template <bool kF32, bool kGather>
__global__ __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) void grad_kernel(GradLaunch g) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_u8*)lds;
  const Fp8bGradArgs& a = g.a;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  // Workgroup b runs on XCD b % 8, which takes a contiguous eighth of an expert's
  // tiles, in panels of eight k tiles: a compact block that shares its rows in L2.
  const int tiles = g.ntn * g.ntk, per = (tiles + 7) / 8, tile = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (tile >= tiles) return;  // uniform: before any barrier
  const int panel = tile / (g.ntn * kPanelTiles), rest = tile - panel * (g.ntn * kPanelTiles);
  const int wide = min(kPanelTiles, g.ntk - panel * kPanelTiles);
  const int tn = rest / wide, tk = panel * kPanelTiles + rest % wide, e = (int)blockIdx.y, part = (int)blockIdx.z;
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

  // The largest product of scales of a row of the group, for each pair of the tile's
  // blocks of dy and x, as a power of two: that of blocks i and j is below
  // 2^top[2 i + j].
  const int nb0 = min(2 * tn, a.N / 128 - 1), nb1 = min(2 * tn + 1, a.N / 128 - 1);
  const int kb0 = min(2 * tk, a.K / 128 - 1), kb1 = min(2 * tk + 1, a.K / 128 - 1);
  auto x_row = [&](int s) { return kGather ? g.xrows[s] : s; };
  int top[4] = {-252, -252, -252, -252};
  {
    const float* p[4] = {a.ys + (size_t)nb0 * a.P, a.ys + (size_t)nb1 * a.P, a.xs + (size_t)kb0 * a.X,
                         a.xs + (size_t)kb1 * a.X};
    for (long first = begin + tid; first < end; first += 4 * 512) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int s = (int)min(first + 512 * u, (long)end - 1), x = x_row(s);
        int exp[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) exp[i] = scale_exponent(p[i][i < 2 ? s : x]);
#pragma unroll
        for (int i = 0; i < 4; ++i) top[i] = max(top[i], exp[i >> 1] + exp[2 + (i & 1)]);
      }
    }
    int(*tops)[4] = reinterpret_cast<int(*)[4]>(lds + kOffTop);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = wave_max_i32(top[i]);
      if (lane == 0) tops[wave][i] = m;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      int m = tops[0][i];
#pragma unroll
      for (int w = 1; w < 8; ++w) m = max(m, tops[w][i]);
      top[i] = (int)wave_u32((uint32_t)m);
    }
  }

  const int wn = wave >> 1, wk = wave & 1;  // columns 64 wn of dy, 128 wk of x
  v16f acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int v = 0; v < 16; ++v) acc[i][j][v] = 0.0f;

  if (steps > 0) {
    const int o = wave & 3;
    GradCtx c{lds0, lane, wave, begin, end, steps, a.yq, a.N, tn, nullptr, g.xrows, 0, 0};
    if (wave >= 4) {
      c.codes = a.xq;
      c.width = a.K;
      c.tile = tk;
      run_rows<true, kGather>(c, acc);
    } else {
      c.scales = o < 2 ? a.ys + (size_t)(o ? nb1 : nb0) * a.P : a.xs + (size_t)(o == 3 ? kb1 : kb0) * a.X;
      // half to each scale: with exponents of -126 to 128 neither passes 2^128
      const int t = o == 0 ? top[0] : o == 1 ? top[1] : o == 2 ? top[2] : top[3];
      c.up_y = -t >> 1;
      c.up_x = -t - c.up_y;
      run_rows<false, kGather>(c, acc);
    }
  }
  const int down = (wn >> 1 ? (wk ? top[3] : top[2]) : (wk ? top[1] : top[0])) - kUp;

  // Element v of a lane: column n = lane % 32 of dy, column 8 (v / 4) + 4 (lane / 32) +
  // v % 4 of x.  They go through LDS (piece q of 16 bytes of row n at q ^ n), so that
  // whole rows of the wave's 128 columns are stored, past the caches: 64 experts of
  // 432 rows, 4096 x 1536, 447 us; 474 with cached stores, 530 with stores of 32 bytes of
  // a row at a time from the registers.
  __syncthreads();  // nobody reads codes any more
  const int n0 = kTile * tn + 64 * wn, k0 = kTile * tk + 128 * wk, h = lane >> 5, n = lane & 31;
  if (n0 >= a.N || k0 >= a.K) return;
  const size_t plane = (size_t)a.N * a.K, first = (size_t)n0 * a.K + k0;
  const uint32_t mine = lds0 + (uint32_t)(wave * kOut);
  auto words = [&](int row, int bytes, int q) {
    return reinterpret_cast<lds_words*>((uintptr_t)(mine + (uint32_t)(row * bytes) + 16u * (uint32_t)(q ^ (row & (bytes / 16 - 1)))));
  };
  if (kF32 || g.parts > 1) {
    float* out = (g.parts > 1 ? g.partial + ((size_t)part * a.E + e) * plane : static_cast<float*>(a.dw) + (size_t)e * plane) + first;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v4f s;
#pragma unroll
          for (int v = 0; v < 4; ++v) s[v] = __builtin_amdgcn_ldexpf(acc[c][i][4 * j + v], down);
          *words(n, 512, 8 * c + 2 * j + h) = __builtin_bit_cast(v4u, s);
        }
#pragma unroll
      for (int t = 0; t < 16; ++t)
        __builtin_nontemporal_store((v4u)*words(2 * t + h, 512, n), reinterpret_cast<global<v4u>*>((uintptr_t)(out + (size_t)(32 * i + 2 * t + h) * a.K + 4 * n)));
    }
  } else {
    uint16_t* out = static_cast<uint16_t*>(a.dw) + (size_t)e * plane + first;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t s[4];
#pragma unroll
          for (int v = 0; v < 4; ++v)
            s[v] = f32x2_to_bf16(__builtin_amdgcn_ldexpf(acc[c][i][8 * w + 2 * v], down),
                                 __builtin_amdgcn_ldexpf(acc[c][i][8 * w + 2 * v + 1], down));
          // lanes of the lower half get columns 0-7 of 16, those of the upper one 8-15
          const auto lo = __builtin_amdgcn_permlane32_swap(s[0], s[2], false, false);
          const auto hi = __builtin_amdgcn_permlane32_swap(s[1], s[3], false, false);
          *words(32 * i + n, 256, 4 * c + 2 * w + h) = v4u{lo[0], hi[0], lo[1], hi[1]};
        }
#pragma unroll
    for (int t = 0; t < 16; ++t) {
      const int row = 4 * t + (lane >> 4);
      __builtin_nontemporal_store((v4u)*words(row, 256, lane & 15), reinterpret_cast<global<v4u>*>((uintptr_t)(out + (size_t)row * a.K + 8 * (lane & 15))));
    }
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
  int k = 1;
  for (; k + 7 <= parts; k += 7) {  // seven loads in flight
    v4f t[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) t[i] = __builtin_nontemporal_load(p + (k + i) * n4);
#pragma unroll
    for (int i = 0; i < 7; ++i) s += t[i];
  }
  for (; k < parts; ++k) s += p[k * n4];
  if constexpr (kF32)
    static_cast<v4f*>(dw)[i] = s;
  else
    static_cast<v2u*>(dw)[i] = v2u{f32x2_to_bf16(s[0], s[1]), f32x2_to_bf16(s[2], s[3])};
}

// Row ranges of each group: as many as there are idle CUs for, each of 256 rows
// and more on average, at most 32 (us with 8, 32 and 64 of them: 16384 rows, 512 x
// 512, 4 tiles: 60, 41 and 53; 2000 rows, where 256 a part leave 7: 20).
int row_parts(long P, int E, int N, int K) {
  const long tiles = (long)E * ((N + kTile - 1) / kTile) * ((K + kTile - 1) / kTile);
  return (int)max(min(min((long)256 / tiles, P / E / 256), 32l), 1l);
}

}  // namespace

// Workspace: the x row of each row, then the parts' sums.
size_t fp8b_grad_ws_bytes(long P, int E, int N, int K) {
  const int parts = row_parts(P, E, N, K);
  return PackedLayout::align256(4 * (size_t)P) + (parts > 1 ? 4 * (size_t)parts * E * N * K : 0);
}

hipError_t launch_fp8b_grad(const Fp8bGradArgs& a, bool fp32_out, void* ws, hipStream_t st) {
  const int parts = row_parts(a.P, a.E, a.N, a.K);
  int32_t* xrows = static_cast<int32_t*>(ws);
  const GradLaunch g{a, a.rows ? xrows : nullptr, (a.N + kTile - 1) / kTile, (a.K + kTile - 1) / kTile, parts,
                     reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + PackedLayout::align256(4 * (size_t)a.P))};
  if (a.rows && a.P > 0) {
    hipLaunchKernelGGL(entries_kernel, dim3(((unsigned)a.P + 1023u) / 1024), dim3(1024), 0, st, a, xrows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
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
