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
#include <utility>

#include "fp8b.h"
#include "tiled.h"

namespace moe {
namespace {

constexpr int kTile = 256;
constexpr int kStepRows = 32;
constexpr int kPanel = kTile * kStepRows * 2;  // bytes of one operand's step in fp16
constexpr int kBuf = 3 * kPanel;               // dy for each block of k, x
constexpr int kCodes = kTile * kStepRows;      // bytes of one operand's step as codes
constexpr int kRawSteps = 3;
constexpr int kPanelTiles = 8;                 // k tiles of a panel of the walk
// LDS: two steps in fp16, three steps of codes (dy, x), four of scales (dy's blocks 0
// and 1, x's; 32 rows each, twice), two of their products, eight of row indices
constexpr int kOffRaw = 2 * kBuf, kOffScale = kOffRaw + kRawSteps * 2 * kCodes, kOffProd = kOffScale + 4 * 1024;
constexpr int kOffIdx = kOffProd + 2 * 256, kOffTop = kOffIdx + 8 * 256, kLds = kOffTop + 128;
static_assert(kLds <= 160 * 1024, "LDS");

struct GradLaunch {
  Fp8bGradArgs a;
  const int32_t* xrows;  // x row of each row of dy, or null: the same row
  int ntn, ntk;          // tiles of an expert
  int parts;             // row ranges of each group
  float* partial;        // their sums, where there are several
};

typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

__device__ __forceinline__ v16f mfma_f16(v4u a, v4u b, v16f c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}
__device__ __forceinline__ uint32_t mul_pair(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, a) * __builtin_bit_cast(v2h, b));
}

// x row of each row of dy
__global__ __launch_bounds__(1024) void entries_kernel(Fp8bGradArgs a, int32_t* __restrict__ xrows) {
  const int p = (int)(blockIdx.x * 1024 + threadIdx.x);
  if (p < a.P) xrows[p] = entry_row(a.rows, p, a.div, a.X);
}

// LDS-DMA of 16 bytes, or a dword, for each lane from an address of its own.
__device__ __forceinline__ void dma16_lanes(const uint8_t* p, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %0, off"
      :
      : "v"(p), "s"(wave_u32(lds))
      : "memory");
}

__device__ __forceinline__ void dma4_from(const uint8_t* p, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %0, off"
      :
      : "v"(p), "s"(wave_u32(lds))
      : "memory");
}

// f(0), f(1), ... with constants, so that what it indexes is in registers from the start.
template <class F, int... I>
__device__ __forceinline__ void each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}

// What the loop is given.
struct GradCtx {
  uint32_t lds0;
  int lane, wave;
  int begin, end, steps;  // rows of the group (or its part), and their steps
  const uint8_t* codes;   // of what this wave moves: dy or x
  int width, tile;        // its columns, and the tile's place among them
  const float* scales;    // of the blocks that a dy wave moves
  const int32_t* xrows;
  int up_y, up_x;         // powers of two for a dy wave's products
};

// The loop of a wave that moves and converts x (kIsX) or dy: rows 8 o .. 8 o + 7 of
// a step, by LDS-DMA as they are, then four columns a thread.
template <bool kIsX, bool kGather>
__device__ __forceinline__ void run_rows(const GradCtx& g, v16f (&acc)[2][4]) {
  const uint32_t lds0 = g.lds0;
  const int lane = g.lane, wave = g.wave, begin = g.begin, steps = g.steps, width = g.width;
  // products: n rows 4 q + c for q of half wn % 2 (block wn % 2), c = 2 (wn / 2) + {0, 1}; k columns of block wk
  const int wn = wave >> 1, wk = wave & 1, r = lane & 31, h = lane >> 5;
  const int o = wave & 3;
  // (columns past the last one read the last 16: not stored)
  const uint32_t piece = (uint32_t)min(kTile * g.tile + 16 * (lane & 15), width - 16);
  const uint8_t* base = g.codes;
  const uint32_t last = (uint32_t)(g.end - 1);
  auto row_at = [&](int step, int r) { return min((uint32_t)begin + (uint32_t)(kStepRows * step + r), last); };
  auto entry = [&](int step, int r) {  // of the index ring
    return (uint32_t)lds_i32(lds0 + kOffIdx + 256u * (uint32_t)(step & 7) + 4u * (uint32_t)r);
  };
  auto load_codes = [&](int step, int slot) {
    const uint32_t to = lds0 + (uint32_t)(kOffRaw + (2 * slot + (kIsX ? 1 : 0)) * kCodes + 2048 * o);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int r = 8 * o + 4 * t + (lane >> 4);
      if constexpr (kIsX && kGather) {
        dma16_lanes(base + (size_t)entry(step, r) * (size_t)width + piece, to + 1024u * t);
      } else {
        const uint32_t first = wave_u32(row_at(step, 0));
        dma16(base + (size_t)first * (size_t)width, (row_at(step, r) - first) * (uint32_t)width + piece, to + 1024u * t);
      }
    }
  };
  // scales: dy wave o those of dy's block o, or of x's block o - 2
  auto load_scales = [&](int step) {
    if constexpr (!kIsX) {
      uint32_t r = row_at(step, lane & 31);
      if (kGather && o >= 2) r = entry(step, lane & 31);
      dma4_from(reinterpret_cast<const uint8_t*>(g.scales + r), lds0 + (uint32_t)(kOffScale + 1024 * (step & 3) + 256 * o));
    }
  };
  auto load_entries = [&](int step) {
    if constexpr (kIsX && kGather)
      dma4_from(reinterpret_cast<const uint8_t*>(g.xrows + row_at(step, lane & 31)),
                lds0 + (uint32_t)(kOffIdx + 256 * (step & 7)));
  };
  constexpr int kLoads = kIsX ? (kGather ? 3 : 2) : 3;  // of a step
  auto load = [&](int j, int slot) {  // behind step j's barrier
    load_codes(j + 4, slot);
    load_scales(j + 5);
    load_entries(j + 8);
  };
  // products of the scales, one of the four pairs of blocks a dy wave, for 32 rows (the upper lanes repeat them)
  const int sn = o >> 1, sk = o & 1;
  float fy, fx;
  auto get_scales = [&](int step) {
    if constexpr (!kIsX) {
      const uint32_t at = lds0 + (uint32_t)(kOffScale + 1024 * (step & 3)) + 4u * (uint32_t)(lane & 31);
      fy = __int_as_float(lds_i32(at + 256u * sn));
      fx = __int_as_float(lds_i32(at + 512u + 256u * sk));
    }
  };
  auto put_products = [&](int step) {
    if constexpr (!kIsX) {
      const float k = __builtin_amdgcn_ldexpf(fy, g.up_y) * __builtin_amdgcn_ldexpf(fx, g.up_x);
      const bool live = (uint32_t)begin + (uint32_t)(kStepRows * step + (lane & 31)) <= last;
      *reinterpret_cast<__attribute__((address_space(3))) _Float16*>((uintptr_t)(
          lds0 + (uint32_t)(kOffProd + 256 * (step & 1) + 64 * (2 * sn + sk) + 2 * (lane & 31)))) = (_Float16)(live ? k : 0.0f);
    }
  };
  // a step's conversion in pieces: its codes; two rows to fp16; the scales' products; each column
  uint32_t raw[8], v[8][2], k[2][4];
  auto get_codes = [&](int slot) {
    const uint32_t at = lds0 + (uint32_t)(kOffRaw + (2 * slot + (kIsX ? 1 : 0)) * kCodes + 2048 * o) + 4u * (uint32_t)lane;
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i] = (uint32_t)lds_i32(at + 256u * i);
  };
  auto rows_to_half = [&](int m) {
#pragma unroll
    for (int i = 2 * m; i < 2 * m + 2; ++i) {
      v[i][0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)raw[i], 1.0f, false));
      v[i][1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)raw[i], 1.0f, true));
    }
  };
  auto get_products = [&](int step) {
    if constexpr (!kIsX) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const v4u t = lds_v4(lds0 + (uint32_t)(kOffProd + 256 * (step & 1) + 64 * b + 16 * o) + 128u * (uint32_t)(lane >> 5));
        k[b][0] = t.x, k[b][1] = t.y, k[b][2] = t.z, k[b][3] = t.w;
      }
    }
  };
  const uint32_t my_column = lds0 + (uint32_t)((kIsX ? 2 * kPanel : 0) + o * kTile * 16) + 16u * (uint32_t)lane;
  auto put_column = [&](int step, int c) {
    lds_words* to = reinterpret_cast<lds_words*>((uintptr_t)(my_column + (uint32_t)((step & 1) * kBuf + 1024 * c)));
    v4u w;
#pragma unroll
    for (int i = 0; i < 4; ++i)  // halves c % 2 of rows 2 i and 2 i + 1
      w[i] = __builtin_amdgcn_perm(v[2 * i + 1][c >> 1], v[2 * i][c >> 1], c & 1 ? 0x07060302u : 0x05040100u);
    if constexpr (kIsX) {
      *to = w;
    } else {
#pragma unroll
      for (int b = 0; b < 2; ++b)
        to[b * (kPanel / 16)] =
            v4u{mul_pair(w[0], k[b][0]), mul_pair(w[1], k[b][1]), mul_pair(w[2], k[b][2]), mul_pair(w[3], k[b][3])};
    }
  };
  // fragments of 16 rows u of a step
  v4u fa[2], fb[4];
  const uint32_t pa = lds0 + (uint32_t)(wk * kPanel) + 16u * (uint32_t)(h * kTile + 128 * (wn >> 1) + 32 * (wn & 1) + r);
  const uint32_t pb = lds0 + (uint32_t)(2 * kPanel) + 16u * (uint32_t)(h * kTile + 32 * wk + r);
  auto read_a = [&](int step, int u, int i) { fa[i] = lds_v4(pa + (uint32_t)((step & 1) * kBuf + (2 * u * kTile + 64 * i) * 16)); };
  auto read_b = [&](int step, int u, int c) { fb[c] = lds_v4(pb + (uint32_t)((step & 1) * kBuf + (2 * u * kTile + 64 * c) * 16)); };
  // Step j: its products, while step j + 1 is converted and the scales' products of
  // step j + 2 are made.  Behind three quarters of the MFMAs a barrier publishes
  // these, and the codes of step j + 2, which have had two steps to arrive; their
  // place takes those of step j + 4, and the next step's fragments are read under
  // the last MFMAs.  (Loads past the last step read its rows again; a step past the
  // last has products of zero.)
  auto iterate = [&](int j, int slot) __attribute__((always_inline)) {  // slot: (j + 1) % 3
    each([&](auto at) __attribute__((always_inline)) {
      constexpr int m = decltype(at)::value, u = m >> 3, i = (m >> 2) & 1, c = m & 3;
      acc[i][c] = mfma_f16(fa[i], fb[c], acc[i][c]);
      if (m == 0) {
        get_codes(slot);
        get_products(j + 1);
        get_scales(j + 2);
      }
      // the second 16 rows' fragments, each behind its register's last use
      if (u == 0 && c == 3) read_a(j, 1, i);
      if (u == 0 && i == 1) read_b(j, 1, c);
      if (m >= 2 && m < 6) rows_to_half(m - 2);
      if (m >= 6 && m < 10) put_column(j + 1, m - 6);
      if (m == 10) put_products(j + 2);
      if (m == 12) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads) : "memory");
        load(j, slot);
        read_a(j + 1, 0, 0);
      }
      if (u == 1 && i == 1) read_b(j + 1, 0, c);
      if (m == 15) read_a(j + 1, 0, 1);
      if (c == 3) __builtin_amdgcn_sched_barrier(0);  // (four MFMAs at a time are the compiler's to order)
    }, std::make_integer_sequence<int, 16>{});
  };
  // the first steps' codes, scales and (by plain loads) indices
  if constexpr (kIsX && kGather) {
#pragma unroll
    for (int q = 0; q < 8; ++q)
      *reinterpret_cast<__attribute__((address_space(3))) int*>((uintptr_t)(lds0 + (uint32_t)(kOffIdx + 256 * q) + 4u * (uint32_t)lane)) =
          g.xrows[row_at(q, lane & 31)];
  }
  __syncthreads();
#pragma unroll
  for (int q = 0; q < 3; ++q) load_codes(q, q);
#pragma unroll
  for (int q = 0; q < 4; ++q) load_scales(q);
  asm volatile("s_waitcnt vmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    get_scales(q);
    put_products(q);
  }
  get_codes(0);
  __syncthreads();
  get_products(0);
#pragma unroll
  for (int m = 0; m < 4; ++m) rows_to_half(m);
#pragma unroll
  for (int c = 0; c < 4; ++c) put_column(0, c);
  __syncthreads();
  load(-1, 0);
#pragma unroll
  for (int i = 0; i < 2; ++i) read_a(0, 0, i);
#pragma unroll
  for (int c = 0; c < 4; ++c) read_b(0, 0, c);
  for (int j = 0, slot = 1; j < steps; ++j, slot = slot == 2 ? 0 : slot + 1) iterate(j, slot);
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

  // The largest scales of the group's rows in the tile's blocks, as powers of two:
  // y_exp and x_exp with scale < 2^exp.
  const int nb0 = min(2 * tn, a.N / 128 - 1), nb1 = min(2 * tn + 1, a.N / 128 - 1);
  const int kb0 = min(2 * tk, a.K / 128 - 1), kb1 = min(2 * tk + 1, a.K / 128 - 1);
  auto x_row = [&](int s) { return kGather ? g.xrows[s] : s; };
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
    float(*tops)[4] = reinterpret_cast<float(*)[4]>(lds + kOffTop);
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
      c.up_y = -(o >> 1 ? y_exp[1] : y_exp[0]);
      c.up_x = kUp - (o & 1 ? x_exp[1] : x_exp[0]);
      run_rows<false, kGather>(c, acc);
    }
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
