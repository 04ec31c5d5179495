// MXFP4 x MXFP4 products for many rows (the operators of mx4_stream.hip, the
// same packed weights): LDS-tiled, bound by the FP4 matrix rate, or by HBM
// where an expert's rows are few.
//
// A work item is 256 rows of one group x 8 weight tiles (256 weight rows).
// Eight waves, two per SIMD, in a 4 x 2 grid, each with up to two 32-token
// sub-tiles x four weight tiles: 8 accumulators of 32 x 32 (128 registers).
// v_mfma_scale_f32_32x32x64_f8f6f4 rather than 16x16x128: it lasts 32 clocks
// instead of 16, so that the other instructions find room beside it, and reads
// half as many operand registers per flop (back to back on random operands:
// 6.2-6.6 PFLOP/s, where the power limit holds the clock; the smaller one
// 4.4-5.1 with one wave per SIMD, 6.5 with two).
//
// K runs in steps of 128, two to a stage: 32 KiB of row pieces (128 bytes of
// each row: at 64 bytes a row the L2 requests alone take as long as the
// MFMAs), four weight half-stages and the scales go from global memory to LDS
// by LDS-DMA into two stages.  One barrier per step, in its second half,
// publishes what the next step reads and frees what the last one has read,
// which is refilled at once with the data of two stages on: weights of a step
// come three steps before their use, rows and scales two.  Every wave issues
// the same ten loads per stage in the same order, dummy stages past the end, so
// that fixed wait counts serve every stage.  Fragments are read from LDS half a
// step before their use.  Row r's eight 16-byte pieces lie at piece
// p ^ (r / 2 % 8), which spreads the 16 rows that one LDS cycle serves over all
// banks.
//
// The workgroups are persistent: one per CU (its LDS allows no second) walks
// its XCD's contiguous share of the items, and the stages run on across items,
// so that an item's first stages arrive under the last steps and the stores of
// the one before.
#include <atomic>

#include "lds_dma.h"
#include "mx4.h"

namespace moe {
namespace {

constexpr int kBM = 256;                // rows of an item
constexpr int kBT = 8;                  // weight tiles of an item
constexpr int kWaves = 8;
constexpr int kA = kBM * 128;           // row pieces of a stage
constexpr int kW = kBT * 2048;          // weight tiles of a step
constexpr int kSA = kBM * 8;            // eight scale bytes per row
constexpr int kSW = 2 * 1024;           // weight scales of two groups of four tiles
constexpr int kOffW = kA, kOffSA = kA + 2 * kW, kOffSW = kOffSA + kSA;
constexpr int kStage = kA + 2 * kW + kSA + kSW;
constexpr int kIdx = 2 * kStage;        // LDS offset of the next item's row indices
constexpr int kLds = kIdx + kWaves * 256;
static_assert(kStage % 1024 == 0 && kLds <= 160 * 1024, "LDS");

// One entry per 256 rows (at most) of a group, of equal heights.
struct Tile {
  int e, row0, n;
};

// Rows of each tile of a group of n rows, in whole sub-tiles of 32.
__host__ __device__ __forceinline__ int tile_height(int n, int tiles) {
  return ((n + 31) / 32 + tiles - 1) / tiles * 32;
}

// Workspace of a grouped product: the number of tiles, from byte 16 on four
// words per tile, and from scales_at() on the activation scales by stage: the
// eight bytes of stage d of sorted row p at 8 (d P + p), so that a tile's
// scales of a stage are one run instead of a request to L2 for each row.
long tile_cap(long P, int E) { return P / kBM + (P < E ? P : E); }
size_t scales_at(long P, int E) { return PackedLayout::align256(16 + 16 * (size_t)tile_cap(P, E)); }

// Block 0 lists the tiles, each thread of the others moves kPer stages of one
// row's scales.
constexpr int kPer = 8;
__global__ __launch_bounds__(1024) void tiles_kernel(Mx4Args a, int E, int K, int cap, int32_t* __restrict__ ws,
                                                     uint8_t* __restrict__ scales) {
  const int P = a.P;
  if (blockIdx.x > 0) {
    const int D = (K + 255) / 256, nd = (D + kPer - 1) / kPer;
    const size_t i = (size_t)(blockIdx.x - 1) * 1024 + threadIdx.x;
    const size_t part = i / (size_t)P;
    if (part >= (size_t)nd) return;
    const int p = (int)(i - part * P), d0 = (int)part * kPer, n = min(kPer, D - d0);
    int x = p;
    if (a.rows) x = (int)((uint32_t)a.rows[p] / (uint32_t)a.div);
    x = max(min(x, a.X - 1), 0);
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.xs + (size_t)x * (K / 32)) + 2 * d0;
    const int dwords = K / 128 - 2 * d0;  // left in the row from stage d0 on
    uint2 v[kPer];
#pragma unroll
    for (int d = 0; d < kPer; ++d)
      if (d < n) v[d] = make_uint2(src[2 * d], src[min(2 * d + 1, dwords - 1)]);  // an odd number's last one twice
#pragma unroll
    for (int d = 0; d < kPer; ++d)
      if (d < n) *reinterpret_cast<uint2*>(scales + 8 * ((size_t)(d0 + d) * P + p)) = v[d];
    return;
  }
  const int32_t* offsets = a.offsets;
  __shared__ int wave_tot[16];
  const int e = threadIdx.x, lane = e & 63, w = e >> 6;
  int begin = 0, n = 0;
  if (e < E) {
    begin = min(max(offsets[e], 0), P);
    n = min(max(offsets[e + 1], begin), P) - begin;
  }
  const int nt = (n + kBM - 1) / kBM;
  const int incl = wave_inclusive_scan(nt, lane);
  if (lane == 63) wave_tot[w] = incl;
  __syncthreads();
  int at = incl - nt, total = 0;
  for (int i = 0; i < 16; ++i) {
    if (i < w) at += wave_tot[i];
    total += wave_tot[i];
  }
  if (e == 0) ws[0] = min(total, cap);
  const int h = nt > 0 ? tile_height(n, nt) : 0;
  int4* list = reinterpret_cast<int4*>(ws) + 1;
  // offsets that decrease could name more tiles than the list holds
  for (int i = 0; i < nt && at + i < cap; ++i) list[at + i] = make_int4(e, begin + i * h, min(h, n - i * h), 0);
}

typedef __attribute__((address_space(4))) const int32_t cint;  // read by scalar loads

// Position p of the walk -> the item's tile of rows and its first weight tile.
struct Walk {
  int ntt, ntn;  // row tiles, weight-tile columns of eight
  int lo, hi;    // this XCD's share
};

__device__ __forceinline__ void walk_item(const Walk& k, int p, int& tt, int& tn) {
  // panels of a quarter of the columns, row tiles running inside a panel: the
  // items that an XCD holds at one time share rows and weights in its L2
  const int sn = (k.ntn + 3) / 4;
  const int sc = p / (k.ntt * sn), q = p - sc * (k.ntt * sn);
  const int w = min(sn, k.ntn - sc * sn);
  tt = q / w;
  tn = sc * sn + q % w;
}

__device__ __forceinline__ Tile get_tile(const Mx4Args& a, const int32_t* ws, int tt, int ntt) {
  Tile t;
  if (a.offsets) {
    const cint* p = reinterpret_cast<const cint*>(reinterpret_cast<uintptr_t>(ws)) + 4 + 4 * tt;
    t.e = p[0];
    t.row0 = p[1];
    t.n = p[2];
  } else {
    const int h = tile_height(a.P, ntt);
    t.e = 0;
    t.row0 = tt * h;
    t.n = min(h, a.P - t.row0);
  }
  return t;
}

__device__ __forceinline__ uint32_t opaque(uint32_t x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ v4u lds_v4(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) v4u*>((uintptr_t)addr);
}
__device__ __forceinline__ int lds_i32(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) int*>((uintptr_t)addr);
}

// One MFMA, its accumulator pinned to AGPRs at this point of the program and
// the scheduler fenced, so that every LDS read and DMA stays where the step
// places it.  (The builtin, not asm: the wait states between a vector write
// and an MFMA that reads it are the compiler's then.)
template <int kA, int kB>
__device__ __forceinline__ void mfma(v16f& c, const v4u& a, const v4u& b, uint32_t sa, uint32_t sb) {
  c = mfma_fp4<kA, kB>(a, b, c, sa, sb);
  asm volatile("" : "+a"(c) : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Where the DMA stands: the next stage to load of the item it is in.  The
// pointers (uniform) are that stage's.
struct Cursor {
  const uint8_t* x;   // activation codes
  const uint8_t* w;   // the wave's weight tile
  const uint8_t* xs;  // activation scales
  const uint8_t* ws;  // the wave's part of the weight scales
  uint32_t a[4];      // per lane: its piece of rows 32 w + 8 u + l / 8
  uint32_t sa;        // per lane: its dword of row scales
  int p, left;        // item, stages left of it (this one counted)
};

struct Frag {
  v4u x[2], w[4];
};

struct Ctx {
  const Mx4Args& a;
  const Mx4Layout& L;
  const int32_t* ws;
  // activation scales: of sorted rows by stage (grouped), or of x by row (dense)
  const uint8_t* scales;
  uint32_t scale_row;  // bytes from a row
  size_t scale_stage;  // and from a stage to the next
  Walk walk;
  int stride;  // of the walk
  uint32_t lds;
  int lane, wave;
};

// LDS-DMA: lane l's 16 (4) bytes at base + off go to LDS address lds + 16 l
// (4 l); an instruction offset counts on both sides.  The LDS address goes to
// M0, which nothing else here uses (LDS instructions need none).  The base is
// copied by the scalar unit first: a scalar register that a vector instruction
// has written (v_readfirstlane) must not be read by a load within five wait
// states, and the compiler does not look into the asm; the copy is also the
// wait state that M0 needs.
template <int kOff = 0>
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  const uint8_t* t;
  asm volatile(
      "s_mov_b32 m0, %3\n\t"
      "s_mov_b64 %0, %2\n\t"
      "global_load_lds_dwordx4 %1, %0 offset:%4"
      : "=&s"(t)
      : "v"(off), "s"(wave_ptr(base)), "s"(wave_u32(lds)), "n"(kOff)
      : "memory");
}
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
  const uint8_t* t;
  asm volatile(
      "s_mov_b32 m0, %3\n\t"
      "s_mov_b64 %0, %2\n\t"
      "global_load_lds_dword %1, %0"
      : "=&s"(t)
      : "v"(off), "s"(wave_ptr(base)), "s"(wave_u32(lds))
      : "memory");
}

// Sub-tiles of 32 rows that wave row wm (of four) takes of a tile of n rows:
// how many, and the first one.  Wave rows 0 and 2 share SIMDs, as do 1 and 3.
__device__ __forceinline__ int sub_tiles(int n, int wm) { return ((n + 31) / 32 + 3 - wm) / 4; }
__device__ __forceinline__ int first_sub(int n, int wm) {
  const int n32 = (n + 31) / 32;
  return wm * (n32 / 4) + min(wm, n32 % 4);
}

// Row of the tile whose scale dword (l % 2: which step's) lane l of wave w
// moves: the scales of wave row wm's two sub-tiles lie side by side
// ([row 32][sub-tile 2][8 bytes]), so that one 128-bit read serves both.
__device__ __forceinline__ int scale_row(int n, int wave, int lane) {
  const int at = 64 * (wave & 1) + lane;
  return 32 * (first_sub(n, wave >> 1) + ((at >> 1) & 1)) + (at >> 2);
}

// Row index DMA of item p (if there is one) into the index buffer: each wave
// loads, and later reads, the indices of the 32 rows whose pieces it moves.
__device__ __forceinline__ void fetch_rows(const Ctx& c, int p) {
  if (!c.a.rows || p >= c.walk.hi) return;
  int tt, tn;
  walk_item(c.walk, p, tt, tn);
  const Tile t = get_tile(c.a, c.ws, tt, c.walk.ntt);
  dma4(wave_ptr(reinterpret_cast<const uint8_t*>(c.a.rows + t.row0)),
       4u * (uint32_t)min(32 * c.wave + (c.lane & 31), t.n - 1), wave_u32(c.lds + kIdx + 256u * (uint32_t)c.wave));
}

// The last stage of an odd number of steps has no second step.  Its weights are
// zeros; for the rows, what would lie past their end reads the first step's
// bytes (a block that is NaN there is NaN in the first step too).
__device__ __forceinline__ void clip_tail(const Ctx& c, Cursor& k) {
  if (k.left != 1 || !(c.L.J & 1)) return;
#pragma unroll
  for (int u = 0; u < 4; ++u) k.a[u] -= (((uint32_t)c.lane & 7) ^ (uint32_t)((c.lane >> 4) + 4 * (u & 1))) & 4 ? 64u : 0u;
  if (!c.a.offsets) k.sa -= 4u * (uint32_t)(c.lane & 1);
}

// Points the cursor at item p (whose row indices are in the index buffer).
__device__ __forceinline__ void enter(const Ctx& c, Cursor& k, int p) {
  int tt, tn;
  walk_item(c.walk, p, tt, tn);
  const Tile t = get_tile(c.a, c.ws, tt, c.walk.ntt);
  const Mx4Layout& L = c.L;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = 8 * u + (c.lane >> 3);
    // logical piece of the lane: physical piece l % 8 of a row whose r / 2 % 8 is l / 16 + 4 (u % 2)
    const uint32_t piece = ((uint32_t)c.lane & 7) ^ (uint32_t)((c.lane >> 4) + 4 * (u & 1));
    int x = t.row0 + min(32 * c.wave + r, t.n - 1);  // rows past the tile read its last one
    if (c.a.rows) x = (int)((uint32_t)lds_i32(c.lds + kIdx + 4 * (64 * c.wave + r)) / (uint32_t)c.a.div);
    k.a[u] = (uint32_t)max(min(x, c.a.X - 1), 0) * ((uint32_t)L.K / 2) + 16u * piece;
  }
  k.sa = (uint32_t)min(scale_row(t.n, c.wave, c.lane), t.n - 1) * c.scale_row + 4u * (uint32_t)(c.lane & 1);
  k.x = wave_ptr(c.a.xq);
  k.xs = wave_ptr(c.scales + (size_t)t.row0 * c.scale_row);
  // tiles past the last one read the last one; their columns are not stored
  k.w = wave_ptr(c.a.packed + L.tile_off(t.e, min(tn * kBT + c.wave, L.NT - 1)));
  k.ws = wave_ptr(c.a.packed + L.scale_off(t.e, min(2 * tn + (c.wave >> 2), L.NG - 1)) + 256 * (c.wave & 3));
  k.p = p;
  k.left = L.D;
  clip_tail(c, k);
}

// Load u (< 10) of the wave's share of the cursor's stage into the one at S, in
// the order of their use: 0-1 the first step's weights, 2-5 row pieces, 6-7
// scales, 8-9 the second step's weights.
__device__ __forceinline__ void issue(const Ctx& c, const Cursor& k, uint32_t S, int u) {
  const uint32_t w = (uint32_t)c.wave, l16 = 16u * (uint32_t)c.lane;
  switch (u) {
    case 0: dma16(k.w, l16, S + (uint32_t)kOffW + 2048u * w); break;
    case 1: dma16<1024>(k.w, l16, S + (uint32_t)kOffW + 2048u * w); break;
    case 2: dma16(k.x, k.a[0], S + 4096u * w); break;
    case 3: dma16(k.x, k.a[1], S + 4096u * w + 1024u); break;
    case 4: dma16(k.x, k.a[2], S + 4096u * w + 2048u); break;
    case 5: dma16(k.x, k.a[3], S + 4096u * w + 3072u); break;
    case 6: dma4(k.xs, k.sa, S + (uint32_t)kOffSA + 256u * w); break;
    case 7: dma4(k.ws, 4u * (uint32_t)c.lane, S + (uint32_t)kOffSW + 256u * w); break;
    case 8: dma16(k.w + 2048, l16, S + (uint32_t)(kOffW + kW) + 2048u * w); break;
    default: dma16<1024>(k.w + 2048, l16, S + (uint32_t)(kOffW + kW) + 2048u * w);
  }
}

// After a stage's loads: the next stage, or the next item's first (past the
// last item its last stage is loaded again and never used).
__device__ __forceinline__ void advance(const Ctx& c, Cursor& k) {
  if (k.left > 1) {
    --k.left;
    k.x += 128;
    k.w += 4096;
    k.xs += c.scale_stage;
    k.ws += 1024;
    clip_tail(c, k);
    return;
  }
  const int p = k.p + c.stride;
  if (p >= c.walk.hi) return;
  // the indices were loaded when the cursor entered this item; with three
  // stages or more since then the waits of the steps have covered them
  if (c.a.rows && c.L.D < 3) wait_vmcnt<0>();
  enter(c, k, p);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the indices are read before they are replaced
  fetch_rows(c, p + c.stride);
}

struct Addr {  // per lane, relative to a stage
  uint32_t a[4];   // row r of the wave's first sub-tile, pieces of the four K-halves (sub-tile i at + 4096 i)
  uint32_t sa;     // its sub-tiles' scales
  uint32_t w;      // first step's weight tile 4 wn (+ 2048 t, K-half 1 at + 1024, second step at + kW)
  uint32_t sw;     // the group's scales
  uint32_t shift;  // 16 g: the lane's half of a row's scale dword
};

struct Scales {
  uint32_t x[2][2];  // sub-tile, step
  v4u w;             // two dwords per step
};

// Fragments q (< S + 4) of a K-half: four weight tiles, then S sub-tiles.
__device__ __forceinline__ void read_frag(Frag& f, uint32_t xa, uint32_t wa, int q) {
  if (q < 4)
    f.w[q] = lds_v4(wa + 2048 * q);
  else
    f.x[q - 4] = lds_v4(xa + 4096 * (q - 4));
}

template <int S>
__device__ __forceinline__ void read_scales(Scales& s, uint32_t stage, const Addr& ad, v4u& raw) {
  raw = lds_v4(stage + ad.sa);
  s.w = lds_v4(stage + ad.sw);
}
template <int S>
__device__ __forceinline__ void shift_scales(Scales& s, const Addr& ad, const v4u& raw) {
#pragma unroll
  for (int i = 0; i < S; ++i) {
    s.x[i][0] = raw[2 * i] >> ad.shift;
    s.x[i][1] = raw[2 * i + 1] >> ad.shift;
  }
}

// MFMA m of K-half kHalf of step H: sub-tile m / 4, tile m % 4 (whose scale is
// byte 2 (m % 2) + kHalf of its pair's dword).
template <int H, int kHalf>
__device__ __forceinline__ void multiply(v16f (&acc)[2][4], const Frag& f, const Scales& s, int m) {
  const int i = m >> 2, t = m & 3;
  if (t & 1)
    mfma<kHalf, 2 + kHalf>(acc[i][t], f.x[i], f.w[t], s.x[i][H], s.w[2 * H + (t >> 1)]);
  else
    mfma<kHalf, kHalf>(acc[i][t], f.x[i], f.w[t], s.x[i][H], s.w[2 * H + (t >> 1)]);
}

// Step H (0, 1) of the stage at `cur` for a wave with S live sub-tiles.  On
// entry f0 holds K-half 0's fragments of this step and s the stage's scales;
// on exit the same for the next step.  Loads: the cursor's stage goes to where
// this one is; in step 0 its first step's weights (whose place is free behind
// the barrier), in step 1 the row pieces and, in the next stage's step 0, the
// rest, spread over the MFMAs.
template <int S, int H>
__device__ __forceinline__ void step(const Ctx& c, Cursor& k, const Addr& ad, uint32_t cur, uint32_t nxt,
                                     v16f (&acc)[2][4], Frag& f0, Frag& f1, Scales& s) {
  constexpr int M = 4 * S;  // MFMAs of a half
  constexpr int R = S + 4;  // fragments of a half
  // first half: K-half 1's fragments arrive under K-half 0's MFMAs
  if constexpr (S > 0) {
    const uint32_t xa = cur + ad.a[2 * H + 1], wa = cur + ad.w + (uint32_t)(H * kW + 1024);
#pragma unroll
    for (int m = 0; m < M; ++m) {
      multiply<H, 0>(acc, f0, s, m);
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q * M / R == m) read_frag(f1, xa, wa, q);
      if constexpr (H == 0) {
#pragma unroll
        for (int u = 6; u < 10; ++u)
          if ((u - 6) * M / 4 + M / 8 == m) issue(c, k, nxt, u);
      }
    }
  } else if constexpr (H == 0) {
#pragma unroll
    for (int u = 6; u < 10; ++u) issue(c, k, nxt, u);
  }
  if constexpr (H == 0) advance(c, k);
  auto publish = [&] {
    // This wave's loads of what the next step reads have landed and its reads
    // of this step are done; then everyone's.  In flight may be, behind step 0,
    // the next stage (10) and, behind step 1, the next stage's second weights
    // and the first ones of the stage after it (4).
    if constexpr (H == 0)
      asm volatile("s_waitcnt vmcnt(10) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(4) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  constexpr int kFrom = H == 0 ? 0 : 2, kTo = H == 0 ? 2 : 6;  // this step's loads behind the barrier
  if constexpr (S > 0) {
    constexpr int kLeft = M - 1;  // places behind the barrier, which stands after the first MFMA
    const uint32_t xa = (H == 0 ? cur + ad.a[2] : nxt + ad.a[0]);
    const uint32_t wa = (H == 0 ? cur + ad.w + (uint32_t)kW : nxt + ad.w);
    v4u raw;
    Scales ns;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      multiply<H, 1>(acc, f1, s, m);
      if (m == 0) {
        publish();
        if constexpr (H == 1) read_scales<S>(ns, nxt, ad, raw);
      }
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q * kLeft / R == m) read_frag(f0, xa, wa, q);
#pragma unroll
      for (int u = kFrom; u < kTo; ++u)
        if ((u - kFrom) * kLeft / (kTo - kFrom) + kLeft / 8 == m) issue(c, k, cur, u);
    }
    if constexpr (H == 1) {
      shift_scales<S>(ns, ad, raw);
      s = ns;
    }
  } else {
    publish();
#pragma unroll
    for (int u = kFrom; u < kTo; ++u) issue(c, k, cur, u);
  }
}

// SiLU(g) u for the SwiGLU epilogue, as silu_mul but with the exponential
// straight from the exp2 instruction (whose results below 2^-126 are 0 here,
// as 1 + them is 1 anyway).
__device__ __forceinline__ float glu_out(float g, float u) {
  return g * u * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.44269504f));
}

// Global (not flat) pointers: flat stores would count as LDS traffic too.
template <class T>
using global = __attribute__((address_space(1))) T;
typedef global<uint8_t> gbyte;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// Stores of one sub-tile: element v of a lane is row 8 (v / 4) + 4 g + v % 4;
// the group's f tiles are f neighbouring columns, so a half-wave's store covers
// a whole run of 128 (64 with SwiGLU) outputs.  base (uniform): row 0 of the
// sub-tile, the group's first column; off: the lane's bytes from there (its
// column, and 4 g rows down); left: rows of the sub-tile that exist.
template <bool kGlu, bool kF32, bool kMask>
__device__ __forceinline__ void store_sub(const v16f (&acc)[4], gbyte* base, size_t row_bytes, uint32_t off, int left,
                                          int f) {
  constexpr int kO = kGlu ? 2 : 4;
#pragma unroll
  for (int v = 0; v < 16; ++v) {
    gbyte* y = base + (size_t)(8 * (v >> 2) + (v & 3)) * row_bytes + off;
    float o[kO];
#pragma unroll
    for (int t = 0; t < kO; ++t) o[t] = kGlu ? glu_out(acc[2 * t][v], acc[2 * t + 1][v]) : acc[t][v];
    if (!kMask || 8 * (v >> 2) + (v & 3) < left) {  // left: less the lane's 4 g
      if constexpr (kF32) {
        global<float>* q = reinterpret_cast<global<float>*>(y);
        if (!kMask || f == kO) {
          if constexpr (kGlu)
            *reinterpret_cast<global<v2f>*>(q) = v2f{o[0], o[1]};
          else
            *reinterpret_cast<global<v4f>*>(q) = v4f{o[0], o[1], o[2], o[3]};
        } else {
#pragma unroll
          for (int t = 0; t < kO - 1; ++t)
            if (t < f) q[t] = o[t];
        }
      } else {
        global<uint16_t>* q = reinterpret_cast<global<uint16_t>*>(y);
        if (!kMask || f == kO) {
          if constexpr (kGlu)
            *reinterpret_cast<global<uint32_t>*>(q) = f32x2_to_bf16(o[0], o[1]);
          else
            *reinterpret_cast<global<v2u>*>(q) = v2u{f32x2_to_bf16(o[0], o[1]), f32x2_to_bf16(o[2], o[3])};
        } else {
#pragma unroll
          for (int t = 0; t < kO - 1; ++t)
            if (t < f) q[t] = f32_to_bf16(o[t]);
        }
      }
    }
    if ((v & 3) == 3) __builtin_amdgcn_sched_barrier(0);  // four rows at a time out of the accumulators
  }
}

template <int S, bool kGlu, bool kF32>
__device__ __forceinline__ void run_item(const Ctx& c, Cursor& k, const Addr& ad, int& stage, const Tile& t, int sub0,
                                         int group) {
  v16f acc[2][4];
  Frag f0, f1;
  Scales s;
  uint32_t cur = wave_u32(c.lds + (uint32_t)(stage * kStage)), nxt;
  if constexpr (S > 0) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][q][v] = 0.0f;
    v4u raw;
    read_scales<S>(s, cur, ad, raw);
#pragma unroll
    for (int q = 0; q < S + 4; ++q) read_frag(f0, cur + ad.a[0], cur + ad.w, q);
    shift_scales<S>(s, ad, raw);
  }
  for (int d = 0; d < c.L.D; ++d) {
    cur = wave_u32(c.lds + (uint32_t)(stage * kStage));
    nxt = wave_u32(c.lds + (uint32_t)((stage ^ 1) * kStage));
    step<S, 0>(c, k, ad, cur, nxt, acc, f0, f1, s);
    step<S, 1>(c, k, ad, cur, nxt, acc, f0, f1, s);
    stage ^= 1;
  }
  if constexpr (S > 0) {
    constexpr int kO = kGlu ? 2 : 4;
    constexpr uint32_t kB = kF32 ? 4 : 2;
    const int g = c.lane >> 5, left = c.L.N / 32 - kO * group, f = min(left, kO);
    const size_t row_bytes = (size_t)c.L.N * kB;
    const uint32_t off = ((uint32_t)(4 * g) * (uint32_t)c.L.N + (uint32_t)f * (uint32_t)(c.lane & 31)) * kB;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int m = 32 * (sub0 + i);
      uint8_t* base = static_cast<uint8_t*>(c.a.y) + ((size_t)(t.row0 + m) * c.L.N + (size_t)(32 * kO) * group) * kB;
      gbyte* gb = reinterpret_cast<gbyte*>(reinterpret_cast<uintptr_t>(wave_ptr(base)));
      if (f == kO && m + 32 <= t.n)
        store_sub<kGlu, kF32, false>(acc[i], gb, row_bytes, off, 32, f);
      else if (f > 0)
        store_sub<kGlu, kF32, true>(acc[i], gb, row_bytes, off, t.n - m - 4 * g, f);
    }
  }
}

template <bool kGlu, bool kF32>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void tiled_kernel(
    Mx4Args a, Mx4Layout L, const int32_t* ws, const uint8_t* scales, int dense_tiles) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  Ctx c{a, L, ws, scales ? scales : a.xs, scales ? 8u : (uint32_t)L.K / 32, scales ? 8 * (size_t)a.P : 8, {},
        (int)(gridDim.x >> 3), (uint32_t)(uintptr_t)(lds_u8*)lds, lane, wave};
  c.walk.ntt = a.offsets ? *reinterpret_cast<const cint*>(reinterpret_cast<uintptr_t>(ws)) : dense_tiles;
  c.walk.ntn = (L.NT + kBT - 1) / kBT;
  const int items = c.walk.ntt * c.walk.ntn, per = (items + 7) / 8;
  // workgroup b runs on XCD b % 8, which owns the run [x per, x per + per)
  c.walk.lo = min((int)(blockIdx.x & 7) * per, items);
  c.walk.hi = min(c.walk.lo + per, items);
  const int first = c.walk.lo + (int)(blockIdx.x >> 3);
  if (first >= c.walk.hi) return;  // uniform: before any barrier

  Cursor k;
  fetch_rows(c, first);
  wait_vmcnt<0>();
  enter(c, k, first);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  fetch_rows(c, first + c.stride);
  const uint32_t s0 = wave_u32(c.lds), s1 = wave_u32(c.lds + (uint32_t)kStage);
#pragma unroll
  for (int u = 0; u < 10; ++u) issue(c, k, s0, u);
  advance(c, k);
#pragma unroll
  for (int u = 0; u < 6; ++u) issue(c, k, s1, u);
  // stage 0 is there but for its second weights: they and six loads of stage 1 may be in flight
  asm volatile("s_waitcnt vmcnt(8)\n\ts_barrier" ::: "memory");

  Addr ad;
  const int r = lane & 31, g = lane >> 5;
  const uint32_t sz = (uint32_t)((r >> 1) & 7);
  ad.w = opaque((uint32_t)(kOffW + 8192 * wn + 16 * lane));
  ad.sa = opaque((uint32_t)(kOffSA + 512 * wm + 16 * r));
  ad.sw = opaque((uint32_t)(kOffSW + 1024 * wn + 16 * lane));
  ad.shift = (uint32_t)(16 * g);
  int stage = 0;
  for (int p = first; p < c.walk.hi; p += c.stride) {
    int tt, tn;
    walk_item(c.walk, p, tt, tn);
    const Tile t = get_tile(a, ws, tt, c.walk.ntt);
    const int sub0 = first_sub(t.n, wm), live = sub_tiles(t.n, wm);
    const uint32_t row = (uint32_t)(32 * sub0 + r);
#pragma unroll
    for (int h = 0; h < 4; ++h)  // piece of K-half h % 2 of step h / 2
      ad.a[h] = opaque(row * 128 + (((uint32_t)(4 * (h >> 1) + 2 * g + (h & 1)) ^ sz) << 4));
    const int group = tn * 2 + wn;
    switch (live) {
      case 0: run_item<0, kGlu, kF32>(c, k, ad, stage, t, sub0, group); break;
      case 1: run_item<1, kGlu, kF32>(c, k, ad, stage, t, sub0, group); break;
      default: run_item<2, kGlu, kF32>(c, k, ad, stage, t, sub0, group); break;
    }
  }
  wait_vmcnt<0>();  // the dummy stages land before the LDS is given back
}

// CUs of the current device, a multiple of eight (one share per XCD).
int workgroups() {
  static std::atomic<int> cached[64];
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  int n = cached[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 8) n = 256;
    n = n / 8 * 8;
    cached[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

}  // namespace

size_t mx4_tiled_ws_bytes(long P, int E, int K) { return scales_at(P, E) + 8 * (size_t)P * ((K + 255) / 256); }

hipError_t launch_mx4_tiled(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, void* ws, hipStream_t st) {
  int32_t* list = static_cast<int32_t*>(ws);
  uint8_t* scales = nullptr;
  if (a.offsets) {
    scales = static_cast<uint8_t*>(ws) + scales_at(a.P, L.E);
    const size_t threads = (size_t)a.P * ((L.D + kPer - 1) / kPer);
    hipLaunchKernelGGL(tiles_kernel, dim3((unsigned)(1 + (threads + 1023) / 1024)), dim3(1024), 0, st, a, L.E, L.K,
                       (int)tile_cap(a.P, L.E), list, scales);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int dense_tiles = (a.P + kBM - 1) / kBM;
  const dim3 grid((unsigned)workgroups()), block(64 * kWaves);
  if (L.glu) {
    if (fp32_out)
      hipLaunchKernelGGL((tiled_kernel<true, true>), grid, block, 0, st, a, L, list, scales, dense_tiles);
    else
      hipLaunchKernelGGL((tiled_kernel<true, false>), grid, block, 0, st, a, L, list, scales, dense_tiles);
  } else {
    if (fp32_out)
      hipLaunchKernelGGL((tiled_kernel<false, true>), grid, block, 0, st, a, L, list, scales, dense_tiles);
    else
      hipLaunchKernelGGL((tiled_kernel<false, false>), grid, block, 0, st, a, L, list, scales, dense_tiles);
  }
  return hipGetLastError();
}

}  // namespace moe
