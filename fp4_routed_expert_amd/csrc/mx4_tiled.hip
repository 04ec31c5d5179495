// MXFP4 x MXFP4 products for many rows (the operators of mx4_stream.hip, the
// same packed weights): LDS-tiled, bound by the FP4 matrix rate, or by HBM
// where an expert's rows are few.
//
// A work item is up to 256 rows of one group x 8 weight tiles (256 weight rows).
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
//
// Measured (one call): 4604 rows, K 16384, N 7168: 239 us, 4.5 PFLOP/s with the
// matrix units 65 % busy at the 1.58 GHz that the power limit leaves.  SwiGLU
// of 4604 tokens x 8 of 256 experts, K 7168, N 2048: 816 us, 5.8 TB/s of HBM.
// 16384 tokens x 8 of 256 experts (Zipf), K 2048, N 7168: 1215 us, 3.2 PFLOP/s
// and 3.5 TB/s.  The same tile by four waves of 64 x 256, one per SIMD: 277, 1058 and
// 1490 us before the later steps, against 283, 960 and 1362 with eight waves
// and stages of 128 bytes a row; 192 rows with three row stages is 3-15 %
// slower.
#include "tiled.h"

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
constexpr int kInfo = kIdx + kWaves * 256;   // for each wave eight items' (first row, rows, column)
constexpr int kState = kInfo + kWaves * 128; // and where its cursor goes next
constexpr int kLds = kState + kWaves * 64;
static_assert(kStage % 1024 == 0 && kLds <= 160 * 1024, "LDS");

// Rows of an item.  A group's tiles of at most 256 rows are of equal heights.
struct Tile {
  int row0, n;
};

// Rows of each tile of a group of n rows, in whole sub-tiles of 32.
__host__ __device__ __forceinline__ int tile_height(int n, int tiles) {
  return ((n + 31) / 32 + tiles - 1) / tiles * 32;
}

// How long tiles x ntn items take whose rows are at most s sub-tiles per SIMD
// (64 s rows): they run in rounds of one per CU, an item takes about 7 + 2 s
// units (what does not shrink is the wait for its loads: K 7168, N 2048, 512
// rows: 39 us with s = 4, 28 with 2, 23 with 1).  The s of the fewest units is
// taken, the largest on a tie.  Dense, K 7168, N 2048, 1024 rows: 24 us against
// 39 with tiles of 256 rows; K 4096, N 1536, 4604 rows: 25 against 29.
__host__ __device__ __forceinline__ float item_units(uint32_t tiles, int ntn, float per_cu, int s) {
  return ceilf((float)tiles * (float)ntn * per_cu) * (float)(7 + 2 * s);  // per_cu: 1 / CUs
}

// Workspace of a grouped product: the number of tiles, from byte 16 on four
// words per tile, from rows_at() on the x row of each sorted row, and from
// scales_at() on the activation scales by stage: the eight bytes of stage d of
// sorted row p at 8 (d P + p), so that a tile's scales of a stage are one run
// instead of a request to L2 for each row.
long tile_cap(long P, int E) { return P / 64 + (P < E ? P : E); }
size_t rows_at(long P, int E) { return PackedLayout::align256(16 + 16 * (size_t)tile_cap(P, E)); }
size_t scales_at(long P, int E) { return PackedLayout::align256(rows_at(P, E) + 4 * (size_t)P); }

// Block 0 lists the tiles, each thread of the others moves kPer stages of one
// row's scales (SwiGLU of 4604 x 8 rows, K 7168: 9.3 us; 16 without the wide
// loads).
constexpr int kPer = 4;
__global__ __launch_bounds__(1024) void tiles_kernel(Mx4Args a, int E, int K, int ntn, float per_cu, int cap,
                                                     bool wide, int32_t* __restrict__ ws,
                                                     int32_t* __restrict__ xrows, uint8_t* __restrict__ scales) {
  const int P = a.P;
  if (blockIdx.x > 0) {
    const int D = (K + 255) / 256;
    const int p = (int)((blockIdx.x - 1) * 1024 + threadIdx.x);
    const int d0 = (int)blockIdx.y * kPer, n = min(kPer, D - d0);
    if (p >= P) return;
    int x = p;
    if (a.rows) x = (int)((uint32_t)a.rows[p] / (uint32_t)a.div);
    x = max(min(x, a.X - 1), 0);
    if (a.rows && d0 == 0) xrows[p] = x;
    const uint32_t* src = reinterpret_cast<const uint32_t*>(a.xs + (size_t)x * (K / 32)) + 2 * d0;
    const int dwords = K / 128 - 2 * d0;  // left in the row from stage d0 on
    uint2 v[kPer];
    if (wide) {  // rows of whole pairs of stages, 16-byte aligned
#pragma unroll
      for (int d = 0; d < kPer; d += 2)
        if (d < n) {
          const v4u t = *reinterpret_cast<const v4u*>(src + 2 * d);
          v[d] = make_uint2(t.x, t.y);
          v[d + 1] = make_uint2(t.z, t.w);
        }
    } else {
#pragma unroll
      for (int d = 0; d < kPer; ++d)
        if (d < n) v[d] = make_uint2(src[2 * d], src[min(2 * d + 1, dwords - 1)]);  // an odd number's last one twice
    }
#pragma unroll
    for (int d = 0; d < kPer; ++d)
      if (d < n) *reinterpret_cast<uint2*>(scales + 8 * ((size_t)(d0 + d) * P + p)) = v[d];
    return;
  }
  if (blockIdx.y > 0) return;
  const int32_t* offsets = a.offsets;
  __shared__ v4u wave_tot[16];
  const int e = threadIdx.x, lane = e & 63, w = e >> 6;
  int begin = 0, n = 0;
  if (e < E) {
    begin = min(max(offsets[e], 0), P);
    n = min(max(offsets[e + 1], begin), P) - begin;
  }
  uint32_t count[4], incl[4];  // tiles of at most 64 (i + 1) rows (a wave's sum stays below 2^32)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    count[i] = (n + 64 * i + 63) / (64 * (i + 1));
    incl[i] = (uint32_t)wave_inclusive_scan((int)count[i], lane);
  }
  if (lane == 63) wave_tot[w] = v4u{incl[0], incl[1], incl[2], incl[3]};
  __syncthreads();
  // offsets that decrease could name more tiles than the list holds, or than 32 bits count
  v4u before = {0, 0, 0, 0}, all = {0, 0, 0, 0};
  for (int v = 0; 64 * v < E; ++v) {
    const v4u t = wave_tot[v];
    if (v == w) before = all;
    all = __builtin_elementwise_add_sat(all, t);
  }
  uint32_t nt = 0, at = 0, total = 0;
  float best = 0.0f;
#pragma unroll
  for (int i = 3; i >= 0; --i) {
    const float units = item_units(all[i], ntn, per_cu, i + 1);
    if (i == 3 || units < best)
      best = units, nt = count[i], at = __builtin_elementwise_add_sat(before[i], incl[i] - nt), total = all[i];
  }
  if (e == 0) ws[0] = min(total, (uint32_t)cap);
  const int h = nt > 0 ? tile_height(n, nt) : 0;
  int4* list = reinterpret_cast<int4*>(ws) + 1;
  for (int i = 0; i < (int)nt; ++i)
    if (__builtin_elementwise_add_sat(at, (uint32_t)i) < (uint32_t)cap) list[at + i] = make_int4(e, begin + i * h, min(h, n - i * h), 0);
}

// What a launch is given.  Only a few of these values are needed at every
// stage; the others are read again from the kernel's arguments (by scalar
// loads) where an item begins or ends, since scalar registers that are kept
// over the K loop spill, and vector registers with them.
struct Launch {
  Mx4Args a;
  Mx4Layout L;
  const int32_t* ws;      // tile list (grouped)
  const int32_t* xrows;   // x row of each sorted row, or null: the same row
  const uint8_t* scales;  // activation scales: of sorted rows by stage (grouped), or of x by row (dense)
  size_t scale_stage;     // bytes from a stage to the next
  int scale_row;          // and from a row to the next
  int tiles, height;      // dense: row tiles and their height
};
typedef __attribute__((address_space(4))) const Launch claunch;

__device__ __forceinline__ void look_up(const claunch* g, Walk& k) {
  if (g->a.offsets) {
    const cint* p = reinterpret_cast<const cint*>(reinterpret_cast<uintptr_t>(g->ws)) + 4 + 4 * k.tt;
    k.e = p[0];
    k.row0 = p[1];
    k.n = p[2];
  } else {
    k.e = 0;
    k.row0 = k.tt * g->height;
    k.n = min(g->height, g->a.P - k.row0);
  }
}
__device__ __forceinline__ void next_item(const claunch* g, Walk& k) {
  k.p += k.stride;
  ++k.count;
  k.more = k.p < k.hi;
  if (!k.more) return;
  k.tt += k.st;
  k.off += k.so;
  if (k.off >= k.w) {
    k.off -= k.w;
    ++k.tt;
  }
  if (k.tt >= k.ntt) locate(k);
  look_up(g, k);
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
  int left;           // stages left of the item (this one counted)
};

struct Frag {
  v4u x[2], w[4];
};

struct Ctx {
  uint32_t lds;
  int lane, wave;
  int D;               // stages of an item
  bool odd;            // an odd number of steps
  bool clip_scales;    // the activation scales lie by row
  size_t scale_stage;  // bytes from a stage's to the next one's

  // the kernel's arguments, read where this is called
  __device__ __forceinline__ const claunch* launch() const {
    const claunch* g = (const claunch*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(g));
    return g;
  }
};

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

__device__ __forceinline__ Walk load_walk(const Ctx& c) { return read_walk(c.lds + kState + 64u * (uint32_t)c.wave); }
__device__ __forceinline__ void store_walk(const Ctx& c, const Walk& k) {
  write_walk(c.lds + kState + 64u * (uint32_t)c.wave, k);
}

// Row index DMA of the walk's item into the index buffer: each wave loads, and
// later reads, the indices of the 32 rows whose pieces it moves.
__device__ __forceinline__ void fetch_rows(const Ctx& c, const Walk& k) {
  const int32_t* xrows = c.launch()->xrows;
  if (!xrows || !k.more) return;
  dma4(reinterpret_cast<const uint8_t*>(xrows + k.row0), 4u * (uint32_t)min(32 * c.wave + (c.lane & 31), k.n - 1),
       c.lds + kIdx + 256u * (uint32_t)c.wave);
}

// The last stage of an odd number of steps has no second step.  Its weights are
// zeros; for the rows, what would lie past their end reads the first step's
// bytes (a block that is NaN there is NaN in the first step too).
__device__ __forceinline__ void clip_tail(const Ctx& c, Cursor& k) {
  if (k.left != 1 || !c.odd) return;
#pragma unroll
  for (int u = 0; u < 4; ++u) k.a[u] -= (((uint32_t)c.lane & 7) ^ (uint32_t)((c.lane >> 4) + 4 * (u & 1))) & 4 ? 64u : 0u;
  if (c.clip_scales) k.sa -= 4u * (uint32_t)(c.lane & 1);
}

// Moves the cursor to the walk's item (whose row indices are in the index
// buffer), notes it for the wave's own use when it gets there, and the walk to
// the one after it.
__device__ __forceinline__ void enter(const Ctx& c, Cursor& k, Walk& walk) {
  const claunch* g = c.launch();
  const int tn = walk.base + walk.off;
  const size_t J2 = (size_t)c.D * 2048;  // half the bytes of a weight tile
  *reinterpret_cast<lds_words*>((uintptr_t)(c.lds + kInfo + 128u * (uint32_t)c.wave + 16u * (uint32_t)(walk.count & 7))) =
      v4u{(uint32_t)walk.row0, (uint32_t)walk.n, (uint32_t)tn, 0u};
  const uint32_t row_bytes = (uint32_t)g->L.K / 2;
  const bool gather = g->xrows != nullptr;
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const int r = 8 * u + (c.lane >> 3);
    // logical piece of the lane: physical piece l % 8 of a row whose r / 2 % 8 is l / 16 + 4 (u % 2)
    const uint32_t piece = ((uint32_t)c.lane & 7) ^ (uint32_t)((c.lane >> 4) + 4 * (u & 1));
    // rows past the tile read its last one
    const int x = gather ? lds_i32(c.lds + kIdx + 4 * (64 * c.wave + r)) : walk.row0 + min(32 * c.wave + r, walk.n - 1);
    k.a[u] = (uint32_t)x * row_bytes + 16u * piece;
  }
  k.sa = (uint32_t)min(scale_row(walk.n, c.wave, c.lane), walk.n - 1) * (uint32_t)g->scale_row +
         4u * (uint32_t)(c.lane & 1);
  k.x = wave_ptr(g->a.xq);
  k.xs = wave_ptr(g->scales + (size_t)walk.row0 * g->scale_row);
  // tiles past the last one read the last one; their columns are not stored
  const int nt = min(tn * kBT + c.wave, g->L.NT - 1), q = min(2 * tn + (c.wave >> 2), g->L.NG - 1);
  k.w = wave_ptr(g->a.packed + ((size_t)walk.e * g->L.NT + nt) * (2 * J2));
  k.ws = wave_ptr(g->a.packed + g->L.s_off + ((size_t)walk.e * g->L.NG + q) * (J2 / 2) + 256 * (c.wave & 3));
  k.left = c.D;
  clip_tail(c, k);
  next_item(g, walk);
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
    case 5: dma16(k.x, k.a[3], S + 4096u * w + 3u * 1024u); break;
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
    // a stage after the item was entered, when its successor's tile is known
    if (k.left == c.D) fetch_rows(c, load_walk(c));
    --k.left;
    k.x += 128;
    k.w += 4096;
    k.xs += c.scale_stage;
    k.ws += 1024;
    clip_tail(c, k);
    return;
  }
  Walk walk = load_walk(c);
  if (!walk.more) return;
  // the indices were loaded a stage after the cursor entered this item; with
  // four stages or more since then the waits of the steps have covered them
  if (c.D < 5) {
    if (c.D == 1) fetch_rows(c, walk);
    wait_vmcnt<0>();
  }
  enter(c, k, walk);
  store_walk(c, walk);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the indices are read before they are replaced
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
        if constexpr (H == 1) read_scales(ns, nxt, ad, raw);
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

// Stores of one sub-tile: element v of a lane is row 8 (v / 4) + 4 g + v % 4;
// the group's f tiles are f neighbouring columns, so a half-wave's store covers
// a whole run of 128 (64 with SwiGLU) outputs.  base (uniform): row 0 of the
// sub-tile, the group's first column; off: the lane's bytes from there (its
// column, and 4 g rows down); left: rows of the sub-tile that exist.  The stores
// are non-temporal: the outputs would push rows and weights out of L2 (16384
// tokens Zipf 1279 -> 1247 us, SwiGLU 867 -> 853, dense 282 -> 277, back to back).
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
            __builtin_nontemporal_store(v2f{o[0], o[1]}, reinterpret_cast<global<v2f>*>(q));
          else
            __builtin_nontemporal_store(v4f{o[0], o[1], o[2], o[3]}, reinterpret_cast<global<v4f>*>(q));
        } else {
#pragma unroll
          for (int t = 0; t < kO - 1; ++t)
            if (t < f) q[t] = o[t];
        }
      } else {
        global<uint16_t>* q = reinterpret_cast<global<uint16_t>*>(y);
        if (!kMask || f == kO) {
          if constexpr (kGlu)
            __builtin_nontemporal_store((uint32_t)f32x2_to_bf16(o[0], o[1]), reinterpret_cast<global<uint32_t>*>(q));
          else
            __builtin_nontemporal_store(v2u{f32x2_to_bf16(o[0], o[1]), f32x2_to_bf16(o[2], o[3])},
                                        reinterpret_cast<global<v2u>*>(q));
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
  uint32_t cur = wave_u32(c.lds + (uint32_t)(stage * kStage)), nxt = wave_u32(c.lds + (uint32_t)((stage ^ 1) * kStage));
  if constexpr (S > 0) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][q][v] = 0.0f;
    v4u raw;
    read_scales(s, cur, ad, raw);
#pragma unroll
    for (int q = 0; q < S + 4; ++q) read_frag(f0, cur + ad.a[0], cur + ad.w, q);
    shift_scales<S>(s, ad, raw);
  }
  for (int d = 0; d < c.D; ++d) {
    cur = wave_u32(c.lds + (uint32_t)(stage * kStage));
    nxt = wave_u32(c.lds + (uint32_t)((stage ^ 1) * kStage));
    step<S, 0>(c, k, ad, cur, nxt, acc, f0, f1, s);
    step<S, 1>(c, k, ad, cur, nxt, acc, f0, f1, s);
    stage ^= 1;
  }
  if constexpr (S > 0) {
    constexpr int kO = kGlu ? 2 : 4;
    constexpr uint32_t kB = kF32 ? 4 : 2;
    const claunch* launch = c.launch();
    const int N = launch->L.N, g = c.lane >> 5, f = min(N / 32 - kO * group, kO);
    const size_t row_bytes = (size_t)N * kB;
    const uint32_t off = ((uint32_t)(4 * g) * (uint32_t)N + (uint32_t)f * (uint32_t)(c.lane & 31)) * kB;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int m = 32 * (sub0 + i);
      uint8_t* base = static_cast<uint8_t*>(launch->a.y) + ((size_t)(t.row0 + m) * N + (size_t)(32 * kO) * group) * kB;
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
    Launch launch) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  const Ctx c{(uint32_t)(uintptr_t)(lds_u8*)lds, lane, wave, launch.L.D, (launch.L.J & 1) != 0, !launch.a.offsets,
              launch.scale_stage};
  Cursor k;
  int mine;  // items of this workgroup
  {
    const claunch* g = c.launch();
    Walk walk;
    walk.ntt = g->a.offsets ? *reinterpret_cast<const cint*>(reinterpret_cast<uintptr_t>(g->ws)) : g->tiles;
    walk.ntn = (g->L.NT + kBT - 1) / kBT;
    const int items = walk.ntt * walk.ntn, per = (items + 7) / 8;
    // workgroup b runs on XCD b % 8, which owns the run [x per, x per + per)
    const int lo = min((int)(blockIdx.x & 7) * per, items);
    walk.hi = min(lo + per, items);
    walk.stride = (int)(gridDim.x >> 3);
    walk.p = lo + (int)(blockIdx.x >> 3);
    if (walk.p >= walk.hi) return;  // uniform: before any barrier
    mine = (walk.hi - walk.p + walk.stride - 1) / walk.stride;
    walk.count = 0;
    walk.more = 1;
    locate(walk);
    look_up(g, walk);
    fetch_rows(c, walk);
    wait_vmcnt<0>();
    enter(c, k, walk);
    store_walk(c, walk);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
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
  for (int i = 0; i < mine; ++i) {
    // as the cursor noted it
    const v4u info = lds_v4(c.lds + kInfo + 128 * wave + 16 * (i & 7));
    const Tile t{(int)wave_u32(info.x), (int)wave_u32(info.y)};
    const int tn = (int)wave_u32(info.z);
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

// Row tiles of a dense product of P rows and ntn columns of items.
int dense_tiles(int P, int ntn) {
  int tiles = 0;
  float best = 0.0f;
  for (int s = 4; s > 0; --s) {
    const int t = (P + 64 * s - 1) / (64 * s);
    const float units = item_units(t, ntn, 1.0f / (float)workgroups(), s);
    if (s == 4 || units < best) best = units, tiles = t;
  }
  return tiles;
}

}  // namespace

size_t mx4_tiled_ws_bytes(long P, int E, int K) { return scales_at(P, E) + 8 * (size_t)P * ((K + 255) / 256); }

hipError_t launch_mx4_tiled(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, void* ws, hipStream_t st) {
  const int ntn = (L.NT + kBT - 1) / kBT;
  Launch g{a, L, nullptr, nullptr, a.xs, 8, L.K / 32, 0, 0};
  if (a.offsets) {
    int32_t* list = static_cast<int32_t*>(ws);
    int32_t* xrows = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + rows_at(a.P, L.E));
    uint8_t* scales = static_cast<uint8_t*>(ws) + scales_at(a.P, L.E);
    const dim3 movers(1 + ((unsigned)a.P + 1023u) / 1024, (unsigned)(L.D + kPer - 1) / kPer);
    const bool wide = L.K % 512 == 0 && (uintptr_t)a.xs % 16 == 0;
    hipLaunchKernelGGL(tiles_kernel, movers, dim3(1024), 0, st, a, L.E, L.K, ntn, 1.0f / (float)workgroups(),
                       (int)tile_cap(a.P, L.E), wide, list, xrows, scales);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.ws = list;
    g.xrows = a.rows ? xrows : nullptr;
    g.scales = scales;
    g.scale_stage = 8 * (size_t)a.P;
    g.scale_row = 8;
  } else {
    g.tiles = dense_tiles(a.P, ntn);
    g.height = tile_height(a.P, g.tiles);
  }
  const dim3 grid((unsigned)workgroups()), block(64 * kWaves);
  if (L.glu) {
    if (fp32_out)
      hipLaunchKernelGGL((tiled_kernel<true, true>), grid, block, 0, st, g);
    else
      hipLaunchKernelGGL((tiled_kernel<true, false>), grid, block, 0, st, g);
  } else {
    if (fp32_out)
      hipLaunchKernelGGL((tiled_kernel<false, true>), grid, block, 0, st, g);
    else
      hipLaunchKernelGGL((tiled_kernel<false, false>), grid, block, 0, st, g);
  }
  return hipGetLastError();
}

}  // namespace moe
