// FP8 products with block scales of 128 for many rows (the operators of
// fp8b_stream.hip, the same packed weights), and the gated feed-forward block and
// its backward pass on them: LDS-tiled, bound by the FP8 matrix rate and the
// vector unit beside it, or by HBM where an expert's rows are few.
//
// A work item is up to 256 rows of one group x 16 weight tiles (256 weight rows:
// two scale blocks of 128 columns, or one of gate and up).  Eight waves, two per
// SIMD, in a 4 x 2 grid, each with up to four token tiles of 16 x eight weight
// tiles.  One v_mfma_f32_16x16x128_f8f6f4 sums one scale block of K into fresh
// registers; an fp32 multiply-add per element then adds it to the accumulator,
// times the product of the row's and the weight block's scale.  Weights are the
// A operand, so that a lane's elements are all of one token: its scale products
// are one multiplication per token tile and block.  The multiply-adds of an MFMA
// (4 per lane, 16 clocks of the vector unit) run three MFMAs (of 32 clocks) later,
// where their wait states are covered.  The accumulators have to lie in vector
// registers, 128 of them.
//
// Stages are one block of K: 32 KiB of row pieces (128 bytes of each row), two
// halves of 16 KiB of weight tiles and the scales, from global memory to LDS by
// LDS-DMA.  A wave's token tiles go to registers before the stage begins, so the
// row pieces are free in its middle: two places of them and five of weight halves
// keep the loads of a stage two stages ahead (with two places of everything the
// loads had one stage, and a stage took 1.2 us however few its rows: K 16384, N
// 7168, 256 rows 178 us, now 119).  Two barriers a stage: behind its first quarter,
// which publishes the second weight half and frees the row pieces and the first
// half, and behind its third, which publishes the next stage's rows and first half
// and frees the second.  Every wave issues the same nine loads per stage
// in the same order, dummy stages past the end, so that one wait count serves every
// barrier.  Row r's eight 16-byte pieces lie at piece p ^ (r / 2 % 8), which spreads
// the 16 rows that one LDS cycle serves over all banks.
//
// The workgroups are persistent: one per CU (its LDS allows no second) walks its
// XCD's contiguous share of the items, and the stages run on across items.
//
// 4604 rows, K 16384, N 7168: 440 us, 2.46 PFLOP/s, the MFMAs busy 61 % at the 1.8 GHz
// that the power limit leaves.  A stage is 32 MFMAs of 32 clocks for each of a SIMD's
// two waves and about 285 instructions, which take a wave eight clocks each: 2048
// clocks of the matrix cores beside 2280 of each wave's issue, and what a wave waits at
// the barriers on top.  With K 2048 an item is 16 stages and its stores 7 % of
// it (16 experts of 8192 rows: 1886 us, 1758 with nothing stored).  SwiGLU of 256
// experts of 144 rows, K 7168, N 2048: 1.43-1.54 ms, 7.8 GB at 5.2-5.6 TB/s.
#include "fp8b.h"
#include "tiled.h"

namespace moe {
namespace {

constexpr int kBM = 256;              // rows of an item
constexpr int kBT = 16;               // weight tiles of an item
constexpr int kWaves = 8;
constexpr int kX = kBM * 128;         // row pieces of a stage
constexpr int kS = kWaves * 256;      // scales: each wave's 32 rows and the item's two row blocks
constexpr int kHalf = kBT / 2 * 2048; // half the weight tiles: the first or the last four of either wave column
constexpr int kHalves = 5;
constexpr int kOffS = 2 * kX;                  // behind two places of row pieces two of scales
constexpr int kOffW = kOffS + 2 * kS;          // and five of weight halves
constexpr int kIdx = kOffW + kHalves * kHalf;  // the next item's row indices
constexpr int kInfo = kIdx + kWaves * 256;     // for each wave eight items' (first row, rows, column)
constexpr int kState = kInfo + kWaves * 128;   // and where its cursor goes next
constexpr int kTop = kState + kWaves * 64;     // largest magnitudes that the waves of a row exchange
constexpr int kLds = kTop + kWaves * 256;
static_assert(kLds <= 160 * 1024, "LDS");

// With exact products (results that stay in fp32) a wave takes at most two token
// tiles, whose bf16 values it keeps: 128 rows an item.
constexpr int kWideSubs = 2;

// Rows of an item.  A group's tiles are of equal heights.
struct Tile {
  int row0, n;
};

// Rows of each tile of a group of n rows, in whole token tiles of 16.
__host__ __device__ __forceinline__ int tile_height(int n, int tiles) {
  return ((n + 15) / 16 + tiles - 1) / tiles * 16;
}

// How long tiles x ntn items take whose rows are at most 64 s: they run in rounds
// of one per CU.  The s of the fewest units is taken, the largest on a tie (us, with s 4
// always: K 7168, N 2048, 1024 rows 44 and 79; K 16384, N 7168, 512 rows 116 and 170; K
// 4096, N 1536, 5000 rows 37 and 51; 4 experts of 256 rows, K 7168, N 2048, 47 and 82;
// with 0, 2 or 7 for the 4 units of an item that do not shrink the same within 1 %).
__host__ __device__ __forceinline__ float item_units(uint32_t tiles, int ntn, float per_cu, int s) {
  return ceilf((float)tiles * (float)ntn * per_cu) * (float)(4 + 2 * s);  // per_cu: 1 / CUs
}

// Workspace of a grouped product: the number of tiles, from byte 16 on four words
// per tile, from rows_at() on the x row of each sorted row.
long tile_cap(long P, int E) { return P / 64 + (P < E ? P : E); }
size_t rows_at(long P, int E) { return PackedLayout::align256(16 + 16 * (size_t)tile_cap(P, E)); }

// Block 0 lists the tiles (of at most 64 `most` rows), the others look the rows up.
__global__ __launch_bounds__(1024) void tiles_kernel(Fp8bArgs a, int E, int ntn, float per_cu, int most, int cap,
                                                     int32_t* __restrict__ ws, int32_t* __restrict__ xrows) {
  const int P = a.P;
  if (blockIdx.x > 0) {
    const int p = (int)((blockIdx.x - 1) * 1024 + threadIdx.x);
    if (p < P) xrows[p] = entry_row(a.rows, p, a.div, a.X);
    return;
  }
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
    if (i >= most) continue;
    const float units = item_units(all[i], ntn, per_cu, i + 1);
    if (i == most - 1 || units < best)
      best = units, nt = count[i], at = __builtin_elementwise_add_sat(before[i], incl[i] - nt), total = all[i];
  }
  if (e == 0) ws[0] = min(total, (uint32_t)cap);
  const int h = nt > 0 ? tile_height(n, nt) : 0;
  int4* list = reinterpret_cast<int4*>(ws) + 1;
  for (int i = 0; i < (int)nt; ++i)
    if (__builtin_elementwise_add_sat(at, (uint32_t)i) < (uint32_t)cap)
      list[at + i] = make_int4(e, begin + i * h, min(h, n - i * h), 0);
}

// What a launch is given.  Only a few of these values are needed at every stage;
// the others are read again from the kernel's arguments (by scalar loads) where
// an item begins or ends, since scalar registers that are kept over the K loop
// spill.
struct Launch {
  Fp8bArgs a;
  Fp8bLayout L;
  const int32_t* ws;     // tile list (grouped)
  const int32_t* xrows;  // x row of each sorted row, or null: the same row
  int tiles, height;     // one group: row tiles and their height
  int panels;            // of the walk
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
  if (k.tt >= k.ntt) locate(k, g->panels);
  look_up(g, k);
}

// Where the DMA stands: the next stage to load of the item it is in.
struct Cursor {
  const uint8_t* x;   // activation codes (uniform)
  const uint8_t* w;   // the wave's weight tile of the first half (uniform)
  uint32_t w1;        // bytes from it to the second half's
  const uint8_t* s;   // per lane: its scale (lanes 0-31 of rows 32 w + l, the others of a weight block)
  uint32_t a[4];      // per lane: its piece of rows 32 w + 8 u + l / 8
  int left;           // stages left of the item (this one counted)
};

struct Ctx {
  uint32_t lds;
  int wave;
  int J;         // stages of an item
  uint32_t row;  // bytes from a block's row scales to the next one's
  // 16 x lane, made anew at every stage: what is derived from it would otherwise
  // be computed in front of the K loop and kept, or spilled, over it
  uint32_t l16;
  __device__ __forceinline__ int lane() const { return (int)(l16 >> 4); }

  // the kernel's arguments, read where this is called
  __device__ __forceinline__ const claunch* launch() const {
    const claunch* g = (const claunch*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(g));
    return g;
  }
};

// Token tiles that wave row wm (of four) takes of a tile of n rows: how many, and
// the first one.  Wave rows 0 and 2 share SIMDs, as do 1 and 3.
__device__ __forceinline__ int sub_tiles(int n, int wm) { return ((n + 15) / 16 + 3 - wm) / 4; }
__device__ __forceinline__ int first_sub(int n, int wm) {
  const int n16 = (n + 15) / 16;
  return wm * (n16 / 4) + min(wm, n16 % 4);
}

__device__ __forceinline__ Walk load_walk(const Ctx& c) { return read_walk(c.lds + kState + 64u * (uint32_t)c.wave); }
__device__ __forceinline__ void store_walk(const Ctx& c, const Walk& k) {
  write_walk(c.lds + kState + 64u * (uint32_t)c.wave, k);
}

// Row index DMA of the walk's item into the index buffer: each wave loads, and
// later reads, the indices of the 32 rows whose pieces and scales it moves.
__device__ __forceinline__ void fetch_rows(const Ctx& c, const Walk& k) {
  const int32_t* xrows = c.launch()->xrows;
  if (!xrows || !k.more) return;
  dma4(reinterpret_cast<const uint8_t*>(xrows + k.row0), 4u * (uint32_t)min(32 * c.wave + (c.lane() & 31), k.n - 1),
       c.lds + kIdx + 256u * (uint32_t)c.wave);
}

// Moves the cursor to the walk's item (whose row indices are in the index
// buffer), notes it for the wave's own use when it gets there, and the walk to
// the one after it.
__device__ __forceinline__ void enter(const Ctx& c, Cursor& k, Walk& walk) {
  const claunch* g = c.launch();
  const int tn = walk.base + walk.off;
  *reinterpret_cast<lds_words*>((uintptr_t)(c.lds + kInfo + 128u * (uint32_t)c.wave + 16u * (uint32_t)(walk.count & 7))) =
      v4u{(uint32_t)walk.row0, (uint32_t)walk.n, (uint32_t)tn, 0u};
  const bool gather = g->xrows != nullptr;
  const int K = g->L.K, J = g->L.J;
  // rows past the tile read its last one
  auto row = [&](int r) {
    return gather ? lds_i32(c.lds + kIdx + 256u * (uint32_t)c.wave + 4u * (uint32_t)r)
                  : walk.row0 + min(32 * c.wave + r, walk.n - 1);
  };
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    // logical piece of the lane: physical piece l % 8 of a row whose r / 2 % 8 is l / 16 + 4 (u % 2)
    const uint32_t piece = ((uint32_t)c.lane() & 7) ^ (uint32_t)((c.lane() >> 4) + 4 * (u & 1));
    k.a[u] = (uint32_t)row(8 * u + (c.lane() >> 3)) * (uint32_t)K + 16u * piece;
  }
  const int block = min(2 * tn + (c.lane() & 1), g->L.NB - 1);  // row blocks past the last one: as the tiles below
  const float* ws = reinterpret_cast<const float*>(g->a.packed + g->L.s_off) + ((size_t)walk.e * g->L.NB + block) * J;
  k.s = reinterpret_cast<const uint8_t*>(c.lane() < 32 ? g->a.xs + row(c.lane() & 31) : ws);
  k.x = wave_ptr(g->a.xq);
  // tiles past the last one read that; their columns are not stored
  const int nt = min(tn * kBT + c.wave + 4 * (c.wave >> 2), g->L.NT - 1), nt1 = min(nt + 4, g->L.NT - 1);
  k.w = wave_ptr(g->a.packed + ((size_t)walk.e * g->L.NT + nt) * ((size_t)J * 2048));
  k.w1 = wave_u32((uint32_t)(nt1 - nt) * (uint32_t)J * 2048u);
  k.left = c.J;
  next_item(g, walk);
}

// Load u (< 9) of the wave's share of the cursor's stage: 0-1 the first weight
// half into place W0, 2-5 row pieces and 6 scales into place p (0, 1), 7-8 the
// second weight half into place W1.
constexpr int kLoads = 9;
__device__ __forceinline__ void issue(const Ctx& c, const Cursor& k, int p, uint32_t W0, uint32_t W1, int u) {
  const uint32_t w = (uint32_t)c.wave, l16 = c.l16, X = c.lds + (uint32_t)(p * kX) + 4096u * w;
  switch (u) {
    case 0: dma16(k.w, l16, W0 + 2048u * w); break;
    case 1: dma16<1024>(k.w, l16, W0 + 2048u * w); break;
    case 2: dma16(k.x, k.a[0], X); break;
    case 3: dma16(k.x, k.a[1], X + 1024u); break;
    case 4: dma16(k.x, k.a[2], X + 2048u); break;
    case 5: dma16(k.x, k.a[3], X + 3u * 1024u); break;
    case 6: dma4_lanes(k.s, c.lds + (uint32_t)(kOffS + p * kS) + 256u * w); break;
    case 7: dma16(k.w + k.w1, l16, W1 + 2048u * w); break;
    default: dma16<1024>(k.w + k.w1, l16, W1 + 2048u * w);
  }
}

// After a stage's loads: the next stage, or the next item's first (past the last
// item its last stage is loaded again and never used).
__device__ __forceinline__ void advance(const Ctx& c, Cursor& k) {
  if (k.left > 1) {
    // a stage after the item was entered, when its successor's tile is known
    if (k.left == c.J) fetch_rows(c, load_walk(c));
    --k.left;
    k.x += 128;
    k.w += 2048;
    k.s += c.lane() < 32 ? c.row : 4u;
    return;
  }
  Walk walk = load_walk(c);
  if (!walk.more) return;
  // the indices were loaded a stage after the cursor entered this item; two stages
  // of loads behind them, the waits have covered them
  if (c.J < 3) {
    if (c.J == 1) fetch_rows(c, walk);
    wait_vmcnt<0>();
  }
  enter(c, k, walk);
  store_walk(c, walk);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the indices are read before they are replaced
}

// LDS addresses of a lane, moved from place to place as the loop goes on.
struct Addr {
  uint32_t x0, x1;  // the two pieces of row r of the wave's first token tile (tile i at + 2048 i)
  uint32_t w;       // the wave's first weight tile of a half (tile i at + 2048 i, its second half at + 1024)
  uint32_t sw;      // the first of the wave's weight scales
  uint32_t s0, s1;  // the row's scale in the first and the second token tile (two tiles on: + 256)
};

// Where the loop stands: the stage's parity, and the places of its first weight
// half and of the one that is loaded next.
struct Place {
  int p;
  int read, load;
  int slack, stores;  // barriers that need not wait for the last item's stores, and how many those are, in fours
};
__device__ __forceinline__ int next_half(int h) { return h == kHalves - 1 ? 0 : h + 1; }
__device__ __forceinline__ uint32_t half_at(const Ctx& c, int h) { return wave_u32(c.lds + (uint32_t)(kOffW + h * kHalf)); }

template <int S>
struct Regs {
  v8i a[4];  // weight tiles
  v8i b[S];  // token tiles of a stage
};
template <>
struct Regs<0> {};

// weight tile i of a half
__device__ __forceinline__ v8i read_w(const Addr& ad, int i) {
  return cat_pieces(lds_v4(ad.w + 2048 * i), lds_v4(ad.w + 2048 * i + 1024));
}
__device__ __forceinline__ v8i read_x(const Addr& ad, int i) {
  return cat_pieces(lds_v4(ad.x0 + 2048 * i), lds_v4(ad.x1 + 2048 * i));
}
__device__ __forceinline__ float lds_f32(uint32_t addr) { return __int_as_float(lds_i32(addr)); }

// A barrier of the loop: the loads that it publishes have landed (kBehind more have
// been issued behind them), and this wave's LDS reads are done; then everyone's.
// The first one of a stage publishes its second weight half, the last loads of two
// stages before; the other one the next stage's rows, scales and first half, the
// first seven loads of the stage before.  Behind an item's end stand its stores too
// (vector memory operations complete in order): the loads that the next three
// barriers publish are older, so that as many more may be outstanding and nothing
// waits for the stores.
constexpr int kFirst = kLoads + 2, kSecond = 2 + 7;
template <int kBehind>
__device__ __forceinline__ void wait_and_meet() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kBehind) : "memory");
}
template <int kBehind>
__device__ __forceinline__ void publish(Place& at) {
  if (at.slack == 0) {
    wait_and_meet<kBehind>();
    return;
  }
  --at.slack;
  switch (at.stores) {
    case 1: wait_and_meet<kBehind + 4>(); break;
    case 2: wait_and_meet<kBehind + 8>(); break;
    case 3: wait_and_meet<kBehind + 12>(); break;
    case 4: wait_and_meet<kBehind + 16>(); break;
    case 5: wait_and_meet<kBehind + 20>(); break;
    case 6: wait_and_meet<kBehind + 24>(); break;
    case 7: wait_and_meet<kBehind + 28>(); break;
    default: wait_and_meet<kBehind + 32>();
  }
}
// After an item: at least n stores have been issued since its last loads.
__device__ __forceinline__ void stored(Place& at, int n) {
  at.stores = min(n / 4, 8);
  at.slack = at.stores > 0 ? 3 : 0;
}

// One stage for a wave with S live token tiles.  On entry f holds its first two
// weight tiles and its token tiles, ad.w is in its first weight half, the scales'
// addresses in its scales, ad.x0 and ad.x1 in the next stage's rows.  On exit the
// same for the next stage.
template <int S, bool kGlu, bool kWide>
__device__ __forceinline__ void step(Ctx& c, Cursor& k, Addr& ad, Place& at, v4f (&acc)[8][4], Regs<S>& f) {
  c.l16 = opaque(c.l16);
  const int load1 = next_half(at.load), read1 = next_half(at.read), read2 = next_half(read1);
  const uint32_t W0 = half_at(c, at.load), W1 = half_at(c, load1);
  auto load = [&](int u) { issue(c, k, at.p, W0, W1, u); };
  if constexpr (S == 0) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) {
      if (u == 2) publish<kFirst>(at);
      if (u == 7) publish<kSecond>(at);
      load(u);
    }
    advance(c, k);
  } else {
    // addresses on from a place to the next one
    const uint32_t hop1 = wave_u32((uint32_t)((read1 - at.read) * kHalf)), hop2 = wave_u32((uint32_t)((read2 - read1) * kHalf));
    const uint32_t flip = wave_u32((uint32_t)(at.p ? -1 : 1));
    float ks[S], ku[S], sx[S];
    const float w0 = lds_f32(ad.sw), w1 = kGlu ? lds_f32(ad.sw + 4) : 0.0f;
#pragma unroll
    for (int t = 0; t < S; ++t) sx[t] = lds_f32((t & 1 ? ad.s1 : ad.s0) + 256 * (t >> 1));
    auto scale_products = [&] {
#pragma unroll
      for (int t = 0; t < S; ++t) {
        ks[t] = sx[t] * w0;
        if constexpr (kGlu) ku[t] = sx[t] * w1;
      }
    };
    // The weight tiles go in pairs, and a pair's MFMAs token tile by token tile, so
    // that a token tile's registers are free for the next stage's six MFMAs before
    // that needs them.  Behind the first MFMA of the second and the fourth pair stand
    // the barriers: the tiles read from there on lie in another half.
    auto turn = [&](int p) {
      if (p == 1) publish<kFirst>(at);
      if (p == 3) publish<kSecond>(at);
      if (p == 1 || p == 3) {
        ad.w = opaque(ad.w + (p == 1 ? hop1 : hop2));
      }
    };
    // tile 2 p + 2 + h, read in pair p
    auto ahead = [&](int p, int h) { f.a[(2 * p + 2 + h) & 3] = read_w(ad, (2 * p + 2 + h) & 3); };
    if constexpr (kWide) {
      Wide x[S];
#pragma unroll
      for (int t = 0; t < S; ++t) x[t] = widen(f.b[t]);
      scale_products();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const Wide w = widen(f.a[i & 3]);
        if ((i & 1) == 0) {
          turn(i >> 1);
          ahead(i >> 1, 0);
          ahead(i >> 1, 1);
        }
        if (i == 6) {
#pragma unroll
          for (int t = 0; t < S; ++t) f.b[t] = read_x(ad, t);
        }
#pragma unroll
        for (int t = 0; t < S; ++t) {
          const v4f d = mfma_wide(w, x[t]);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][t][v] = fmaf(d[v], ks[t], acc[i][t][v]);
          asm volatile("" : "+v"(acc[i][t]));
        }
        // (two in front of the first barrier, five in front of the second, two behind it)
        if (i < 2) load(i);
        if (i >= 2 && i < 6) load(i);
        if (i == 5) load(6);
        if (i >= 6) load(i + 1);
      }
    } else {
      constexpr int kLag = 3;  // MFMAs between one and its multiply-adds
      constexpr int M = 8 * S;
      v4f d[kLag + 1];
      auto add = [&](int m) {
        const int i = 2 * (m / (2 * S)) + (m & 1), t = m / 2 % S;
        const float s = kGlu && (i & 1) ? ku[t] : ks[t];
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][t][v] = fmaf(d[m & kLag][v], s, acc[i][t][v]);
        asm volatile("" : "+v"(acc[i][t]));  // here, not behind the branches of advance()
      };
#pragma unroll
      for (int m = 0; m < M; ++m) {
        const int p = m / (2 * S), at_p = m % (2 * S), h = m & 1, t = m / 2 % S;
        d[m & kLag] = mfma_block(f.a[(2 * p + h) & 3], f.b[t]);
        __builtin_amdgcn_sched_barrier(0);  // in front of a barrier, not behind it
        if (m == kLag - 1) scale_products();  // their reads come back under the first MFMAs
        if (m >= kLag) add(m - kLag);
        if (at_p == 0) {
          turn(p);
          ahead(p, 0);
        }
        if (at_p == 1) ahead(p, 1);
        if (p == 3 && h == 1) f.b[t] = read_x(ad, t);
        // the loads of two stages on, spread over the stage: in front of the first
        // barrier the first weight half, in front of the second rows and scales, behind
        // it the second half
#pragma unroll
        for (int u = 0; u < kLoads; ++u)
          if ((u < 2 ? (2 * u + 1) * S / 2 : u < 7 ? 2 * S + (4 * u - 7) * S / 5 : 6 * S + (2 * u - 13) * S / 2) == m) load(u);
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int m = (M > kLag ? M - kLag : 0); m < M; ++m) add(m);
    }
    advance(c, k);  // here, where the fewest registers are taken
    ad.x0 = opaque(ad.x0 - flip * kX);
    ad.x1 = opaque(ad.x1 - flip * kX);
    ad.sw = opaque(ad.sw + flip * kS);
    ad.s0 = opaque(ad.s0 + flip * kS);
    ad.s1 = opaque(ad.s1 + flip * kS);
  }
  at.p ^= 1;
  at.read = read2;
  at.load = next_half(load1);
}

// (Cached stores: non-temporal ones were 2 % slower for the sums, 16 experts of 8192
// rows, K 2048, N 7168, 1886 us against 1936, and 12 % in the backward pass, 32 experts of
// 2048 rows, K 4096, N 1536, 554 against 620; its non-temporal loads another 2 %.)
__device__ __forceinline__ void store16(void* p, v4u v) { *reinterpret_cast<global<v4u>*>((uintptr_t)p) = v; }
__device__ __forceinline__ void store8(void* p, uint32_t a, uint32_t b) {
  *reinterpret_cast<global<v2u>*>((uintptr_t)p) = v2u{a, b};
}

// Sums as they are: a lane's pair of tiles is eight neighbouring columns of its
// token, a quad of lanes (g = 0..3) 32.
template <int S, bool kF32>
__device__ __forceinline__ int store_sums(const Ctx& c, const v4f (&acc)[8][4], const Tile& t, int sub0, int tn) {
  constexpr size_t kB = kF32 ? 4 : 2;
  const claunch* g = c.launch();
  const int N = g->L.N, r = c.lane() & 15, q = c.lane() >> 4, col0 = 256 * tn + 128 * (c.wave & 1);
  const int pairs = min((N - col0) / 32, 4);  // N is a multiple of 32; none at all where col0 >= N
  uint8_t* y = static_cast<uint8_t*>(g->a.y) + ((size_t)(t.row0 + 16 * sub0 + r) * N + col0 + 8 * q) * kB;
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (16 * (sub0 + i) + r < t.n) {
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (p < pairs) {
          const v4f lo = acc[2 * p][i], hi = acc[2 * p + 1][i];
          uint8_t* o = y + ((size_t)(16 * i) * N + 32 * p) * kB;
          if constexpr (kF32) {
            store16(o, __builtin_bit_cast(v4u, lo));
            store16(o + 16, __builtin_bit_cast(v4u, hi));
          } else {
            store16(o, v4u{f32x2_to_bf16(lo[0], lo[1]), f32x2_to_bf16(lo[2], lo[3]), f32x2_to_bf16(hi[0], hi[1]),
                           f32x2_to_bf16(hi[2], hi[3])});
          }
        }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  return pairs > 0 ? S * pairs * (kF32 ? 2 : 1) : 0;
}

// SwiGLU, and the codes of its rows.  A wave has 64 columns of an item's 128; the
// two waves of a row exchange their largest magnitudes through LDS.
template <int S>
__device__ __forceinline__ int store_glu(const Ctx& c, v4f (&acc)[8][4], const Tile& t, int sub0, int tn) {
  const claunch* g = c.launch();
  const int N = g->L.N, r = c.lane() & 15, q = c.lane() >> 4;
  const size_t P = (size_t)g->a.P;
  const size_t row0 = (size_t)(t.row0 + 16 * sub0 + r);
  const int col0 = 128 * tn + 64 * (c.wave & 1) + 8 * q;
  uint32_t top[S > 0 ? S : 1];
  if constexpr (S > 0) {
    uint16_t* gate = g->a.gate;
    uint16_t* up = g->a.up;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      if (gate && 16 * (sub0 + i) + r < t.n) {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const size_t at = (row0 + 16 * i) * N + col0 + 32 * p;
          const v4f a = acc[4 * p][i], b = acc[4 * p + 2][i], d = acc[4 * p + 1][i], e = acc[4 * p + 3][i];
          store16(gate + at, v4u{f32x2_to_bf16(a[0], a[1]), f32x2_to_bf16(a[2], a[3]), f32x2_to_bf16(b[0], b[1]),
                                 f32x2_to_bf16(b[2], b[3])});
          store16(up + at, v4u{f32x2_to_bf16(d[0], d[1]), f32x2_to_bf16(d[2], d[3]), f32x2_to_bf16(e[0], e[1]),
                               f32x2_to_bf16(e[2], e[3])});
        }
      }
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const float h = glu_out(acc[2 * p][i][v], acc[2 * p + 1][i][v]);
          acc[2 * p][i][v] = h;
          m = max(m, magnitude_bits(h));
        }
      top[i] = max_lanes_xor16_32_u32(m);
      if (q == 0)
        *reinterpret_cast<__attribute__((address_space(3))) uint32_t*>(
            (uintptr_t)(c.lds + kTop + 256u * (uint32_t)c.wave + 4u * (uint32_t)(16 * i + r))) = top[i];
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
  if constexpr (S > 0) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const uint32_t other = (uint32_t)lds_i32(c.lds + kTop + 256u * (uint32_t)(c.wave ^ 1) + 4u * (uint32_t)(16 * i + r));
      const BlockScale k = block_scale(max(top[i], other));
      if (16 * (sub0 + i) + r < t.n) {
        uint8_t* o = g->a.q + (row0 + 16 * i) * N + col0;
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          const v4f lo = acc[4 * p][i], hi = acc[4 * p + 2][i];
          store8(o + 32 * p, block_codes(lo[0], lo[1], lo[2], lo[3], k), block_codes(hi[0], hi[1], hi[2], hi[3], k));
        }
        if (q == 0 && (c.wave & 1) == 0) g->a.s[(size_t)tn * P + row0 + 16 * i] = k.scale;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  return S * (g->a.gate ? 6 : 2);
}

// The sums are dh: dg and du of the wave's 128 columns, and their codes.
template <int S>
__device__ __forceinline__ int store_grad(const Ctx& c, v4f (&acc)[8][4], const Tile& t, int sub0, int tn) {
  const claunch* g = c.launch();
  const int N = g->L.N, r = c.lane() & 15, q = c.lane() >> 4, nb = 2 * tn + (c.wave & 1), NB = N / 128;
  if (nb >= NB) return 0;
  const size_t P = (size_t)g->a.P;
  v4u eg[2][4], eu[2][4];
  auto row_of = [&](int i) { return (size_t)(t.row0 + min(16 * (sub0 + i) + r, t.n - 1)); };
  auto fetch = [&](int i) {
    const size_t at = row_of(i) * N + 128 * nb + 8 * q;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      eg[i & 1][p] = *reinterpret_cast<const global<v4u>*>((uintptr_t)(g->a.gate + at + 32 * p));
      eu[i & 1][p] = *reinterpret_cast<const global<v4u>*>((uintptr_t)(g->a.up + at + 32 * p));
    }
  };
  if constexpr (S > 0) fetch(0);
#pragma unroll
  for (int i = 0; i < S; ++i) {
    if (i + 1 < S) fetch(i + 1);  // in front of this tile's stores, which its values would otherwise wait for
    const int m = 16 * (sub0 + i) + r;
    const size_t row = row_of(i);
    float du[32];
    uint32_t tg = 0, tu = 0;
#pragma unroll
    for (int p = 0; p < 4; ++p)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t wg = eg[i & 1][p][e >> 1], wu = eu[i & 1][p][e >> 1];
        const float gv = __uint_as_float(e & 1 ? wg & 0xFFFF0000u : wg << 16);
        const float uv = __uint_as_float(e & 1 ? wu & 0xFFFF0000u : wu << 16);
        float dg;
        glu_grad(acc[2 * p + (e >> 2)][i][e & 3], gv, uv, dg, du[8 * p + e]);
        acc[2 * p + (e >> 2)][i][e & 3] = dg;
        tg = max(tg, magnitude_bits(dg));
        tu = max(tu, magnitude_bits(du[8 * p + e]));
      }
    const BlockScale kg = block_scale(max_lanes_xor16_32_u32(tg)), ku = block_scale(max_lanes_xor16_32_u32(tu));
    if (m < t.n) {
      uint8_t* o = g->a.q + row * (2 * (size_t)N) + 128 * nb + 8 * q;
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const v4f lo = acc[2 * p][i], hi = acc[2 * p + 1][i];
        store8(o + 32 * p, block_codes(lo[0], lo[1], lo[2], lo[3], kg), block_codes(hi[0], hi[1], hi[2], hi[3], kg));
        const float* u = du + 8 * p;
        store8(o + N + 32 * p, block_codes(u[0], u[1], u[2], u[3], ku), block_codes(u[4], u[5], u[6], u[7], ku));
      }
      if (q == 0) {
        g->a.s[(size_t)nb * P + row] = kg.scale;
        g->a.s[(size_t)(NB + nb) * P + row] = ku.scale;
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  return 8 * S;
}

template <int S, Fp8bOut kOut>
__device__ __forceinline__ void run_item(Ctx& c, Cursor& k, Place& at, const Tile& t, int sub0, int tn) {
  constexpr bool kGlu = kOut == Fp8bOut::kGlu;
  v4f acc[8][4];
  Regs<S> f;
  Addr ad;
  if constexpr (S > 0) {
    const int r = c.lane() & 15, g = c.lane() >> 4, wn = c.wave & 1;
    const uint32_t X = c.lds + (uint32_t)(at.p * kX), sc = c.lds + (uint32_t)(kOffS + at.p * kS);
    ad.x0 = opaque(X + (uint32_t)(16 * sub0 + r) * 128 + (((uint32_t)(g ^ (r >> 1)) & 7) << 4));
    ad.x1 = opaque(X + (uint32_t)(16 * sub0 + r) * 128 + (((uint32_t)(g ^ (r >> 1) ^ 4) & 7) << 4));
    ad.w = opaque(half_at(c, at.read) + (uint32_t)(8192 * wn) + c.l16);
    ad.sw = opaque(sc + (uint32_t)(256 * c.wave + 128 + (kGlu ? 0 : 4 * wn)));
    ad.s0 = opaque(sc + (uint32_t)(256 * (sub0 >> 1) + 64 * (sub0 & 1) + 4 * r));
    ad.s1 = opaque(sc + (uint32_t)(256 * ((sub0 + 1) >> 1) + 64 * ((sub0 + 1) & 1) + 4 * r));
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int q = 0; q < S; ++q) acc[i][q] = v4f{0.f, 0.f, 0.f, 0.f};
    f.a[0] = read_w(ad, 0);
    f.a[1] = read_w(ad, 1);
#pragma unroll
    for (int q = 0; q < S; ++q) f.b[q] = read_x(ad, q);
    const uint32_t flip = (uint32_t)(at.p ? -kX : kX);
    ad.x0 = opaque(ad.x0 + flip);
    ad.x1 = opaque(ad.x1 + flip);
  }
  for (int j = 0; j < c.J; ++j) step<S, kGlu, kOut == Fp8bOut::kFp32>(c, k, ad, at, acc, f);
  int n;
  if constexpr (kOut == Fp8bOut::kGlu)
    n = store_glu<S>(c, acc, t, sub0, tn);
  else if constexpr (kOut == Fp8bOut::kGluGrad)
    n = store_grad<S>(c, acc, t, sub0, tn);
  else
    n = store_sums<S, kOut == Fp8bOut::kFp32>(c, acc, t, sub0, tn);
  stored(at, n);
}

template <Fp8bOut kOut>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2))) void tiled_kernel(Launch launch) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int tid = threadIdx.x;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1;
  Ctx c{(uint32_t)(uintptr_t)(lds_u8*)lds, wave, launch.L.J, 4u * (uint32_t)launch.a.X, opaque(16u * (uint32_t)(tid & 63))};
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
    locate(walk, g->panels);
    look_up(g, walk);
    fetch_rows(c, walk);
    wait_vmcnt<0>();
    enter(c, k, walk);
    store_walk(c, walk);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
  // two stages ahead, into the places 0, 1 and 2, 3 of the weight halves
#pragma unroll
  for (int p = 0; p < 2; ++p) {
#pragma unroll
    for (int u = 0; u < kLoads; ++u) issue(c, k, p, half_at(c, 2 * p), half_at(c, 2 * p + 1), u);
    advance(c, k);
  }
  wait_and_meet<kLoads + 2>();  // stage 0 but for its second half
  Place at{0, 0, 4, 0, 0};
  for (int i = 0; i < mine; ++i) {
    // as the cursor noted it
    const v4u info = lds_v4(c.lds + kInfo + 128 * wave + 16 * (i & 7));
    const Tile t{(int)wave_u32(info.x), (int)wave_u32(info.y)};
    const int tn = (int)wave_u32(info.z);
    const int sub0 = first_sub(t.n, wm), live = sub_tiles(t.n, wm);
    if (live == 0) {
      run_item<0, kOut>(c, k, at, t, sub0, tn);
    } else if (live == 1) {
      run_item<1, kOut>(c, k, at, t, sub0, tn);
    } else if (kOut == Fp8bOut::kFp32 || live == 2) {
      run_item<2, kOut>(c, k, at, t, sub0, tn);
    } else if constexpr (kOut != Fp8bOut::kFp32) {
      if (live == 3)
        run_item<3, kOut>(c, k, at, t, sub0, tn);
      else
        run_item<4, kOut>(c, k, at, t, sub0, tn);
    }
  }
  wait_vmcnt<0>();  // the dummy stages land before the LDS is given back
}

// Row tiles of a product of one group of P rows and ntn columns of items.
int dense_tiles(int P, int ntn, int most) {
  int tiles = 0;
  float best = 0.0f;
  for (int s = most; s > 0; --s) {
    const int t = (P + 64 * s - 1) / (64 * s);
    const float units = item_units(t, ntn, 1.0f / (float)workgroups(), s);
    if (s == most || units < best) best = units, tiles = t;
  }
  return tiles;
}

}  // namespace

size_t fp8b_tiled_ws_bytes(long P, int E) { return rows_at(P, E) + 4 * (size_t)P; }

hipError_t launch_fp8b_tiled(const Fp8bArgs& a, const Fp8bLayout& L, Fp8bOut out, void* ws, hipStream_t st) {
  const int ntn = (L.NT + kBT - 1) / kBT;
  const int most = out == Fp8bOut::kFp32 ? kWideSubs : 4;
  // Where a group is a tile on average its weights are read once whatever the walk, and
  // one panel keeps its rows in L2 (us, one panel and four, three runs in turn: 256
  // experts of 144 rows, K 7168, N 2048, SwiGLU 1548 and 1559, its backward pass 849 and
  // 863, K 2048, N 7168 806 and 816; 64 experts of 96 rows, K 4096, N 1536, SwiGLU 153 and
  // 158, but K 1536, N 4096, 102 and 99); else panels share weights between row tiles
  // (T16384 to 256 experts, skewed, K 2048, N 7168: 2338 and 2165; dense, 4604 rows, K
  // 16384, N 7168, 455 and 437; two, six, seven, eight and fourteen panels 0-5 % slower).
  Launch g{a, L, nullptr, nullptr, 0, 0, a.offsets && a.P <= kBM * (long)L.E ? 1 : 4};
  if (a.offsets) {
    int32_t* list = static_cast<int32_t*>(ws);
    int32_t* xrows = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + rows_at(a.P, L.E));
    hipLaunchKernelGGL(tiles_kernel, dim3(1 + (a.rows ? ((unsigned)a.P + 1023u) / 1024 : 0)), dim3(1024), 0, st, a, L.E,
                       ntn, 1.0f / (float)workgroups(), most, (int)tile_cap(a.P, L.E), list, xrows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    g.ws = list;
    g.xrows = a.rows ? xrows : nullptr;
  } else {
    g.tiles = dense_tiles(a.P, ntn, most);
    g.height = tile_height(a.P, g.tiles);
  }
  const dim3 grid((unsigned)workgroups()), block(64 * kWaves);
  switch (out) {
    case Fp8bOut::kBf16: hipLaunchKernelGGL(tiled_kernel<Fp8bOut::kBf16>, grid, block, 0, st, g); break;
    case Fp8bOut::kFp32: hipLaunchKernelGGL(tiled_kernel<Fp8bOut::kFp32>, grid, block, 0, st, g); break;
    case Fp8bOut::kGlu: hipLaunchKernelGGL(tiled_kernel<Fp8bOut::kGlu>, grid, block, 0, st, g); break;
    default: hipLaunchKernelGGL(tiled_kernel<Fp8bOut::kGluGrad>, grid, block, 0, st, g);
  }
  return hipGetLastError();
}

}  // namespace moe
