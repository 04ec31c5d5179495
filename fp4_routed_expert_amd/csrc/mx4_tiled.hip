// MXFP4 x MXFP4 products for many rows (the operators of mx4_stream.hip, the
// same packed weights): LDS-tiled, bound by the FP4 matrix rate, or by HBM
// where an expert's rows are few.
//
// A work item is 256 rows of one group x 8 weight tiles (256 weight rows).
// Four waves, one per SIMD, in a 2 x 2 grid, each with up to four 32-token
// sub-tiles x four weight tiles: 16 accumulators of 32 x 32 (256 registers).
// v_mfma_scale_f32_32x32x64_f8f6f4 rather than 16x16x128: with one wave per
// SIMD the larger instruction issues at 6.2-6.6 PFLOP/s on random operands,
// the smaller one at 4.4-5.1 (it lasts 16 clocks, too few to issue anything
// else under), and it reads half as many operand registers per flop.
//
// K runs in steps of 128.  A step's 34 KiB (row pieces, weight tiles, both
// sides' scales) go from global memory to LDS by LDS-DMA into a ring of four
// slots, three steps ahead; one barrier per step, in its second half,
// publishes the next step and frees the current one's slot, which is refilled
// at once.  Fragments are read from LDS half a step before their use.  Row r's
// four 16-byte pieces lie at piece p ^ (r / 4 % 4), which spreads the 16 rows
// that one LDS cycle serves over all banks.
//
// The workgroups are persistent: one per CU (its LDS allows no second) walks
// its XCD's contiguous share of the items, and the ring runs on across items,
// so that an item's first steps arrive under the last steps and the stores of
// the one before.  Every wave issues the same ten loads per step, dummy steps
// past the end, so one fixed wait count serves all steps.
#include <atomic>

#include "lds_dma.h"
#include "mx4.h"

namespace moe {
namespace {

constexpr int kBM = 256;                // rows of an item
constexpr int kBT = 8;                  // weight tiles of an item
constexpr int kA = kBM * 64;            // row pieces of a step
constexpr int kW = kBT * 2048;          // weight tiles
constexpr int kSA = kBM * 4;            // four scale bytes per row
constexpr int kSW = kBT * 128;          // 64 lanes x 2 bytes per tile
constexpr int kStage = kA + kW + kSA + kSW;
constexpr int kSlots = 4;
constexpr int kIdx = kSlots * kStage;   // LDS offset of the next item's row indices
constexpr int kLds = kIdx + kBM * 4;
static_assert(kStage % 1024 == 0 && kLds <= 160 * 1024, "LDS");

// One entry per 256 rows (at most) of a group, of equal heights.
struct Tile {
  int e, row0, n;
};

// Rows of each tile of a group of n rows, in whole sub-tiles of 32.
__host__ __device__ __forceinline__ int tile_height(int n, int tiles) {
  return ((n + 31) / 32 + tiles - 1) / tiles * 32;
}

// ws: the number of tiles, then from byte 16 on four words per tile.
__global__ __launch_bounds__(1024) void tiles_kernel(const int32_t* __restrict__ offsets, int E, int P, int cap,
                                                     int32_t* __restrict__ ws) {
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
__device__ __forceinline__ uint32_t lds_u16(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) uint16_t*>((uintptr_t)addr);
}
__device__ __forceinline__ int lds_i32(uint32_t addr) {
  return *reinterpret_cast<const __attribute__((address_space(3))) int*>((uintptr_t)addr);
}

// One MFMA, its accumulator pinned to AGPRs at this point of the program and
// the scheduler fenced, so that every LDS read and DMA stays where the step
// places it.  (The builtin, not asm: the wait states between a vector write
// and an MFMA that reads it are the compiler's then.)
template <int kByte>
__device__ __forceinline__ void mfma(v16f& c, const v4u& a, const v4u& b, uint32_t sa, uint32_t sb) {
  c = mfma_fp4<kByte>(a, b, c, sa, sb);
  asm volatile("" : "+a"(c) : : "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// Where the DMA stands: the next step to load of the item it is in.
struct Cursor {
  const uint8_t* w0;  // the wave's two weight tiles at K-step 0
  const uint8_t* w1;
  const uint8_t* sw;  // and their pair's scales
  uint32_t a[4];      // per lane: byte offset of its piece of rows 64 w + 16 u + l / 4
  uint32_t sa;        // of row 64 w + l's scales
  int p, j;           // item, step
};

struct Frag {
  v4u x[4], w[4];
};

struct Ctx {
  const Mx4Args& a;
  const Mx4Layout& L;
  const int32_t* ws;
  Walk walk;
  int stride;  // of the walk
  uint32_t lds;
  int lane, wave;
};

// LDS-DMA blocks: the LDS address goes to M0 (restored after), the instruction
// offset counts on both sides.  The base is copied by the scalar unit first: a
// scalar register that a vector instruction has written (v_readfirstlane) must
// not be read by a load within five wait states, and the compiler does not look
// into the asm; the copy is also the wait state that M0 needs.
__device__ __forceinline__ void dma_rows(const uint8_t* base, const uint32_t (&off)[4], uint32_t lds) {
  const uint8_t* t;
  uint32_t m;
  asm volatile(
      "s_mov_b32 %1, m0\n\t"
      "s_mov_b32 m0, %7\n\t"
      "s_mov_b64 %0, %6\n\t"
      "global_load_lds_dwordx4 %2, %0\n\t"
      "global_load_lds_dwordx4 %3, %0 offset:1024\n\t"
      "global_load_lds_dwordx4 %4, %0 offset:2048\n\t"
      "global_load_lds_dwordx4 %5, %0 offset:3072\n\t"
      "s_mov_b32 m0, %1"
      : "=&s"(t), "=&s"(m)
      : "v"(off[0]), "v"(off[1]), "v"(off[2]), "v"(off[3]), "s"(base), "s"(lds)
      : "memory");
}
__device__ __forceinline__ void dma_tile(const uint8_t* base, uint32_t off, uint32_t lds) {
  const uint8_t* t;
  uint32_t m;
  asm volatile(
      "s_mov_b32 %1, m0\n\t"
      "s_mov_b32 m0, %4\n\t"
      "s_mov_b64 %0, %3\n\t"
      "global_load_lds_dwordx4 %2, %0\n\t"
      "global_load_lds_dwordx4 %2, %0 offset:1024\n\t"
      "s_mov_b32 m0, %1"
      : "=&s"(t), "=&s"(m)
      : "v"(off), "s"(base), "s"(lds)
      : "memory");
}
__device__ __forceinline__ void dma_dwords(const uint8_t* base, uint32_t off, uint32_t lds) {
  const uint8_t* t;
  uint32_t m;
  asm volatile(
      "s_mov_b32 %1, m0\n\t"
      "s_mov_b32 m0, %4\n\t"
      "s_mov_b64 %0, %3\n\t"
      "global_load_lds_dword %2, %0\n\t"
      "s_mov_b32 m0, %1"
      : "=&s"(t), "=&s"(m)
      : "v"(off), "s"(base), "s"(lds)
      : "memory");
}

// Row index DMA of item p (if there is one) into the index buffer; each wave
// loads and later reads the 64 rows whose pieces it moves.
__device__ __forceinline__ void fetch_rows(const Ctx& c, int p) {
  if (!c.a.rows || p >= c.walk.hi) return;
  int tt, tn;
  walk_item(c.walk, p, tt, tn);
  const Tile t = get_tile(c.a, c.ws, tt, c.walk.ntt);
  const uint32_t local = (uint32_t)min(64 * c.wave + c.lane, t.n - 1);
  dma_dwords(wave_ptr(reinterpret_cast<const uint8_t*>(c.a.rows + t.row0)), 4u * local,
             wave_u32(c.lds + kIdx + 256u * (uint32_t)c.wave));
}

// Points the cursor at item p (whose row indices are in the index buffer).
__device__ __forceinline__ void enter(const Ctx& c, Cursor& k, int p) {
  int tt, tn;
  walk_item(c.walk, p, tt, tn);
  const Tile t = get_tile(c.a, c.ws, tt, c.walk.ntt);
  const Mx4Layout& L = c.L;
  const uint32_t rowb = (uint32_t)L.K / 2, K32 = (uint32_t)L.K / 32;
  // logical piece of the lane: physical piece l % 4 of a row whose r / 4 % 4 is l / 16
  const uint32_t piece = (uint32_t)(((c.lane & 3) ^ (c.lane >> 4)) << 4);
#pragma unroll
  for (int u = 0; u < 5; ++u) {
    const int r = 64 * c.wave + (u < 4 ? 16 * u + (c.lane >> 2) : c.lane);
    const int m = min(r, t.n - 1);  // rows past the tile read its last one
    int x = t.row0 + m;
    if (c.a.rows) x = (int)((uint32_t)lds_i32(c.lds + kIdx + 4 * r) / (uint32_t)c.a.div);
    x = max(min(x, c.a.X - 1), 0);
    if (u < 4)
      k.a[u] = (uint32_t)x * rowb + piece + 3072u - 1024u * (uint32_t)u;
    else
      k.sa = (uint32_t)x * K32;
  }
  const int nt = tn * kBT + 2 * c.wave;
  k.w0 = wave_ptr(c.a.packed + L.tile_off(t.e, min(nt, L.NT - 1)));
  k.w1 = wave_ptr(c.a.packed + L.tile_off(t.e, min(nt + 1, L.NT - 1)));
  k.sw = wave_ptr(c.a.packed + L.scale_off(t.e, min(nt, L.NT - 1) >> 1));
  k.p = p;
  k.j = 0;
}

// Block u (< 4) of the wave's share of the cursor's step into the slot at S:
// its row pieces (4 loads), its weight tiles (2 and 2), both scales.
constexpr int kBlocks = 4;
__device__ __forceinline__ void issue1(const Ctx& c, const Cursor& k, uint32_t S, int j, int u) {
  if (u == 0) {
    // the rows' offsets have 1024 u taken off (and 3072 put on)
    dma_rows(wave_ptr(c.a.xq + (size_t)j * 64 - 3072), k.a, S + 4096u * (uint32_t)c.wave);
  } else if (u < 3) {
    dma_tile(wave_ptr((u == 1 ? k.w0 : k.w1) + (size_t)j * 2048), 16u * (uint32_t)c.lane,
             S + (uint32_t)kA + 4096u * (uint32_t)c.wave + 2048u * (uint32_t)(u - 1));
  } else {
    dma_dwords(wave_ptr(c.a.xs + (size_t)j * 4), k.sa, S + (uint32_t)(kA + kW) + 256u * (uint32_t)c.wave);
    dma_dwords(wave_ptr(k.sw + (size_t)j * 256), 4u * (uint32_t)c.lane,
               S + (uint32_t)(kA + kW + kSA) + 256u * (uint32_t)c.wave);
  }
}

// After a step's loads: the next step, or the next item's first (past the
// last item its steps are loaded again and never used).
__device__ __forceinline__ void advance(const Ctx& c, Cursor& k) {
  if (++k.j < c.L.J) return;
  const int p = k.p + c.stride;
  if (p >= c.walk.hi) {
    k.j = 0;
    return;
  }
  // the indices were loaded when the cursor entered this item; with more steps
  // than the prologue's four the per-step waits have covered them
  if (c.a.rows && c.L.J <= kSlots) wait_vmcnt<0>();
  enter(c, k, p);
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the indices are read before they are replaced
  fetch_rows(c, p + c.stride);
}

struct Addr {  // per lane, relative to a slot
  uint32_t a0, a1;  // row r of the wave's first sub-tile, pieces of K-halves 0 and 1 (sub-tile i at + 2048 i)
  uint32_t sa;      // its scale pair (+ 128 i)
  uint32_t w;       // weight tile 4 wn (+ 2048 t, K-half 1 at + 1024)
  uint32_t sw;      // its scale pair (+ 128 t)
};

// One K-step of a wave with S live sub-tiles.  On entry f0 and the scales hold
// K-half 0's fragments of this step; on exit those of the next one.
template <int S>
__device__ __forceinline__ void step(const Ctx& c, Cursor& k, const Addr& ad, int slot, v16f (&acc)[4][4], Frag& f0,
                                     Frag& f1, uint32_t (&sx)[4], uint32_t (&sw)[4]) {
  const uint32_t cur = wave_u32(c.lds + (uint32_t)(slot * kStage));
  const uint32_t nxt = wave_u32(c.lds + (uint32_t)(((slot + 1) & 3) * kStage));
  constexpr int M = 4 * S;       // MFMAs of a half
  constexpr int R = S + 4;       // fragments of a half
  if constexpr (S > 0) {
    // first half: K-half 1's fragments arrive under K-half 0's MFMAs
    const uint32_t xa = cur + ad.a1, wa = cur + ad.w + 1024;
#pragma unroll
    for (int m = 0; m < M; ++m) {
      mfma<0>(acc[m >> 2][m & 3], f0.x[m >> 2], f0.w[m & 3], sx[m >> 2], sw[m & 3]);
#pragma unroll
      for (int q = 0; q < R; ++q)
        if (q * M / (2 * R) == m) {
          if (q < 4)
            f1.w[q] = lds_v4(wa + 2048 * q);
          else
            f1.x[q - 4] = lds_v4(xa + 2048 * (q - 4));
        }
    }
  }
  uint32_t nsx[4], nsw[4];
  const int kj = __builtin_amdgcn_readfirstlane(k.j);
  const uint32_t xa = nxt + ad.a0, wa = nxt + ad.w, sxa = nxt + ad.sa, swa = nxt + ad.sw;
  // what follows the barrier: the next step's K-half 0 and this slot's refill
  constexpr int kFirst = 2;                                // MFMAs in the pipe across the barrier
  constexpr int kLeft = S > 0 ? M - kFirst : 1;            // MFMAs after it
  auto after = [&](int m) {
    // m-th of kLeft places: its share of the fragments (in the first half of
    // the places) and of the ten loads
#pragma unroll
    for (int q = 0; q < R; ++q)
      if (S > 0 && q * kLeft / (2 * R) == m) {
        if (q < 4) {
          f0.w[q] = lds_v4(wa + 2048 * q);
          nsw[q] = lds_u16(swa + 128 * q);
        } else {
          f0.x[q - 4] = lds_v4(xa + 2048 * (q - 4));
          nsx[q - 4] = lds_u16(sxa + 128 * (q - 4));
        }
      }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u)
      if (u * kLeft / kBlocks == m) issue1(c, k, cur, kj, u);
  };
  auto publish = [&] {
    // this wave's loads of the next step have landed (20 newer ones may be in
    // flight) and its reads of this step are done; then everyone's
    asm volatile("s_waitcnt vmcnt(20) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  };
  if constexpr (S > 0) {
#pragma unroll
    for (int m = 0; m < M; ++m) {
      mfma<1>(acc[m >> 2][m & 3], f1.x[m >> 2], f1.w[m & 3], sx[m >> 2], sw[m & 3]);
      if (m == kFirst - 1) publish();
      if (m >= kFirst - 1 && m < M - 1) after(m - (kFirst - 1));
    }
#pragma unroll
    for (int i = 0; i < S; ++i) sx[i] = nsx[i];
#pragma unroll
    for (int t = 0; t < 4; ++t) sw[t] = nsw[t];
  } else {
    publish();
    after(0);
  }
  advance(c, k);
}

// Stores of a wave's S sub-tiles: element v of a lane is row 8 (v / 4) + 4 g +
// v % 4 of its sub-tile; the group's f tiles are f neighbouring columns, so a
// half-wave's store covers a whole run of 128 (64 with SwiGLU) outputs.
template <bool kGlu, bool kF32>
__device__ __forceinline__ void store_row(const Ctx& c, const float (&v)[4], size_t row, int group, int f, int n) {
  constexpr int kO = kGlu ? 2 : 4;
  float o[kO];
#pragma unroll
  for (int t = 0; t < kO; ++t) o[t] = kGlu ? silu_mul(v[2 * t], v[2 * t + 1]) : v[t];
  const size_t at = row * c.L.N + 32 * kO * group + f * n;
  if constexpr (kF32) {
    float* y = static_cast<float*>(c.a.y) + at;
    if (f == kO) {
      if constexpr (kGlu)
        *reinterpret_cast<v2f*>(y) = v2f{o[0], o[1]};
      else
        *reinterpret_cast<v4f*>(y) = v4f{o[0], o[1], o[2], o[3]};
    } else {
#pragma unroll
      for (int t = 0; t < kO - 1; ++t)
        if (t < f) y[t] = o[t];
    }
  } else {
    uint16_t* y = static_cast<uint16_t*>(c.a.y) + at;
    if (f == kO) {
      if constexpr (kGlu)
        *reinterpret_cast<uint32_t*>(y) = f32x2_to_bf16(o[0], o[1]);
      else
        *reinterpret_cast<uint2*>(y) = make_uint2(f32x2_to_bf16(o[0], o[1]), f32x2_to_bf16(o[2], o[3]));
    } else {
#pragma unroll
      for (int t = 0; t < kO - 1; ++t)
        if (t < f) y[t] = f32_to_bf16(o[t]);
    }
  }
}

template <int S, bool kGlu, bool kF32>
__device__ __forceinline__ void run_item(const Ctx& c, Cursor& k, const Addr& ad, int& slot, const Tile& t, int sub0,
                                         int group) {
  v16f acc[4][4];
  Frag f0, f1;
  uint32_t sx[4], sw[4];
  if constexpr (S > 0) {
#pragma unroll
    for (int i = 0; i < S; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
#pragma unroll
        for (int v = 0; v < 16; ++v) acc[i][q][v] = 0.0f;
      }
    const uint32_t s = c.lds + (uint32_t)(slot * kStage);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      f0.w[q] = lds_v4(s + ad.w + 2048 * q);
      sw[q] = lds_u16(s + ad.sw + 128 * q);
    }
#pragma unroll
    for (int i = 0; i < S; ++i) {
      f0.x[i] = lds_v4(s + ad.a0 + 2048 * i);
      sx[i] = lds_u16(s + ad.sa + 128 * i);
    }
  }
  for (int j = 0; j < c.L.J; ++j) {
    step<S>(c, k, ad, slot, acc, f0, f1, sx, sw);
    slot = (slot + 1) & 3;
  }
  if constexpr (S > 0) {
    const int n = c.lane & 31, g = c.lane >> 5;
    constexpr int kO = kGlu ? 2 : 4;
    const int left = c.L.N / 32 - kO * group, f = left < kO ? left : kO;
    if (f > 0) {
#pragma unroll
      for (int i = 0; i < S; ++i)
#pragma unroll
        for (int v = 0; v < 16; ++v) {
          const int m = 32 * (sub0 + i) + 8 * (v >> 2) + 4 * g + (v & 3);
          const float o[4] = {acc[i][0][v], acc[i][1][v], acc[i][2][v], acc[i][3][v]};
          if (m < t.n) store_row<kGlu, kF32>(c, o, (size_t)t.row0 + m, group, f, n);
          __builtin_amdgcn_sched_barrier(0);  // one row at a time out of the accumulators
        }
    }
  }
}

template <bool kGlu, bool kF32>
__global__ __launch_bounds__(256) __attribute__((amdgpu_waves_per_eu(1, 1))) void tiled_kernel(
    Mx4Args a, Mx4Layout L, const int32_t* ws, int dense_tiles) {
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 1, wn = wave & 1;
  Ctx c{a, L, ws, {}, (int)(gridDim.x >> 3), (uint32_t)(uintptr_t)(lds_u8*)lds, lane, wave};
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
  for (int s = 0; s < kSlots; ++s) {
    const uint32_t S = wave_u32(c.lds + (uint32_t)(s * kStage));
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) issue1(c, k, S, __builtin_amdgcn_readfirstlane(k.j), u);
    advance(c, k);
  }
  asm volatile("s_waitcnt vmcnt(30)\n\ts_barrier" ::: "memory");  // step 0 is there

  Addr ad;
  const int r = lane & 31, g = lane >> 5;
  const uint32_t sz = (uint32_t)((r >> 2) & 3);
  ad.w = opaque((uint32_t)(kA + 8192 * wn + 16 * lane));
  ad.sw = opaque((uint32_t)(kA + kW + kSA + 512 * wn + 2 * lane));
  int slot = 0;
  for (int p = first; p < c.walk.hi; p += c.stride) {
    int tt, tn;
    walk_item(c.walk, p, tt, tn);
    const Tile t = get_tile(a, ws, tt, c.walk.ntt);
    // the live sub-tiles in halves: the first wave row takes the odd one
    const int n32 = (t.n + 31) / 32, h0 = (n32 + 1) / 2;
    const int sub0 = wm == 0 ? 0 : h0, live = wm == 0 ? h0 : n32 - h0;
    const uint32_t row = (uint32_t)(32 * sub0 + r);
    ad.a0 = opaque(row * 64 + (((uint32_t)(2 * g) ^ sz) << 4));
    ad.a1 = opaque(row * 64 + (((uint32_t)(2 * g + 1) ^ sz) << 4));
    ad.sa = opaque((uint32_t)(kA + kW) + row * 4 + 2 * g);
    const int group = tn * 2 + wn;
    switch (live) {
      case 0: run_item<0, kGlu, kF32>(c, k, ad, slot, t, sub0, group); break;
      case 1: run_item<1, kGlu, kF32>(c, k, ad, slot, t, sub0, group); break;
      case 2: run_item<2, kGlu, kF32>(c, k, ad, slot, t, sub0, group); break;
      case 3: run_item<3, kGlu, kF32>(c, k, ad, slot, t, sub0, group); break;
      default: run_item<4, kGlu, kF32>(c, k, ad, slot, t, sub0, group); break;
    }
  }
  wait_vmcnt<0>();  // the dummy steps land before the LDS is given back
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

long tile_cap(long P, int E) { return P / kBM + (P < E ? P : E); }

}  // namespace

size_t mx4_tiled_ws_bytes(long P, int E) { return 16 + 16 * (size_t)tile_cap(P, E); }

hipError_t launch_mx4_tiled(const Mx4Args& a, const Mx4Layout& L, bool fp32_out, void* ws, hipStream_t st) {
  int32_t* list = static_cast<int32_t*>(ws);
  if (a.offsets) {
    hipLaunchKernelGGL(tiles_kernel, dim3(1), dim3(1024), 0, st, a.offsets, L.E, a.P, (int)tile_cap(a.P, L.E), list);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  const int dense_tiles = (a.P + kBM - 1) / kBM;
  const dim3 grid((unsigned)workgroups()), block(256);
  if (L.glu) {
    if (fp32_out)
      hipLaunchKernelGGL((tiled_kernel<true, true>), grid, block, 0, st, a, L, list, dense_tiles);
    else
      hipLaunchKernelGGL((tiled_kernel<true, false>), grid, block, 0, st, a, L, list, dense_tiles);
  } else {
    if (fp32_out)
      hipLaunchKernelGGL((tiled_kernel<false, true>), grid, block, 0, st, a, L, list, dense_tiles);
    else
      hipLaunchKernelGGL((tiled_kernel<false, false>), grid, block, 0, st, a, L, list, dense_tiles);
  }
  return hipGetLastError();
}

}  // namespace moe
