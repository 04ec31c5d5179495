// What the LDS-tiled products of mx4_tiled.hip and fp8b_tiled.hip share: the
// walk of persistent workgroups over their items, LDS and LDS-DMA access.
#pragma once

#include <atomic>

#include "lds_dma.h"
#include "mx4.h"

namespace moe {

typedef __attribute__((address_space(4))) const int32_t cint;  // read by scalar loads

// Global (not flat) pointers: flat stores would count as LDS traffic too.
template <class T>
using global = __attribute__((address_space(1))) T;
typedef global<uint8_t> gbyte;
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

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

// LDS-DMA of a dword for each lane from an address of its own.
__device__ __forceinline__ void dma4_lanes(const uint8_t* p, uint32_t lds) {
  asm volatile(
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dword %0, off"
      :
      : "v"(p), "s"(wave_u32(lds))
      : "memory");
}

// Where a wave's walk over the items stands (in LDS between items).  The items
// go by panels of columns (a quarter of them), row tiles running inside a panel,
// so that the items that an XCD holds at one time share rows and weights in
// its L2.  Steps inside a panel need no division.
struct Walk {
  int p, hi, stride;  // item, end of this XCD's share, items from one to the next
  int ntt, ntn;       // row tiles, columns of items
  int tt, off;        // row tile, column inside the panel
  int base, w;        // the panel's first column and its width
  int st, so;         // stride / w, stride % w
  int e, row0, n;     // the item's tile of rows
  int count, more;    // items before it; whether there is one
};
static_assert(sizeof(Walk) == 64, "four 128-bit words");

__device__ __forceinline__ void locate(Walk& k, int panels = 4) {
  const int sn = (k.ntn + panels - 1) / panels, sc = k.p / (k.ntt * sn), q = k.p - sc * (k.ntt * sn);
  k.base = sc * sn;
  k.w = max(min(sn, k.ntn - k.base), 1);
  k.tt = q / k.w;
  k.off = q - k.tt * k.w;
  k.st = k.stride / k.w;
  k.so = k.stride - k.st * k.w;
}
// The walk in LDS: a wave's own 64 bytes.
typedef __attribute__((address_space(3))) v4u lds_words;
__device__ __forceinline__ Walk read_walk(uint32_t lds) {
  const lds_words* p = reinterpret_cast<const lds_words*>((uintptr_t)lds);
  v4u w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = p[i];
  Walk k;
  int* f = reinterpret_cast<int*>(&k);
#pragma unroll
  for (int i = 0; i < 16; ++i) f[i] = (int)wave_u32(w[i >> 2][i & 3]);
  return k;
}
__device__ __forceinline__ void write_walk(uint32_t lds, const Walk& k) {
  lds_words* p = reinterpret_cast<lds_words*>((uintptr_t)lds);
  const int* f = reinterpret_cast<const int*>(&k);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    p[i] = v4u{(uint32_t)f[4 * i], (uint32_t)f[4 * i + 1], (uint32_t)f[4 * i + 2], (uint32_t)f[4 * i + 3]};
}

// CUs of the current device, a multiple of eight (one share per XCD).
inline int workgroups() {
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

}  // namespace moe
