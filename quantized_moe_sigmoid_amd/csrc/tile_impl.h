// tile_impl.h — what the LDS-tiled products share (mxfp4_tile.hip, int8_tile.hip): loads straight
// into LDS that the kernel counts itself, the order of tiles over the XCDs, the row tiles of a route.
#pragma once

#include "mxfp4_impl.h"

namespace coli {

// Loads of 64 lanes straight into LDS: 16 (4) bytes from each lane's address base + off to
// consecutive LDS bytes at the wave-uniform address lds; the pair: two, 4096 LDS bytes apart
// (the instruction's offset moves both addresses, so o0 is 4096 high). Lanes outside hi : lo
// load nothing, and a load without lanes is counted like the others. Written as asm because
// the compiler would wait for every such load before the next LDS read; the kernel counts them
// itself. No register is loaded; M0 and the active lanes are put back.
__device__ __forceinline__ uint64_t lanes_of(int lo, int hi) {  // in scalar registers
  return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(hi) << 32 | (uint32_t)__builtin_amdgcn_readfirstlane(lo);
}
__device__ __forceinline__ void dma16_pair(const uint8_t *base, uint32_t o0, uint32_t o1, uint32_t lds, int lo, int hi) {
  uint64_t active;
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %1, m0\n\ts_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\t"
      "global_load_lds_dwordx4 %4, %6 offset:-4096\n\tglobal_load_lds_dwordx4 %5, %6\n\t"
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %0"
      : "=&s"(active), "=&s"(m0)
      : "s"(lds + 4096), "s"(lanes_of(lo, hi)), "v"(o0), "v"(o1), "s"(base)
      : "memory", "scc");
}
// The same, for what no other workgroup will read: past the caches
__device__ __forceinline__ void dma16_pair_once(const uint8_t *base, uint32_t o0, uint32_t o1, uint32_t lds, int lo, int hi) {
  uint64_t active;
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %1, m0\n\ts_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\t"
      "global_load_lds_dwordx4 %4, %6 offset:-4096 nt\n\tglobal_load_lds_dwordx4 %5, %6 nt\n\t"
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %0"
      : "=&s"(active), "=&s"(m0)
      : "s"(lds + 4096), "s"(lanes_of(lo, hi)), "v"(o0), "v"(o1), "s"(base)
      : "memory", "scc");
}
__device__ __forceinline__ void dma16(const uint8_t *base, uint32_t off, uint32_t lds, int lo, int hi) {
  uint64_t active;
  uint32_t m0;
  asm volatile(
      "s_mov_b32 %1, m0\n\ts_mov_b32 m0, %2\n\ts_and_saveexec_b64 %0, %3\n\tglobal_load_lds_dwordx4 %4, %5\n\t"
      "s_mov_b32 m0, %1\n\ts_mov_b64 exec, %0"
      : "=&s"(active), "=&s"(m0)
      : "s"(lds), "s"(lanes_of(lo, hi)), "v"(off), "s"(base)
      : "memory", "scc");
}

// A pointer that is the same in all lanes, in scalar registers
__device__ __forceinline__ const uint8_t *uniform(const uint8_t *p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)u), hi = __builtin_amdgcn_readfirstlane((uint32_t)(u >> 32));
  return reinterpret_cast<const uint8_t *>((uint64_t)hi << 32 | lo);
}

template <int N>
__device__ __forceinline__ void wait_loads() {  // all but the last N loads of this wavefront have arrived
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

typedef uint32_t v2u32 __attribute__((ext_vector_type(2)));
typedef uint32_t v4u32 __attribute__((ext_vector_type(4)));

// Slot of chunk (block) c of an LDS row of eight is c ^ swizzle: the rows that one LDS access
// reads at the same chunk fall on different banks.
__device__ __forceinline__ int tile_swizzle(int row) { return (row & 7) ^ ((row >> 3) & 1); }

// Workgroup id -> tile (x of nx, y of ny) of a dense product. Consecutive ids go to different
// XCDs (id % 8); each XCD gets a run of tiles in strips of TILE_STRIP columns, so that the
// tiles it works on at a time share rows and columns in its L2.
constexpr int TILE_STRIP = 4;
__device__ __forceinline__ void tile_of(int id, int nx, int ny, int &x, int &y) {
  const int n = nx * ny, xcd = id & 7, q = n >> 3, r = n & 7;
  const int t = xcd * q + min(xcd, r) + (id >> 3);
  const int strip = t / (TILE_STRIP * ny), in = t - strip * TILE_STRIP * ny;
  const int w = min(TILE_STRIP, nx - strip * TILE_STRIP);
  y = in / w;
  x = strip * TILE_STRIP + in - y * w;
}

// AUX 2: 16-byte pieces pass the caches by
template <int AUX = 0, typename W>
__device__ __forceinline__ void store_out(W w, __amdgpu_buffer_rsrc_t out, uint32_t off) {
  if constexpr (sizeof(W) == 16)
    __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u32, w), out, off, 0, AUX);
  else if constexpr (sizeof(W) == 4)
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(uint32_t, w), out, off, 0, 0);
  else
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, w), out, off, 0, 0);
}

// Row tiles of an expert that go through a column strip together, so that its weights come from
// the fabric once (4.23 -> 3.95 GB for gate/up of 2048 tokens); 2 and 8: 833 and 825 us
constexpr int EXP_GROUP = 8;

// Tile c of an expert's `all`: its w entry, routed | place in its group << 8 | size of the group << 16
__device__ __forceinline__ int tile_place(int c, int all, int routed) {
  const int i = c % EXP_GROUP;
  return routed | i << 8 | min(EXP_GROUP, all - (c - i)) << 16;
}

// Args: the grouping of a launch, with tiles and ntiles to write.
// Tiles of a route: {expert, first (of perm, or token), rows, place}, the shared expert's first.
template <typename Args>
__global__ __launch_bounds__(1024) void route_tiles_kernel(Args a, int bm, int cap) {
  __shared__ int wsum[16];
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int na = hit_experts(a.nact, a.off, a.E);
  const int shared = a.has_shared ? (a.M + bm - 1) / bm : 0;
  int e = 0, first = 0, n = 0;
  if (tid < na) {
    e = a.active[tid];
    first = a.off[e];
    n = a.off[e + 1] - first;
  }
  const int mine = (n + bm - 1) / bm;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(incl, o);
    if (lane >= o) incl += t;
  }
  if (lane == 63) wsum[wv] = incl;
  __syncthreads();
  int base = shared, total = shared;
  for (int i = 0; i < 16; i++) {
    if (i < wv) base += wsum[i];
    total += wsum[i];
  }
  for (int c = tid; c < shared && c < cap; c += 1024)
    a.tiles[c] = make_int4(a.E, c * bm, min(bm, a.M - c * bm), tile_place(c, shared, 0));
  int g = base + incl - mine;
  for (int c = 0; c < mine; c++, g++)
    if (g < cap) a.tiles[g] = make_int4(e, first + c * bm, min(bm, n - c * bm), tile_place(c, mine, 1));
  if (tid == 0) *a.ntiles = min(total, cap);
}

}  // namespace coli
