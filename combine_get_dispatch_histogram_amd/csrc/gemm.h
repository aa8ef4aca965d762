// gemm.h -- device building blocks of the grouped matrix products on gfx950:
// asynchronous global -> LDS tiles, MFMA operand reads, and the walk from a
// tile number to its group of rows.
//
// Both operands of a product are named by their place in the MFMA: P gives
// the rows of the 16 x 16 result (four consecutive ones to a lane), Q its
// columns (one to a lane).  The result of a rows kernel is out[q][p]: with the
// weights as P and the tokens as Q a lane holds consecutive output channels of
// one token, so results go to memory as row-contiguous vectors without a trip
// through LDS, and a token's scale is one value a lane.
#pragma once

#include "device.h"
#include "kernels.h"

namespace miep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) uint8_t lds_byte;

// The kernels' lambdas: one that is called instead of inlined keeps what it
// captures in scratch memory.
#define MIEP_INLINE __attribute__((always_inline))

// A tile's K extent is 128 bytes a row in every type (64 bf16, 128 E4M3).
constexpr int kStepBytes = 128;

// Sixteen zero bytes in device memory: the source of every element of a tile
// that lies past the contraction's end (0 * NaN would not be 0, so both
// operands read zeros there).
__device__ __attribute__((aligned(16))) const uint32_t g_zero16[4] = {0u, 0u, 0u, 0u};

// One wavefront's 1 KiB of a tile: lane i's 16 bytes go to lds + 16 * i.  The
// loads carry no register results; the kernel waits for them by count
// (wait_tiles) before the barrier that publishes the tile.
__device__ __forceinline__ void dma16(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(src) : "memory");
}
// The same from a scalar base and a 32-bit lane offset.  (A scalar register that
// a vector instruction wrote, as when a spilled one comes back, may be a vector
// load's base after five wait states: the pause and the move before it.)
__device__ __forceinline__ void dma16s(const void* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 3\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(lds), "v"(off), "s"(base) : "memory");
}
// 4 bytes a lane to lds + 4 * i.
__device__ __forceinline__ void dma4(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(lds), "v"(src) : "memory");
}

// One byte a lane, zero-extended to the dword at lds + 4 * i.
__device__ __forceinline__ void dma1(const void* src, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_ubyte %1, off" ::"s"(lds), "v"(src) : "memory");
}

// A transposed tile has 64 contraction rows of BP channels.  A transposing
// read takes 32 bytes of each of 4 rows a 16-lane group: rows 0-3, 8-11 (then
// 4-7, 12-15) by half wavefront; f spreads those 8 rows over the line.
__device__ __forceinline__ int swz_t(int row) { return ((row & 3) | ((row >> 1) & 4)) << 1; }

// One store of 16 bytes a lane, whatever surrounds it: for results that a later
// wait counts.  (A vector write to the data registers of a store of more than 8
// bytes may follow it after two wait states; the compiler, which sees to that
// elsewhere, does not look into the statement.)
__device__ __forceinline__ void store16(void* p, const v4u& v) {
  const u32x4 t = {v.x, v.y, v.z, v.w};
  asm volatile("global_store_dwordx4 %0, %1, off\n\ts_nop 1" ::"v"(p), "v"(t) : "memory");
}

// Waits until at most N vector memory operations of this wavefront are in
// flight and its LDS reads have returned, then for the workgroup: tiles whose
// loads every wavefront has waited for may be read, and tiles that every
// wavefront has read may be overwritten.
template <int N>
__device__ __forceinline__ void wait_tiles() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <class T>
__device__ __forceinline__ T lds_read(uint32_t at) {
  return *reinterpret_cast<const __attribute__((address_space(3))) T*>(at);
}
template <class T>
__device__ __forceinline__ void lds_write(uint32_t at, const T& v) {
  *reinterpret_cast<__attribute__((address_space(3))) T*>(at) = v;
}
__device__ __forceinline__ i16x4 lds_read_tr(uint32_t at) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<__attribute__((address_space(3))) i16x4*>(at));
}

// Two 16 x 16 results of neighbouring P tiles (four consecutive p to a lane,
// four lanes 16 apart to a tile's 16) as 8 consecutive p to a lane: lanes of
// the even quarters take the first tile's p from 4 * quarter on, those of the
// odd ones the second's from 4 * (quarter - 1) on, so that a store of 16 bytes
// a lane writes 64 whole bytes of each of 16 rows.
__device__ __forceinline__ v4u pack_pair(const f32x4& a, const f32x4& b) {
  const auto x = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[0], a[1]), pack_bf16x2(b[0], b[1]), false, false);
  const auto y = __builtin_amdgcn_permlane16_swap(pack_bf16x2(a[2], a[3]), pack_bf16x2(b[2], b[3]), false, false);
  return v4u{static_cast<uint32_t>(x[0]), static_cast<uint32_t>(y[0]), static_cast<uint32_t>(x[1]), static_cast<uint32_t>(y[1])};
}

// Waits until every wavefront's LDS reads have returned.
__device__ __forceinline__ void all_read() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// What the matrix instructions' sums keep.  bf16: products and sums in fp32.
// E4M3 (with or without scales; 16x16x32's are no better than 16x16x128's): the
// products of 8 consecutive channels are first cut, toward zero, to multiples of
// 2^(e - 13), e the largest sum of two exponents among those products that are
// not zero, then added exactly; the groups of 8 and the running sum are fp32.
// A group so loses less than 7 * 2^(e - 13), and a product 2^13 times smaller
// than a neighbour may vanish beside it.  On the whole: 1.5e-5 (rms) of
// a sum of 128 products of normal numbers, a hundredth of the result's bf16
// rounding.  Full fp32 sums would need bf16 MFMAs of converted codes, at half the
// rate: the cut is taken for the rate.

// Keeps the arithmetic that makes v where it is written: left alone, the
// compiler moves the multiplications by FP8 scales behind a step's branches
// and holds every MFMA's result until then.
__device__ __forceinline__ void pin(f32x4& v) { asm volatile("" : "+v"(v)); }

// ---- the groups' rows, never trusted: a group reads as the part of
// [begin, begin + rows) inside [0, limit).
__device__ __forceinline__ void group_range(const GroupArgs& g, int i, int64_t* begin, int* rows) {
  const int64_t b = g.begin ? g.begin[i] : static_cast<int64_t>(i) * g.stride;
  int64_t n = g.rows[i];
  if (!g.begin && n > g.stride) n = g.stride;
  if (b < 0 || b >= g.limit) n = 0;
  else if (n > g.limit - b) n = g.limit - b;
  *begin = b;
  *rows = n > 0 ? static_cast<int>(n) : 0;
}

struct TileAt {
  int group;       // -1: past the last tile
  int first;       // the tile's place among the group's tiles
  int64_t begin;
  int rows;
};

__device__ __forceinline__ int row_tiles(int n, int bq) { return (n + bq - 1) / bq; }

// Tile t of the sequence in which group i has row_tiles(rows, bq) * per tiles.
// Every wavefront walks for itself: one load a lane for each 64 groups and a
// scan of the lane counts.
__device__ __forceinline__ TileAt find_tile(const GroupArgs& g, int bq, int per, int t) {
  const int lane = lane_id();
  int before = 0;
  TileAt r;
  r.group = -1;
  r.first = 0;
  r.begin = 0;
  r.rows = 0;
  for (int g0 = 0; g0 < g.G; g0 += kWave) {
    int64_t b = 0;
    int n = 0;
    if (g0 + lane < g.G) group_range(g, g0 + lane, &b, &n);
    const int tiles = row_tiles(n, bq) * per;
    const int inc = wave_inclusive_scan(tiles);
    const uint64_t past = ballot(before + inc > t && tiles > 0);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      r.group = g0 + l;
      r.first = t - before - (readlane(inc, l) - readlane(tiles, l));
      r.rows = readlane(n, l);
      r.begin = (static_cast<int64_t>(readlane(static_cast<int>(b >> 32), l)) << 32) |
                static_cast<uint32_t>(readlane(static_cast<int>(b), l));
      return r;
    }
    before += readlane(inc, 63);
  }
  return r;
}

// How many they are.  Groups that overlap may have more than the layout's rows
// make; past kMostTiles, where a walk's own steps would overflow, they are not
// counted.
__device__ __forceinline__ int count_tiles(const GroupArgs& g, int bq, int per) {
  const int lane = lane_id();
  int64_t total = 0;
  for (int g0 = 0; g0 < g.G; g0 += kWave) {
    int64_t b = 0;
    int n = 0;
    if (g0 + lane < g.G) group_range(g, g0 + lane, &b, &n);
    const int sum = readlane(wave_inclusive_scan(row_tiles(n, bq) * per), 63);
    total += sum < 0 ? kMostTiles : sum;
  }
  return static_cast<int>(total < kMostTiles ? total : kMostTiles);
}

}  // namespace miep
