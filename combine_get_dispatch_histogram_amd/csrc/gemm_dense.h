// gemm_dense.h -- dense products: one weight for all rows, sizes known to the host.
#pragma once

#include "gemm_rows.h"

namespace miep {

// The rows kernel's product for few tiles: a workgroup computes 64 x 64, each of
// its 8 wavefronts all of it over every eighth step of the contraction, through
// a buffer of its own, so without barriers; their sums are added up in
// wavefront order in LDS.  A wavefront that has read one operand of a step into
// registers starts the next step's loads of it, and multiplies under them (both
// operands together: 4096 x 256 x 7168 24.1 us, so 23.4).  Against
// tiles whose wavefronts share each step, an operand leaves LDS once instead of
// up to four times, which is what bounds a 64 x 64 tile.
struct DenseSplit {
  static constexpr int kWaves = 8, kSide = 64, kTiles = kSide / 16;
  static constexpr int kBytes = kSide * kStepBytes;                   // of one operand's step
  static constexpr int kLoads = kBytes / 1024;
  static constexpr int kLds = kWaves * 2 * kBytes;
};

// Transposed P: 64 contraction rows of 64 channels, 128 bytes each; the four even
// (or odd) rows of a half wavefront's transposing read lie in different quarters.
__device__ __forceinline__ int swz_t64(int row) { return (row & 2) | ((row >> 1) & 4); }

template <bool PT, int EPI>
__global__ __launch_bounds__(512, 2) void gemm_dense_split_kernel(GemmRowsArgs a) {
  using S = DenseSplit;
  constexpr int T = S::kTiles;
  __shared__ __align__(1024) uint8_t lds_mem[S::kLds];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const uint32_t mine = (uint32_t)(uintptr_t)(lds_byte*)lds_mem + wave * 2 * S::kBytes;

  const int NO = a.NO, C = a.C, nk = (C + 63) / 64;
  const int64_t rows = a.g.limit, ldq = static_cast<int64_t>(C) * 2, ldp = static_cast<int64_t>(PT ? NO : C) * 2;
  // XCD x computes the x-th eighth of the tiles, in bands of 8 row tiles, so that
  // tiles that share rows or weights meet in one L2
  const int ntiles = (NO + 63) / 64, mtiles = static_cast<int>((rows + 63) / 64);
  const int64_t total = static_cast<int64_t>(ntiles) * mtiles;
  const int xcd = blockIdx.x & 7;
  const int64_t t = total * xcd / 8 + (blockIdx.x >> 3);
  if (t >= total * (xcd + 1) / 8) return;
  constexpr int kBand = 8;
  const int band = static_cast<int>(t / (kBand * ntiles)), in_band = static_cast<int>(t - static_cast<int64_t>(band) * kBand * ntiles);
  const int bh = min(kBand, mtiles - band * kBand);
  const int p0 = in_band / bh * 64;
  const int64_t q0 = (static_cast<int64_t>(band) * kBand + in_band % bh) * 64;
  const int live = static_cast<int>(rows - q0 < 64 ? rows - q0 : 64);

  const uint8_t* pbase = static_cast<const uint8_t*>(a.p) + (PT ? p0 * 2ll : static_cast<int64_t>(EPI == kEpiSwiglu ? p0 / 2 : p0) * ldp);
  const uint8_t* qbase = static_cast<const uint8_t*>(a.q) + q0 * ldq;
  uint32_t poff[S::kLoads], qoff[S::kLoads];
#pragma unroll
  for (int i = 0; i < S::kLoads; ++i) {
    const int row = i * 8 + lane / 8;
    if constexpr (PT) {
      int col = ((lane & 7) ^ swz_t64(row)) * 16;
      if (p0 + col / 2 >= NO) col = 0;
      poff[i] = static_cast<uint32_t>(row * ldp + col);
    } else {
      const int at = EPI == kEpiSwiglu ? swiglu_row(p0, row, NO) : min(row, NO - 1 - p0);
      poff[i] = static_cast<uint32_t>(at * ldp) + ((lane & 7) ^ swz(row)) * 16;
    }
    qoff[i] = static_cast<uint32_t>(min(row, live - 1) * ldq) + ((lane & 7) ^ swz(row)) * 16;
  }
  auto issue_p = [&](int step) MIEP_INLINE {
    const uint8_t* pb = pbase + static_cast<int64_t>(step) * (PT ? 64 * ldp : kStepBytes);
    if ((step + 1) * 64 <= C) {
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) dma16s(pb, poff[i], mine + i * 1024);
    } else {                                                          // behind the contraction's end: zeros
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const int row = i * 8 + lane / 8;
        const bool in = PT ? step * 64 + row < C : step * 64 + ((lane & 7) ^ swz(row)) * 8 < C;
        dma16(in ? static_cast<const void*>(pb + poff[i]) : static_cast<const void*>(g_zero16), mine + i * 1024);
      }
    }
  };
  auto issue_q = [&](int step) MIEP_INLINE {
    const uint8_t* qb = qbase + static_cast<int64_t>(step) * kStepBytes;
    if ((step + 1) * 64 <= C) {
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) dma16s(qb, qoff[i], mine + S::kBytes + i * 1024);
    } else {
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const bool in = step * 64 + ((lane & 7) ^ swz(i * 8 + lane / 8)) * 8 < C;
        dma16(in ? static_cast<const void*>(qb + qoff[i]) : static_cast<const void*>(g_zero16), mine + S::kBytes + i * 1024);
      }
    }
  };

  f32x4 acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (wave < nk) {
    issue_p(wave);
    issue_q(wave);
  }
  for (int step = wave; step < nk; step += S::kWaves) {
    const bool more = step + S::kWaves < nk;
    bf16x8 p[2][T], q[2][T];
    // P has come; its operands have left the buffer before the next step's come
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kLoads) : "memory");
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const uint32_t at = (i * 16 + m) * kStepBytes + (((h * 4 + quarter) ^ swz(m)) * 16);
        if constexpr (PT) {
          const int r = h * 32 + quarter * 8 + m / 4;
          const uint32_t tr = mine + r * kStepBytes + ((i * 2 + (m & 3) / 2) ^ swz_t64(r)) * 16 + (m & 1) * 8;
          struct { i16x4 lo, hi; } v;
          v.lo = lds_read_tr(tr);
          v.hi = lds_read_tr(tr + 4 * kStepBytes);
          p[h][i] = __builtin_bit_cast(bf16x8, v);
        } else {
          p[h][i] = lds_read<bf16x8>(mine + at);
        }
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (more) {
      issue_p(step + S::kWaves);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kLoads) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i)
        q[h][i] = lds_read<bf16x8>(mine + S::kBytes + (i * 16 + m) * kStepBytes + (((h * 4 + quarter) ^ swz(m)) * 16));
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    if (more) issue_q(step + S::kWaves);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int j = 0; j < T; ++j) acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p[h][i], q[h][j], acc[i][j], 0, 0, 0);
  }

  // a wavefront's sums take the place of its own buffer: [row][16 pieces of 4
  // columns], the pieces of a row exchanged so that rows meet different banks
  float* sums = reinterpret_cast<float*>(lds_mem + wave * 2 * S::kBytes);
#pragma unroll
  for (int j = 0; j < T; ++j)
#pragma unroll
    for (int i = 0; i < T; ++i) *reinterpret_cast<f32x4*>(sums + (j * 16 + m) * 64 + ((i * 4 + quarter) ^ m) * 4) = acc[i][j];
  __syncthreads();
  auto whole = [&](int row, int piece, float (&v)[4]) MIEP_INLINE {
    const float* s = reinterpret_cast<const float*>(lds_mem) + row * 64 + (piece ^ (row & 15)) * 4;
    f32x4 x = *reinterpret_cast<const f32x4*>(s);
#pragma unroll
    for (int w = 1; w < S::kWaves; ++w) {
      const f32x4 y = *reinterpret_cast<const f32x4*>(s + w * (2 * S::kBytes / 4));
#pragma unroll
      for (int r = 0; r < 4; ++r) x[r] += y[r];
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = x[r];
  };
  constexpr int PIECES = EPI == kEpiSwiglu ? 8 : 16;                  // of 4 columns of the result
  const int width = EPI == kEpiSwiglu ? NO / 2 : NO;
#pragma unroll
  for (int k = 0; k < 64 * PIECES / 512; ++k) {
    const int item = k * 512 + threadIdx.x, row = item / PIECES, piece = item % PIECES;
    const int c = (EPI == kEpiSwiglu ? p0 / 2 : p0) + piece * 4;
    if (row >= live || c >= width) continue;
    float v[4];
    if constexpr (EPI == kEpiSwiglu) {
      float u[4];
      whole(row, piece / 4 * 8 + piece % 4, v);
      whole(row, piece / 4 * 8 + piece % 4 + 4, u);
      EpilogueRow(a.epi, a.out, q0 + row, NO).swiglu(c, v, u);
    } else {
      whole(row, piece, v);
      EpilogueRow(a.epi, a.out, q0 + row, NO).plain(c, v);
    }
  }
}

template <bool PT, int EPI>
hipError_t launch_dense_split(const GemmRowsArgs& a, hipStream_t st) {
  const int64_t total = ((a.g.limit + 63) / 64) * ((a.NO + 63) / 64);
  gemm_dense_split_kernel<PT, EPI><<<static_cast<unsigned>((total + 7) / 8 * 8), 512, 0, st>>>(a);
  return hipGetLastError();
}

// A tile's time by measurement: `rounds` of (steps * step + fixed) us, a round
// being as many tiles as the GPU holds at a time.  `busy` is what a step takes
// longer with every CU at work than with few (power, L2).  All bf16, weights not
// in a cache; us by the tiles 32x32 / 64x64 (both split over wavefronts) / 128x64 /
// 128x128 / 128x192 / 128x256 / 256x192 / 256x256, the rule's choice marked (of the
// last two the wide kernel's own rule takes one, by rounds):
//   1000 x  256 x 7168   *14.4 /  22.9 /  37.6 /  46.3 /  56.9 /  73.3 /  97.9 / 127.7
//    128 x 4096 x 7168    40.3 / *33.8 /  55.3 /  70.0 /  72.2 /  74.5 / 106.5 / 107.3
//   4096 x  256 x 7168    61.0 / *32.3 /  53.4 /  66.9 /  81.0 /  98.6 / 108.1 / 141.0
//   4096 x 1024 x 1024    48.3 /  24.9 /  13.7 / *13.4 /  15.2 /  17.0 /  20.9 /  26.7
//   1024 x 4096 x 7168   229.2 / 106.6 /  86.6 / *67.6 /  78.6 /  94.7 / 105.2 / 137.4
//    700 x 7168 x 2048    98.0 /  48.8 /  37.6 /  38.3 / *26.5 /  30.2 /  36.6 /  45.8
//   1003 x 7168 x 2048   136.2 /  67.9 /  50.0 /  42.2 /  44.7 / *32.0 /  36.6 /  46.9
//   3000 x 4096 x 4096   513.0 / 171.0 / 122.2 / 105.7 /  92.4 / 103.9 / *77.9 /  90.3
//   2000 x 8192 x 2048   328.8 / 150.0 /  95.5 /  82.0 /  74.1 /  64.9 /  72.8 / *54.8
//   8192 x 4096 x 7168    2167 / 747.1 / 587.2 / 507.3 / 450.3 / 395.0 / 373.9 /*341.3
// Gradients of the rows (C = N):
//    777 x 4096 -> 1024   42.5 / *17.1 /  22.8 /  29.5 /  36.5 /  46.0 /  59.7 /  77.5
//    500 x 4096 -> 7168  175.8 /  68.5 /  53.7 / *40.6 /  44.7 /  52.6 /  62.9 /  82.0
//   1024 x 4096 -> 7168  291.4 / 119.0 / 101.4 /  79.5 /  80.7 / *55.7 /  65.3 /  81.1
//   3000 x 4096 -> 4096  577.4 / 169.7 / 128.6 / 105.9 /  92.1 / 104.3 / *78.0 /  88.9
//   4096 x 4096 -> 7168   1148 / 445.9 / 349.8 / 277.1 / 229.1 / 222.9 / 212.4 /*191.8
struct DenseTile {
  int p, q, slots;
  float step, busy, fixed;
};
enum { kDense32, kDense64, kDense128x64, kDense128, kDense128x192, kDense128x256, kDense192, kDense256, kDenseTiles };
constexpr DenseTile kDenseTile[kDenseTiles] = {
    {32, 32, 256, 0.14f, 0.f, 0.8f},   {64, 64, 256, 0.22f, 0.f, 2.2f},    {128, 64, 512, 0.45f, 0.27f, 1.5f}, {128, 128, 256, 0.55f, 0.06f, 2.5f},
    {128, 192, 256, 0.68f, 0.06f, 2.5f}, {128, 256, 256, 0.85f, 0.1f, 3.f}, {256, 192, 256, 0.85f, 0.45f, 4.f}, {256, 256, 256, 1.f, 0.55f, 5.f}};

inline int dense_tile(int64_t rows, int NO, int C) {
  int best = kDense256;
  float least = 0.f;
  for (int i = 0; i < kDenseTiles; ++i) {
    const DenseTile& t = kDenseTile[i];
    const int64_t tiles = (rows + t.q - 1) / t.q * ((NO + t.p - 1) / t.p);
    const float full = static_cast<float>(tiles) / t.slots;
    // two workgroups a CU take turns: their rounds need not be whole
    const float rounds = t.slots > 256 ? (full > 1.f ? full : 1.f) : static_cast<float>((tiles + t.slots - 1) / t.slots);
    const float us = rounds * ((C + 63) / 64 * (t.step + t.busy * (full < 1.f ? full : 1.f)) + t.fixed);
    if (i == 0 || us < least) {
      least = us;
      best = i;
    }
  }
  return best;
}

template <bool PT, int EPI>
hipError_t launch_dense(const GemmRowsArgs& a, hipStream_t st) {
  constexpr int EL = kGemmBf16;
  switch (dense_tile(a.g.limit, a.NO, a.C)) {
    case kDense32: return launch_rows_split<EL, PT, false, EPI>(a, st);
    case kDense64: return launch_dense_split<PT, EPI>(a, st);
    case kDense128x64: return launch_rows_tile<EL, PT, false, 128, 64, 2, 2, 3, 3, EPI>(a, st);
    case kDense128: return launch_rows_tile<EL, PT, false, 128, 128, 2, 4, 5, 5, EPI>(a, st);
    case kDense128x192: return launch_rows_tile<EL, PT, false, 128, 192, 2, 4, 4, 4, EPI>(a, st);
    case kDense128x256: return launch_rows_tile<EL, PT, false, 128, 256, 2, 4, 3, 3, EPI>(a, st);
    default: break;                                                   // 192 or 256 rows: the kernel's own count of rounds
  }
  gemm_rows_wide_kernel<EL, PT, false, EPI><<<256, 8 * kWave, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace miep
