// gemm_rows_split.h -- the rows kernel for few tiles over a long contraction.
//
// With fewer tiles than CUs a tile's time is its steps' latency, one after the
// other.  Here a workgroup computes only 32 output channels x 32 rows, and its
// 8 wavefronts take every eighth step of the contraction each, through buffers
// of their own (so without barriers); their sums are added up in wavefront
// order in LDS at the end.
#pragma once

#include "gemm.h"

namespace miep {

template <int EL>
struct RowsSplit {
  static constexpr bool kFp8 = EL != kGemmBf16;
  static constexpr int kWaves = 8, kSide = 32;
  static constexpr int kBytes = kSide * kStepBytes;                  // of one operand's step
  static constexpr int kLoads = kBytes / 1024;
  static constexpr int kStage = 2 * kBytes + (kFp8 ? 256 : 0);       // P, Q, scales (32 rows', then the P block's)
  static constexpr int kPitch = kSide + 4;
  static constexpr int kLds = kWaves * 2 * kStage;
  static_assert(kLds <= 163840 && kSide * kPitch * 4 <= 2 * kStage, "buffers");
};

// Transposed P: 64 contraction rows of 32 channels, 64 bytes each.
__device__ __forceinline__ int swz_t32(int row) { return (row >> 2) & 2; }

template <int EL, bool PT, bool GATHER>
__global__ __launch_bounds__(512, 2) void gemm_rows_split_kernel(GemmRowsArgs a) {
  using S = RowsSplit<EL>;
  constexpr int EB = S::kFp8 ? 1 : 2, KE = kStepBytes / EB;
  __shared__ __align__(1024) uint8_t lds_mem[S::kLds];
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_byte*)lds_mem;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const uint32_t mine = lds + wave * 2 * S::kStage;

  const int NO = a.NO, C = a.C;
  const int ntiles = (NO + S::kSide - 1) / S::kSide;
  const int64_t ldq = static_cast<int64_t>(C) * EB;
  const int64_t ldp = static_cast<int64_t>(PT ? NO : C) * EB;
  const int cbytes = C * EB;
  const int nk = (C + KE - 1) / KE;
  const int64_t kb = C / kFp8Group;
  constexpr int SB = EL == kGemmFp8 ? 4 : 1;

  const int total = count_tiles(a.g, S::kSide, ntiles);
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const TileAt at = find_tile(a.g, S::kSide, ntiles, t);
    if (at.group < 0) break;
    const int mtiles = max(row_tiles(at.rows, S::kSide), 1);
    const int first = min(max(at.first, 0), mtiles * ntiles - 1);
    const int p0 = first / mtiles * S::kSide, q0 = first % mtiles * S::kSide;
    const int live = min(S::kSide, at.rows - q0);
    const int64_t row0 = at.begin + q0;
    const uint8_t* pg = static_cast<const uint8_t*>(a.p) + static_cast<int64_t>(at.group) * NO * C * EB;

    // this lane's 16 bytes of load i: where its first step's lie, and its chunk
    const uint8_t *pptr[S::kLoads], *qptr[S::kLoads];
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      if constexpr (PT) {
        const int row = i * 16 + lane / 4;
        int col = ((lane & 3) ^ swz_t32(row)) * 16;
        if (p0 + col / 2 >= NO) col = 0;
        pptr[i] = pg + row * ldp + static_cast<int64_t>(p0) * EB + col;
      } else {
        const int row = i * 8 + lane / 8;
        pptr[i] = pg + static_cast<int64_t>(min(p0 + row, NO - 1)) * ldp + ((lane & 7) ^ ((row >> 1) & 7)) * 16;
      }
      const int row = i * 8 + lane / 8;
      int64_t src = row0 + min(row, live - 1);
      if constexpr (GATHER) {
        src = a.row_index[src];
        if (src >= a.q_rows) src = -1;
      }
      qptr[i] = (src >= 0 ? static_cast<const uint8_t*>(a.q) + src * ldq : pg) + ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    }
    const uint8_t* sptr = nullptr;
    if constexpr (S::kFp8) {
      const uint8_t* ps = static_cast<const uint8_t*>(a.p_scales) +
                          (static_cast<int64_t>(at.group) * ((NO + 127) / 128) + p0 / 128) * kb * SB;
      int64_t src = row0 + min(lane & 31, live - 1);
      if constexpr (GATHER) {
        src = a.row_index[src];
        if (src >= a.q_rows) src = -1;
      }
      sptr = lane < 32 && src >= 0 ? static_cast<const uint8_t*>(a.q_scales) + src * kb * SB : ps;
    }
    auto issue = [&](int step, int buf) MIEP_INLINE {
      const uint32_t to = mine + buf * S::kStage;
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        bool in;
        if constexpr (PT) in = step * KE + i * 16 + lane / 4 < C;
        else in = step * kStepBytes + ((lane & 7) ^ (((i * 8 + lane / 8) >> 1) & 7)) * 16 < cbytes;
        const uint8_t* p = pptr[i] + static_cast<int64_t>(step) * (PT ? (kStepBytes / 2) * ldp : kStepBytes);
        dma16(in ? static_cast<const void*>(p) : static_cast<const void*>(g_zero16), to + i * 1024);
      }
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const bool in = step * kStepBytes + ((lane & 7) ^ (((i * 8 + lane / 8) >> 1) & 7)) * 16 < cbytes;
        const uint8_t* q = qptr[i] + static_cast<int64_t>(step) * kStepBytes;
        dma16(in ? static_cast<const void*>(q) : static_cast<const void*>(g_zero16), to + S::kBytes + i * 1024);
      }
      if constexpr (S::kFp8) {
        if constexpr (SB == 4) dma4(sptr + static_cast<int64_t>(step) * 4, to + 2 * S::kBytes);
        else dma1(sptr + step, to + 2 * S::kBytes);
      }
    };

    f32x4 acc[2][2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

    if (wave < nk) issue(wave, 0);
    int buf = 0;
    for (int step = wave; step < nk; step += S::kWaves, buf ^= 1) {
      if (step + S::kWaves < nk) {
        issue(step + S::kWaves, buf ^ 1);
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * S::kLoads + (S::kFp8 ? 1 : 0)) : "memory");
      } else {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      }
      const uint32_t from = mine + buf * S::kStage;
      struct half { i32x4 v[2]; };
      half p[2], q[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int row = i * 16 + m;
          const uint32_t chunk = ((h * 4 + quarter) ^ ((row >> 1) & 7)) * 16;
          q[i].v[h] = lds_read<i32x4>(from + S::kBytes + row * kStepBytes + chunk);
          if constexpr (PT) {
            const int r = h * 32 + quarter * 8 + m / 4;
            const uint32_t at32 = from + r * 64 + ((i * 2 + (m & 3) / 2) ^ swz_t32(r)) * 16 + (m & 1) * 8;
            struct { i16x4 lo, hi; } v;
            v.lo = lds_read_tr(at32);
            v.hi = lds_read_tr(at32 + 4 * 64);
            p[i].v[h] = __builtin_bit_cast(i32x4, v);
          } else {
            p[i].v[h] = lds_read<i32x4>(from + row * kStepBytes + chunk);
          }
        }
      }
      if constexpr (!S::kFp8) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p[i].v[h]),
                                                                  __builtin_bit_cast(bf16x8, q[j].v[h]), acc[i][j], 0, 0, 0);
      } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t sat = from + 2 * S::kBytes;
          if constexpr (EL == kGemmFp8) {
            const float s = lds_read<float>(sat + 32 * 4) * lds_read<float>(sat + (j * 16 + m) * 4);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const f32x4 z = {0.f, 0.f, 0.f, 0.f};
              const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, p[i]),
                                                                              __builtin_bit_cast(i32x8, q[j]), z, 0, 0, 0, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s, acc[i][j][r]);
            }
          } else {
            const int ep = lds_read<int>(sat + 32 * 4), e = lds_read<int>(sat + (j * 16 + m) * 4);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(__builtin_bit_cast(i32x8, p[i]),
                                                                          __builtin_bit_cast(i32x8, q[j]), acc[i][j], 0, 0, 0, ep, 0, e);
          }
        }
      }
      // the operands have left this buffer before the next turn loads into it
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    }

    // a wavefront's sums take the place of its own buffers
    float* sums = reinterpret_cast<float*>(lds_mem + wave * 2 * S::kStage);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        *reinterpret_cast<f32x4*>(sums + (j * 16 + m) * S::kPitch + i * 16 + quarter * 4) = acc[i][j];
    __syncthreads();
    {
      const int row = threadIdx.x / 16, p = threadIdx.x % 16 * 2;
      float x = 0.f, y = 0.f;
#pragma unroll
      for (int w = 0; w < S::kWaves; ++w) {
        const float* s = reinterpret_cast<const float*>(lds_mem + w * 2 * S::kStage) + row * S::kPitch + p;
        x += s[0];
        y += s[1];
      }
      if (row < live && p0 + p < NO) {
        bool none = false;
        if constexpr (GATHER) {
          const int src = a.row_index[row0 + row];
          none = src < 0 || src >= a.q_rows;
        }
        *reinterpret_cast<uint32_t*>(a.out + (row0 + row) * NO + p0 + p) = none ? 0u : pack_bf16x2(x, y);
      }
    }
    __syncthreads();
  }
}

// The most tiles that disjoint groups can have.
inline int64_t split_tiles(const GemmRowsArgs& a) {
  return ((a.g.limit + 31) / 32 + a.g.G) * ((static_cast<int64_t>(a.NO) + 31) / 32);
}

template <int EL, bool PT, bool GATHER>
hipError_t launch_rows_split(const GemmRowsArgs& a, hipStream_t st) {
  const int64_t most = split_tiles(a);
  gemm_rows_split_kernel<EL, PT, GATHER><<<static_cast<unsigned>(most < 256 ? most : 256), 512, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace miep
