// gemm_weight.hip -- grouped bf16 product over the rows: the weights' gradient.
//
//   dW_g[n][k] (+)= sum over the rows i of group g of dY[i][n] * X[src(i)][k]
//
// The contraction runs over rows, so both operands are read through LDS's
// transposing loads: tiles of 64 rows come in as they lie in memory (rows of
// 512 or 256 bytes) and a lane reads 4 rows of one channel at a time.  X gives
// the MFMA's rows, so that a lane holds 4 consecutive k of one n.
#include "gemm.h"

namespace miep {

template <int BP, int BQ, int WP, int WQ, int NST>
struct WeightTile {
  static constexpr int kRows = 64;                                   // contraction rows of a stage
  static constexpr int kWaves = WP * WQ;
  static constexpr int kTP = BP / WP / 16, kTQ = BQ / WQ / 16;
  static constexpr int kPBytes = BP * 2 * kRows, kQBytes = BQ * 2 * kRows;
  static constexpr int kStage = kPBytes + kQBytes;
  static constexpr int kPLoads = kPBytes / 1024 / kWaves, kQLoads = kQBytes / 1024 / kWaves;
  static constexpr int kLoads = kPLoads + kQLoads;
  static constexpr int kPChunks = BP / 8, kQChunks = BQ / 8;         // 16-byte chunks of a tile row
  static_assert(kPChunks >= 16 && kQChunks >= 16 && kLoads * (NST - 1) < 64, "tile shape");
};

template <bool GATHER, bool F32, int BP, int BQ, int WP, int WQ, int NST>
__global__ __launch_bounds__(WP * WQ * kWave, 2) void gemm_weight_kernel(GemmWeightArgs a) {
  using S = WeightTile<BP, BQ, WP, WQ, NST>;
  constexpr int TP = S::kTP, TQ = S::kTQ;
  __shared__ __align__(1024) uint8_t lds_mem[NST * S::kStage];
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_byte*)lds_mem;

  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int wp = wave % WP, wq = wave / WP;
  const int m = lane & 15, quarter = lane >> 4;

  // XCD x takes the x-th eighth of the tiles: neighbours share dY or X columns in its L2
  const int ptiles = (a.K + BP - 1) / BP, qtiles = (a.N + BQ - 1) / BQ;
  const int64_t total = static_cast<int64_t>(ptiles) * qtiles * a.g.G;
  const int64_t chunk = (total + 7) / 8;
  const int64_t t = (blockIdx.x & 7) * chunk + (blockIdx.x >> 3);
  if ((blockIdx.x >> 3) >= chunk || t >= total) return;
  const int group = static_cast<int>(t / (ptiles * qtiles));
  const int in_group = static_cast<int>(t - static_cast<int64_t>(group) * (ptiles * qtiles));
  const int q0 = in_group / ptiles * BQ, p0 = in_group % ptiles * BP;

  int64_t begin;
  int rows;
  group_range(a.g, group, &begin, &rows);
  begin = (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(begin >> 32))) << 32) |
          static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(begin)));
  rows = __builtin_amdgcn_readfirstlane(rows);
  if (rows == 0 && a.accumulate) return;
  const int nk = (rows + S::kRows - 1) / S::kRows;

  const int64_t ldq = 2 * static_cast<int64_t>(a.N), ldp = 2 * static_cast<int64_t>(a.K);
  const uint8_t* qbase = reinterpret_cast<const uint8_t*>(a.q) + begin * ldq + 2 * static_cast<int64_t>(q0);
  const uint8_t* pbase = reinterpret_cast<const uint8_t*>(a.p) + (GATHER ? 0 : begin * ldp) + 2 * static_cast<int64_t>(p0);
  int prow[S::kPLoads], pcol[S::kPLoads], qrow[S::kQLoads], qcol[S::kQLoads];
#pragma unroll
  for (int i = 0; i < S::kPLoads; ++i) {
    prow[i] = (i * S::kWaves + wave) * (64 / S::kPChunks) + lane / S::kPChunks;
    pcol[i] = ((lane % S::kPChunks) ^ ((prow[i] & 3) | ((prow[i] >> 1) & 4)) << 1) * 16;
    if (p0 + pcol[i] / 2 >= a.K) pcol[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < S::kQLoads; ++i) {
    qrow[i] = (i * S::kWaves + wave) * (64 / S::kQChunks) + lane / S::kQChunks;
    qcol[i] = ((lane % S::kQChunks) ^ ((qrow[i] & 3) | ((qrow[i] >> 1) & 4)) << 1) * 16;
    if (q0 + qcol[i] / 2 >= a.N) qcol[i] = 0;
  }
  // gathered rows' sources, read one stage ahead of the loads that use them
  int src[GATHER ? S::kPLoads : 1];
  auto sources = [&](int step) {
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < S::kPLoads; ++i) {
        const int r = step * S::kRows + prow[i];
        src[i] = r < rows ? a.row_index[begin + r] : -1;
      }
    }
  };
  auto issue = [&](int step, int buf) {
    const uint32_t st = lds + buf * S::kStage;
    const int r0 = step * S::kRows;
    const bool tail = rows - r0 < S::kRows;
#pragma unroll
    for (int i = 0; i < S::kPLoads; ++i) {
      const uint32_t to = st + (i * S::kWaves + wave) * 1024;
      if constexpr (GATHER) {
        const bool in = src[i] >= 0 && src[i] < a.p_rows;
        dma16(in ? static_cast<const void*>(pbase + src[i] * ldp + pcol[i]) : static_cast<const void*>(g_zero16), to);
      } else {
        const uint32_t off = static_cast<uint32_t>(prow[i] * ldp + pcol[i]);
        const uint8_t* pb = pbase + r0 * ldp;
        if (!tail) dma16s(pb, off, to);
        else dma16(r0 + prow[i] < rows ? static_cast<const void*>(pb + off) : static_cast<const void*>(g_zero16), to);
      }
    }
#pragma unroll
    for (int i = 0; i < S::kQLoads; ++i) {
      const uint32_t to = st + S::kPBytes + (i * S::kWaves + wave) * 1024;
      const uint32_t off = static_cast<uint32_t>(qrow[i] * ldq + qcol[i]);
      const uint8_t* qb = qbase + r0 * ldq;
      if (!tail) dma16s(qb, off, to);
      else dma16(r0 + qrow[i] < rows ? static_cast<const void*>(qb + off) : static_cast<const void*>(g_zero16), to);
    }
  };

  f32x4 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  uint32_t pa[TP], qa[TQ];
  {
    const int row = quarter * 8 + m / 4;
    const int s = ((row & 3) | ((row >> 1) & 4)) << 1;
#pragma unroll
    for (int i = 0; i < TP; ++i)
      pa[i] = row * (2 * BP) + ((wp * 2 * TP + i * 2 + (m & 3) / 2) ^ s) * 16 + (m & 1) * 8;
#pragma unroll
    for (int j = 0; j < TQ; ++j)
      qa[j] = S::kPBytes + row * (2 * BQ) + ((wq * 2 * TQ + j * 2 + (m & 3) / 2) ^ s) * 16 + (m & 1) * 8;
  }

#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s < nk) {
      sources(s);
      issue(s, s);
    }
  sources(NST - 1);
  int buf = 0;
  for (int step = 0; step < nk; ++step) {
    if (!GATHER && step + NST - 2 < nk) wait_tiles<(NST - 2) * S::kLoads>();
    else wait_tiles<0>();
    const int ahead = step + NST - 1;
    if (ahead < nk) issue(ahead, buf == 0 ? NST - 1 : buf - 1);
    sources(ahead + 1);
    const uint32_t st = lds + buf * S::kStage;
    buf = buf == NST - 1 ? 0 : buf + 1;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 pf[TP], qf[TQ];
#pragma unroll
      for (int j = 0; j < TQ; ++j) {
        struct { i16x4 lo, hi; } v;
        v.lo = lds_read_tr(st + qa[j] + h * 32 * 2 * BQ);
        v.hi = lds_read_tr(st + qa[j] + (h * 32 + 4) * 2 * BQ);
        qf[j] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        struct { i16x4 lo, hi; } v;
        v.lo = lds_read_tr(st + pa[i] + h * 32 * 2 * BP);
        v.hi = lds_read_tr(st + pa[i] + (h * 32 + 4) * 2 * BP);
        pf[i] = __builtin_bit_cast(bf16x8, v);
      }
#pragma unroll
      for (int i = 0; i < TP; ++i)
#pragma unroll
        for (int j = 0; j < TQ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[i], qf[j], acc[i][j], 0, 0, 0);
    }
  }

#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    const int n = q0 + (wq * TQ + j) * 16 + m;
    if (n >= a.N) continue;
    const int64_t o = (static_cast<int64_t>(group) * a.N + n) * a.K;
#pragma unroll
    for (int i = 0; i < TP; ++i) {
      if constexpr (F32) {
        const int k = p0 + (wp * TP + i) * 16 + quarter * 4;
        if (k >= a.K) continue;
        f32x4* at = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o + k);
        f32x4 v = acc[i][j];
        if (a.accumulate) {
          const f32x4 old = *at;
          v = f32x4{old[0] + v[0], old[1] + v[1], old[2] + v[2], old[3] + v[3]};
        }
        *at = v;
      } else if ((i & 1) == 0) {
        const int kk = p0 + (wp * TP + i + (quarter & 1)) * 16 + (quarter >> 1) * 8;
        const v4u v = pack_pair(acc[i][j], acc[i + 1][j]);
        if (kk < a.K) *reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.out) + o + kk) = v;
      }
    }
  }
}

template <bool GATHER, bool F32, int BP, int BQ, int WP, int WQ, int NST>
hipError_t launch_weight_tile(const GemmWeightArgs& a, hipStream_t st) {
  const int64_t tiles = static_cast<int64_t>((a.K + BP - 1) / BP) * ((a.N + BQ - 1) / BQ) * a.g.G;
  const int64_t grid = (tiles + 7) / 8 * 8;
  if (grid > max_blocks(WP * WQ * kWave)) return hipErrorInvalidConfiguration;
  gemm_weight_kernel<GATHER, F32, BP, BQ, WP, WQ, NST><<<static_cast<unsigned>(grid), WP * WQ * kWave, 0, st>>>(a);
  return hipGetLastError();
}

template <bool GATHER, bool F32>
hipError_t launch_weight(const GemmWeightArgs& a, hipStream_t st) {
  const int64_t big = static_cast<int64_t>((a.K + 255) / 256) * ((a.N + 255) / 256) * a.g.G;
  if (big < 256) return launch_weight_tile<GATHER, F32, 128, 128, 2, 2, 2>(a, st);
  return launch_weight_tile<GATHER, F32, 256, 256, 2, 4, 2>(a, st);
}

hipError_t launch_gemm_weight(const GemmWeightArgs& a, hipStream_t st) {
  if (a.g.G == 0) return hipSuccess;
  if (a.row_index) return a.out_f32 ? launch_weight<true, true>(a, st) : launch_weight<true, false>(a, st);
  return a.out_f32 ? launch_weight<false, true>(a, st) : launch_weight<false, false>(a, st);
}

}  // namespace miep
