// gemm_weight.hip -- grouped bf16 product over the rows: the weights' gradient.
//
//   dW_g[n][k] (+)= sum over the rows i of group g of dY[i][n] * X[src(i)][k]
//
// The contraction runs over rows, so both operands are read through LDS's
// transposing loads: tiles of 64 rows come in as they lie in memory (rows of
// 512 or 256 bytes) and a lane reads 4 rows of one channel at a time.  X gives
// the MFMA's rows (P), so that a lane holds 4 consecutive k of one n.
//
// With few rows a group the fp32 result is most of the traffic (4 N K bytes a
// group), so it leaves in whole 128-byte lines (see the stores): 32 ragged groups
// of 8192 rows, 7168 x 2048, take 496 us, of which the stores alone 308 and the
// rest alone 271 (a bf16 result 403, added to an fp32 one 998, gathered 514).
// With many rows the MFMAs and their LDS reads bound it: 16384 rows over 4
// groups 404 us, 1,190 TFLOP/s, of 4096 x 7168 785 us, 1,225.
#include <type_traits>

#include "gemm.h"

namespace miep {

template <bool GATHER, int BP, int BQ, int WP, int WQ, int NSP, int NSQ>
struct WeightTile {
  static constexpr int kRows = 64;                                   // contraction rows of a step
  static constexpr int kWaves = WP * WQ;
  static constexpr int kTP = BP / WP / 16, kTQ = BQ / WQ / 16;
  static constexpr int kPBytes = BP * 2 * kRows, kQBytes = BQ * 2 * kRows;
  static constexpr int kIndexBytes = GATHER ? 4 * kRows : 0;         // source rows that come with a step of Q
  static constexpr int kLds = NSP * kPBytes + NSQ * (kQBytes + kIndexBytes);
  static constexpr int kPLoads = kPBytes / 1024 / kWaves, kQLoads = kQBytes / 1024 / kWaves + (GATHER ? 1 : 0);
  static constexpr int kPChunks = BP / 8, kQChunks = BQ / 8;         // 16-byte chunks of a tile row
  // loads in flight behind the tile that a barrier publishes, as in the rows kernel
  static constexpr int kBehind = (NSP > NSQ ? NSQ - 1 : NSQ - 2) * kPLoads + (NSQ - 2) * kQLoads;
  static_assert(kPChunks >= 16 && kQChunks >= 16 && NSQ >= 2 && NSP >= NSQ && kLds <= 163840, "tile shape");
  static_assert(!GATHER || (NSP == 2 && NSQ == 2), "indices come two steps ahead");
};

template <bool GATHER, bool F32, int BP, int BQ, int WP, int WQ, int NSP, int NSQ>
__global__ __launch_bounds__(WP * WQ * kWave, 2) void gemm_weight_kernel(GemmWeightArgs a) {
  using S = WeightTile<GATHER, BP, BQ, WP, WQ, NSP, NSQ>;
  constexpr int TP = S::kTP, TQ = S::kTQ;
  __shared__ __align__(1024) uint8_t lds_mem[S::kLds];
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_byte*)lds_mem;

  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int wp = wave % WP, wq = wave / WP;
  const int m = lane & 15, quarter = lane >> 4;

  // Groups differ in rows, so every XCD (workgroups go to the 8 in turn) takes
  // an eighth of each group's tiles, in order, so that they share dY's and
  // X's columns in its L2; groups of few tiles are dealt out one by one.
  const int ptiles = (a.K + BP - 1) / BP, qtiles = (a.N + BQ - 1) / BQ;
  const int per_group = ptiles * qtiles;
  int group, tile;
  if (per_group >= 64) {
    const int part = (per_group + 7) / 8, at = blockIdx.x >> 3;
    group = at / part;
    tile = (blockIdx.x & 7) * part + at % part;
  } else {
    group = blockIdx.x / per_group;
    tile = blockIdx.x - group * per_group;
  }
  if (group >= a.g.G || tile >= per_group) return;
  const int q0 = tile / ptiles * BQ, p0 = tile % ptiles * BP;

  int64_t begin;
  int rows;
  group_range(a.g, group, &begin, &rows);
  begin = (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(begin >> 32))) << 32) |
          static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(begin)));
  rows = __builtin_amdgcn_readfirstlane(rows);
  if (rows == 0 && a.accumulate) return;
  const int nk = (rows + S::kRows - 1) / S::kRows;
  const bool ragged_end = rows % S::kRows != 0;

  const int64_t ldq = 2 * static_cast<int64_t>(a.N), ldp = 2 * static_cast<int64_t>(a.K);
  const uint8_t* qbase = reinterpret_cast<const uint8_t*>(a.q) + begin * ldq + 2 * static_cast<int64_t>(q0);
  const uint8_t* pbase = reinterpret_cast<const uint8_t*>(a.p) + (GATHER ? 0 : begin * ldp) + 2 * static_cast<int64_t>(p0);
  // Of load i of a step: the lane's row of the tile (rows of load i + 1 lie
  // 64 / chunks * waves further) and its 16 bytes of that row.
  constexpr int QL = S::kQBytes / 1024 / S::kWaves;
  constexpr int PR = 64 / S::kPChunks * S::kWaves, QR = 64 / S::kQChunks * S::kWaves;
  const int prow = wave * (64 / S::kPChunks) + lane / S::kPChunks, qrow = wave * (64 / S::kQChunks) + lane / S::kQChunks;
  uint32_t poff[S::kPLoads], qoff[QL];
#pragma unroll
  for (int i = 0; i < S::kPLoads; ++i) {
    const int row = prow + i * PR;
    int col = ((lane % S::kPChunks) ^ swz_t(row)) * 16;
    if (p0 + col / 2 >= a.K) col = 0;
    poff[i] = static_cast<uint32_t>((GATHER ? 0 : row * ldp) + col);
  }
#pragma unroll
  for (int i = 0; i < QL; ++i) {
    const int row = qrow + i * QR;
    int col = ((lane % S::kQChunks) ^ swz_t(row)) * 16;
    if (q0 + col / 2 >= a.N) col = 0;
    qoff[i] = static_cast<uint32_t>(row * ldq + col);
  }
  auto p_at = [&](int buf) MIEP_INLINE { return lds + buf * S::kPBytes; };
  auto q_at = [&](int buf) MIEP_INLINE { return lds + NSP * S::kPBytes + buf * (S::kQBytes + S::kIndexBytes); };
  // A gathered row's address; a row behind the group's last, or without a
  // source, reads zeros.
  auto sourced = [&](int src) MIEP_INLINE { return src >= 0 && src < a.p_rows; };
  auto gathered = [&](int i, int step, int src) MIEP_INLINE {
    const bool in = step * S::kRows + prow + i * PR < rows && sourced(src);
    return in ? static_cast<const void*>(pbase + src * ldp + poff[i]) : static_cast<const void*>(g_zero16);
  };
  // Load i of a step of 64 whole rows (gathered: of any).  The indices of a
  // gathered step come with the Q loads two steps before its own loads, those
  // of step u + 1 in the place behind Q's step u.
  auto index_at = [&](int step, int row) MIEP_INLINE { return lds_read<int>(q_at((step - 1) & 1) + S::kQBytes + row * 4); };
  auto load_p = [&](int i, int step, int buf) MIEP_INLINE {
    const uint32_t to = p_at(buf) + (i * S::kWaves + wave) * 1024;
    if constexpr (GATHER) {
      dma16(gathered(i, step, index_at(step, prow + i * PR)), to);
    } else {
      dma16s(pbase + static_cast<int64_t>(step) * S::kRows * ldp, poff[i], to);
    }
  };
  auto load_q = [&](int i, int step, int buf) MIEP_INLINE {
    if (i < QL) dma16s(qbase + static_cast<int64_t>(step) * S::kRows * ldq, qoff[i], q_at(buf) + (i * S::kWaves + wave) * 1024);
    else if constexpr (GATHER)
      dma4(a.row_index + begin + min((step + 1) * S::kRows + lane, rows - 1), q_at(buf) + S::kQBytes);
  };
  // A step's loads, if there is such a step; the last one may have fewer rows.
  auto issue_p = [&](int step, int buf) MIEP_INLINE {
    if (step >= nk) return;
#pragma unroll
    for (int i = 0; i < S::kPLoads; ++i) {
      if (GATHER || !ragged_end || step != nk - 1) {
        load_p(i, step, buf);
      } else {
        const uint8_t* src = pbase + static_cast<int64_t>(step) * S::kRows * ldp + poff[i];
        dma16(step * S::kRows + prow + i * PR < rows ? static_cast<const void*>(src) : static_cast<const void*>(g_zero16),
              p_at(buf) + (i * S::kWaves + wave) * 1024);
      }
    }
  };
  auto issue_q = [&](int step, int buf) MIEP_INLINE {
    if (step >= nk) return;
#pragma unroll
    for (int i = 0; i < S::kQLoads; ++i) {
      if (i >= QL || !ragged_end || step != nk - 1) {
        load_q(i, step, buf);
      } else {
        const uint8_t* src = qbase + static_cast<int64_t>(step) * S::kRows * ldq + qoff[i];
        dma16(step * S::kRows + qrow + i * QR < rows ? static_cast<const void*>(src) : static_cast<const void*>(g_zero16),
              q_at(buf) + (i * S::kWaves + wave) * 1024);
      }
    }
  };

  // dY's row that goes with one without a source may hold NaN or infinities,
  // which zeros on the other side do not take away: once it has come, and
  // before the barrier that publishes it, its place is overwritten with zeros,
  // by the lanes that loaded it.  (Rows without a source are rare: choosing
  // every load's address instead took 4% of a long group's time.)
  auto clear_lost = [&](uint64_t lost, int buf) MIEP_INLINE {
    if (lost == 0) return;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
    for (int i = 0; i < QL; ++i)
      if (lost >> (qrow + i * QR) & 1) lds_write(q_at(buf) + (i * S::kWaves + wave) * 1024 + lane * 16, i32x4{0, 0, 0, 0});
  };

  f32x4 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};

  if (nk > 0) {
    uint32_t pa[TP], qa[TQ];
    {
      const int row = quarter * 8 + m / 4;
#pragma unroll
      for (int i = 0; i < TP; ++i)
        pa[i] = row * (2 * BP) + ((wp * 2 * TP + i * 2 + (m & 3) / 2) ^ swz_t(row)) * 16 + (m & 1) * 8;
#pragma unroll
      for (int j = 0; j < TQ; ++j)
        qa[j] = row * (2 * BQ) + ((wq * 2 * TQ + j * 2 + (m & 3) / 2) ^ swz_t(row)) * 16 + (m & 1) * 8;
    }

    // The order of loads, waits and barriers is the rows kernel's: step t
    // issues P's step t - 1 + NSP over its MFMAs and, behind its barrier, Q's
    // step t + NSQ.
    uint64_t lost = 0;
#pragma unroll
    for (int t = -NSP; t < 0; ++t) {
      if (t - 1 + NSP >= 0) {
        if constexpr (GATHER) {                                       // step 0: its indices straight from memory
          const int src = a.row_index[begin + min(lane, rows - 1)];
          lost = ballot(!sourced(src));
          int from[S::kPLoads];
#pragma unroll
          for (int i = 0; i < S::kPLoads; ++i) from[i] = __shfl(src, prow + i * PR);
#pragma unroll
          for (int i = 0; i < S::kPLoads; ++i) dma16(gathered(i, 0, from[i]), p_at(0) + (i * S::kWaves + wave) * 1024);
        } else {
          issue_p(t - 1 + NSP, t - 1 + NSP);
        }
      }
      if (t + NSQ >= 0) issue_q(t + NSQ, t + NSQ);
    }
    if constexpr (GATHER) clear_lost(lost, 0);
    if (nk >= NSP) wait_tiles<S::kBehind + S::kQLoads>();
    else wait_tiles<0>();
    auto publish = [&](int step) MIEP_INLINE {
      if (step - 1 + NSP < nk) wait_tiles<S::kBehind>();
      else wait_tiles<0>();
    };
    int step = 0, pbuf = 0, qbuf = 0;
    auto before = [&](int buf) MIEP_INLINE { return buf == 0 ? NSP - 1 : buf - 1; };

    // Slots, operand ring and barrier as in the rows kernel; halves are 32 rows.
    constexpr int SLOTS = 2 * TP, D = 3, RING = 4;
    static_assert(SLOTS % RING == 0 && TQ <= SLOTS - D && D <= TP, "operand ring");
    bf16x8 pf[RING], qf[2][TQ];
    auto operand = [&](uint32_t at, int row_bytes) MIEP_INLINE {
      struct { i16x4 lo, hi; } t;
      t.lo = lds_read_tr(at);
      t.hi = lds_read_tr(at + 4 * row_bytes);
      return __builtin_bit_cast(bf16x8, t);
    };
    auto read_q = [&](int h, uint32_t at, int j) MIEP_INLINE { qf[h][j] = operand(at + qa[j] + h * 32 * 2 * BQ, 2 * BQ); };
    auto read_p = [&](int k, uint32_t at) MIEP_INLINE { pf[k % RING] = operand(at + pa[k % TP] + k / TP * 32 * 2 * BP, 2 * BP); };
#pragma unroll
    for (int j = 0; j < TQ; ++j) read_q(0, q_at(0), j);
#pragma unroll
    for (int k = 0; k < D; ++k) read_p(k, p_at(0));
    auto body = [&](auto more, auto last) MIEP_INLINE {
      const int pb = pbuf, qb = qbuf;
      pbuf = pbuf == NSP - 1 ? 0 : pbuf + 1;
      qbuf = qbuf == NSQ - 1 ? 0 : qbuf + 1;
      if constexpr (!more) issue_p(step - 1 + NSP, before(pb));
      int src = 0;
      if constexpr (GATHER && !last) src = index_at(step + 1, lane);
#pragma unroll
      for (int k = 0; k < SLOTS; ++k) {
        const int late = k - (SLOTS - D);
        if constexpr (!last)
          if (late == 0) {
            if constexpr (GATHER) clear_lost(ballot(!sourced(src)), qbuf);
            publish(step);
          }
        if (k + D < SLOTS) read_p(k + D, p_at(pb));
        else if constexpr (!last) read_p(k + D - SLOTS, p_at(pbuf));
        if (k < TP) {
#pragma unroll
          for (int j = k * TQ / TP; j < (k + 1) * TQ / TP; ++j) read_q(1, q_at(qb), j);
        }
        if (late >= 0) {
          if constexpr (!last) {
#pragma unroll
            for (int j = late * TQ / D; j < (late + 1) * TQ / D; ++j) read_q(0, q_at(qbuf), j);
          }
          if constexpr (more) {
#pragma unroll
            for (int l = late * S::kQLoads / D; l < (late + 1) * S::kQLoads / D; ++l) load_q(l, step + NSQ, qb);
          }
        } else if constexpr (more) {
          constexpr int n = SLOTS - D;
#pragma unroll
          for (int l = 0; l < S::kPLoads; ++l)
            if (l * n / S::kPLoads == k) load_p(l, step - 1 + NSP, before(pb));
        }
#pragma unroll
        for (int j = 0; j < TQ; ++j)
          acc[k % TP][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[k % RING], qf[k / TP][j], acc[k % TP][j], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (!more && !last) issue_q(step + NSQ, qb);
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    const int whole = nk - (ragged_end ? 1 : 0);
    constexpr int ahead = NSP - 1 > NSQ ? NSP - 1 : NSQ;
    for (; step + ahead < whole; ++step) body(yes, no);
    for (; step + 1 < nk; ++step) body(no, no);
    body(no, yes);
  }

  // Stores.  fp32: lanes of even and odd m exchange halves of two neighbouring
  // tiles, so that 8 lanes write 128 consecutive bytes of one n: half lines
  // take 522 us where whole ones take 488 (32 groups of 256 rows, 7168 x 2048;
  // stores past the caches the same 488).
  const bool odd = m & 1;
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
#pragma unroll
    for (int i = 0; i < TP; i += 2) {
      if constexpr (F32) {
        const int k = p0 + (wp * TP + i + (m & 1)) * 16 + quarter * 4;
        f32x4 v[2];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float x = acc[i][j][r], y = acc[i + 1][j][r];
          const float other = dpp_f32<0xB1>(odd ? x : y);             // quad_perm [1,0,3,2]
          v[0][r] = odd ? other : x;
          v[1][r] = odd ? y : other;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n = q0 + (wq * TQ + j) * 16 + (m & ~1) + h;
          if (n >= a.N || k >= a.K) continue;
          f32x4* at = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + (static_cast<int64_t>(group) * a.N + n) * a.K + k);
          if (a.accumulate) {
            const f32x4 old = *at;
            v[h] = f32x4{old[0] + v[h][0], old[1] + v[h][1], old[2] + v[h][2], old[3] + v[h][3]};
          }
          *at = v[h];
        }
      } else {
        const int n = q0 + (wq * TQ + j) * 16 + m;
        const int k = p0 + (wp * TP + i + (quarter & 1)) * 16 + (quarter >> 1) * 8;
        const v4u v = pack_pair(acc[i][j], acc[i + 1][j]);
        if (n < a.N && k < a.K)
          *reinterpret_cast<v4u*>(static_cast<uint16_t*>(a.out) + (static_cast<int64_t>(group) * a.N + n) * a.K + k) = v;
      }
    }
  }
}

// Few tiles under many rows: the rows are split.  A workgroup computes 64 x 64
// of dW; its 8 wavefronts take every eighth step of 32 rows each, through
// buffers of their own (so without barriers), and their sums are added up in
// wavefront order in LDS at the end.
struct SplitTile {
  static constexpr int kRows = 32, kWaves = 8, kSide = 64, kT = kSide / 16;
  static constexpr int kBytes = kSide * 2 * kRows;                   // of one operand's step
  static constexpr int kLoads = kBytes / 1024;
  static constexpr int kPitch = kSide + 4;                           // of a wavefront's sums, floats: rows in different banks
  static constexpr int kSums = kSide * kPitch * 4;
  static constexpr int kLds = kWaves * (kSums > 4 * kBytes ? kSums : 4 * kBytes);
  static_assert(kLds <= 163840, "buffers");
};

// Rows of 128 bytes: the 8 rows of a half wavefront's transposing read (0-3 and
// 8-11) differ in parity, bit 1 and bit 3.
__device__ __forceinline__ int swz_t64(int row) { return (((row >> 1) & 1) | ((row >> 2) & 2)) << 1; }

template <bool GATHER, bool F32>
__global__ __launch_bounds__(512, 2) void gemm_weight_split_kernel(GemmWeightArgs a) {
  using S = SplitTile;
  __shared__ __align__(1024) uint8_t lds_mem[S::kLds];
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_byte*)lds_mem;
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const int ptiles = (a.K + S::kSide - 1) / S::kSide, qtiles = (a.N + S::kSide - 1) / S::kSide;
  const int group = blockIdx.x / (ptiles * qtiles), tile = blockIdx.x - group * (ptiles * qtiles);
  const int q0 = tile / ptiles * S::kSide, p0 = tile % ptiles * S::kSide;

  int64_t begin;
  int rows;
  group_range(a.g, group, &begin, &rows);
  begin = (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(begin >> 32))) << 32) |
          static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(begin)));
  rows = __builtin_amdgcn_readfirstlane(rows);
  if (rows == 0 && a.accumulate) return;

  const int64_t ldq = 2 * static_cast<int64_t>(a.N), ldp = 2 * static_cast<int64_t>(a.K);
  const uint8_t* qbase = reinterpret_cast<const uint8_t*>(a.q) + begin * ldq + 2 * static_cast<int64_t>(q0);
  const uint8_t* pbase = reinterpret_cast<const uint8_t*>(a.p) + (GATHER ? 0 : begin * ldp) + 2 * static_cast<int64_t>(p0);
  const uint32_t mine = lds + wave * 4 * S::kBytes;                  // [buffer][P, Q]
  int src[GATHER ? S::kLoads : 1];
  auto sources = [&](int step) MIEP_INLINE {
    if constexpr (GATHER) {
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i) {
        const int r = step * S::kRows + i * 8 + lane / 8;
        src[i] = r < rows ? a.row_index[begin + r] : -1;
      }
    }
  };
  auto issue = [&](int step, int buf) MIEP_INLINE {
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int row = i * 8 + lane / 8, r = step * S::kRows + row;
      int pc = ((lane & 7) ^ swz_t64(row)) * 16, qc = pc;
      if (p0 + pc / 2 >= a.K) pc = 0;
      if (q0 + qc / 2 >= a.N) qc = 0;
      bool in = r < rows;
      const uint8_t* p;
      if constexpr (GATHER) {                                         // a row without a source: zeros from both
        in = in && src[i] >= 0 && src[i] < a.p_rows;
        p = pbase + src[i] * ldp + pc;
      } else {
        p = pbase + r * ldp + pc;
      }
      const uint8_t* q = qbase + r * ldq + qc;
      dma16(in ? static_cast<const void*>(q) : static_cast<const void*>(g_zero16), mine + (2 * buf + 1) * S::kBytes + i * 1024);
      dma16(in ? static_cast<const void*>(p) : static_cast<const void*>(g_zero16), mine + 2 * buf * S::kBytes + i * 1024);
    }
  };

  f32x4 acc[S::kT][S::kT];
#pragma unroll
  for (int i = 0; i < S::kT; ++i)
#pragma unroll
    for (int j = 0; j < S::kT; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint32_t at[S::kT];
  {
    const int row = quarter * 8 + m / 4;
#pragma unroll
    for (int i = 0; i < S::kT; ++i) at[i] = row * 128 + ((i * 2 + (m & 3) / 2) ^ swz_t64(row)) * 16 + (m & 1) * 8;
  }
  auto operand = [&](uint32_t from) MIEP_INLINE {
    struct { i16x4 lo, hi; } t;
    t.lo = lds_read_tr(from);
    t.hi = lds_read_tr(from + 4 * 128);
    return __builtin_bit_cast(bf16x8, t);
  };

  const int nk = (rows + S::kRows - 1) / S::kRows;
  int buf = 0;
  if (wave < nk) {
    sources(wave);
    issue(wave, 0);
    sources(wave + S::kWaves);
  }
  for (int step = wave; step < nk; step += S::kWaves, buf ^= 1) {
    if (step + S::kWaves < nk) {
      issue(step + S::kWaves, buf ^ 1);
      sources(step + 2 * S::kWaves);
      // (gathered: the sources' own loads are behind these, so all have come when they are used)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * S::kLoads) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    bf16x8 pf[S::kT], qf[S::kT];
#pragma unroll
    for (int i = 0; i < S::kT; ++i) {
      pf[i] = operand(mine + 2 * buf * S::kBytes + at[i]);
      qf[i] = operand(mine + (2 * buf + 1) * S::kBytes + at[i]);
    }
#pragma unroll
    for (int i = 0; i < S::kT; ++i)
#pragma unroll
      for (int j = 0; j < S::kT; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(pf[i], qf[j], acc[i][j], 0, 0, 0);
    // the operands have left this buffer before the next turn loads into it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  all_read();
  float* sums = reinterpret_cast<float*>(lds_mem);
#pragma unroll
  for (int j = 0; j < S::kT; ++j)
#pragma unroll
    for (int i = 0; i < S::kT; ++i)
      *reinterpret_cast<f32x4*>(sums + wave * (S::kSums / 4) + (j * 16 + m) * S::kPitch + i * 16 + quarter * 4) = acc[i][j];
  __syncthreads();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int x = threadIdx.x + h * 512, n = x / 16, k = x % 16 * 4;
    f32x4 v = *reinterpret_cast<const f32x4*>(sums + n * S::kPitch + k);
#pragma unroll
    for (int w = 1; w < S::kWaves; ++w) {
      const f32x4 u = *reinterpret_cast<const f32x4*>(sums + w * (S::kSums / 4) + n * S::kPitch + k);
      v = f32x4{v[0] + u[0], v[1] + u[1], v[2] + u[2], v[3] + u[3]};
    }
    if (q0 + n >= a.N || p0 + k >= a.K) continue;
    const int64_t o = (static_cast<int64_t>(group) * a.N + q0 + n) * a.K + p0 + k;
    if constexpr (F32) {
      f32x4* to = reinterpret_cast<f32x4*>(static_cast<float*>(a.out) + o);
      if (a.accumulate) {
        const f32x4 old = *to;
        v = f32x4{old[0] + v[0], old[1] + v[1], old[2] + v[2], old[3] + v[3]};
      }
      *to = v;
    } else {
      *reinterpret_cast<v2u*>(static_cast<uint16_t*>(a.out) + o) = v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
  }
}

template <bool GATHER, bool F32, int BP, int BQ, int WP, int WQ, int NSP, int NSQ>
hipError_t launch_weight_tile(const GemmWeightArgs& a, hipStream_t st) {
  const int64_t per_group = static_cast<int64_t>((a.K + BP - 1) / BP) * ((a.N + BQ - 1) / BQ);
  const int64_t grid = per_group >= 64 ? (per_group + 7) / 8 * 8 * a.g.G : per_group * a.g.G;
  if (grid > max_blocks(WP * WQ * kWave) || grid > (1ll << 31) - 1) return hipErrorInvalidConfiguration;
  gemm_weight_kernel<GATHER, F32, BP, BQ, WP, WQ, NSP, NSQ><<<static_cast<unsigned>(grid), WP * WQ * kWave, 0, st>>>(a);
  return hipGetLastError();
}

template <bool GATHER, bool F32>
hipError_t launch_weight(const GemmWeightArgs& a, hipStream_t st) {
  auto tiles = [&](int64_t side) { return (a.K + side - 1) / side * ((a.N + side - 1) / side) * a.g.G; };
  // Splitting the rows: 8000 rows of 512 x 512 89 -> 35 us, of 1024 x 1024 92
  // -> 37; but of 2048 x 2048 103 -> 118, 8 groups of 1000 of 512 x 512 18.5
  // -> 20, and 500 rows of 512 x 512 the same 11.
  if (tiles(64) <= 256 && a.g.limit / a.g.G >= 512) {
    gemm_weight_split_kernel<GATHER, F32><<<static_cast<unsigned>(tiles(64)), 512, 0, st>>>(a);
    return hipGetLastError();
  }
  // 128 x 128 tiles, two at a time on a CU, or 256 x 256 ones, one at a time:
  // whose rounds are the shorter together, one of 128s taking 5/8 of one of 256s
  // (us in 128s / 256s: 2 groups of 2048 rows, 4096 x 2048, 75 / 63; one of 4096
  // rows 69 / 95; 4 of 2000, 1408 x 2048, 66 / 54; 8 of 500, 2048 x 1408, 42 / 46).
  if ((tiles(128) + 511) / 512 * 5 < (tiles(256) + 255) / 256 * 8)
    return launch_weight_tile<GATHER, F32, 128, 128, 2, 2, 2, 2>(a, st);
  return launch_weight_tile<GATHER, F32, 256, 256, 2, 4, GATHER ? 2 : 3, 2>(a, st);
}

hipError_t launch_gemm_weight(const GemmWeightArgs& a, hipStream_t st) {
  if (a.g.G == 0) return hipSuccess;
  if (a.row_index) return a.out_f32 ? launch_weight<true, true>(a, st) : launch_weight<true, false>(a, st);
  return a.out_f32 ? launch_weight<false, true>(a, st) : launch_weight<false, false>(a, st);
}

}  // namespace miep
