// gemm_rows.h -- the rows kernel of the grouped products (forward, and the
// rows' gradient), instantiated for bf16 in gemm.hip and for E4M3 in
// gemm_fp8.hip.
//
//   out[i][p] = sum_c Q[src(i)][c] * P_g[p][c]        for the rows i of group g
//
// A workgroup computes BQ rows x BP output channels.  Each 128-byte step of
// the contraction comes to LDS by asynchronous 16-byte loads, several buffers deep,
// with one barrier a step; wavefront (wp, wq) multiplies its BP/WP x BQ/WQ part
// with 16x16 MFMAs.  16384 rows over 4 even groups of 4096 x 7168: bf16 726 us,
// 1,325 TFLOP/s at 1.9 GHz (a library's large product reaches 1,450), E4M3 463
// us, 2,080 TFLOP/s, with power-of-two scales 405 us, 2,370 (library 3,180).  A
// few rows a group: bound by the weights' bytes (8 x 4096 x 7168: bf16 79 us,
// 6.0 TB/s; E4M3 42 us, 5.6 TB/s, and 34 us where the last-level cache still
// holds part of the same weights from the call before).
#pragma once

#include <cmath>
#include <type_traits>

#include "gemm.h"
#include "gemm_epilogue.h"
#include "gemm_rows_split.h"

namespace miep {

template <int EL, bool PT, bool GATHER, int BP, int BQ, int WP, int WQ, int NSP, int NSQ>
struct RowsTile {
  static constexpr int kWaves = WP * WQ;
  static constexpr int kTP = BP / WP / 16, kTQ = BQ / WQ / 16;       // 16 x 16 results a wavefront
  static constexpr bool kFp8 = EL != kGemmBf16;
  static constexpr int kEB = kFp8 ? 1 : 2;                           // bytes of an element
  static constexpr int kPBytes = BP * kStepBytes, kQBytes = BQ * kStepBytes;
  // FP8 scales of a stage, a dword each: the rows' (BQ, at least one load's
  // 64), then the P blocks' (one load; a tile has at most 2)
  static constexpr int kQScales = BQ < kWave ? kWave : BQ;
  static constexpr int kScaleBytes = kFp8 ? kQScales * 4 + 256 : 0;
  static_assert(!kFp8 || kQScales / kWave < kWaves, "one scale load a wavefront");
  static constexpr int kQStage = kQBytes + kScaleBytes;
  static constexpr int kLds = NSP * kPBytes + NSQ * kQStage;
  static constexpr int kPLoads = kPBytes / 1024 / kWaves;            // a wavefront's loads of a step
  static constexpr int kQLoads = kQBytes / 1024 / kWaves + (kFp8 ? 1 : 0);
  // Few results a wavefront (so registers to spare) and equally deep buffers:
  // a whole step's operands are read a step ahead.
  static constexpr bool kShort = kTP <= 4;
  // Loads that may be in flight behind the tile that a barrier publishes (see
  // `publish`): the buffers that are deeper than the two of every tile.
  static constexpr int kBehind = (NSP > NSQ ? NSQ - 1 : NSQ - 2) * kPLoads + (NSQ - 2) * kQLoads;
  static_assert(!kShort || NSP == NSQ, "short steps load both operands at once");
  static_assert(kPLoads * kWaves * 1024 == kPBytes && kQBytes % (kWaves * 1024) == 0, "whole loads a wavefront");
  static_assert(kTP % 2 == 0 && kTQ >= 1 && NSQ >= 2 && NSP >= NSQ && kLds <= 163840, "tile shape");
  static_assert(kBehind + kPLoads + kQLoads < 64, "loads in flight");
  static_assert(!(PT && kFp8), "the transposed operand is bf16");
};

// Swizzle: the 16-byte chunk c of a tile row is kept at chunk c ^ s(row), so
// that the 16 consecutive rows of one operand read lie in 16 different 16-byte
// places of the 256-byte LDS line (rows are 128 bytes: their parity is one bit
// of the place, s the other three).
__device__ __forceinline__ int swz(int row) { return (row >> 1) & 7; }

// One workgroup's tiles, of `total`; its LDS from `lds` on (kLds bytes).  EPI:
// what happens to the results (gemm_epilogue.h).
template <int EL, bool PT, bool GATHER, int BP, int BQ, int WP, int WQ, int NSP, int NSQ, int EPI>
__device__ __forceinline__ void rows_tiles(const GemmRowsArgs& a, int total, uint32_t lds) {
  using S = RowsTile<EL, PT, GATHER, BP, BQ, WP, WQ, NSP, NSQ>;
  constexpr int TP = S::kTP, TQ = S::kTQ, EB = S::kEB;

  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  // consecutive wavefronts share their rows of Q, so that the wavefronts a
  // short tile leaves idle are spread evenly over the four SIMDs
  const int wp = wave % WP, wq = wave / WP;
  const int m = lane & 15, quarter = lane >> 4;

  const int NO = a.NO, C = a.C;
  const int ntiles = (NO + BP - 1) / BP;
  const int64_t ldq = static_cast<int64_t>(C) * EB;                   // bytes
  const int64_t ldp = static_cast<int64_t>(PT ? NO : C) * EB;
  const int cbytes = C * EB;                                          // contraction, bytes of a k-major row
  const int KE = kStepBytes / EB;
  const int nk = (C + KE - 1) / KE;
  const bool ragged_end = C % KE != 0;
  const int64_t kb = C / kFp8Group;                                       // scale blocks of a row (FP8)

  // Workgroups go to the 8 XCDs in turn: XCD x walks the x-th eighth of the
  // tiles, so tiles that share weights or rows meet in one L2.  (The groups'
  // last, short tiles stay among the others: all at the end, they fill up the
  // last round but read their weights again, 32 groups of 300 rows, 4096 x 2048
  // 193 -> 183 us, of about 400 252 -> 225.)
  const int xcd = blockIdx.x & 7, stride = gridDim.x >> 3;
  const int end = static_cast<int>(static_cast<int64_t>(total) * (xcd + 1) / 8);
  int turn = static_cast<int>(static_cast<int64_t>(total) * xcd / 8) + (blockIdx.x >> 3);
  auto next_tile = [&]() MIEP_INLINE {
    TileAt r;
    r.group = -1;
    if (turn < end) r = find_tile(a.g, BQ, ntiles, turn);
    turn += stride;
    return r;
  };

  // The tile that is being loaded and multiplied; the previous one's results
  // are stored while its first loads are under way.
  int p0, live;
  int64_t row0;
  const uint8_t *pg, *pbase, *qbase;
  uint32_t poff[S::kPLoads];
  constexpr int QL = S::kQBytes / 1024 / S::kWaves;
  uint32_t qoff[QL];
  uint32_t lost;                                                      // bit i: load i's row has no source
  uint32_t none = 0;                                                  // bit j: nor has this lane's row of results j
  constexpr int SB = EL == kGemmFp8 ? 4 : 1;                          // bytes of an FP8 scale
  const uint8_t* sptr;
  uint32_t sto;
  auto set_tile = [&](const TileAt& at) MIEP_INLINE {
    // bands of kBand row tiles, in a band the row tiles of one column of tiles
    // after the other: the 32 tiles that an XCD works on at a time share 8
    // tiles of rows and 4 of weights
    constexpr int kBand = 8;
    const int mtiles = max(row_tiles(at.rows, BQ), 1);
    const int first = min(max(at.first, 0), mtiles * ntiles - 1);
    const int band = first / (kBand * ntiles), in_band = first - band * (kBand * ntiles);
    const int bh = min(kBand, mtiles - band * kBand);
    const int pt = in_band / bh, qt = band * kBand + in_band - pt * bh;
    const int q0 = qt * BQ;
    p0 = pt * BP;
    live = min(BQ, at.rows - q0);                                     // rows of this tile
    row0 = at.begin + q0;
    pg = static_cast<const uint8_t*>(a.p) + static_cast<int64_t>(at.group) * NO * C * EB;

    // Sources of this lane's 16 bytes of every load of a stage.
    pbase = pg + (PT ? static_cast<int64_t>(p0) * EB : static_cast<int64_t>(EPI == kEpiSwiglu ? p0 / 2 : p0) * ldp);
#pragma unroll
    for (int i = 0; i < S::kPLoads; ++i) {
      const int l = i * S::kWaves + wave;
      if constexpr (PT) {
        constexpr int CH = BP * 2 / 16;                               // chunks of a tile row
        const int row = l * (64 / CH) + lane / CH;
        int col = ((lane % CH) ^ swz_t(row)) * 16;
        if (p0 + col / 2 >= NO) col = 0;
        poff[i] = static_cast<uint32_t>(row * ldp + col);
      } else {
        int row = l * 8 + lane / 8;
        const int c = (lane & 7) ^ swz(row);
        if constexpr (EPI == kEpiSwiglu) row = swiglu_row(p0, row, NO);
        else if (p0 + row >= NO) row = NO - 1 - p0;
        poff[i] = static_cast<uint32_t>(row * ldp + c * 16);
      }
    }
    // Q's rows: at a fixed stride, or anywhere in the gathered source (its
    // offsets in 16-byte units, so that 32 bits reach 64 GiB).  A row without
    // a source reads row 0 of the weights, and stores zeros.
    qbase = static_cast<const uint8_t*>(a.q) + (GATHER ? 0 : row0 * ldq);
    if constexpr (GATHER) {
      none = 0;
#pragma unroll
      for (int j = 0; j < TQ; ++j) {
        const int src = a.row_index[row0 + min((wq * TQ + j) * 16 + m, live - 1)];
        if (src < 0 || src >= a.q_rows) none |= 1u << j;
      }
    }
    lost = 0;
#pragma unroll
    for (int i = 0; i < QL; ++i) {
      int row = (i * S::kWaves + wave) * 8 + lane / 8;
      const int c = (lane & 7) ^ swz(row);
      row = min(row, live - 1);
      if constexpr (GATHER) {
        const int64_t src = a.row_index[row0 + row];
        const bool ok = src >= 0 && src < a.q_rows;
        qoff[i] = static_cast<uint32_t>((ok ? src * ldq / 16 : 0) + c);
        if (!ok) lost |= 1u << i;
      } else {
        qoff[i] = static_cast<uint32_t>(row * ldq + c * 16);
      }
    }
    // FP8: this wavefront's one load of a stage's scales -- 64 rows of Q's, or
    // the P blocks' (every further wavefront repeats those)
    if constexpr (S::kFp8) {
      constexpr int SL = S::kQScales / kWave;
      const int64_t pb = static_cast<int64_t>(at.group) * ((NO + 127) / 128);
      const uint8_t* ps = static_cast<const uint8_t*>(a.p_scales) + pb * kb * SB;
      if (wave < SL) {
        int64_t src = row0 + min((wave * kWave + lane) % BQ, live - 1);
        if constexpr (GATHER) {
          src = a.row_index[src];
          if (src >= a.q_rows) src = -1;
        }
        sptr = src >= 0 ? static_cast<const uint8_t*>(a.q_scales) + src * kb * SB : ps;
      } else {
        sptr = ps + static_cast<int64_t>(min(p0 / 128 + lane, (NO - 1) / 128)) * kb * SB;
      }
      sto = S::kQBytes + min(wave, SL) * 256;
    }

  };

    auto p_at = [&](int buf) MIEP_INLINE { return lds + buf * S::kPBytes; };
    auto q_at = [&](int buf) MIEP_INLINE { return lds + NSP * S::kPBytes + buf * S::kQStage; };
    // Load i of this wavefront's loads of a step of 128 whole bytes.
    auto load_p = [&](int i, int step, int buf) MIEP_INLINE {
      dma16s(pbase + static_cast<int64_t>(step) * (PT ? (kStepBytes / 2) * ldp : kStepBytes), poff[i],
             p_at(buf) + (i * S::kWaves + wave) * 1024);
    };
    auto load_q = [&](int i, int step, int buf) MIEP_INLINE {
      if (i < QL) {
        const uint32_t to = q_at(buf) + (i * S::kWaves + wave) * 1024;
        if constexpr (GATHER) {
          const uint8_t* base = (lost >> i) & 1 ? pg : qbase;
          dma16(base + static_cast<int64_t>(step) * kStepBytes + (static_cast<uint64_t>(qoff[i]) << 4), to);
        } else {
          dma16s(qbase + static_cast<int64_t>(step) * kStepBytes, qoff[i], to);
        }
      } else if constexpr (S::kFp8) {
        if constexpr (SB == 4) dma4(sptr + static_cast<int64_t>(step) * 4, q_at(buf) + sto);
        else dma1(sptr + step, q_at(buf) + sto);
      }
    };
    // All of a step's loads, if there is such a step; the last step of a
    // contraction that is not whole reads zeros behind its end.  (Its lane
    // constants are computed anew: kept through the loop they would cost it
    // registers.)
    auto issue_p = [&](int step, int buf) MIEP_INLINE {
      if (step >= nk) return;
      if (S::kFp8 || !ragged_end || step != nk - 1) {
#pragma unroll
        for (int i = 0; i < S::kPLoads; ++i) load_p(i, step, buf);
        return;
      }
      int ln = lane;
      asm volatile("" : "+v"(ln));
      const uint8_t* pb = pbase + static_cast<int64_t>(step) * (PT ? (kStepBytes / 2) * ldp : kStepBytes);
#pragma unroll
      for (int i = 0; i < S::kPLoads; ++i) {
        const int l = i * S::kWaves + wave;
        bool in;
        if constexpr (PT) in = step * KE + l * (64 / (BP * 2 / 16)) + ln / (BP * 2 / 16) < C;
        else in = step * kStepBytes + ((ln & 7) ^ swz(l * 8 + ln / 8)) * 16 < cbytes;
        dma16(in ? static_cast<const void*>(pb + poff[i]) : static_cast<const void*>(g_zero16), p_at(buf) + l * 1024);
      }
    };
    auto issue_q = [&](int step, int buf) MIEP_INLINE {
      if (step >= nk) return;
      if (S::kFp8 || !ragged_end || step != nk - 1) {
#pragma unroll
        for (int i = 0; i < S::kQLoads; ++i) load_q(i, step, buf);
        return;
      }
      int ln = lane;
      asm volatile("" : "+v"(ln));
#pragma unroll
      for (int q = 0; q < QL; ++q) {
        const int l = q * S::kWaves + wave;
        const bool in = step * kStepBytes + ((ln & 7) ^ swz(l * 8 + ln / 8)) * 16 < cbytes;
        const uint8_t* src;
        if constexpr (GATHER) src = ((lost >> q) & 1 ? pg : qbase) + (static_cast<uint64_t>(qoff[q]) << 4);
        else src = qbase + qoff[q];
        dma16(in ? static_cast<const void*>(src + static_cast<int64_t>(step) * kStepBytes) : static_cast<const void*>(g_zero16),
              q_at(buf) + l * 1024);
      }
    };

    // lane addresses of the operand reads, within a buffer
    uint32_t pa[PT ? TP : 2], qa[2];
    if constexpr (PT) {
#pragma unroll
      for (int i = 0; i < TP; ++i) {
        const int row = quarter * 8 + m / 4;
        const int ch = wp * 2 * TP + i * 2 + (m & 3) / 2;
        pa[i] = row * (2 * BP) + (ch ^ swz_t(row)) * 16 + (m & 1) * 8;
      }
    } else {
      const int row = wp * 16 * TP + m;
      pa[0] = row * kStepBytes + (quarter ^ swz(row)) * 16;
      pa[1] = pa[0] ^ 64;
    }
    {
      const int row = wq * 16 * TQ + m;
      qa[0] = row * kStepBytes + (quarter ^ swz(row)) * 16;
      qa[1] = qa[0] ^ 64;
    }

    // P's buffers may be deeper than Q's: the weights stream from memory, the
    // rows mostly come from L2.  Step t issues the loads of P's step t - 1 +
    // NSP, spread over its MFMAs, and behind its barrier those of Q's step t +
    // NSQ; before the first step come those that steps before it would have
    // issued, in that order.  (Short steps issue both behind the barrier, P's
    // of step t + NSP.)
    auto issue_first = [&]() MIEP_INLINE {
#pragma unroll
      for (int t = -NSP; t < 0; ++t) {
        if constexpr (S::kShort) issue_p(t + NSP, t + NSP);
        else if (t - 1 + NSP >= 0) issue_p(t - 1 + NSP, t - 1 + NSP);
        if (t + NSQ >= 0) issue_q(t + NSQ, t + NSQ);
      }
    };

    f32x4 acc[TP][TQ];
    // A whole tile's results leave in exactly kStores stores a wavefront behind
    // the next tile's first loads; the waits for those let the stores be (16384
    // rows of 7168 x 2048: 408 -> 394 us, of 4096 x 7168, ragged: 956 -> 924).
    constexpr int kStores = TP / 2 * TQ;
    bool stored = false;
    TileAt at = next_tile();
    if (at.group < 0) return;
    set_tile(at);
    issue_first();
    while (true) {
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    const bool busy = wq * 16 * TQ < live;
    at = next_tile();
    constexpr int kFirst = S::kBehind + S::kQLoads + (S::kShort ? S::kPLoads : 0);
    if (nk < NSP) wait_tiles<0>();
    else if (stored) wait_tiles<kFirst + kStores>();
    else wait_tiles<kFirst>();
    // The barrier of a step: the next step's tile has come (while the loads
    // behind it may be in flight; at the contraction's end there are fewer),
    // and every wavefront has read this step's.
    auto publish = [&](int step) MIEP_INLINE {
      // (step 0: the next step's loads are older than the stores, but for long
      // steps with equally deep buffers)
      if ((S::kShort || NSP > NSQ) && step == 0 && stored && NSP <= nk) wait_tiles<S::kBehind + kStores>();
      else if (step - 1 + NSP < nk) wait_tiles<S::kBehind>();
      else wait_tiles<0>();
    };
    int step = 0, pbuf = 0, qbuf = 0;
    auto before = [&](int buf) MIEP_INLINE { return buf == 0 ? NSP - 1 : buf - 1; };
    auto next_buffers = [&]() MIEP_INLINE {
      pbuf = pbuf == NSP - 1 ? 0 : pbuf + 1;
      qbuf = qbuf == NSQ - 1 ? 0 : qbuf + 1;
    };
    if (!busy) {
      for (; step + 1 < nk; ++step) {
        if constexpr (!S::kShort) issue_p(step - 1 + NSP, before(pbuf));
        publish(step);
        if constexpr (S::kShort) issue_p(step + NSP, pbuf);
        issue_q(step + NSQ, qbuf);
        next_buffers();
      }
    } else if constexpr (S::kShort) {
      // All operands of a step (32 bytes a lane each: 64 bf16 channels in two
      // halves, or 128 E4M3) are in registers when it begins; its barrier comes
      // first, and the next step's operands are read under its MFMAs, into
      // the other of two sets.
      i32x8 pf[2][TP], qf[2][TQ];
      float s[2][TQ];
      int e[2][TQ], ep[2] = {0, 0};
      auto read_p = [&](int set, int i, uint32_t at) MIEP_INLINE {
        if constexpr (PT) {
          struct { i16x4 v[4]; } t;
#pragma unroll
          for (int r = 0; r < 4; ++r) t.v[r] = lds_read_tr(at + pa[i] + (r / 2 * 32 + r % 2 * 4) * 2 * BP);
          pf[set][i] = __builtin_bit_cast(i32x8, t);
        } else {
          struct { i32x4 lo, hi; } t;
          t.lo = lds_read<i32x4>(at + pa[0] + i * 16 * kStepBytes);
          t.hi = lds_read<i32x4>(at + pa[1] + i * 16 * kStepBytes);
          pf[set][i] = __builtin_bit_cast(i32x8, t);
        }
      };
      auto read_q = [&](int set, int j, uint32_t at) MIEP_INLINE {
        struct { i32x4 lo, hi; } t;
        t.lo = lds_read<i32x4>(at + qa[0] + j * 16 * kStepBytes);
        t.hi = lds_read<i32x4>(at + qa[1] + j * 16 * kStepBytes);
        qf[set][j] = __builtin_bit_cast(i32x8, t);
      };
      auto read_scales = [&](int set, uint32_t at) MIEP_INLINE {
        const uint32_t psat = at + S::kQBytes + S::kQScales * 4 + wp * 16 * TP / 128 * 4;
        if constexpr (EL == kGemmFp8) {
          const float sp = lds_read<float>(psat);
#pragma unroll
          for (int j = 0; j < TQ; ++j) s[set][j] = sp * lds_read<float>(at + S::kQBytes + ((wq * TQ + j) * 16 + m) * 4);
        } else if constexpr (S::kFp8) {
          ep[set] = lds_read<int>(psat);
#pragma unroll
          for (int j = 0; j < TQ; ++j) e[set][j] = lds_read<int>(at + S::kQBytes + ((wq * TQ + j) * 16 + m) * 4);
        }
      };
#pragma unroll
      for (int j = 0; j < TQ; ++j) read_q(0, j, q_at(0));
#pragma unroll
      for (int i = 0; i < TP; ++i) read_p(0, i, p_at(0));
      read_scales(0, q_at(0));
      const int whole = nk - (ragged_end ? 1 : 0);                    // steps of 128 whole bytes
      auto body = [&](auto parity, auto more, auto last) MIEP_INLINE {
        constexpr int now = parity, then = 1 - parity;
        const int pb = pbuf, qb = qbuf;
        if constexpr (!last) publish(step);
        if constexpr (!more && !last) {
          issue_p(step + NSP, pb);
          issue_q(step + NSQ, qb);
        }
        next_buffers();
#pragma unroll
        for (int i = 0; i < TP; ++i) {
          if constexpr (!last) {
            if (i == 0) read_scales(then, q_at(qbuf));
#pragma unroll
            for (int j = i * TQ / TP; j < (i + 1) * TQ / TP; ++j) read_q(then, j, q_at(qbuf));
            read_p(then, i, p_at(pbuf));
          }
          if constexpr (more) {
            constexpr int all = S::kPLoads + S::kQLoads;
#pragma unroll
            for (int l = i * all / TP; l < (i + 1) * all / TP; ++l) {
              if (l < S::kQLoads) load_q(l, step + NSQ, qb);
              else load_p(l - S::kQLoads, step + NSP, pb);
            }
          }
#pragma unroll
          for (int j = 0; j < TQ; ++j) {
            if constexpr (EL == kGemmBf16) {
              struct operand { bf16x8 lo, hi; };
              const operand p = __builtin_bit_cast(operand, pf[now][i]), q = __builtin_bit_cast(operand, qf[now][j]);
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p.lo, q.lo, acc[i][j], 0, 0, 0);
              acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p.hi, q.hi, acc[i][j], 0, 0, 0);
            } else if constexpr (EL == kGemmFp8) {
              const f32x4 z = {0.f, 0.f, 0.f, 0.f};
              const f32x4 d = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[now][i], qf[now][j], z, 0, 0, 0, 0, 0, 0);
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[r], s[now][j], acc[i][j][r]);
            } else {
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[now][i], qf[now][j], acc[i][j], 0, 0, 0, ep[now], 0, e[now][j]);
            }
          }
#pragma unroll
          for (int j = 0; j < TQ; ++j) pin(acc[i][j]);
          __builtin_amdgcn_sched_barrier(0);
        }
        ++step;
      };
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      constexpr std::integral_constant<int, 0> even{};
      constexpr std::integral_constant<int, 1> odd{};
      while (step + 1 + NSP < whole) {
        body(even, yes, no);
        body(odd, yes, no);
      }
      while (step + 2 < nk) {
        body(even, no, no);
        body(odd, no, no);
      }
      if (step + 1 < nk) {
        body(even, no, no);
        body(odd, no, yes);
      } else {
        body(even, no, yes);
      }
    } else if constexpr (!S::kFp8) {
      // A step is 2 * TP slots: slot k multiplies P's operand k % TP of the
      // half k / TP (32 channels) with the half's TQ operands of Q.  Operands
      // come from LDS D slots ahead of their use, P's through a ring of four.
      // The barrier lies D slots before the step's end: behind it every
      // wavefront holds the last operands of this step's buffers, and the next
      // step's first operands are read under the last MFMAs.
      constexpr int SLOTS = 2 * TP, D = TP < 3 ? TP : 3, RING = 4;
      static_assert(SLOTS % RING == 0 && D < RING && D <= TP, "operand ring");
      bf16x8 pf[RING], qf[2][TQ];
      auto read_q = [&](int h, uint32_t at, int j) MIEP_INLINE { qf[h][j] = lds_read<bf16x8>(at + qa[h] + j * 16 * kStepBytes); };
      auto read_p = [&](int k, uint32_t at) MIEP_INLINE {
        const int h = k / TP, i = k % TP;
        if constexpr (PT) {
          struct { i16x4 lo, hi; } t;
          t.lo = lds_read_tr(at + pa[i] + h * 32 * 2 * BP);
          t.hi = lds_read_tr(at + pa[i] + (h * 32 + 4) * 2 * BP);
          pf[k % RING] = __builtin_bit_cast(bf16x8, t);
        } else {
          pf[k % RING] = lds_read<bf16x8>(at + pa[h] + i * 16 * kStepBytes);
        }
      };
#pragma unroll
      for (int j = 0; j < TQ; ++j) read_q(0, q_at(0), j);
#pragma unroll
      for (int k = 0; k < D; ++k) read_p(k, p_at(0));
      auto body = [&](auto more, auto last) MIEP_INLINE {
        const int pb = pbuf, qb = qbuf;
        next_buffers();
        if constexpr (!more) issue_p(step - 1 + NSP, before(pb));
#pragma unroll
        for (int k = 0; k < SLOTS; ++k) {
          const int late = k - (SLOTS - D);                           // slots behind the barrier
          if constexpr (!last)
            if (late == 0) publish(step);
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
      const int whole = nk - (ragged_end ? 1 : 0);                    // steps of 128 whole bytes
      constexpr int ahead = NSP - 1 > NSQ ? NSP - 1 : NSQ;
      for (; step + ahead < whole; ++step) body(yes, no);
      for (; step + 1 < nk; ++step) body(no, no);
      body(no, yes);
    } else {
      // A step is TP slots: slot i multiplies P's operand i (128 channels, 32
      // bytes a lane) with all of Q's.  P's operands come a slot ahead through
      // a ring of two; Q's are held over the step and each replaced by the
      // next step's behind its last use, so the barrier lies before the last
      // slot.  fp32 scales multiply each block's sum into the result in fp32
      // (the MFMAs start from zero); power-of-two scales go into the MFMAs as
      // their exponent bytes, and the running sum through them.  What the MFMAs
      // keep of their products is said in gemm.h.
      i32x8 pf[2], qf[TQ];
      float s[TQ];
      int e[TQ], ep = 0;
      auto operand = [&](uint32_t at0, uint32_t at1) MIEP_INLINE {
        struct { i32x4 lo, hi; } t;
        t.lo = lds_read<i32x4>(at0);
        t.hi = lds_read<i32x4>(at1);
        return __builtin_bit_cast(i32x8, t);
      };
      auto read_p = [&](int i, uint32_t at) MIEP_INLINE {
        pf[i & 1] = operand(at + pa[0] + i * 16 * kStepBytes, at + pa[1] + i * 16 * kStepBytes);
      };
      auto read_q = [&](int j, uint32_t at) MIEP_INLINE {
        qf[j] = operand(at + qa[0] + j * 16 * kStepBytes, at + qa[1] + j * 16 * kStepBytes);
      };
      const uint32_t psat = S::kQBytes + S::kQScales * 4 + wp * 16 * TP / 128 * 4;
      auto read_scales = [&](uint32_t at) MIEP_INLINE {
        if constexpr (EL == kGemmFp8) {
          const float sp = lds_read<float>(at + psat);
#pragma unroll
          for (int j = 0; j < TQ; ++j) s[j] = sp * lds_read<float>(at + S::kQBytes + ((wq * TQ + j) * 16 + m) * 4);
        } else {
          ep = lds_read<int>(at + psat);
#pragma unroll
          for (int j = 0; j < TQ; ++j) e[j] = lds_read<int>(at + S::kQBytes + ((wq * TQ + j) * 16 + m) * 4);
        }
      };
#pragma unroll
      for (int j = 0; j < TQ; ++j) read_q(j, q_at(0));
      read_p(0, p_at(0));
      read_scales(q_at(0));
      auto body = [&](auto more, auto last) MIEP_INLINE {
        const int pb = pbuf, qb = qbuf;
        next_buffers();
        if constexpr (!more) issue_p(step - 1 + NSP, before(pb));
#pragma unroll
        for (int i = 0; i < TP; ++i) {
          const bool end = i == TP - 1;
          if constexpr (!last)
            if (end) publish(step);
          if (!end) read_p(i + 1, p_at(pb));
          else if constexpr (!last) read_p(0, p_at(pbuf));
          if constexpr (more) {
            if (end) {
#pragma unroll
              for (int l = 0; l < S::kQLoads; ++l) load_q(l, step + NSQ, qb);
            } else {
#pragma unroll
              for (int l = 0; l < S::kPLoads; ++l)
                if (i == (l / 2 < TP - 2 ? l / 2 : TP - 2)) load_p(l, step - 1 + NSP, before(pb));
            }
          }
          f32x4 d[TQ];
#pragma unroll
          for (int j = 0; j < TQ; ++j) {
            if constexpr (EL == kGemmFp8) {
              const f32x4 z = {0.f, 0.f, 0.f, 0.f};
              d[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[i & 1], qf[j], z, 0, 0, 0, 0, 0, 0);
            } else {
              acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(pf[i & 1], qf[j], acc[i][j], 0, 0, 0, ep, 0, e[j]);
            }
            if constexpr (!last) {
              if (end) {
                __builtin_amdgcn_sched_barrier(0);
                read_q(j, q_at(qbuf));
              }
            }
          }
          if constexpr (EL == kGemmFp8) {
#pragma unroll
            for (int j = 0; j < TQ; ++j)
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[j][r], s[j], acc[i][j][r]);
          }
#pragma unroll
          for (int j = 0; j < TQ; ++j) pin(acc[i][j]);
          if constexpr (!last)
            if (end) read_scales(q_at(qbuf));
          __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (!more && !last) issue_q(step + NSQ, qb);
      };
      constexpr std::true_type yes{};
      constexpr std::false_type no{};
      constexpr int ahead = NSP - 1 > NSQ ? NSP - 1 : NSQ;
      for (; step + ahead < nk; ++step) body(yes, no);
      for (; step + 1 < nk; ++step) body(no, no);
      body(no, yes);
    }

    const int out_p0 = p0, out_live = live;
    const int64_t out_row0 = row0;
    const uint32_t out_none = none;
    if (at.group >= 0) {
      all_read();                                                     // this tile's last buffers
      set_tile(at);
      issue_first();
    }
    auto result = [&](int j, int i) MIEP_INLINE {                     // lanes exchange: not under a lane's own condition
      const v4u v = pack_pair(acc[i][j], acc[i + 1][j]);
      return GATHER && (out_none >> j & 1) ? v4u{0u, 0u, 0u, 0u} : v;
    };
    stored = EPI == kEpiNone && out_live == BQ && out_p0 + BP <= NO;
    if constexpr (EPI != kEpiNone) {
      if (busy) epilogue_tile<EPI>(a.epi, a.out, NO, out_row0 + wq * 16 * TQ, out_live - wq * 16 * TQ, out_p0 + wp * 16 * TP, acc);
    } else if (stored) {
#pragma unroll
      for (int j = 0; j < TQ; ++j) {
        uint16_t* o = a.out + (out_row0 + (wq * TQ + j) * 16 + m) * NO + out_p0 + (wp * TP + (quarter & 1)) * 16 + (quarter >> 1) * 8;
#pragma unroll
        for (int i = 0; i < TP; i += 2) store16(o + i * 16, result(j, i));
      }
    } else if (busy) {
#pragma unroll
      for (int j = 0; j < TQ; ++j) {
        const int row = (wq * TQ + j) * 16 + m;
        if (row >= out_live) continue;
        uint16_t* o = a.out + (out_row0 + row) * NO;
#pragma unroll
        for (int i = 0; i < TP; i += 2) {
          const int p = out_p0 + (wp * TP + i + (quarter & 1)) * 16 + (quarter >> 1) * 8;
          const v4u v = result(j, i);
          if (p < NO) *reinterpret_cast<v4u*>(o + p) = v;
        }
      }
    }
    if (at.group < 0) return;
  }
}

template <int EL, bool PT, bool GATHER, int BP, int BQ, int WP, int WQ, int NSP, int NSQ, int EPI>
__global__ __launch_bounds__(WP * WQ * kWave, 2) void gemm_rows_kernel(GemmRowsArgs a) {
  __shared__ __align__(1024) uint8_t lds_mem[RowsTile<EL, PT, GATHER, BP, BQ, WP, WQ, NSP, NSQ>::kLds];
  rows_tiles<EL, PT, GATHER, BP, BQ, WP, WQ, NSP, NSQ, EPI>(a, count_tiles(a.g, BQ, (a.NO + BP - 1) / BP),
                                                       (uint32_t)(uintptr_t)(lds_byte*)lds_mem);
}

// Tiles of 256 channels, of 192 or 256 rows by what the groups hold: the one
// whose rounds of one tile a workgroup are the shorter together, a tile of 192
// taking 5/6 of the time of one of 256 (both by measurement: 46 and 56 us of
// 4096 x 2048, 151 and 190 of 7168 x 2048's gradient).  32 groups, bf16: of 256
// rows each 218 us in 256s and 321 in 192s (gradient of 7168 x 2048); of 300
// rows 224 and 183 (4096 x 2048).
template <int EL, bool PT, bool GATHER, int EPI>
__global__ __launch_bounds__(8 * kWave, 2) void gemm_rows_wide_kernel(GemmRowsArgs a) {
  constexpr int NSP = EL == kGemmBf16 ? 3 : 2;
  constexpr int kLds192 = RowsTile<EL, PT, GATHER, 256, 192, 2, 4, 3, 2>::kLds;
  constexpr int kLds256 = RowsTile<EL, PT, GATHER, 256, 256, 2, 4, NSP, 2>::kLds;
  __shared__ __align__(1024) uint8_t lds_mem[kLds192 > kLds256 ? kLds192 : kLds256];
  const uint32_t lds = (uint32_t)(uintptr_t)(lds_byte*)lds_mem;
  const int ntiles = (a.NO + 255) / 256;
  const int t192 = count_tiles(a.g, 192, ntiles), t256 = count_tiles(a.g, 256, ntiles);
  const int64_t grid = gridDim.x;
  if ((t192 + grid - 1) / grid * 5 < (t256 + grid - 1) / grid * 6)
    rows_tiles<EL, PT, GATHER, 256, 192, 2, 4, 3, 2, EPI>(a, t192, lds);
  else
    rows_tiles<EL, PT, GATHER, 256, 256, 2, 4, NSP, 2, EPI>(a, t256, lds);
}

template <int EL, bool PT, bool GATHER, int BP, int BQ, int WP, int WQ, int NSP, int NSQ, int EPI = kEpiNone>
hipError_t launch_rows_tile(const GemmRowsArgs& a, hipStream_t st) {
  const int64_t per = (a.NO + BP - 1) / BP;
  const int64_t most = ((a.g.limit + BQ - 1) / BQ + a.g.G) * per;     // disjoint groups have no more tiles
  int per_cu = 0;
  // resident workgroups: by LDS (160 KiB a CU) and two wavefronts a SIMD
  per_cu = 163840 / RowsTile<EL, PT, GATHER, BP, BQ, WP, WQ, NSP, NSQ>::kLds;
  const int by_waves = 8 / (WP * WQ);
  per_cu = per_cu < by_waves ? per_cu : by_waves;
  int64_t grid = 256ll * (per_cu > 0 ? per_cu : 1);
  if (grid > (most + 7) / 8 * 8) grid = (most + 7) / 8 * 8;
  gemm_rows_kernel<EL, PT, GATHER, BP, BQ, WP, WQ, NSP, NSQ, EPI><<<static_cast<unsigned>(grid), WP * WQ * kWave, 0, st>>>(a);
  return hipGetLastError();
}

template <int EL, bool PT, bool GATHER>
hipError_t launch_rows(const GemmRowsArgs& a, hipStream_t st) {
  constexpr bool F8 = EL != kGemmBf16;
  // Few tiles over a long contraction: split it (bf16, us against the tiles
  // below: 16 rows of 1 x 4096 x 7168 28 -> 15, 100 rows of 1 x 256 x 7168 46 ->
  // 13, 16 rows of 2 x 4096 x 7168 28 -> 22; of 4 x 4096 x 7168 37 -> 38, and
  // 16 steps only, 100 rows of 1 x 256 x 1024, 13 -> 14.5).
  const int64_t tiles32 = a.g.G * ((static_cast<int64_t>(a.expected) + 31) / 32) * ((a.NO + 31) / 32);
  if (tiles32 <= 256 && a.C / (F8 ? 128 : 64) >= 24 && split_tiles(a) <= kMostTiles)
    return launch_rows_split<EL, PT, GATHER, kEpiNone>(a, st);
  // Rows that most groups stay under when e are expected and chance spreads
  // them (a binomial count's deviation is at most sqrt(e)).
  const int64_t e = a.expected + static_cast<int64_t>(std::sqrt(static_cast<double>(a.expected)));
  // Measured in us on 8 experts of 4096 x 7168 weights unless said otherwise,
  // bf16, tiles written channels x rows.
  //   A few rows: the weights stream past them.  128 x 32, two workgroups a
  //   CU, against 128 x 128: 16 rows 84 / 85.5, 4 rows 82 / 81, 16 rows of
  //   7168 x 2048 36 / 38, E4M3 21.2 / 25.7.
  if (e <= 24) return launch_rows_tile<EL, PT, GATHER, 128, 32, 4, 1, F8 ? 3 : 4, F8 ? 3 : 4>(a, st);
  const int64_t wide = (a.NO + 255) / 256, narrow = (a.NO + 127) / 128;
  if (a.g.G * wide * ((e + 255) / 256) >= 192) {
    // enough tiles of 256 channels for the GPU's 256 CUs
    gemm_rows_wide_kernel<EL, PT, GATHER, kEpiNone><<<256, 8 * kWave, 0, st>>>(a);
    return hipGetLastError();
  }
  //   Fewer: 128 channels, as many rows as a group needs: 128 x 128 / 192 /
  //   256 at 64 rows 92 / 92 / 100, at 128 rows 160 / 106 / 110, at 180 rows
  //   (some groups more than 192) 145 / 186 / 123.
  if (e <= 108 || a.g.G * narrow * ((e + 127) / 128) <= 256)
    return launch_rows_tile<EL, PT, GATHER, 128, 128, 2, 4, F8 ? 4 : 5, F8 ? 4 : 5>(a, st);
  if (e <= 192) return launch_rows_tile<EL, PT, GATHER, 128, 192, 2, 4, F8 ? 3 : 4, F8 ? 3 : 4>(a, st);
  return launch_rows_tile<EL, PT, GATHER, 128, 256, 2, 4, 3, 3>(a, st);
}

}  // namespace miep
