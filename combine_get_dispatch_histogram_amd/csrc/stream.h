// stream.h -- products of a few rows, where reading the weights is the cost.
//
//   acc[tp][tq] = sum_c W[row(tp, i)][c] * X[col(tq, j)][c]      16 x 16 each
//
// The weights go from memory straight to registers (each is used by one
// wavefront once, so LDS would only add a trip), 16 bytes a lane: a load takes 64
// consecutive bytes of each of 16 rows.  The contraction's order is free, so E4M3
// codes need no reordering for the bf16 MFMAs that they are converted to: a
// lane's 16 codes meet the 16 channels of X at the same places.  A wavefront
// keeps kAhead steps of 128 bytes a row in flight; the wavefronts of a workgroup
// share a tile's contraction and add their sums up in LDS, in order.
#pragma once

#include "gemm.h"

namespace miep {

// E4M3 codes (products of a converted code and a bf16 number are exact in fp32,
// so unlike the E4M3 MFMA's nothing is cut) with a scale a 128 x 128 block.
template <int EL>
struct StreamType {
  static constexpr bool kFp8 = EL != kGemmBf16;
  static constexpr int kStep = kFp8 ? 128 : 64;                       // channels
  static constexpr int kXLoads = kFp8 ? 4 : 2;                        // 16-byte loads of X a step and lane
};

template <int EL, int TP, int TQ>
struct StreamFrag {
  u32x4 w[TP][2];
  u32x4 x[TQ][StreamType<EL>::kXLoads];
  float s[TP];
};

// Two E4M3 codes of v (the low or the high half) as bf16, exactly.
template <bool HIGH>
__device__ __forceinline__ uint32_t bf16x2_of_e4m3(uint32_t v) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 r = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(v, 1.0f, HIGH);
  return __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ bf16x8 bf16x8_of_e4m3(uint32_t lo, uint32_t hi) {
  const u32x4 t = {bf16x2_of_e4m3<false>(lo), bf16x2_of_e4m3<true>(lo), bf16x2_of_e4m3<false>(hi), bf16x2_of_e4m3<true>(hi)};
  return __builtin_bit_cast(bf16x8, t);
}

__device__ __forceinline__ u32x4 load16(const uint8_t* base, uint32_t off) {
  return *reinterpret_cast<const u32x4*>(base + off);
}

// A scale of block (row, step): fp32, or the exponent byte of a power of two.
template <int EL>
__device__ __forceinline__ float block_scale(const void* s, int64_t at) {
  if constexpr (EL == kGemmFp8) return static_cast<const float*>(s)[at];
  else return __uint_as_float(static_cast<uint32_t>(static_cast<const uint8_t*>(s)[at]) << 23);
}

// What a wavefront multiplies: bases are uniform, offsets a lane's own (row *
// pitch + 16 * quarter for W; X's of a step's first 16 bytes).
template <int EL, int TP, int TQ>
struct StreamSource {
  const uint8_t* w;
  const uint8_t* x;
  uint32_t woff[TP], xoff[TQ];
  const void* scales;          // E4M3: of the weight's matrix
  int64_t srow[TP];            // E4M3: first scale of the tile's block of rows
  int C;                       // channels; bf16: behind them both operands read as zeros

  // A step of whole 128 bytes a row.
  __device__ __forceinline__ void load(StreamFrag<EL, TP, TQ>& f, int step) const {
    constexpr bool F8 = StreamType<EL>::kFp8;
    const uint8_t* wb = w + static_cast<int64_t>(step) * 128;
    const uint8_t* xb = x + static_cast<int64_t>(step) * (F8 ? 256 : 128);
#pragma unroll
    for (int i = 0; i < TP; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) f.w[i][h] = load16(wb + h * 64, woff[i]);
#pragma unroll
    for (int j = 0; j < TQ; ++j)
#pragma unroll
      for (int h = 0; h < StreamType<EL>::kXLoads; ++h)
        f.x[j][h] = load16(xb + (F8 ? (h >> 1) * 128 + (h & 1) * 16 : h * 64), xoff[j]);
    if constexpr (F8) {
#pragma unroll
      for (int i = 0; i < TP; ++i) f.s[i] = block_scale<EL>(scales, srow[i] + step);
    }
  }
  // bf16, the last step of a contraction that is not whole: behind its end both
  // operands are zeros (0 * NaN would not be 0).
  __device__ __forceinline__ void load_end(StreamFrag<EL, TP, TQ>& f, int step) const {
    const u32x4 zero = {0u, 0u, 0u, 0u};
    const int c = step * 64 + (lane_id() >> 4) * 8;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool in = c + h * 32 < C;
      const int64_t at = static_cast<int64_t>(step) * 128 + h * 64;
#pragma unroll
      for (int i = 0; i < TP; ++i) f.w[i][h] = in ? load16(w + at, woff[i]) : zero;
#pragma unroll
      for (int j = 0; j < TQ; ++j) f.x[j][h] = in ? load16(x + at, xoff[j]) : zero;
    }
  }
};

template <int EL, int TP, int TQ>
__device__ __forceinline__ void stream_multiply(const StreamFrag<EL, TP, TQ>& f, f32x4 (&acc)[TP][TQ]) {
#pragma unroll
  for (int i = 0; i < TP; ++i) {
    if constexpr (StreamType<EL>::kFp8) {
      f32x4 d[TQ];
#pragma unroll
      for (int j = 0; j < TQ; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const bf16x8 p = bf16x8_of_e4m3(f.w[i][h >> 1][(h & 1) * 2], f.w[i][h >> 1][(h & 1) * 2 + 1]);
#pragma unroll
        for (int j = 0; j < TQ; ++j)
          d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(p, __builtin_bit_cast(bf16x8, f.x[j][h]), d[j], 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < TQ; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[j][r], f.s[i], acc[i][j][r]);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < TQ; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.w[i][h]),
                                                              __builtin_bit_cast(bf16x8, f.x[j][h]), acc[i][j], 0, 0, 0);
    }
  }
}

// acc += the steps first, first + stride, ... below `end`, AHEAD of them in
// flight.
template <int AHEAD, int EL, int TP, int TQ>
__device__ __forceinline__ void stream_steps(const StreamSource<EL, TP, TQ>& src, int first, int stride, int end, f32x4 (&acc)[TP][TQ]) {
  const int whole = min(end, src.C / StreamType<EL>::kStep);
  const int n = first < whole ? (whole - first + stride - 1) / stride : 0;
  StreamFrag<EL, TP, TQ> f[AHEAD + 1];
  // (The first loads stand apart in either branch: where the compiler sees that
  // they may be missing, it has the loop wait for all loads, not for its own.)
  int i = 0;
  if (n > 2 * AHEAD) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) src.load(f[k], first + k * stride);
    do {
#pragma unroll
      for (int d = 0; d <= AHEAD; ++d) {
        src.load(f[(d + AHEAD) % (AHEAD + 1)], first + (i + d + AHEAD) * stride);
        __builtin_amdgcn_sched_barrier(0);
        stream_multiply(f[d], acc);
        __builtin_amdgcn_sched_barrier(0);
      }
      i += AHEAD + 1;
    } while (i + 2 * AHEAD < n);
  } else {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (k < n) src.load(f[k], first + k * stride);
  }
  // AHEAD .. 2 * AHEAD steps are left (or as many as there are), the first of
  // them under way
#pragma unroll
  for (int d = 0; d < 2 * AHEAD; ++d) {
    if (d < AHEAD && i + d + AHEAD < n) src.load(f[(d + AHEAD) % (AHEAD + 1)], first + (i + d + AHEAD) * stride);
    if (i + d < n) stream_multiply(f[d % (AHEAD + 1)], acc);
  }
  if constexpr (!StreamType<EL>::kFp8) {
    if (whole < end && first <= whole && (whole - first) % stride == 0) {
      src.load_end(f[0], whole);
      stream_multiply(f[0], acc);
    }
  }
}

}  // namespace miep
