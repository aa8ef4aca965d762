// stream.h -- products of a few rows, where reading the weights is the cost.
//
//   acc[i] = sum_c W[row(i, m)][c] * X[col(n)][c]      16 rows of W x 16 of X each
//
// Every step of 128 bytes a row of W comes to LDS by asynchronous loads, into a
// ring that a wavefront has for itself, so without barriers; the wavefronts of a
// workgroup share a contraction's steps and add their sums up in LDS, in order.
// The loads are what a CU has too little of: a load whose four neighbouring lanes
// lie in different 128-byte lines (an MFMA operand straight into registers) took
// 57 cycles a KiB, 18 bytes a cycle and CU; eight lanes a line take under half of
// that.  The contraction's order is free, so E4M3 codes need no reordering for
// the bf16 MFMAs that they are converted to: a lane's 16 codes meet the 16
// channels of X at the same places.
#pragma once

#include "gemm.h"

namespace miep {

__device__ __forceinline__ int swz8(int row) { return (row >> 1) & 7; }

// Two E4M3 codes of v (the low or the high half) as bf16, exactly: their products
// with bf16 numbers are exact in fp32, so nothing is cut as the E4M3 MFMA cuts.
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

// A pointer that is the same in all lanes, in scalar registers.
__device__ __forceinline__ const uint8_t* uniform(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>(static_cast<uint64_t>(hi) << 32 | lo);
}

// A wavefront's ring of steps in BYTES bytes of LDS: the rows of W that WL loads of
// 1 KiB bring (8 each), those of X that XL loads bring (8 each, E4M3 4: its step is
// 128 channels), and E4M3's two scales, of the blocks that the rows of W lie in
// (read when they are needed, they would stop a wavefront for a memory's latency at
// every tile and expert: 64 tokens over 55 experts, second product, 260 -> 150 us).
template <int EL, int WL, int XL, int BYTES, int TQ = 1>
struct StreamRing {
  static constexpr int TP = (WL + 1) / 2;                             // 16 x 16 results
  static constexpr bool kFp8 = EL != kGemmBf16;
  static constexpr int kChannels = kFp8 ? 128 : 64;                   // of a step
  static constexpr int kXRow = kChannels * 2, kXRows = XL * 1024 / kXRow;
  static constexpr int kWBytes = WL * 1024, kScales = kWBytes + XL * 1024, kStep = kScales + (kFp8 ? 256 : 0);
  static constexpr int kDepth = BYTES / kStep < 8 ? BYTES / kStep : 8;
  static constexpr int kLoads = WL + XL + (kFp8 ? 1 : 0);
  static_assert(kDepth >= 1 && kDepth * kLoads < 64, "ring");
  static_assert(TQ == 1 || kXRows == 16 * TQ, "whole tiles of X");

  uint32_t lds;
  int head, tail;                                                     // buffers: next to fill, next to read

  struct Frag {
    u32x4 w[TP][2];
    u32x4 x[TQ][kFp8 ? 4 : 2];
    float s[2];
  };

  __device__ __forceinline__ explicit StreamRing(uint32_t at) : lds(at), head(0), tail(0) {}

  // Where the lane's 16 bytes of W load i lie in a step of 128 bytes a row (row
  // i * 8 + lane / 8), and of X load i.
  static __device__ __forceinline__ int w_row(int i) { return i * 8 + lane_id() / 8; }
  static __device__ __forceinline__ int w_chunk(int i) { return (lane_id() & 7) ^ swz8(w_row(i) & 15); }
  static __device__ __forceinline__ int x_row(int i) { return kFp8 ? i * 4 + lane_id() / 16 : i * 8 + lane_id() / 8; }
  static __device__ __forceinline__ int x_chunk(int i) {
    if constexpr (kFp8) return (lane_id() & 15) ^ (x_row(i) & 15);
    else return (lane_id() & 7) ^ swz8(x_row(i) & 15);
  }

  // The next step's loads.  `scale`: the lane's, of the first block in even lanes
  // and of the second in odd ones (any in bf16).  `left`: channels of the contraction from this step
  // on; bf16 behind its end reads zeros in both operands (0 * NaN would not be 0).
  __device__ __forceinline__ void issue(const uint8_t* w, const uint32_t (&woff)[WL], const uint8_t* x, const uint32_t (&xoff)[XL], const uint8_t* scale, int left) {
    w = uniform(w);
    x = uniform(x);
    const uint32_t to = __builtin_amdgcn_readfirstlane(lds + head * kStep);
    head = head == kDepth - 1 ? 0 : head + 1;
    if (kFp8 || left >= kChannels) {
#pragma unroll
      for (int i = 0; i < WL; ++i) dma16s(w, woff[i], to + i * 1024);
#pragma unroll
      for (int i = 0; i < XL; ++i) dma16s(x, xoff[i], to + kWBytes + i * 1024);
      if constexpr (EL == kGemmFp8) dma4(scale, to + kScales);
      else if constexpr (kFp8) dma1(scale, to + kScales);
    } else {
#pragma unroll
      for (int i = 0; i < WL; ++i)
        dma16(w_chunk(i) * 8 < left ? static_cast<const void*>(w + woff[i]) : static_cast<const void*>(g_zero16), to + i * 1024);
#pragma unroll
      for (int i = 0; i < XL; ++i)
        dma16(x_chunk(i) * 8 < left ? static_cast<const void*>(x + xoff[i]) : static_cast<const void*>(g_zero16), to + kWBytes + i * 1024);
    }
  }

  // Waits for the oldest step, of which `more` say that kDepth - 1 others have been
  // issued behind it, and takes it to registers; its buffer is free then.
  __device__ __forceinline__ void take(Frag& f, bool more) {
    if (more) asm volatile("s_waitcnt vmcnt(%0)" ::"n"((kDepth - 1) * kLoads) : "memory");
    else asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    const uint32_t at = lds + tail * kStep;
    tail = tail == kDepth - 1 ? 0 : tail + 1;
    const int m = lane_id() & 15, quarter = lane_id() >> 4;
    // (rows that were not loaded: any)
    const int wm = WL == 1 ? m & 7 : m, xm = m & (kXRows - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < TP; ++i) f.w[i][h] = lds_read<u32x4>(at + i * 2048 + wm * 128 + ((h * 4 + quarter) ^ swz8(wm)) * 16);
#pragma unroll
    for (int h = 0; h < (kFp8 ? 4 : 2); ++h) {
      const int chunk = kFp8 ? (((h >> 1) * 4 + quarter) * 2 + (h & 1)) ^ xm : (h * 4 + quarter) ^ swz8(xm);
#pragma unroll
      for (int j = 0; j < TQ; ++j) f.x[j][h] = lds_read<u32x4>(at + kWBytes + (j * 16 + xm) * kXRow + chunk * 16);
    }
    if constexpr (kFp8) {
      const u32x2 t = lds_read<u32x2>(at + kScales);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (EL == kGemmFp8) f.s[i] = __uint_as_float(t[i]);
        else f.s[i] = __uint_as_float(t[i] << 23 | ((t[i] + 1 & 0xfe) == 0 ? 1u << 22 : 0u));   // exponent byte: 0 is 2^-127, 255 NaN
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }

  // acc += W * X of a step; E4M3: second(i, r) says whether row r of result i's four
  // lies in the second block.
  template <class SECOND>
  static __device__ __forceinline__ void multiply(const Frag& f, SECOND second, f32x4 (&acc)[TP][TQ]) {
#pragma unroll
    for (int i = 0; i < TP; ++i) {
      if constexpr (kFp8) {
        f32x4 d[TQ];
#pragma unroll
        for (int j = 0; j < TQ; ++j) d[j] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const bf16x8 w = bf16x8_of_e4m3(f.w[i][h >> 1][(h & 1) * 2], f.w[i][h >> 1][(h & 1) * 2 + 1]);
#pragma unroll
          for (int j = 0; j < TQ; ++j) d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, __builtin_bit_cast(bf16x8, f.x[j][h]), d[j], 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < TQ; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = __builtin_fmaf(d[j][r], second(i, r) ? f.s[1] : f.s[0], acc[i][j][r]);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < TQ; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, f.w[i][h]), __builtin_bit_cast(bf16x8, f.x[j][h]), acc[i][j], 0, 0, 0);
      }
    }
  }
};

}  // namespace miep
