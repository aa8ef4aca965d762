// swiglu.hip -- the activation between an expert's two products, over the
// rows of ragged groups:
//
//   a = silu(gate) * up,  silu(g) = g * s,  s = 1 / (1 + exp(-g))
//   d gate = da * up * s * (1 + g * (1 - s)),  d up = da * g * s
//
// in fp32 from bf16, rounded once: to bf16, or cast to E4M3 by the dispatch's
// rule (a scale per 128 channels) straight from the fp32 value, so that the
// low-latency path's second product reads codes that were rounded once.
// Bound by memory at I = 2048 and more: a row is 4*I bytes read and I to 2*I
// written (backward 6*I and 4*I: 16384 rows of 2 x 2048 take 54 us, 6.2 TB/s).
// A lane owns 8 channels (16-byte loads of gate and up); sixteen lanes hold one
// scale's 128.
#include "gemm.h"

namespace miep {

// exp(-g) to fp32 accuracy from the hardware's exp2: the product g * log2(e)
// is carried in two parts, the low one applied to first order.  |g| is capped
// where the sigmoid is 1 (or exp(-g) overflows and it is 0) to fp32.
__device__ __forceinline__ float sigmoid(float g) {
  const float c = -fminf(fmaxf(g, -100.f), 100.f);
  const float hi = c * 1.44269502f;                                   // log2(e), rounded to fp32
  const float lo = fmaf(c, 1.44269502f, -hi) + c * 1.92596299e-8f;    // and its rest
  const float e = __builtin_amdgcn_exp2f(hi) * fmaf(lo, 0.693147182f, 1.f);   // infinity stays infinity
  return __builtin_amdgcn_rcpf(1.f + e);
}

__device__ __forceinline__ void widen(const v4u& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ v4u narrow(const float (&f)[8]) {
  return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// 16 bytes to memory; past the caches where the result is as large as half the
// last-level cache (see launch_swiglu).
template <bool STREAM>
__device__ __forceinline__ void put(uint16_t* p, const v4u& v) {
  const u32x4 t = {v.x, v.y, v.z, v.w};
  if constexpr (STREAM) __builtin_nontemporal_store(t, reinterpret_cast<u32x4*>(p));
  else *reinterpret_cast<u32x4*>(p) = t;
}

template <int KIND, bool STREAM>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluArgs a) {
  const int total = count_tiles(a.g, a.rows_per_tile, 1);
  const int per_row = a.I / 8;
  for (int t = blockIdx.x; t < total; t += gridDim.x) {
    const TileAt at = find_tile(a.g, a.rows_per_tile, 1, t);
    if (at.group < 0) return;
    const int r0 = max(at.first, 0) * a.rows_per_tile;
    const int n = min(a.rows_per_tile, at.rows - r0);
    const int items = n > 0 ? n * per_row : 0;
    for (int i = threadIdx.x; i < items; i += 256) {
      const int r = i / per_row, c = i - r * per_row;
      const int64_t row = at.begin + r0 + r;
      const uint16_t* h = a.h + row * 2 * a.I + c * 8;
      float gate[8], up[8], v[8];
      widen(ld16(h), gate);
      widen(ld16(h + a.I), up);
      if constexpr (KIND == kSwigluBackward) {
        float da[8], dg[8];
        widen(ld16(a.da + row * a.I + c * 8), da);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float s = sigmoid(gate[k]);
          dg[k] = da[k] * up[k] * s * (1.f + gate[k] * (1.f - s));
          v[k] = da[k] * (gate[k] * s);
        }
        uint16_t* o = static_cast<uint16_t*>(a.out) + row * 2 * a.I + c * 8;
        put<STREAM>(o, narrow(dg));
        put<STREAM>(o + a.I, narrow(v));
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = gate[k] * sigmoid(gate[k]) * up[k];
        if constexpr (KIND == kSwigluBf16) {
          put<STREAM>(static_cast<uint16_t*>(a.out) + row * a.I + c * 8, narrow(v));
        } else {
          // items of one row are a multiple of 16: the sixteen lanes of a DPP row are active together
          float top = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) top = fmaxf(top, fabsf(v[k]));
          top = group8_max(top);
          top = fmaxf(top, dpp_f32<0x140>(top));                      // row_mirror: the other eight lanes
          float inv;
          const float scale = fp8_scales(top, a.round_scale != 0, &inv);
          const v2u code{e4m3x4(v[0] * scale, v[1] * scale, v[2] * scale, v[3] * scale),
                         e4m3x4(v[4] * scale, v[5] * scale, v[6] * scale, v[7] * scale)};
          *reinterpret_cast<v2u*>(static_cast<uint8_t*>(a.out) + row * a.I + c * 8) = code;
          if ((c & 15) == 0) {
            const int64_t s = row * (a.I / kFp8Group) + c / 16;
            a.scales[s] = inv;
            if (a.scales_ue8m0) a.scales_ue8m0[s] = ue8m0_byte(inv);
          }
        }
      }
    }
  }
}

hipError_t launch_swiglu(const SwigluArgs& args, int kind, hipStream_t st) {
  SwigluArgs a = args;
  if (a.g.G == 0 || a.g.limit == 0) return hipSuccess;
  // One row a workgroup at a time (16384 rows of 2 x 2048, backward: 61 us; 4
  // rows 65, 8 rows 72).  Chosen at that width, where a row is 256 lanes' work;
  // narrower rows leave lanes idle, and 16384 rows take (bf16 / E4M3 / backward)
  // 35 / 37 / 52 us at 2048, 28 / 32 / 39 at 1408, 23 / 26 / 30 at 768 and 21 /
  // 22 / 26 at 512, where their bytes would take 8 / 7 / 13.
  a.rows_per_tile = 1;
  const int64_t most = a.g.limit + a.g.G;
  const unsigned grid = static_cast<unsigned>(most < 2048 ? most : 2048);
  // A result of half the 256 MiB last-level cache or more is stored past it:
  // 16384 rows 63 -> 52 us (with a copy that reads it behind, 122 -> 115);
  // smaller ones are read from the cache again (4096 rows and a copy: 27 us,
  // streamed 30).
  const int64_t bytes = a.g.limit * a.I * (kind == kSwigluBackward ? 4 : 2);
  const bool stream = bytes >= (128ll << 20);
  if (kind == kSwigluFp8) swiglu_kernel<kSwigluFp8, false><<<grid, 256, 0, st>>>(a);
  else if (kind == kSwigluBf16 && stream) swiglu_kernel<kSwigluBf16, true><<<grid, 256, 0, st>>>(a);
  else if (kind == kSwigluBf16) swiglu_kernel<kSwigluBf16, false><<<grid, 256, 0, st>>>(a);
  else if (stream) swiglu_kernel<kSwigluBackward, true><<<grid, 256, 0, st>>>(a);
  else swiglu_kernel<kSwigluBackward, false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace miep
