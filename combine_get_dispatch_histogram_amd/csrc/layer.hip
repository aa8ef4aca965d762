// layer.hip -- a few tokens through their experts and back, without dispatch:
//
//   y[t] = residual[t] + sum_k w[t][k] * W2_e (silu(g) * u),  [g | u] = W1_e x[t],  e = idx[t][k]
//
// Bound by the chosen experts' weights, which are read once.  Two launches: all
// first products and their activation to `a` (bf16, a row an expert and token),
// then all second products; a token's experts meet in the second, where a
// workgroup owns 16 output channels and walks every expert, so their sum needs no
// atomics and has one order.  Either kernel finds the experts' tokens itself, in
// LDS: a bit a token for every expert, and the bits' order is the tokens'.
#include "act.h"
#include "stream.h"

namespace miep {

namespace {

constexpr int kLayerWaves = 8, kLayerThreads = kLayerWaves * kWave;

// The experts that some token chose, ascending, with their tokens, in dynamic LDS.
struct Lists {
  uint64_t* mask;              // [E][words] a bit a token
  int* off;                    // [most + 1] first position of each listed expert
  uint16_t* active;            // [most] the experts
  uint16_t* token;             // [N*K] a position's token
  uint16_t* expert;            // [N*K] and expert
  float* weight;               // [N*K] its weight (an expert named twice: their sum)
  int count;                   // listed experts
};

template <bool WEIGHTS>
__device__ __forceinline__ Lists make_lists(const LayerArgs& a, uint8_t* lds, int* wave_sums) {
  const ListsLayout at = lists_layout(a.N, a.K, a.E);
  Lists l;
  l.mask = reinterpret_cast<uint64_t*>(lds);
  l.off = reinterpret_cast<int*>(lds + at.off);
  l.active = reinterpret_cast<uint16_t*>(lds + at.active);
  l.token = reinterpret_cast<uint16_t*>(lds + at.token);
  l.expert = reinterpret_cast<uint16_t*>(lds + at.expert);
  l.weight = reinterpret_cast<float*>(lds + at.weight);
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  for (int i = tid; i < a.E * at.words; i += kLayerThreads) l.mask[i] = 0;
  __syncthreads();
  for (int i = tid; i < at.entries; i += kLayerThreads) {
    const int64_t e = a.idx[i] - a.first;
    const int t = i / a.K;
    if (e >= 0 && e < a.E)
      atomicOr(reinterpret_cast<unsigned long long*>(l.mask + e * at.words + t / 64), 1ull << (t & 63));
  }
  __syncthreads();
  int before = 0;                                                     // listed << 16 | positions
  for (int e0 = 0; e0 < a.E; e0 += kLayerThreads) {
    const int e = e0 + tid;
    int n = 0;
    if (e < a.E)
      for (int w = 0; w < at.words; ++w) n += __builtin_popcountll(l.mask[e * at.words + w]);
    const int both = n > 0 ? 1 << 16 | n : 0;
    const int inc = wave_inclusive_scan(both);
    if (lane == 63) wave_sums[wave] = inc;
    __syncthreads();
    int mine = before + inc - both;
    for (int w = 0; w < kLayerWaves; ++w) {
      if (w < wave) mine += wave_sums[w];
      before += wave_sums[w];
    }
    if (n > 0) {
      const int place = mine >> 16;
      int p = mine & 0xffff;
      l.active[place] = static_cast<uint16_t>(e);
      l.off[place] = p;
      for (int w = 0; w < at.words; ++w)
        for (uint64_t bits = l.mask[e * at.words + w]; bits; bits &= bits - 1) {
          l.token[p] = static_cast<uint16_t>(w * 64 + __builtin_ctzll(bits));
          l.expert[p++] = static_cast<uint16_t>(e);
        }
    }
    __syncthreads();
  }
  l.count = before >> 16;
  if (tid == 0) l.off[l.count] = before & 0xffff;
  if constexpr (WEIGHTS) {
    for (int p = tid; p < (before & 0xffff); p += kLayerThreads) {
      const int64_t t = l.token[p], e = a.first + l.expert[p];
      float w = 0.f;
      for (int k = 0; k < a.K; ++k) w += a.idx[t * a.K + k] == e ? a.wts[t * a.K + k] : 0.f;
      l.weight[p] = w;
    }
  }
  __syncthreads();
  return l;
}

// ---- first products: units of 16 gate and 16 up channels of an expert
template <int EL, int TQ>
__device__ __forceinline__ void up_unit(const LayerArgs& a, const Lists& l, int place, int i0, int c0, int n, float* sums) {
  constexpr bool F8 = EL != kGemmBf16;
  constexpr int EB = F8 ? 1 : 2;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const int e = l.active[place], first = l.off[place] + c0;
  const uint32_t ldw = static_cast<uint32_t>(a.H) * EB;
  StreamSource<EL, 2, TQ> src;
  src.w = static_cast<const uint8_t*>(a.w1) + static_cast<int64_t>(__builtin_amdgcn_readfirstlane(e)) * 2 * a.I * ldw;
  src.x = reinterpret_cast<const uint8_t*>(a.x);
  src.C = a.H;
  const int row = min(i0 + m, a.I - 1);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    src.woff[p] = static_cast<uint32_t>(p * a.I + row) * ldw + quarter * 16;
    if constexpr (F8) {
      const int kb = a.H / kFp8Group;
      src.scales = a.s1;
      src.srow[p] = (static_cast<int64_t>(__builtin_amdgcn_readfirstlane(e)) * (2 * a.I / kFp8Group) + (p * a.I + i0) / kFp8Group) * kb;
    }
  }
#pragma unroll
  for (int j = 0; j < TQ; ++j)
    src.xoff[j] = static_cast<uint32_t>(l.token[first + min(j * 16 + m, n - 1)]) * (a.H * 2u) + quarter * (F8 ? 32 : 16);
  f32x4 acc[2][TQ];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[p][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  constexpr int S = StreamType<EL>::kStep;
  stream_steps<F8 ? 1 : 2>(src, wave, kLayerWaves, (a.H + S - 1) / S, acc);
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int j = 0; j < TQ; ++j)
      *reinterpret_cast<f32x4*>(sums + (((wave * TQ + j) * 16 + m) * 2 + p) * 16 + quarter * 4) = acc[p][j];
  __syncthreads();
  for (int i = threadIdx.x; i < TQ * 128; i += kLayerThreads) {
    const int col = i / 8, p = i % 8 * 2;
    if (col >= n || i0 + p >= a.I) continue;
    float gx = 0.f, gy = 0.f, ux = 0.f, uy = 0.f;
#pragma unroll
    for (int w = 0; w < kLayerWaves; ++w) {
      const float* s = sums + (w * TQ * 16 + col) * 32 + p;
      gx += s[0];
      gy += s[1];
      ux += s[16];
      uy += s[17];
    }
    *reinterpret_cast<uint32_t*>(a.a + static_cast<int64_t>(first + col) * a.I + i0 + p) =
        pack_bf16x2(gx * sigmoid(gx) * ux, gy * sigmoid(gy) * uy);
  }
  __syncthreads();
}

template <int EL, int MOST>
__global__ __launch_bounds__(kLayerThreads, MOST == 1 ? 4 : 2) void layer_up_kernel(LayerArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ __align__(16) float sums[kLayerWaves * MOST * 16 * 32];
  __shared__ int wave_sums[kLayerWaves];
  const Lists l = make_lists<false>(a, lds, wave_sums);
  const int tiles = (a.I + 15) / 16;
  for (int u = blockIdx.x; u < l.count * tiles; u += gridDim.x) {
    const int place = u / tiles, i0 = (u - place * tiles) * 16;
    const int n = l.off[place + 1] - l.off[place];
    for (int c0 = 0; c0 < n; c0 += MOST * 16) {
      const int left = n - c0;
      if (MOST == 1 || left <= 16) up_unit<EL, 1>(a, l, place, i0, c0, min(left, 16), sums);
      else if constexpr (MOST > 1) {
        if (left <= 32) up_unit<EL, 2>(a, l, place, i0, c0, left, sums);
        else up_unit<EL, 4>(a, l, place, i0, c0, min(left, 64), sums);
      }
    }
  }
}

// ---- second products: 16 output channels a workgroup; the experts' steps one
// after the other are cut evenly over its wavefronts
template <int EL, int TQ>
__device__ __forceinline__ void down_part(const LayerArgs& a, const Lists& l, int place, int h0, int s0, int s1, int c0, int n, float* out) {
  constexpr bool F8 = EL != kGemmBf16;
  constexpr int EB = F8 ? 1 : 2;
  const int lane = lane_id(), m = lane & 15, quarter = lane >> 4;
  const int e = __builtin_amdgcn_readfirstlane(static_cast<int>(l.active[place]));
  const int first = l.off[place] + c0;
  const uint32_t ldw = static_cast<uint32_t>(a.I) * EB;
  StreamSource<EL, 1, TQ> src;
  src.w = static_cast<const uint8_t*>(a.w2) + (static_cast<int64_t>(e) * a.H + h0) * ldw;
  src.x = reinterpret_cast<const uint8_t*>(a.a);
  src.C = a.I;
  src.woff[0] = static_cast<uint32_t>(min(m, a.H - 1 - h0)) * ldw + quarter * 16;
  if constexpr (F8) {
    src.scales = a.s2;
    src.srow[0] = (static_cast<int64_t>(e) * (a.H / kFp8Group) + h0 / kFp8Group) * (a.I / kFp8Group);
  }
#pragma unroll
  for (int j = 0; j < TQ; ++j)
    src.xoff[j] = static_cast<uint32_t>(first + min(j * 16 + m, n - 1)) * (a.I * 2u) + quarter * (F8 ? 32 : 16);
  f32x4 acc[1][TQ];
#pragma unroll
  for (int j = 0; j < TQ; ++j) acc[0][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  stream_steps<F8 ? (TQ == 4 ? 1 : 2) : (TQ == 1 ? 4 : 2)>(src, s0, 1, s1, acc);
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    const int col = j * 16 + m;
    if (col < n) {
      const float w = l.weight[first + col];
      f32x4* o = reinterpret_cast<f32x4*>(out + l.token[first + col] * 16 + quarter * 4);
      f32x4 v = *o;
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(w, acc[0][j][r], v[r]);
      *o = v;
    }
  }
}

template <int EL, int MOST>
__global__ __launch_bounds__(kLayerThreads, MOST == 1 ? 4 : 2) void layer_down_kernel(LayerArgs a) {
  extern __shared__ __align__(16) uint8_t lds[];
  __shared__ int wave_sums[kLayerWaves];
  const Lists l = make_lists<true>(a, lds, wave_sums);
  float* sums = reinterpret_cast<float*>(lds + lists_layout(a.N, a.K, a.E).end);      // [wavefront][token][16]
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  float* out = sums + wave * a.N * 16;
  for (int i = lane_id(); i < a.N * 4; i += kWave) reinterpret_cast<f32x4*>(out)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  __builtin_amdgcn_wave_barrier();
  constexpr int S = StreamType<EL>::kStep;
  const int h0 = blockIdx.x * 16, steps = (a.I + S - 1) / S;
  const int64_t total = static_cast<int64_t>(l.count) * steps;
  int64_t at = total * wave / kLayerWaves;
  const int64_t end = total * (wave + 1) / kLayerWaves;
  while (at < end) {
    const int place = static_cast<int>(at / steps), s0 = static_cast<int>(at - static_cast<int64_t>(place) * steps);
    const int s1 = static_cast<int>(end - at < steps - s0 ? s0 + (end - at) : steps);
    const int n = __builtin_amdgcn_readfirstlane(l.off[place + 1] - l.off[place]);
    for (int c0 = 0; c0 < n; c0 += MOST * 16) {
      const int left = n - c0;
      if (MOST == 1 || left <= 16) down_part<EL, 1>(a, l, place, h0, s0, s1, c0, min(left, 16), out);
      else if constexpr (MOST > 1) {
        if (left <= 32) down_part<EL, 2>(a, l, place, h0, s0, s1, c0, left, out);
        else down_part<EL, 4>(a, l, place, h0, s0, s1, c0, min(left, 64), out);
      }
    }
    at += s1 - s0;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.N * 8; i += kLayerThreads) {
    const int t = i / 8, p = i % 8 * 2;
    if (h0 + p >= a.H) continue;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < kLayerWaves; ++w) {
      x += sums[(w * a.N + t) * 16 + p];
      y += sums[(w * a.N + t) * 16 + p + 1];
    }
    const int64_t o = static_cast<int64_t>(t) * a.H + h0 + p;
    if (a.residual) {
      const uint32_t r = *reinterpret_cast<const uint32_t*>(a.residual + o);
      x += bf16_lo(r);
      y += bf16_hi(r);
    }
    *reinterpret_cast<uint32_t*>(a.y + o) = pack_bf16x2(x, y);
  }
}

template <int EL, int MOST>
hipError_t launch_sized(const LayerArgs& a, hipStream_t st) {
  const ListsLayout at = lists_layout(a.N, a.K, a.E);
  const int64_t units = static_cast<int64_t>(at.most) * ((a.I + 15) / 16);
  const unsigned most = MOST == 1 ? 512 : 256;
  layer_up_kernel<EL, MOST><<<static_cast<unsigned>(units < most ? units : most), kLayerThreads, static_cast<unsigned>(at.end), st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  layer_down_kernel<EL, MOST><<<(a.H + 15) / 16, kLayerThreads, static_cast<unsigned>(at.end + kLayerWaves * a.N * 64), st>>>(a);
  return hipGetLastError();
}

template <int EL>
hipError_t launch_typed(const LayerArgs& a, hipStream_t st) {
  return a.N <= 16 ? launch_sized<EL, 1>(a, st) : launch_sized<EL, 4>(a, st);
}

}  // namespace

hipError_t launch_layer(const LayerArgs& a, hipStream_t st) {
  if (a.N == 0) return hipSuccess;
  if (a.type == kGemmFp8) return launch_typed<kGemmFp8>(a, st);
  if (a.type == kGemmFp8Ue8m0) return launch_typed<kGemmFp8Ue8m0>(a, st);
  return launch_typed<kGemmBf16>(a, st);
}

}  // namespace miep
