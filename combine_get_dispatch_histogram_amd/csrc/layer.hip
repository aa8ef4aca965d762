// layer.hip -- a few tokens through their experts and back, without dispatch:
//
//   y[t] = residual[t] + sum_k w[t][k] * W2_e (silu(g) * u),  [g | u] = W1_e x[t],  e = idx[t][k]
//
// Bound by the chosen experts' weights, which are read once.  Two launches: all
// first products and their activation to `a` (bf16, a row an expert and token),
// then all second products; a token's experts meet in the second, where a
// workgroup owns 8 to 32 output channels and walks every expert, so their sum needs
// no atomics and has one order.  Either kernel finds the experts' tokens itself, in
// LDS: a bit a token for every expert, and the bits' order is the tokens'.
// Hidden 7168, inner 2048: one token over 8 experts, bf16, 123 us (705 MB, 5.8
// TB/s); 64 tokens over 55 experts, E4M3, 389 us (2.4 GB, 6.2 TB/s).  3 tokens, 8
// of 64 experts each, of 256 x 384, E4M3 (6 MB): 19 us, of which each kernel's lists take 1.7,
// its rings' first loads 2 to 4, and the second's steps half a us each.
#include "act.h"
#include "stream.h"

namespace miep {

namespace {

// LDS of a workgroup: RING bytes of rings, its wavefronts' sums, the lists; the
// shorter rings where long lists leave no room for the others.
constexpr int kUpWaves = 8, kMostLds = 163840;
constexpr int kUpRing = 137216, kUpRingShort = 69632, kDownRing = 104448, kDownRingShort = 49152;
constexpr int kUpSums = kUpWaves * 2048, kScratch = 128;
static_assert(kUpRingShort + kUpSums + kScratch + kLayerListBytes <= kMostLds, "the longest lists");
static_assert(kDownRingShort + 4 * kLayerTokens * 2 * 64 + kScratch + kLayerListBytes <= kMostLds, "the longest lists");

// The experts that some token chose, ascending, with their tokens, in dynamic LDS:
// a share is at most 16 tokens of one expert, what a pass over its weights serves.
struct Share {
  int expert, first, n;        // its tokens are those of the positions from `first` on
};
struct Lists {
  v2u* share;                  // [count] expert | first << 16, n
  uint16_t* token;             // [positions] a position's token
  float* weight;               // [positions] its weight (an expert named twice: their sum)
  int count, most;             // shares, the most tokens of one
  __device__ __forceinline__ Share at(int i) const {
    const v2u s = share[i];
    const int x = __builtin_amdgcn_readfirstlane(static_cast<int>(s.x)), n = __builtin_amdgcn_readfirstlane(static_cast<int>(s.y));
    return Share{x & 0xffff, static_cast<int>(static_cast<uint32_t>(x) >> 16), n};
  }
};

// A bit a token for every expert, then the bits' ranks: no order depends on which
// entry comes first.  Entries that are looked at twice are read once where a
// thread has one (together with the weights, under the clearing of the masks).
template <int WAVES, bool WEIGHTS>
__device__ __forceinline__ Lists make_lists(const LayerArgs& a, uint8_t* lds, int* scratch) {
  constexpr int THREADS = WAVES * kWave;
  const ListsLayout at = lists_layout(a.N, a.K, a.E);
  uint64_t* mask = reinterpret_cast<uint64_t*>(lds);
  uint16_t* start = reinterpret_cast<uint16_t*>(lds + at.start);      // [E] first position
  Lists l;
  l.share = reinterpret_cast<v2u*>(lds + at.share);
  l.token = reinterpret_cast<uint16_t*>(lds + at.token);
  l.weight = reinterpret_cast<float*>(lds + at.weight);
  int *sums = scratch, *valid = scratch + WAVES, *most = scratch + 2 * WAVES;      // [WAVES] each
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave, words = at.words;
  const int64_t own = tid < at.entries ? a.idx[tid] - a.first : -1;
  const float own_weight = WEIGHTS && tid < at.entries ? a.wts[tid] : 0.f;
  for (int i = tid; i < a.E * words; i += THREADS) mask[i] = 0;
  __syncthreads();
  int named = 0;
  for (int i0 = 0; i0 < at.entries; i0 += THREADS) {
    const int i = i0 + tid;
    const int64_t e = i0 == 0 ? own : i < at.entries ? a.idx[i] - a.first : -1;
    const int t = i / a.K;
    const bool here = e >= 0 && e < a.E;
    if (here) atomicOr(reinterpret_cast<unsigned long long*>(mask + e * words + t / 64), 1ull << (t & 63));
    named += __builtin_popcountll(ballot(here));
  }
  if (lane == 0) valid[wave] = named;
  __syncthreads();
  int before = 0, fullest = 0;                                        // shares << 16 | positions
  for (int e0 = 0; e0 < a.E; e0 += THREADS) {
    const int e = e0 + tid;
    int n = 0;
    if (e < a.E)
      for (int w = 0; w < words; ++w) n += __builtin_popcountll(mask[e * words + w]);
    fullest = max(fullest, n);
    const int both = (n + 15) / 16 << 16 | n;
    const int inc = wave_inclusive_scan(both);
    if (lane == 63) sums[wave] = inc;
    __syncthreads();
    int mine = before + inc - both;
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) mine += sums[w];
      before += sums[w];
    }
    if (n > 0) start[e] = static_cast<uint16_t>(mine & 0xffff);
    for (int c = 0; c < n; c += 16)
      l.share[(mine >> 16) + c / 16] = v2u{static_cast<uint32_t>(e | ((mine & 0xffff) + c) << 16), static_cast<uint32_t>(min(n - c, 16))};
    if (e0 + THREADS < a.E) __syncthreads();
  }
  l.count = before >> 16;
  for (int d = 32; d > 0; d >>= 1) fullest = max(fullest, __shfl_xor(fullest, d));
  if (lane == 0) most[wave] = fullest;
  __syncthreads();
  named = 0;
  for (int w = 0; w < WAVES; ++w) {
    named += valid[w];
    fullest = max(fullest, most[w]);
  }
  l.most = min(__builtin_amdgcn_readfirstlane(fullest), 16);
  for (int i = tid; i < at.entries; i += THREADS) {
    const int64_t e = i == tid ? own : a.idx[i] - a.first;
    if (e < 0 || e >= a.E) continue;
    const int t = i / a.K;
    int p = start[e];
    for (int w = 0; w < t / 64; ++w) p += __builtin_popcountll(mask[e * words + w]);
    p += __builtin_popcountll(mask[e * words + t / 64] & ((1ull << (t & 63)) - 1));
    l.token[p] = static_cast<uint16_t>(t);
    if constexpr (WEIGHTS) {
      float w = i == tid ? own_weight : a.wts[i];
      if (named != (before & 0xffff)) {                                     // some token names an expert twice: all of its entries' sum
        w = 0.f;
        for (int k = 0; k < a.K; ++k) w += a.idx[t * a.K + k] - a.first == e ? a.wts[t * a.K + k] : 0.f;
      }
      l.weight[p] = w;
    }
  }
  // No load is left open: the compiler would wait for all loads, the rings' too,
  // wherever one's register is used again (fp8, 64 tokens, the second product: 139 -> 198 us).
  __builtin_amdgcn_s_waitcnt(0x0f70);                                 // vmcnt(0)
  __syncthreads();
  return l;
}

// ---- first products: units of 16 gate and 16 up channels of an expert, for 16 of
// its tokens.  A workgroup's units come one after the other through its rings: the
// next unit's first loads are under way while this one's sums are added up.
template <int EL, int XL, int RING>
__device__ __forceinline__ void up_units(const LayerArgs& a, const Lists& l, uint8_t* ring_mem, float* sums) {
  constexpr bool F8 = EL != kGemmBf16;
  using Ring = StreamRing<EL, 4, XL, RING / kUpWaves>;
  constexpr int EB = F8 ? 1 : 2;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const uint32_t ldw = static_cast<uint32_t>(a.H) * EB;
  const int tiles = (a.I + 15) / 16, kb = a.H / kFp8Group;
  const int steps = (a.H + Ring::kChannels - 1) / Ring::kChannels;
  const int mine = wave < steps ? (steps - wave + kUpWaves - 1) / kUpWaves : 0;         // this wavefront's steps of a unit

  const int units = l.count * tiles;                                  // every share's tiles
  // the issuing side
  Ring ring((uint32_t)(uintptr_t)(lds_byte*)ring_mem + wave * (RING / kUpWaves));
  int ahead = blockIdx.x, ahead_step = 0;
  const uint8_t *w = nullptr, *scale = nullptr;
  constexpr int SB = EL == kGemmFp8 ? 4 : 1;                          // bytes of a scale
  uint32_t woff[4], xoff[XL];
  auto set_unit = [&]() MIEP_INLINE {
    const int place = ahead / tiles, i0 = (ahead - place * tiles) * 16;
    const Share u = l.at(place);
    w = static_cast<const uint8_t*>(a.w1) + (static_cast<int64_t>(u.expert) * 2 * a.I + i0) * ldw;
    if constexpr (F8)                                                 // of the gate rows' block, and of the up rows'
      scale = static_cast<const uint8_t*>(a.s1) +
              (static_cast<int64_t>(u.expert) * (2 * a.I / kFp8Group) + ((lane & 1) * a.I + i0) / kFp8Group) * kb * SB;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = Ring::w_row(i);
      woff[i] = static_cast<uint32_t>(min(row & 15, a.I - 1 - i0) + (row >> 4) * a.I) * ldw + Ring::w_chunk(i) * 16;
    }
#pragma unroll
    for (int i = 0; i < XL; ++i)
      xoff[i] = static_cast<uint32_t>(l.token[u.first + min(Ring::x_row(i), u.n - 1)]) * (a.H * 2u) + Ring::x_chunk(i) * 16;
  };
  auto issue = [&]() MIEP_INLINE {
    if (ahead >= units) return;
    if (ahead_step == 0) set_unit();
    const int step = wave + ahead_step * kUpWaves;
    ring.issue(w + step * 128ll, woff, reinterpret_cast<const uint8_t*>(a.x) + step * static_cast<int64_t>(Ring::kXRow), xoff, scale + step * SB,
               a.H - step * Ring::kChannels);
    if (++ahead_step == mine) {
      ahead_step = 0;
      ahead += gridDim.x;
    }
  };
  if (mine > 0) {
#pragma unroll 1
    for (int i = 0; i < Ring::kDepth; ++i) issue();
  }

  for (int at = blockIdx.x; at < units; at += gridDim.x) {
    const int place = at / tiles, i0 = (at - place * tiles) * 16;
    const Share u = l.at(place);
    f32x4 acc[2][1] = {{f32x4{0.f, 0.f, 0.f, 0.f}}, {f32x4{0.f, 0.f, 0.f, 0.f}}};
    for (int i = 0; i < mine; ++i) {
      typename Ring::Frag f;
      ring.take(f, ahead < units);
      issue();
      Ring::multiply(f, [](int p, int) { return p == 1; }, acc);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) *reinterpret_cast<f32x4*>(sums + ((wave * 16 + m) * 2 + p) * 16 + quarter * 4) = acc[p][0];
    all_read();
    for (int i = threadIdx.x; i < 128; i += kUpWaves * kWave) {
      const int col = i / 8, p = i % 8 * 2;
      if (col >= u.n || i0 + p >= a.I) continue;
      float gx = 0.f, gy = 0.f, ux = 0.f, uy = 0.f;
#pragma unroll
      for (int k = 0; k < kUpWaves; ++k) {
        const float* v = sums + (k * 16 + col) * 32 + p;
        gx += v[0];
        gy += v[1];
        ux += v[16];
        uy += v[17];
      }
      *reinterpret_cast<uint32_t*>(a.a + static_cast<int64_t>(u.first + col) * a.I + i0 + p) =
          pack_bf16x2(gx * sigmoid(gx) * ux, gy * sigmoid(gy) * uy);
    }
    all_read();
  }
}

template <int EL, int RING>
__global__ __launch_bounds__(kUpWaves * kWave) void layer_up_kernel(LayerArgs a) {
  extern __shared__ __align__(1024) uint8_t lds[];                    // rings, sums, lists
  float* sums = reinterpret_cast<float*>(lds + RING);
  const Lists l = make_lists<kUpWaves, false>(a, lds + RING + kUpSums + kScratch, reinterpret_cast<int*>(lds + RING + kUpSums));
  const int most = l.most;
  // as few of X's rows as the fullest expert has tokens
  if constexpr (EL == kGemmBf16) {
    if (most <= 8) up_units<EL, 1, RING>(a, l, lds, sums);
    else up_units<EL, 2, RING>(a, l, lds, sums);
  } else {
    if (most <= 4) up_units<EL, 1, RING>(a, l, lds, sums);
    else if (most <= 8) up_units<EL, 2, RING>(a, l, lds, sums);
    else up_units<EL, 4, RING>(a, l, lds, sums);
  }
}

// ---- second products: a.tile output channels a workgroup; the shares' steps one
// after the other go to its wavefronts in turn, so that together they read whole
// rows.  At a share's end a wavefront adds its results, times the gate weights, to
// its own sums of every token.  Of 16 tokens or fewer eight wavefronts have room for
// their sums, which halves the steps of each (the 3 tokens above: 14.5 ->
// 10.7 us; one token over 8 of 7168 x 2048 45.4 -> 43.5), of more of them four.
template <int EL, int WAVES, int WL, int XL, int RING>
__device__ __forceinline__ void down_part(const LayerArgs& a, const Lists& l, uint8_t* ring_mem, float* out) {
  constexpr bool F8 = EL != kGemmBf16;
  using Ring = StreamRing<EL, WL, XL, RING / WAVES>;
  constexpr int EB = F8 ? 1 : 2, TP = Ring::TP, P = 16 * TP;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const int h0 = blockIdx.x * a.tile, kb = a.I / kFp8Group;
  const uint32_t ldw = static_cast<uint32_t>(a.I) * EB, ldx = static_cast<uint32_t>(a.I) * 2;
  const int steps = (a.I + Ring::kChannels - 1) / Ring::kChannels;

  const int total = l.count * steps;                                  // (a share's weights are under 4 GiB, its steps under 2^15)
  struct Walk { int share, step; };
  auto move = [&](Walk& at, int by) MIEP_INLINE {                     // true: to another share
    at.step += by;
    if (at.step < steps) return false;
    while (at.step >= steps) {
      at.step -= steps;
      ++at.share;
    }
    return true;
  };
  const int mine = total > wave ? (total - wave + WAVES - 1) / WAVES : 0;
  Walk at{0, 0};
  move(at, wave);

  Ring ring((uint32_t)(uintptr_t)(lds_byte*)ring_mem + wave * (RING / WAVES));
  uint32_t woff[WL], xoff[XL];
#pragma unroll
  for (int i = 0; i < WL; ++i) woff[i] = static_cast<uint32_t>(min(Ring::w_row(i), min(a.tile, a.H - h0) - 1)) * ldw + Ring::w_chunk(i) * 16;
  // E4M3: the tile's rows lie in one block of 128 or, from row `border` on, in the next
  constexpr int SB = EL == kGemmFp8 ? 4 : 1;                          // bytes of a scale
  const int border = kFp8Group - h0 % kFp8Group;
  const int second = border < min(a.tile, a.H - h0) ? kb : 0;
  Walk ahead = at;
  int issued = 0;
  const uint8_t *w = nullptr, *scale = nullptr;
  bool fresh = true;
  auto issue = [&]() MIEP_INLINE {
    if (issued >= mine) return;
    if (fresh) {
      const Share u = l.at(ahead.share);
      w = static_cast<const uint8_t*>(a.w2) + (static_cast<int64_t>(u.expert) * a.H + h0) * ldw;
      if constexpr (F8)
        scale = static_cast<const uint8_t*>(a.s2) +
                ((static_cast<int64_t>(u.expert) * (a.H / kFp8Group) + h0 / kFp8Group) * kb + (lane & 1) * second) * SB;
#pragma unroll
      for (int i = 0; i < XL; ++i) xoff[i] = static_cast<uint32_t>(u.first + min(Ring::x_row(i), u.n - 1)) * ldx + Ring::x_chunk(i) * 16;
    }
    ring.issue(w + ahead.step * 128ll, woff, reinterpret_cast<const uint8_t*>(a.a) + ahead.step * static_cast<int64_t>(Ring::kXRow), xoff,
               scale + ahead.step * SB, a.I - ahead.step * Ring::kChannels);
    fresh = move(ahead, WAVES);
    ++issued;
  };
#pragma unroll 1
  for (int i = 0; i < Ring::kDepth; ++i) issue();

  f32x4 acc[TP][1];
#pragma unroll
  for (int i = 0; i < TP; ++i) acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int done = 0; done < mine; ++done) {
    const Walk now = at;
    const bool last = move(at, WAVES) || done + 1 == mine;
    typename Ring::Frag f;
    ring.take(f, issued < mine);
    issue();
    Ring::multiply(f, [&](int i, int r) { return i * 16 + quarter * 4 + r >= border; }, acc);
    if (last) {
      const Share u = l.at(now.share);
      if (m < u.n) {
        const int p = u.first + m;
        const float gate = l.weight[p];
#pragma unroll
        for (int i = 0; i < TP; ++i) {
          f32x4* o = reinterpret_cast<f32x4*>(out + l.token[p] * P + i * 16 + quarter * 4);
          f32x4 v = *o;
#pragma unroll
          for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf(gate, acc[i][0][r], v[r]);
          *o = v;
        }
      }
#pragma unroll
      for (int i = 0; i < TP; ++i) acc[i][0] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
  }
}

template <int EL, int WAVES, int WL, int RING>
__global__ __launch_bounds__(WAVES* kWave) void layer_down_kernel(LayerArgs a) {
  constexpr int P = (WL + 1) / 2 * 16, THREADS = WAVES * kWave;
  extern __shared__ __align__(1024) uint8_t lds[];                    // rings, sums, lists
  float* sums = reinterpret_cast<float*>(lds + RING);                 // [wavefront][token][P]
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  float* out = sums + wave * a.N * P;
  for (int i = lane_id(); i < a.N * (P / 4); i += kWave) reinterpret_cast<f32x4*>(out)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  uint8_t* rest = lds + RING + WAVES * a.N * P * 4;
  const Lists l = make_lists<WAVES, true>(a, rest + kScratch, reinterpret_cast<int*>(rest));
  const int most = l.most;
  if constexpr (EL == kGemmBf16) {
    if (most <= 8) down_part<EL, WAVES, WL, 1, RING>(a, l, lds, out);
    else down_part<EL, WAVES, WL, 2, RING>(a, l, lds, out);
  } else {
    if (most <= 4) down_part<EL, WAVES, WL, 1, RING>(a, l, lds, out);
    else if (most <= 8) down_part<EL, WAVES, WL, 2, RING>(a, l, lds, out);
    else down_part<EL, WAVES, WL, 4, RING>(a, l, lds, out);
  }
  __syncthreads();
  const int h0 = blockIdx.x * a.tile, pairs = min(a.tile, a.H - h0) / 2;
  for (int i = threadIdx.x; i < a.N * pairs; i += THREADS) {
    const int t = i / pairs, p = (i - t * pairs) * 2;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
      x += sums[(k * a.N + t) * P + p];
      y += sums[(k * a.N + t) * P + p + 1];
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

template <int EL, int WL>
hipError_t launch_down(const LayerArgs& a, unsigned rest, hipStream_t st) {
  const unsigned tiles = (a.H + a.tile - 1) / a.tile;
  const unsigned sums = a.N * ((WL + 1) / 2) * 64;                    // of a wavefront
  if (kDownRing + 8 * sums + rest <= kMostLds && a.N <= 16) layer_down_kernel<EL, 8, WL, kDownRing><<<tiles, 8 * kWave, kDownRing + 8 * sums + rest, st>>>(a);
  else if (kDownRing + 4 * sums + rest <= kMostLds) layer_down_kernel<EL, 4, WL, kDownRing><<<tiles, 4 * kWave, kDownRing + 4 * sums + rest, st>>>(a);
  else layer_down_kernel<EL, 4, WL, kDownRingShort><<<tiles, 4 * kWave, kDownRingShort + 4 * sums + rest, st>>>(a);
  return hipGetLastError();
}

template <int EL>
hipError_t launch_typed(const LayerArgs& a, hipStream_t st) {
  const ListsLayout lists = lists_layout(a.N, a.K, a.E);
  const int64_t units = static_cast<int64_t>(lists.shares) * ((a.I + 15) / 16);
  const unsigned grid = static_cast<unsigned>(units < 256 ? units : 256), rest = static_cast<unsigned>(lists.end) + kScratch;
  if (kUpRing + kUpSums + rest <= kMostLds) layer_up_kernel<EL, kUpRing><<<grid, kUpWaves * kWave, kUpRing + kUpSums + rest, st>>>(a);
  else layer_up_kernel<EL, kUpRingShort><<<grid, kUpWaves * kWave, kUpRingShort + kUpSums + rest, st>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // as many channels a workgroup as make whole rounds of the 256 CUs, 8 to 32
  LayerArgs d = a;
  const int rounds = (a.H + 256 * 32 - 1) / (256 * 32);
  d.tile = ((a.H + 256 * rounds - 1) / (256 * rounds) + 1) / 2 * 2;
  if (d.tile < 8) d.tile = 8;
  if (d.tile <= 8) return launch_down<EL, 1>(d, rest, st);
  if (d.tile <= 16) return launch_down<EL, 2>(d, rest, st);
  return launch_down<EL, 4>(d, rest, st);
}

}  // namespace

hipError_t launch_layer(const LayerArgs& a, hipStream_t st) {
  if (a.N == 0) return hipSuccess;
  if (a.type == kGemmFp8) return launch_typed<kGemmFp8>(a, st);
  if (a.type == kGemmFp8Ue8m0) return launch_typed<kGemmFp8Ue8m0>(a, st);
  return launch_typed<kGemmBf16>(a, st);
}

}  // namespace miep
