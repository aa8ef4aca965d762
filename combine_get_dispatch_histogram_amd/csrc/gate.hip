// gate.hip -- the router's choice: logits -> top-k experts of every token and
// their weights, and the gradient of the logits.
//
//   s = softmax(l) over the experts, or sigmoid(l) of each
//   choice: the K largest l, or with a bias or groups the K largest s + b among
//   the experts of the best groups (a group's score: the sum of its largest one
//   or two s + b); equal ones by the lower index
//   w_k = scale * s_k, or scale * s_k / (sum of the chosen s)
//
// Backward, for the weights' gradient d (g_k = scale * d_k):
//   softmax                dl_e = s_e * ([e chosen] g_e - sum_k s_k g_k)
//   softmax, renormalised  dl_k = r_k * (g_k - sum_j r_j g_j),  r = w / scale
//   sigmoid                dl_k = g_k * s_k * (1 - s_k)
//   sigmoid, renormalised  dl_k = r_k * (1 - s_k) * (g_k - sum_j r_j g_j)
//
// A choice between s + b is a comparison of rounded sums: in 32 bits about one
// token of 16384 (256 experts) would choose or order its experts otherwise than
// the formula, so those scores are 64-bit.  Without bias and groups s orders the
// experts as l does, and l is compared itself.  Weights are computed in 32 bits.
//
// Up to 512 experts and 16 choices: 16 lanes a token, neighbouring experts a lane,
// in 32 bits with the choice's certainty (gate_rows_kernel): a lane sorts
// its keys once, and the K choices are maxima over 16 lanes' first keys (DPP, no
// LDS).  Otherwise, and for the few tokens whose choice 32 bits leave open, 64
// lanes a token, exactly (gate_token).  16384 tokens, 256 experts in 8 groups: 15 us
// (all of them exactly: 38), of which the logits' 17 MB would take 3: bound by its
// instructions (sorting, and nine rounds of a maximum): 1,370 a wavefront, 9 us at one
// in four cycles, and VALUs busy for 74% of the time that a CU is.  The gradient of a
// softmax over 256 experts, 16384 tokens, 34 MB: 10 us; 650 instructions a wavefront,
// VALUs busy for 69% of a CU's time, behind two loads one after the other (the choices,
// then the logits they name) that nothing covers in a single round of wavefronts.
#include "device.h"
#include "gemm.h"

namespace miep {

namespace {

constexpr float kMost = 3.402823466e38f;
constexpr float kNone = -INFINITY;

template <int CTRL, class T>
__device__ __forceinline__ T dpp(T v) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(T, static_cast<uint64_t>(hi) << 32 | lo);
  } else {
    return __builtin_bit_cast(T, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xF, 0xF, true));
  }
}

// v of the lanes' partners: the pair (a, b) holds, in every lane, the values of
// a lane of the even and of the odd half (of 32 lanes, or of 16).
template <bool ROWS>
__device__ __forceinline__ void swap_halves(uint32_t v, uint32_t* a, uint32_t* b) {
  const auto r = ROWS ? __builtin_amdgcn_permlane16_swap(v, v, false, false) : __builtin_amdgcn_permlane32_swap(v, v, false, false);
  *a = r[0];
  *b = r[1];
}
template <bool ROWS, class T>
__device__ __forceinline__ void swap_halves_of(T v, T* a, T* b) {
  if constexpr (sizeof(T) == 8) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t al, bl, ah, bh;
    swap_halves<ROWS>(static_cast<uint32_t>(u), &al, &bl);
    swap_halves<ROWS>(static_cast<uint32_t>(u >> 32), &ah, &bh);
    *a = __builtin_bit_cast(T, static_cast<uint64_t>(ah) << 32 | al);
    *b = __builtin_bit_cast(T, static_cast<uint64_t>(bh) << 32 | bl);
  } else {
    uint32_t x, y;
    swap_halves<ROWS>(__builtin_bit_cast(uint32_t, v), &x, &y);
    *a = __builtin_bit_cast(T, x);
    *b = __builtin_bit_cast(T, y);
  }
}

// Over the wavefront, every lane active; all lanes get the same bits.
template <class T, class F>
__device__ __forceinline__ T wave_all(T v, F f) {
  v = f(v, dpp<0xB1>(v));    // quad_perm [1,0,3,2]
  v = f(v, dpp<0x4E>(v));    // quad_perm [2,3,0,1]
  v = f(v, dpp<0x141>(v));   // row_half_mirror
  v = f(v, dpp<0x140>(v));   // row_mirror
  T a, b;
  swap_halves_of<true>(v, &a, &b);
  v = f(a, b);
  swap_halves_of<false>(v, &a, &b);
  return f(a, b);
}
template <class T>
__device__ __forceinline__ T bigger(T a, T b) { return a > b ? a : b; }
__device__ __forceinline__ float bigger(float a, float b) { return __builtin_fmaxf(a, b); }
__device__ __forceinline__ double bigger(double a, double b) { return __builtin_fmax(a, b); }
template <class T>
__device__ __forceinline__ T wave_max(T v) { return wave_all(v, [](T a, T b) { return bigger(a, b); }); }
template <class T>
__device__ __forceinline__ T wave_sum(T v) { return wave_all(v, [](T a, T b) { return a + b; }); }

__device__ __forceinline__ double readlane(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), l);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// NaN is a masked expert, like -inf; +inf the largest number of the type.
template <bool F32>
__device__ __forceinline__ float usable(float l) {
  return l == l ? __builtin_fminf(l, F32 ? kMost : 0x1.fep127f) : kNone;
}

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int e) {
  if constexpr (F32) return usable<F32>(static_cast<const float*>(row)[e]);
  else return usable<F32>(__uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[e]) << 16));
}

// Experts in `lanes` lanes, V each: in pieces of PER neighbours that the lanes take
// in turn (16 bytes where V and the type give as many), so that a load's lanes lie
// side by side; single experts where the rows or groups are not whole pieces.
template <int V, bool F32>
constexpr int kPiece = V < (F32 ? 4 : 8) ? V : (F32 ? 4 : 8);
template <int PER>
__device__ __forceinline__ int expert_of(int v, int lanes, int lane, bool wide) {
  return wide ? ((v / PER) * lanes + lane) * PER + v % PER : v * lanes + lane;
}

// The lane's V of the n numbers from row[first] on, -inf behind them.
template <int V, int PER, bool F32>
__device__ __forceinline__ void load_logits(const void* row, int first, int n, int lanes, int lane, bool wide, float (&l)[V]) {
  if (wide) {
#pragma unroll
    for (int v = 0; v < V; v += PER) {
      const int at = expert_of<PER>(v, lanes, lane, true);
      constexpr int BYTES = PER * (F32 ? 4 : 2);
      uint32_t w[BYTES < 4 ? 1 : BYTES / 4] = {};
      if (at < n) {
        const uint8_t* p = static_cast<const uint8_t*>(row) + (first + at) * (F32 ? 4ll : 2ll);
        if constexpr (BYTES >= 16) {
#pragma unroll
          for (int i = 0; i < BYTES / 16; ++i) {
            const v4u t = ld16(p + i * 16);
            w[i * 4] = t.x; w[i * 4 + 1] = t.y; w[i * 4 + 2] = t.z; w[i * 4 + 3] = t.w;
          }
        } else if constexpr (BYTES == 8) {
          const v2u t = *reinterpret_cast<const v2u*>(p);
          w[0] = t.x; w[1] = t.y;
        } else if constexpr (BYTES == 4) {
          w[0] = *reinterpret_cast<const uint32_t*>(p);
        } else {
          w[0] = *reinterpret_cast<const uint16_t*>(p);
        }
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        float x;
        if constexpr (F32) x = __uint_as_float(w[i]);
        else x = i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
        l[v + i] = at < n ? usable<F32>(x) : kNone;
      }
    }
  } else {
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int at = expert_of<PER>(v, lanes, lane, false);
      l[v] = at < n ? logit<F32>(row, first + at) : kNone;
    }
  }
}

// Places of the K largest of the wavefront's values (V a lane, place = lane * V
// + v), the largest first, equal ones by place, to lanes 0 .. K-1; -1 where only
// -inf is left.
template <int V, class T>
__device__ __forceinline__ int choose(T (&val)[V], int K) {
  const int lane = lane_id();
  int mine = -1;
  for (int k = 0; k < K; ++k) {
    T m = val[0];
#pragma unroll
    for (int v = 1; v < V; ++v) m = bigger(m, val[v]);
    const T top = wave_max(m);
    if (!(top > static_cast<T>(kNone))) break;
    const int win = __builtin_ctzll(ballot(m == top));
    int pos = V - 1;
#pragma unroll
    for (int v = V - 2; v >= 0; --v) pos = val[v] == top ? v : pos;
    const int e = miep::readlane(lane * V + pos, win);
    if (lane == k) mine = e;
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (lane == win && v == pos) val[v] = static_cast<T>(kNone);
  }
  return mine;
}

// exp(l - m) with 0 for a masked expert.
__device__ __forceinline__ float rel_exp(float l, float m) { return l > kNone ? expf(l - m) : 0.f; }

// The chosen expert's score over e^m: sigmoid(l), for l < 0 written so that
// far negative logits keep their ratios.
__device__ __forceinline__ float sigmoid_over(float l, float m) {
  return l >= 0.f ? 1.f / (1.f + expf(-l)) : expf(l - m) / (1.f + expf(l));
}

// One token over the wavefront: V experts a lane, scores in 64 bits.  mem: 64 * V
// numbers of LDS.
template <int V, bool F32, bool SCORES>
__device__ __forceinline__ void gate_token(const GateArgs& a, int64_t t, double* mem) {
  const int lane = lane_id();
  const int E = a.E, K = a.K;
  const int64_t pitch = static_cast<int64_t>(E) * (F32 ? 4 : 2);
  const void* row = static_cast<const uint8_t*>(a.logits) + t * pitch;
  constexpr int PER = kPiece<V, F32>;
  float l[V];
  load_logits<V, PER, F32>(row, lane * V, E - lane * V, 1, 0, E % PER == 0, l);
  float top = l[0];
#pragma unroll
  for (int v = 1; v < V; ++v) top = bigger(top, l[v]);
  float sum = 0.f;
  const bool rows_sum = a.score == kGateSoftmax && !a.renorm;
  if (rows_sum) {
    top = wave_max(top);
#pragma unroll
    for (int v = 0; v < V; ++v) sum += rel_exp(l[v], top);
    sum = wave_sum(sum);
  }
  int mine;
  if constexpr (SCORES) {
    double c[V];
    if (a.score == kGateSoftmax) {
      const double m = wave_max(top);
      double s = 0.0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        c[v] = l[v] > kNone ? exp(static_cast<double>(l[v]) - m) : 0.0;
        s += c[v];
      }
      s = wave_sum(s);
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] /= s;
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) c[v] = 1.0 / (1.0 + exp(-static_cast<double>(l[v])));
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int e = lane * V + v;
      if (a.bias && e < E) c[v] += usable<true>(a.bias[e]);
      if (!(l[v] > kNone)) c[v] = kNone;
    }
    if (a.groups > 1) {
      // a lane a group: its best one or two scores, from LDS; lanes start at
      // different members so that they read different banks
#pragma unroll
      for (int v = 0; v < V; ++v) mem[lane * V + v] = c[v];
      __builtin_amdgcn_wave_barrier();
      double one = kNone, two = kNone;
      if (lane < a.groups) {
        int j = lane % a.per_group;
        for (int i = 0; i < a.per_group; ++i) {
          const double x = mem[lane * a.per_group + j];
          two = bigger(two, x < one ? x : one);
          one = bigger(one, x);
          j = j + 1 == a.per_group ? 0 : j + 1;
        }
        if (a.group_best == 2) one += two;
      }
      __builtin_amdgcn_wave_barrier();
      int before = 0;
      for (int g = 0; g < a.groups; ++g) {
        const double x = readlane(one, g);
        before += x > one || (x == one && g < lane);
      }
      const uint64_t in = ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (!(in >> (fdiv(lane * V + v, a.per_div) & 63) & 1)) c[v] = kNone;
    }
    mine = choose<V>(c, K);
  } else {
    mine = choose<V>(l, K);
  }
  // lane k: the weight of choice k
  const bool live = mine >= 0;
  const float own = live ? logit<F32>(row, mine) : kNone;
  float w;
  if (a.score == kGateSoftmax) {
    const float m = rows_sum ? top : wave_max(own);
    w = rel_exp(own, m);
    if (a.renorm) sum = wave_sum(w);
    w = live ? w / sum : 0.f;
  } else {
    const float m = a.renorm ? bigger(wave_max(own), -kMost) : 0.f;
    w = live ? sigmoid_over(own, m < 0.f ? m : 0.f) : 0.f;
    if (a.renorm) {
      sum = wave_sum(w);
      w = live ? w / sum : 0.f;
    }
  }
  if (lane < K) {
    a.idx[t * K + lane] = mine;
    a.w[t * K + lane] = w * a.scale;
  }
}

template <int V, bool F32, bool SCORES>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs a) {
  __shared__ double lds[SCORES ? 4 * 64 * V : 1];
  double* mem = SCORES ? lds + threadIdx.x / kWave * 64 * V : lds;
  for (int64_t t = wave_index(); t < a.N; t += static_cast<int64_t>(gridDim.x) * 4) gate_token<V, F32, SCORES>(a, t, mem);
}

// ---- 16 lanes a token
template <class T, class F>
__device__ __forceinline__ T row_all(T v, F f) {
  v = f(v, dpp<0xB1>(v));
  v = f(v, dpp<0x4E>(v));
  v = f(v, dpp<0x141>(v));
  return f(v, dpp<0x140>(v));
}
__device__ __forceinline__ float row_max(float v) { return row_all(v, [](float a, float b) { return __builtin_fmaxf(a, b); }); }
__device__ __forceinline__ int row_max(int v) { return row_all(v, [](int a, int b) { return max(a, b); }); }
__device__ __forceinline__ float row_sum(float v) { return row_all(v, [](float a, float b) { return a + b; }); }

// Numbers as integers of the same order, and back.
constexpr int kNoKey = static_cast<int>(0x80000000u);
__device__ __forceinline__ int key_of(float f) {
  const int b = __float_as_int(f + 0.f);                              // (-0 is 0)
  return b ^ ((b >> 31) & 0x7fffffff);
}
__device__ __forceinline__ float of_key(int k) { return k == kNoKey ? kNone : __int_as_float(k ^ ((k >> 31) & 0x7fffffff)); }

// exp(x) to 2^-23 and |x| * 2^-24 of itself: enough to choose by, where a choice
// within that is made again.
__device__ __forceinline__ float quick_exp(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }

// Descending, by Batcher's merge exchange.
template <int V>
__device__ __forceinline__ void sort_keys(int (&v)[V]) {
#pragma unroll
  for (int p = 1; p < V; p *= 2)
#pragma unroll
    for (int k = p; k >= 1; k /= 2)
#pragma unroll
      for (int j = k % p; j + k < V; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < V && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const int x = v[i + j], y = v[i + j + k];
            v[i + j] = max(x, y);
            v[i + j + k] = min(x, y);
          }
}

// A token in 16 lanes: a.lanes of them for each group (all without groups), each
// with a.each of its experts, at most V.  A lane's keys are what is compared with
// the place in the lane in the last 4 bits (5 of 32 experts a lane), so that they
// sort by two instructions an exchange:
//   bf16 logits      the logit, exactly, and the expert in the lower 16 bits
//   fp32 logits      the logit, without those bits
//   s + bias         in 32 bits, without those bits
// Where two neighbours among the chosen and the next, or the last chosen group and
// the next, are nearer than the cut and the scores' errors together (a few 2^-23;
// one token in 100 or so), the candidates alone, a lane each, are compared in 64
// bits: as many as are clear of the next one.  What that leaves (more than 16
// candidates, a third one of a group) is chosen again by gate_token.
template <int V, bool F32, bool SCORES, bool WIDE>
__global__ __launch_bounds__(256, V <= 16 ? 4 : 2) void gate_rows_kernel(GateArgs a) {
  __shared__ double exact_mem[SCORES ? 4 * 16 * V : 1];
  __shared__ int chosen[4][4][16];
  __shared__ __align__(16) int sorted[4][64][V];
  const int lane = lane_id(), sub = lane & 15, seg = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x / kWave));
  const int E = a.E, K = a.K;
  const int64_t pitch = static_cast<int64_t>(E) * (F32 ? 4 : 2);
  constexpr int PER = kPiece<V, F32>;
  const int group = sub / a.lanes, in_group = sub % a.lanes, e0 = group * a.per_group;
  const int n = group < a.groups ? a.per_group : 0;                   // experts of the lane's group
  constexpr bool wide = WIDE;                                         // whole pieces
  constexpr int LOW = V <= 16 ? 15 : 31;
  constexpr bool EXACT = !F32 && !SCORES;                             // keys are the logits themselves
  for (int64_t t0 = wave_index() * 4; t0 < a.N; t0 += static_cast<int64_t>(gridDim.x) * 16) {
    const int64_t t = t0 + seg < a.N ? t0 + seg : a.N - 1;
    const void* row = static_cast<const uint8_t*>(a.logits) + t * pitch;
    float c[V];
    load_logits<V, PER, F32>(row, e0, n, a.lanes, in_group, wide, c);
    const bool rows_sum = a.score == kGateSoftmax && (SCORES || !a.renorm);
    float top = 0.f, sum = 0.f;
    if (rows_sum) {
      top = c[0];
#pragma unroll
      for (int v = 1; v < V; ++v) top = __builtin_fmaxf(top, c[v]);
      top = __builtin_fmaxf(row_max(top), -kMost);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const float x = quick_exp(c[v] - top);
        sum += x;
        if constexpr (SCORES) c[v] = c[v] > kNone ? x : kNone;
      }
      sum = row_sum(sum);
    }
    if constexpr (SCORES) {
      // (without a bias the denominator changes no comparison)
      const float inv = a.bias ? __builtin_amdgcn_rcpf(sum) : 1.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (a.score == kGateSoftmax) c[v] *= inv;
        else c[v] = c[v] > kNone ? __builtin_amdgcn_rcpf(1.f + quick_exp(-c[v])) : kNone;
      }
      if (a.bias) {
        float b[V];
        load_logits<V, PER, true>(a.bias, e0, n, a.lanes, in_group, wide, b);
#pragma unroll
        for (int v = 0; v < V; ++v) c[v] += b[v];
      }
    }
    int key[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int b = key_of(c[v]), low = EXACT ? 0xffff - e0 - expert_of<PER>(v, a.lanes, in_group, wide) : LOW - v;
      key[v] = c[v] > kNone ? (EXACT ? b & ~0xffff : b & ~LOW) | low : kNoKey;
    }
    sort_keys(key);
#pragma unroll
    for (int v = 0; v < V; ++v) sorted[wave][lane][v] = key[v];
    auto place = [&](int k) MIEP_INLINE { return EXACT ? 0xffff - (k & 0xffff) : e0 + expert_of<PER>(LOW - (k & LOW), a.lanes, in_group, wide); };
    // the nearest that two keys may be to stand for their order
    constexpr float kStep = V <= 16 ? 0x1p-18f : 0x1p-17f;            // both keys' last bits
    auto apart = [&](float x) MIEP_INLINE {
      const float y = fabsf(x);
      return SCORES ? (kStep + 0x1p-21f) * (y > 1.f ? y : 1.f) : __builtin_fmaxf(kStep * y, 0x1p-120f);
    };
    // what an expert is compared by, in 64 bits
    double denominator = 1.0;
    auto prepare = [&]() MIEP_INLINE {
      if (!SCORES || a.score != kGateSoftmax || !a.bias) return;
      double d = 0.0;
#pragma unroll 1
      for (int e = sub; e < E; e += 16) d += exp(static_cast<double>(logit<F32>(row, e)) - static_cast<double>(top));
      denominator = row_all(d, [](double x, double y) { return x + y; });
    };
    auto exact = [&](int e) MIEP_INLINE {
      const double l = logit<F32>(row, e);
      if constexpr (!SCORES) return l;
      const double s = a.score == kGateSoftmax ? exp(l - static_cast<double>(top)) / denominator : 1.0 / (1.0 + exp(-l));
      return a.bias ? s + static_cast<double>(usable<true>(a.bias[e])) : s;
    };
    bool open = false;                                                // for gate_token
    if constexpr (SCORES) {
      if (a.groups > 1) {
        const int lanes = a.lanes;                                    // 1, 2, 4 or 8
        auto best_two = [&](auto& one, auto& two) MIEP_INLINE {
          auto merge = [&](auto x, auto y) MIEP_INLINE {
            two = bigger(one < x ? one : x, bigger(two, y));
            one = bigger(one, x);
          };
          if (lanes > 1) merge(dpp<0xB1>(one), dpp<0xB1>(two));
          if (lanes > 2) merge(dpp<0x4E>(one), dpp<0x4E>(two));
          if (lanes > 4) merge(dpp<0x141>(one), dpp<0x141>(two));
        };
        auto before = [&](auto score) MIEP_INLINE {                   // better groups
          int n = 0;
          for (int g = 0; g < a.groups; ++g) {
            const auto x = __shfl(score, (lane & 48) + g * lanes);
            n += x > score || (x == score && g < group);
          }
          return n;
        };
        float one = of_key(key[0]), two = of_key(key[1]);
        best_two(one, two);
        // Half a sum (so that none overflows), and its distance from the formula's at most: half of what
        // its members' keys may be off, which goes by each one's own size and not the sum's (s + 1000 and
        // s - 1000 make one near 1); an eighth of a step for roundings and the softmax's denominator (some
        // 30 of 2^-24).  Any two groups farther apart than twice the largest of these are in order.
        const bool both = a.group_best == 2;
        const float score = both ? 0.5f * one + 0.5f * two : one;
        float off = both ? 0.25f * apart(one) + 0.25f * apart(two) : 0.5f * apart(one);
        off = row_max(score > kNone ? off + 0.125f * kStep : 0.f);    // (a group that has none scores -inf, exactly)
        bool in = before(score) < a.top_groups && group < a.groups;
        const float least = -row_max(in ? -score : kNone), next = row_max(in || group >= a.groups ? kNone : score);
        const bool near = least - next <= 2.f * off;                  // (both -inf: by the index)
        if (ballot(near) != 0) {
          // the same from each lane's first two in 64 bits, unless a third may be one of its group's two
          const bool third = key[2] != kNoKey && of_key(key[2]) >= two - 2.f * apart(two);
          const uint32_t any = static_cast<uint32_t>(ballot(third) >> (lane & 48)) & 0xffffu;
          open = near && any != 0;
          prepare();
          {
            const double x = key[0] != kNoKey ? exact(place(key[0])) : kNone, y = key[1] != kNoKey ? exact(place(key[1])) : kNone;
            double p = bigger(x, y), q = x < y ? x : y;
            best_two(p, q);
            const bool sure = before(a.group_best == 2 ? p + q : p) < a.top_groups && group < a.groups;
            in = near ? sure : in;
          }
        }
        if (!in) key[0] = kNoKey;
      }
    }
    float last = 0.f;
    bool near = false;                                                // some neighbours so far
    int count = 0;                                                    // candidates
    int head = key[0], taken = 0;                                     // the lane's first key that is left
    while (true) {
      const int best = row_max(head);
      bool here = false;
      if constexpr (!EXACT) {
        const float x = of_key(best);
        here = count > 0 && last - x <= apart(last);
        last = x;
        near = near || (here && count <= K);
      }
      if (count >= K) {
        // done when the candidates so far are clear of the next
        const bool go_on = here && count < 16;
        open = open || (here && !go_on);
        if (EXACT || ballot(go_on) == 0) break;
      }
      const uint32_t who = static_cast<uint32_t>(ballot(head == best) >> (lane & 48)) & 0xffffu;
      if (__builtin_ctz(who) == sub) {
        chosen[wave][seg][count] = best != kNoKey ? place(best) : -1;
        ++taken;
        head = taken < V && best != kNoKey ? sorted[wave][lane][taken & (V - 1)] : kNoKey;
      }
      ++count;
    }
    if (!EXACT && ballot(near) != 0) {
      prepare();
      __builtin_amdgcn_wave_barrier();
      const int e = sub < count ? chosen[wave][seg][sub] : -1;
      const double d = e >= 0 ? exact(e) : kNone;
      int better = 0;
      for (int j = 0; j < count; ++j) {
        const double x = __shfl(d, (lane & 48) + j);
        const int f = __shfl(e, (lane & 48) + j);
        better += f >= 0 && (x > d || (x == d && f < e));
      }
      __builtin_amdgcn_wave_barrier();
      if (e >= 0) chosen[wave][seg][better] = e;                      // (those that are none stay behind)
    }
    __builtin_amdgcn_wave_barrier();
    // lane k: the weight of choice k
    const int mine = sub < K ? chosen[wave][seg][sub] : -1;
    __builtin_amdgcn_wave_barrier();
    const bool live = mine >= 0;
    const float own = live ? logit<F32>(row, mine) : kNone;
    float w;
    if (a.score == kGateSoftmax) {
      const float m = a.renorm ? row_max(own) : top;
      w = rel_exp(own, m);
      if (a.renorm) sum = row_sum(w);
      w = live ? w / sum : 0.f;
    } else {
      const float m = a.renorm ? __builtin_fmaxf(row_max(own), -kMost) : 0.f;
      w = live ? sigmoid_over(own, m < 0.f ? m : 0.f) : 0.f;
      if (a.renorm) {
        sum = row_sum(w);
        w = live ? w / sum : 0.f;
      }
    }
    if (sub < K && t0 + seg < a.N && !open) {
      a.idx[t * K + sub] = mine;
      a.w[t * K + sub] = w * a.scale;
    }
    uint64_t again = ballot(open && t0 + seg < a.N);
    while (again != 0) {
      const int s = __builtin_ctzll(again) / 16;
      again &= ~(0xffffull << (s * 16));
      gate_token<V / 4, F32, SCORES>(a, t0 + s, SCORES ? exact_mem + wave * 16 * V : exact_mem);
    }
  }
}

// LANES (16 or 64) lanes a token, V neighbouring experts a lane; lane k also has
// choice k (with more than LANES choices: 64 lanes).  The choices' gradients meet
// the experts' in LDS: every choice writes its own place, one that is named twice
// the sum.
template <int LANES, int V, bool F32>
__global__ __launch_bounds__(256) void gate_backward_kernel(GateArgs a) {
  __shared__ __align__(16) float mem[256 / LANES][LANES * V];
  const int lane = lane_id(), sub = lane % LANES;
  const int E = a.E, K = a.K;
  const int64_t pitch = static_cast<int64_t>(E) * (F32 ? 4 : 2);
  const bool dense = a.score == kGateSoftmax && !a.renorm;
  float* at = mem[threadIdx.x / LANES];
  auto all_max = [&](float v) MIEP_INLINE { return LANES == 16 ? row_max(v) : wave_max(v); };
  auto all_sum = [&](float v) MIEP_INLINE { return LANES == 16 ? row_sum(v) : wave_sum(v); };
  constexpr int PER_WAVE = kWave / LANES, PER = kPiece<V, F32>;
  const bool wide = E % PER == 0;
  for (int64_t t0 = wave_index() * PER_WAVE; t0 < a.N; t0 += static_cast<int64_t>(gridDim.x) * 4 * PER_WAVE) {
    const int64_t t = t0 + lane / LANES < a.N ? t0 + lane / LANES : a.N - 1;
    const void* row = static_cast<const uint8_t*>(a.logits) + t * pitch;
    const int64_t e64 = sub < K ? a.idx[t * K + sub] : -1;
    const int mine = e64 >= 0 && e64 < E ? static_cast<int>(e64) : -1;
    const float given = mine >= 0 ? a.d_w[t * K + sub] * a.scale : 0.f;
    const float own = mine >= 0 ? logit<F32>(row, mine) : kNone;
    float g = own > kNone ? given : 0.f;                              // (a masked expert's weight is 0 and stays so, whatever d_w holds there)
    float p[V];
    float dot = 0.f;
    if (dense) {
      load_logits<V, PER, F32>(row, 0, E, LANES, sub, wide, p);
      float top = p[0];
#pragma unroll
      for (int v = 1; v < V; ++v) top = bigger(top, p[v]);
      top = bigger(all_max(top), -kMost);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = rel_exp(p[v], top);
        sum += p[v];
      }
      sum = all_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] *= inv;
      dot = all_sum(rel_exp(own, top) * inv * g);
    } else if (a.score == kGateSoftmax) {
      const float m = all_max(own);
      float r = rel_exp(own, m);
      const float sum = all_sum(r);
      r = own > kNone ? r / sum : 0.f;
      g = r * (g - all_sum(r * g));
    } else {
      const float m = bigger(all_max(own), -kMost);
      const float down = own > kNone ? 1.f / (1.f + expf(own)) : 0.f;      // 1 - s
      if (a.renorm) {
        float r = own > kNone ? sigmoid_over(own, m < 0.f ? m : 0.f) : 0.f;
        const float sum = all_sum(r);
        r = own > kNone ? r / sum : 0.f;
        g = r * down * (g - all_sum(r * g));
      } else {
        g = own > kNone ? g * sigmoid_over(own, 0.f) * down : 0.f;
      }
    }
    // who else names this expert: the last writer's lane stands in its place
#pragma unroll
    for (int v = 0; v < V; ++v) at[sub + v * LANES] = 0.f;
    __builtin_amdgcn_wave_barrier();
    if (mine >= 0) at[mine] = __int_as_float(sub + 1);
    __builtin_amdgcn_wave_barrier();
    const bool twice = mine >= 0 && __float_as_int(at[mine]) != sub + 1;
    if (ballot(twice) != 0) {
      float both = 0.f;
      for (int k = 0; k < K; ++k) {                                   // all of them, in order
        const int e = __shfl(mine, lane - sub + k);
        const float x = __shfl(g, lane - sub + k);
        if (e == mine) both += x;
      }
      g = both;
    }
    __builtin_amdgcn_wave_barrier();
    if (mine >= 0) at[mine] = g;
    __builtin_amdgcn_wave_barrier();
    float d[V];
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = at[expert_of<PER>(v, LANES, sub, wide)];
    __builtin_amdgcn_wave_barrier();
    if (dense) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = p[v] * (d[v] - dot);
    }
    if (t0 + lane / LANES >= a.N) continue;
    uint8_t* out = static_cast<uint8_t*>(a.d_logits) + t * pitch;
    if (wide) {
#pragma unroll
      for (int v = 0; v < V; v += PER) {
        const int e = expert_of<PER>(v, LANES, sub, true);
        if (e >= E) continue;
        uint8_t* to = out + e * (F32 ? 4ll : 2ll);
        if constexpr (F32) {
          *reinterpret_cast<v4u*>(to) = v4u{__float_as_uint(d[v]), __float_as_uint(d[v + 1]), __float_as_uint(d[v + 2]), __float_as_uint(d[v + 3])};
        } else if constexpr (PER == 8) {
          *reinterpret_cast<v4u*>(to) = v4u{pack_bf16x2(d[v], d[v + 1]), pack_bf16x2(d[v + 2], d[v + 3]), pack_bf16x2(d[v + 4], d[v + 5]), pack_bf16x2(d[v + 6], d[v + 7])};
        } else {
          *reinterpret_cast<v2u*>(to) = v2u{pack_bf16x2(d[v], d[v + 1]), pack_bf16x2(d[v + 2], d[v + 3])};
        }
      }
    } else {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int e = expert_of<PER>(v, LANES, sub, false);
        if (e >= E) continue;
        if constexpr (F32) reinterpret_cast<float*>(out)[e] = d[v];
        else reinterpret_cast<uint16_t*>(out)[e] = static_cast<uint16_t>(pack_bf16x2(d[v], 0.f));
      }
    }
  }
}

template <int V>
void launch_tokens(const GateArgs& a, bool scores, unsigned grid, hipStream_t st) {
  if (a.f32 && scores) gate_kernel<V, true, true><<<grid, 256, 0, st>>>(a);
  else if (a.f32) gate_kernel<V, true, false><<<grid, 256, 0, st>>>(a);
  else if (scores) gate_kernel<V, false, true><<<grid, 256, 0, st>>>(a);
  else gate_kernel<V, false, false><<<grid, 256, 0, st>>>(a);
}

template <int LANES, int V>
void launch_backward(const GateArgs& a, hipStream_t st) {
  const int64_t wgs = (a.N + 256 / LANES - 1) / (256 / LANES);
  const unsigned grid = static_cast<unsigned>(wgs < (1 << 20) ? wgs : (1 << 20));
  if (a.f32) gate_backward_kernel<LANES, V, true><<<grid, 256, 0, st>>>(a);
  else gate_backward_kernel<LANES, V, false><<<grid, 256, 0, st>>>(a);
}

template <int V, bool F32, bool SCORES>
void launch_rows_typed(const GateArgs& a, unsigned grid, hipStream_t st) {
  constexpr int PER = kPiece<V, F32>;
  if (a.E % PER == 0 && a.per_group % PER == 0) gate_rows_kernel<V, F32, SCORES, true><<<grid, 256, 0, st>>>(a);
  else gate_rows_kernel<V, F32, SCORES, false><<<grid, 256, 0, st>>>(a);
}

template <int V>
void launch_rows_kernel(const GateArgs& a, bool scores, unsigned grid, hipStream_t st) {
  if (a.f32 && scores) launch_rows_typed<V, true, true>(a, grid, st);
  else if (a.f32) launch_rows_typed<V, true, false>(a, grid, st);
  else if (scores) launch_rows_typed<V, false, true>(a, grid, st);
  else launch_rows_typed<V, false, false>(a, grid, st);
}

}  // namespace

hipError_t launch_gate(const GateArgs& args, bool backward, hipStream_t st) {
  GateArgs a = args;
  if (a.N == 0) return hipSuccess;
  a.per_group = a.E / a.groups;
  a.per_div = make_fastdiv(a.per_group);
  if (a.per_group == 1) a.group_best = 1;                             // there is no second member to add
  const bool scores = a.bias || a.groups > 1;
  const int64_t wgs = (a.N + 3) / 4;
  const unsigned grid = static_cast<unsigned>(wgs < (1 << 20) ? wgs : (1 << 20));
  if (backward) {
    if (a.K <= 16 && a.E <= 256) {
      if (a.E <= 64) launch_backward<16, 4>(a, st);
      else if (a.E <= 128) launch_backward<16, 8>(a, st);
      else launch_backward<16, 16>(a, st);
    } else if (a.E <= 256) {
      launch_backward<64, 4>(a, st);
    } else if (a.E <= 512) {
      launch_backward<64, 8>(a, st);
    } else if (a.E <= 1024) {
      launch_backward<64, 16>(a, st);
    } else {
      launch_backward<64, 32>(a, st);
    }
    return hipGetLastError();
  }
  // 16 lanes a token, if they hold its experts: a power of two of them a group
  a.lanes = 16;
  while (a.lanes * a.groups > 16) a.lanes /= 2;
  if (a.lanes > 0) a.each = (a.per_group + a.lanes - 1) / a.lanes;
  const int piece = a.f32 ? 4 : 8;                                    // whole 16-byte pieces a lane where the groups have them
  if (a.per_group % piece == 0) a.each = (a.each + piece - 1) / piece * piece;
  if (a.lanes > 0 && a.each <= 32 && a.K <= 16) {
    const int64_t rows_wgs = (a.N + 15) / 16;
    const unsigned rows_grid = static_cast<unsigned>(rows_wgs < (1 << 20) ? rows_wgs : (1 << 20));
    if (a.each <= 4) launch_rows_kernel<4>(a, scores, rows_grid, st);
    else if (a.each <= 8) launch_rows_kernel<8>(a, scores, rows_grid, st);
    else if (a.each <= 16) launch_rows_kernel<16>(a, scores, rows_grid, st);
    else launch_rows_kernel<32>(a, scores, rows_grid, st);
    return hipGetLastError();
  }
  if (a.E <= 64) launch_tokens<1>(a, scores, grid, st);
  else if (a.E <= 128) launch_tokens<2>(a, scores, grid, st);
  else if (a.E <= 256) launch_tokens<4>(a, scores, grid, st);
  else if (a.E <= 512) launch_tokens<8>(a, scores, grid, st);
  else if (a.E <= 1024) launch_tokens<16>(a, scores, grid, st);
  else launch_tokens<32>(a, scores, grid, st);
  return hipGetLastError();
}

}  // namespace miep
