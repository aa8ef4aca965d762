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
// One wavefront a token, V neighbouring experts a lane; the K choices are K
// maxima over the wavefront (DPP and permlane exchanges, no LDS).
#include "device.h"

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

__device__ __forceinline__ float readlane(float v, int l) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
}
__device__ __forceinline__ double readlane(double v, int l) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), l);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), l);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}

// NaN is a masked expert, like -inf; +inf the largest number.
__device__ __forceinline__ float usable(float l) { return l == l ? __builtin_fminf(l, kMost) : kNone; }

template <bool F32>
__device__ __forceinline__ float logit(const void* row, int e) {
  if constexpr (F32) return usable(static_cast<const float*>(row)[e]);
  else return usable(__uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(row)[e]) << 16));
}

// The lane's V logits, -inf behind the last expert.
template <int V, bool F32>
__device__ __forceinline__ void load_logits(const void* row, int E, bool wide, float (&l)[V]) {
  const int e0 = lane_id() * V;
  constexpr int PER = F32 ? 4 : 8;                                    // a 16-byte load
  if constexpr (V % PER == 0) {
    if (wide) {
#pragma unroll
      for (int v = 0; v < V; v += PER) {
        if (e0 + v < E) {
          const v4u t = ld16(static_cast<const uint8_t*>(row) + (e0 + v) * (F32 ? 4ll : 2ll));
          const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
          for (int i = 0; i < PER; ++i) {
            if constexpr (F32) l[v + i] = usable(__uint_as_float(w[i]));
            else l[v + i] = usable(i & 1 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]));
          }
        } else {
#pragma unroll
          for (int i = 0; i < PER; ++i) l[v + i] = kNone;
        }
      }
      return;
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) l[v] = e0 + v < E ? logit<F32>(row, e0 + v) : kNone;
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

template <int V, bool F32, bool SCORES>
__global__ __launch_bounds__(256) void gate_kernel(GateArgs a) {
  __shared__ double lds[SCORES ? 4 * 64 * V : 1];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int E = a.E, K = a.K;
  const int64_t pitch = static_cast<int64_t>(E) * (F32 ? 4 : 2);
  for (int64_t t = wave_index(); t < a.N; t += static_cast<int64_t>(gridDim.x) * 4) {
    const void* row = static_cast<const uint8_t*>(a.logits) + t * pitch;
    float l[V];
    load_logits<V, F32>(row, E, a.wide_loads != 0, l);
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
        if (a.bias && e < E) c[v] += a.bias[e];
        if (!(l[v] > kNone) || !(c[v] == c[v])) c[v] = kNone;
      }
      if (a.groups > 1) {
        // a lane a group: its best one or two scores, from LDS; lanes start at
        // different members so that they read different banks
        double* mem = lds + wave * 64 * V;
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
          if (a.group_best == 2 && a.per_group > 1) one += two;
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
}

template <int V, bool F32>
__global__ __launch_bounds__(256) void gate_backward_kernel(GateArgs a) {
  const int lane = lane_id();
  const int E = a.E, K = a.K;
  const int64_t pitch = static_cast<int64_t>(E) * (F32 ? 4 : 2);
  const bool dense = a.score == kGateSoftmax && !a.renorm;
  for (int64_t t = wave_index(); t < a.N; t += static_cast<int64_t>(gridDim.x) * 4) {
    const void* row = static_cast<const uint8_t*>(a.logits) + t * pitch;
    const int64_t e64 = lane < K ? a.idx[t * K + lane] : -1;
    const int mine = e64 >= 0 && e64 < E ? static_cast<int>(e64) : -1;
    float g = mine >= 0 ? a.d_w[t * K + lane] * a.scale : 0.f;
    const float own = mine >= 0 ? logit<F32>(row, mine) : kNone;
    float p[V], d[V];
    float dot = 0.f;
    if (dense) {
      load_logits<V, F32>(row, E, a.wide_loads != 0, p);
      float top = p[0];
#pragma unroll
      for (int v = 1; v < V; ++v) top = bigger(top, p[v]);
      top = wave_max(top);
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        p[v] = rel_exp(p[v], top);
        sum += p[v];
      }
      sum = wave_sum(sum);
      const float inv = sum > 0.f ? 1.f / sum : 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) p[v] *= inv;
      dot = wave_sum(rel_exp(own, top) * inv * g);
    } else if (a.score == kGateSoftmax) {
      const float m = wave_max(own);
      float r = rel_exp(own, m);
      const float sum = wave_sum(r);
      r = own > kNone ? r / sum : 0.f;
      g = r * (g - wave_sum(r * g));
    } else {
      const float m = bigger(wave_max(own), -kMost);
      const float down = own > kNone ? 1.f / (1.f + expf(own)) : 0.f;      // 1 - s
      if (a.renorm) {
        float r = own > kNone ? sigmoid_over(own, m < 0.f ? m : 0.f) : 0.f;
        const float sum = wave_sum(r);
        r = own > kNone ? r / sum : 0.f;
        g = r * down * (g - wave_sum(r * g));
      } else {
        g = own > kNone ? g * sigmoid_over(own, 0.f) * down : 0.f;
      }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) d[v] = 0.f;
    for (int k = 0; k < K; ++k) {                                     // an expert named twice: both, in order
      const int e = miep::readlane(mine, k) - lane * V;
      const float x = readlane(g, k);
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (e == v) d[v] += x;
    }
    if (dense) {
#pragma unroll
      for (int v = 0; v < V; ++v) d[v] = p[v] * (d[v] - dot);
    }
    uint8_t* out = static_cast<uint8_t*>(a.d_logits) + t * pitch;
    const int e0 = lane * V;
    constexpr int PER = F32 ? 4 : 8;
    bool stored = false;
    if constexpr (V % PER == 0) {
      if (a.wide_loads) {
        stored = true;
#pragma unroll
        for (int v = 0; v < V; v += PER) {
          if (e0 + v >= E) continue;
          v4u o;
          if constexpr (F32) o = v4u{__float_as_uint(d[v]), __float_as_uint(d[v + 1]), __float_as_uint(d[v + 2]), __float_as_uint(d[v + 3])};
          else o = v4u{pack_bf16x2(d[v], d[v + 1]), pack_bf16x2(d[v + 2], d[v + 3]), pack_bf16x2(d[v + 4], d[v + 5]), pack_bf16x2(d[v + 6], d[v + 7])};
          *reinterpret_cast<v4u*>(out + (e0 + v) * (F32 ? 4ll : 2ll)) = o;
        }
      }
    }
    if (!stored) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (e0 + v >= E) continue;
        if constexpr (F32) reinterpret_cast<float*>(out)[e0 + v] = d[v];
        else reinterpret_cast<uint16_t*>(out)[e0 + v] = static_cast<uint16_t>(pack_bf16x2(d[v], 0.f));
      }
    }
  }
}

template <int V, bool F32>
void launch(const GateArgs& a, bool backward, bool scores, unsigned grid, hipStream_t st) {
  if (backward) gate_backward_kernel<V, F32><<<grid, 256, 0, st>>>(a);
  else if (scores) gate_kernel<V, F32, true><<<grid, 256, 0, st>>>(a);
  else gate_kernel<V, F32, false><<<grid, 256, 0, st>>>(a);
}

template <int V>
void launch_typed(const GateArgs& a, bool backward, bool scores, unsigned grid, hipStream_t st) {
  if (a.f32) launch<V, true>(a, backward, scores, grid, st);
  else launch<V, false>(a, backward, scores, grid, st);
}

}  // namespace

hipError_t launch_gate(const GateArgs& args, bool backward, hipStream_t st) {
  GateArgs a = args;
  if (a.N == 0) return hipSuccess;
  a.per_group = a.E / a.groups;
  a.per_div = make_fastdiv(a.per_group);
  a.wide_loads = a.E % (a.f32 ? 4 : 8) == 0;                          // whole 16-byte pieces of every row
  const bool scores = a.bias || a.groups > 1;
  const int64_t wgs = (a.N + 3) / 4;
  const unsigned grid = static_cast<unsigned>(wgs < (1 << 20) ? wgs : (1 << 20));
  if (a.E <= 64) launch_typed<1>(a, backward, scores, grid, st);
  else if (a.E <= 128) launch_typed<2>(a, backward, scores, grid, st);
  else if (a.E <= 256) launch_typed<4>(a, backward, scores, grid, st);
  else if (a.E <= 512) launch_typed<8>(a, backward, scores, grid, st);
  else if (a.E <= 1024) launch_typed<16>(a, backward, scores, grid, st);
  else launch_typed<32>(a, backward, scores, grid, st);
  return hipGetLastError();
}

}  // namespace miep
