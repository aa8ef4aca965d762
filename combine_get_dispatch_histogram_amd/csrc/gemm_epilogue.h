// gemm_epilogue.h -- what a dense product's results go through on their way to
// memory: out = f(z + bias) + residual in fp32, rounded once, and z + bias kept
// in bf16 where the backward pass wants it.  A lane of a tile kernel brings four
// consecutive columns of a row (a pair of neighbouring 16 x 16 results gives 8,
// after the exchange of pack_pair), so bias, residual and stores are 8- and
// 16-byte pieces; the kernels that add up sums of several wavefronts bring two.
#pragma once

#include "act.h"
#include "gemm.h"

namespace miep {

enum { kEpiNone = 0, kEpiPlain = 1, kEpiSwiglu = 2 };

// SwiGLU: a tile's 16-row blocks of the weight [gate | up] (NO rows) are gate and
// up in turn, so that a lane holds both of a column.  Row `row` of the tile from
// the virtual row p0 on, counted from gate row p0 / 2.
__device__ __forceinline__ int swiglu_row(int p0, int row, int NO) {
  const int c = min((row >> 5) * 16 + (row & 15), NO / 2 - 1 - p0 / 2);
  return c + ((row >> 4) & 1) * (NO / 2);
}

struct EpilogueRow {
  const Epilogue& e;
  uint16_t* out;               // the row's first column
  const uint16_t* residual;
  uint16_t* z;
  int NO, width;

  __device__ __forceinline__ EpilogueRow(const Epilogue& epi, void* o, int64_t row, int no)
      : e(epi), NO(no), width(epi.act == kActSwiglu ? no / 2 : no) {
    out = static_cast<uint16_t*>(o) + row * width * (epi.out_f32 ? 2 : 1);
    residual = epi.residual ? epi.residual + row * width : nullptr;
    z = epi.z ? epi.z + row * no : nullptr;
  }

  // V (2 or 4) consecutive columns of a row.
  template <int V>
  __device__ __forceinline__ void put16(uint16_t* to, const float (&v)[V]) const {
    if constexpr (V == 2) *reinterpret_cast<uint32_t*>(to) = pack_bf16x2(v[0], v[1]);
    else *reinterpret_cast<v2u*>(to) = v2u{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
  }
  template <int V>
  __device__ __forceinline__ void add_bias(int p, float (&v)[V]) const {
    if (!e.bias) return;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] += e.bias[p + i];
  }
  template <int V>
  __device__ __forceinline__ void store(int p, float (&v)[V]) const {
    if (residual) {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const uint32_t r = *reinterpret_cast<const uint32_t*>(residual + p + i);
        v[i] += bf16_lo(r);
        v[i + 1] += bf16_hi(r);
      }
    }
    if (e.out_f32) {
      float* o = reinterpret_cast<float*>(out) + p;
      if constexpr (V == 2) *reinterpret_cast<float2*>(o) = float2{v[0], v[1]};
      else *reinterpret_cast<f32x4*>(o) = f32x4{v[0], v[1], v[2], v[3]};
    } else {
      put16(out + p, v);
    }
  }
  template <int V>
  __device__ __forceinline__ void plain(int p, float (&v)[V]) const {
    add_bias(p, v);
    if (z) put16(z + p, v);
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = activate(v[i], e.act);
    store(p, v);
  }
  template <int V>
  __device__ __forceinline__ void swiglu(int p, float (&g)[V], float (&u)[V]) const {
    add_bias(p, g);
    add_bias(width + p, u);
    if (z) {
      put16(z + p, g);
      put16(z + width + p, u);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) g[i] = g[i] * sigmoid(g[i]) * u[i];
    store(p, g);
  }
};

// A wavefront's 16 * TP x 16 * TQ results from column p0 and row row0 on, of
// which `rows` exist.  A column's bias is read once, the activation chosen once
// for 16 rows.
template <int EPI, int TP, int TQ>
__device__ __forceinline__ void epilogue_tile(const Epilogue& e, void* out, int NO, int64_t row0, int rows, int p0, f32x4 (&acc)[TP][TQ]) {
  const int lane = lane_id(), m = lane & 15, quarter = lane >> 4;
  const int width = EPI == kEpiSwiglu ? NO / 2 : NO;
  // Results i and i + NEXT are 16 columns apart; a lane's four columns of one
  // (for the loads), and its eight of both after the exchange.
  constexpr int NEXT = EPI == kEpiSwiglu ? 2 : 1;
  const int q4 = (EPI == kEpiSwiglu ? p0 / 2 : p0) + quarter * 4;
  const int q8 = (EPI == kEpiSwiglu ? p0 / 2 : p0) + (quarter & 1) * 16 + (quarter >> 1) * 8;
  if (e.bias) {
#pragma unroll
    for (int i = 0; i < TP; ++i) {
      const int c = min(q4 + i / NEXT * 16, width - 4) + (EPI == kEpiSwiglu ? (i & 1) * width : 0);
      const f32x4 b = *reinterpret_cast<const f32x4*>(e.bias + c);
#pragma unroll
      for (int j = 0; j < TQ; ++j)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] += b[r];
    }
  }
  if (e.z) {
#pragma unroll
    for (int j = 0; j < TQ; ++j) {
      const int row = j * 16 + m;
      if (row >= rows) continue;                                      // a row's lanes are in or out together
      uint16_t* z = e.z + (row0 + row) * NO;
#pragma unroll
      for (int i = 0; i < TP; i += 2 * NEXT) {
        const int c = q8 + i / NEXT * 16;
        const v4u v = pack_pair(acc[i][j], acc[i + NEXT][j]);
        if (c < width) *reinterpret_cast<v4u*>(z + c) = v;
        if constexpr (EPI == kEpiSwiglu) {
          const v4u u = pack_pair(acc[i + 1][j], acc[i + 3][j]);
          if (c < width) *reinterpret_cast<v4u*>(z + width + c) = u;
        }
      }
    }
  }
#pragma unroll
  for (int j = 0; j < TQ; ++j) {
    const int row = j * 16 + m;
    if (row >= rows) continue;
    const int64_t at = (row0 + row) * width;
    if constexpr (EPI == kEpiSwiglu) {
#pragma unroll
      for (int i = 0; i < TP; i += 2)
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[i][j][r] = acc[i][j][r] * sigmoid(acc[i][j][r]) * acc[i + 1][j][r];
    } else {
      auto each = [&](auto f) MIEP_INLINE {
#pragma unroll
        for (int i = 0; i < TP; ++i)
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[i][j][r] = f(acc[i][j][r]);
      };
      switch (e.act) {
        case kActRelu: each([](float v) { return activate(v, kActRelu); }); break;
        case kActSilu: each([](float v) { return activate(v, kActSilu); }); break;
        case kActGelu: each([](float v) { return activate(v, kActGelu); }); break;
        case kActGeluTanh: each([](float v) { return activate(v, kActGeluTanh); }); break;
        default: break;
      }
    }
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < TP; i += NEXT) {
        const v2u r = *reinterpret_cast<const v2u*>(e.residual + at + min(q4 + i / NEXT * 16, width - 4));
        acc[i][j][0] += bf16_lo(r.x);
        acc[i][j][1] += bf16_hi(r.x);
        acc[i][j][2] += bf16_lo(r.y);
        acc[i][j][3] += bf16_hi(r.y);
      }
    }
    if (e.out_f32) {
      float* o = static_cast<float*>(out) + at;
#pragma unroll
      for (int i = 0; i < TP; i += NEXT)
        if (q4 + i / NEXT * 16 < width) *reinterpret_cast<f32x4*>(o + q4 + i / NEXT * 16) = acc[i][j];
    } else {
      uint16_t* o = static_cast<uint16_t*>(out) + at;
#pragma unroll
      for (int i = 0; i < TP; i += 2 * NEXT) {
        const v4u v = pack_pair(acc[i][j], acc[i + NEXT][j]);
        if (q8 + i / NEXT * 16 < width) *reinterpret_cast<v4u*>(o + q8 + i / NEXT * 16) = v;
      }
    }
  }
}

}  // namespace miep
