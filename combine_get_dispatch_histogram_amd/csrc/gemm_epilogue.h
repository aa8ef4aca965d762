// gemm_epilogue.h -- what a dense product's results go through on their way to
// memory: out = f(z + bias) + residual in fp32, rounded once, and z + bias kept
// in bf16 where the backward pass wants it.  A lane brings four consecutive
// columns of a row (a pair of neighbouring 16 x 16 results gives 8, after the
// exchange of pack_pair), so bias, residual and stores are 8- and 16-byte pieces.
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

  __device__ __forceinline__ f32x4 biased(f32x4 v, int p) const {
    if (e.bias) v += *reinterpret_cast<const f32x4*>(e.bias + p);
    return v;
  }
  __device__ __forceinline__ f32x4 with_residual(f32x4 v, int p) const {
    if (residual) {
      const v2u r = *reinterpret_cast<const v2u*>(residual + p);
      v += f32x4{bf16_lo(r.x), bf16_hi(r.x), bf16_lo(r.y), bf16_hi(r.y)};
    }
    return v;
  }
  __device__ __forceinline__ f32x4 activated(f32x4 v) const {
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = activate(v[r], e.act);
    return v;
  }

  // Two neighbouring results: this lane's columns p + 4 * quarter and 16 on, of
  // `wide` columns.
  __device__ __forceinline__ void store(int p, int quarter, const f32x4& a, const f32x4& b) const {
    if (e.out_f32) {
      float* o = reinterpret_cast<float*>(out) + p + quarter * 4;
      if (p + quarter * 4 < width) *reinterpret_cast<f32x4*>(o) = a;
      if (p + 16 + quarter * 4 < width) *reinterpret_cast<f32x4*>(o + 16) = b;
    } else {
      const v4u v = pack_pair(a, b);
      const int at = p + (quarter & 1) * 16 + (quarter >> 1) * 8;
      if (at < width) *reinterpret_cast<v4u*>(out + at) = v;
    }
  }
  __device__ __forceinline__ void keep(int p, int limit, int quarter, const f32x4& a, const f32x4& b) const {
    if (!z) return;
    const v4u v = pack_pair(a, b);
    const int at = p + (quarter & 1) * 16 + (quarter >> 1) * 8;
    if (at < limit) *reinterpret_cast<v4u*>(z + at) = v;
  }

  __device__ __forceinline__ void plain(int p, int quarter, f32x4 a, f32x4 b) const {
    const int pa = min(p + quarter * 4, NO - 4), pb = min(p + 16 + quarter * 4, NO - 4);
    a = biased(a, pa);
    b = biased(b, pb);
    keep(p, NO, quarter, a, b);
    store(p, quarter, with_residual(activated(a), pa), with_residual(activated(b), pb));
  }
  // Columns p on and p + 16 on, gate and up of each.
  __device__ __forceinline__ void swiglu(int p, int quarter, f32x4 ga, f32x4 ua, f32x4 gb, f32x4 ub) const {
    const int pa = min(p + quarter * 4, width - 4), pb = min(p + 16 + quarter * 4, width - 4);
    ga = biased(ga, pa);
    gb = biased(gb, pb);
    ua = biased(ua, width + pa);
    ub = biased(ub, width + pb);
    keep(p, width, quarter, ga, gb);
    if (z) {
      const v4u v = pack_pair(ua, ub);
      const int at = p + (quarter & 1) * 16 + (quarter >> 1) * 8;
      if (at < width) *reinterpret_cast<v4u*>(z + width + at) = v;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      ga[r] = ga[r] * sigmoid(ga[r]) * ua[r];
      gb[r] = gb[r] * sigmoid(gb[r]) * ub[r];
    }
    store(p, quarter, with_residual(ga, pa), with_residual(gb, pb));
  }

  // The same for two consecutive columns of a row's whole sums.
  __device__ __forceinline__ void store2(int p, float x, float y) const {
    if (residual) {
      const uint32_t r = *reinterpret_cast<const uint32_t*>(residual + p);
      x += bf16_lo(r);
      y += bf16_hi(r);
    }
    if (e.out_f32) *reinterpret_cast<float2*>(reinterpret_cast<float*>(out) + p) = float2{x, y};
    else *reinterpret_cast<uint32_t*>(out + p) = pack_bf16x2(x, y);
  }
  __device__ __forceinline__ void plain2(int p, float x, float y) const {
    if (e.bias) {
      x += e.bias[p];
      y += e.bias[p + 1];
    }
    if (z) *reinterpret_cast<uint32_t*>(z + p) = pack_bf16x2(x, y);
    store2(p, activate(x, e.act), activate(y, e.act));
  }
  __device__ __forceinline__ void swiglu2(int p, float gx, float gy, float ux, float uy) const {
    if (e.bias) {
      gx += e.bias[p];
      gy += e.bias[p + 1];
      ux += e.bias[width + p];
      uy += e.bias[width + p + 1];
    }
    if (z) {
      *reinterpret_cast<uint32_t*>(z + p) = pack_bf16x2(gx, gy);
      *reinterpret_cast<uint32_t*>(z + width + p) = pack_bf16x2(ux, uy);
    }
    store2(p, gx * sigmoid(gx) * ux, gy * sigmoid(gy) * uy);
  }
};

}  // namespace miep
