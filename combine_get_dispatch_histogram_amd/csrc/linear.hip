// linear.hip -- dense products with an epilogue for a few rows (more of them:
// gemm_linear.hip), and the gradient through activation and bias.
//
// Up to 16 rows are bound by reading the weight (SwiGLU over 4096 x 7168: 11.2 us,
// 59 MB, 5.3 TB/s).  Of 64 rows two thirds of what a step brings to LDS are x, and
// a ring holds one or two steps, so its loads are not covered (7168 x 2048: 11.2 us,
// 31 MB).  The gradient of 4096 rows of 2 x 2048, SwiGLU, takes 19 us for its 84 MB
// (4.4 TB/s): 16 wavefronts a CU are one round, in each of which the loads of four
// rows, 960 instructions and the stores follow one another.
#include "gemm_epilogue.h"
#include "stream.h"

namespace miep {

namespace {

// At most 64 rows of x (TQ tiles of 16): a workgroup computes 16 * TP of the weight's rows (SwiGLU:
// half of them gate and the same ones of up, so that it has both); its wavefronts
// take every 8th step of the contraction.
template <int TP, int XL, int TQ, bool SWIGLU>
__global__ __launch_bounds__(512) void linear_few_kernel(LinearArgs a) {
  constexpr int WAVES = 8, P = 16 * TP, Q = 16 * TQ, RING = 20480;
  using Ring = StreamRing<kGemmBf16, 2 * TP, XL, RING, TQ>;
  static_assert(Q * P * 4 <= RING, "a wavefront's sums take the place of its ring");
  __shared__ __align__(1024) uint8_t lds_mem[WAVES * RING];
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  const int m = lane & 15, quarter = lane >> 4;
  const int rows = static_cast<int>(a.rows), half = a.N / 2;
  const int p0 = blockIdx.x * (SWIGLU ? P / 2 : P);
  const uint32_t pitch = static_cast<uint32_t>(a.K) * 2;
  const uint8_t* w = reinterpret_cast<const uint8_t*>(a.w) + static_cast<int64_t>(p0) * pitch;
  const uint8_t* x = reinterpret_cast<const uint8_t*>(a.x);
  uint32_t woff[2 * TP], xoff[XL];
#pragma unroll
  for (int i = 0; i < 2 * TP; ++i) {
    const int at = Ring::w_row(i);
    const uint32_t row = SWIGLU ? min(at % (P / 2), half - 1 - p0) + at / (P / 2) * half : min(at, a.N - 1 - p0);
    woff[i] = row * pitch + Ring::w_chunk(i) * 16;
  }
#pragma unroll
  for (int i = 0; i < XL; ++i) xoff[i] = min(Ring::x_row(i), rows - 1) * pitch + Ring::x_chunk(i) * 16;
  f32x4 acc[TP][TQ];
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  Ring ring((uint32_t)(uintptr_t)(lds_byte*)lds_mem + wave * RING);
  const int steps = (a.K + 63) / 64, n = wave < steps ? (steps - wave + WAVES - 1) / WAVES : 0;
  auto issue = [&](int i) MIEP_INLINE {
    const int step = wave + i * WAVES;
    ring.issue(w + step * 128ll, woff, x + step * 128ll, xoff, nullptr, a.K - step * 64);
  };
#pragma unroll
  for (int i = 0; i < Ring::kDepth; ++i)
    if (i < n) issue(i);
  for (int i = 0; i < n; ++i) {
    typename Ring::Frag f;
    ring.take(f, i + Ring::kDepth <= n);
    if (i + Ring::kDepth < n) issue(i + Ring::kDepth);
    Ring::multiply(f, [](int, int) { return false; }, acc);
  }
  // sums[wave][row][P], the pieces of 4 columns exchanged so that rows meet different banks
  constexpr int PIECES = P / 4;
  float* mine = reinterpret_cast<float*>(lds_mem + wave * RING);
#pragma unroll
  for (int i = 0; i < TP; ++i)
#pragma unroll
    for (int j = 0; j < TQ; ++j)
      *reinterpret_cast<f32x4*>(mine + (j * 16 + m) * P + (((i * 4 + quarter) ^ m) & (PIECES - 1)) * 4) = acc[i][j];
  __syncthreads();
  constexpr int PAIRS = SWIGLU ? P / 4 : P / 2;
  for (int i = threadIdx.x; i < rows * PAIRS; i += WAVES * kWave) {
    const int r = i / PAIRS, p = i % PAIRS * 2;
    const EpilogueRow to(a.epi, a.out, r, a.N);
    float v[2] = {}, u[2] = {};
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
      const float* s = reinterpret_cast<const float*>(lds_mem + k * RING) + r * P;
      auto at = [&](int c) MIEP_INLINE { return s + ((c / 4 ^ r) & (PIECES - 1)) * 4 + c % 4; };
      v[0] += at(p)[0];
      v[1] += at(p)[1];
      if constexpr (SWIGLU) {
        u[0] += at(p + P / 2)[0];
        u[1] += at(p + P / 2)[1];
      }
    }
    if constexpr (SWIGLU) {
      if (p0 + p < half) to.swiglu(p0 + p, v, u);
    } else if (p0 + p < a.N) {
      to.plain(p0 + p, v);
    }
  }
}

template <int TP, bool SWIGLU>
void launch_few(const LinearArgs& a, hipStream_t st) {
  const unsigned grid = SWIGLU ? (a.N / 2 + 8 * TP - 1) / (8 * TP) : (a.N + 16 * TP - 1) / (16 * TP);
  if (a.rows <= 8) linear_few_kernel<TP, 1, 1, SWIGLU><<<grid, 512, 0, st>>>(a);
  else if (a.rows <= 16) linear_few_kernel<TP, 2, 1, SWIGLU><<<grid, 512, 0, st>>>(a);
  else if (a.rows <= 32) linear_few_kernel<TP, 4, 2, SWIGLU><<<grid, 512, 0, st>>>(a);
  else linear_few_kernel<TP, 8, 4, SWIGLU><<<grid, 512, 0, st>>>(a);
}

// Gradient through the activation: a lane 8 columns, a wavefront 512, the four
// wavefronts of a workgroup every fourth row of its part.  The bias gradient is
// summed from the unrounded values: by lane, by wavefront, then over the parts.
template <bool DYF32, int ACT>
__global__ __launch_bounds__(256) void act_backward_kernel(ActBackwardArgs a) {
  constexpr bool SWIGLU = ACT == kActSwiglu;
  __shared__ float sums[4][512][SWIGLU ? 2 : 1];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int width = SWIGLU ? a.N / 2 : a.N;
  const int c = blockIdx.x * 512 + lane * 8;
  const int64_t r0 = static_cast<int64_t>(blockIdx.y) * a.rows_per_part;
  const int64_t r1 = r0 + a.rows_per_part < a.rows ? r0 + a.rows_per_part : a.rows;
  float sg[8] = {}, su[8] = {};
  // four rows' loads under way together: a wavefront has as few as four rows
  constexpr int ROWS = 4;
  for (int64_t r = r0 + wave; c < width && r < r1; r += 4 * ROWS) {
    v4u dy[ROWS][DYF32 ? 2 : 1], z[ROWS], u[SWIGLU ? ROWS : 1];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r + 4 * k < r1 ? r + 4 * k : r;
      const uint8_t* d = static_cast<const uint8_t*>(a.dy) + (row * width + c) * (DYF32 ? 4 : 2);
      dy[k][0] = ld16(d);
      if constexpr (DYF32) dy[k][1] = ld16(d + 16);
      if (ACT != kActNone) z[k] = ld16(a.z + row * a.N + c);
      if constexpr (SWIGLU) u[k] = ld16(a.z + row * a.N + width + c);
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r + 4 * k;
      if (row >= r1) break;
      float g[8], d[8];
      if constexpr (DYF32) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          g[i * 4] = __uint_as_float(dy[k][i].x); g[i * 4 + 1] = __uint_as_float(dy[k][i].y);
          g[i * 4 + 2] = __uint_as_float(dy[k][i].z); g[i * 4 + 3] = __uint_as_float(dy[k][i].w);
        }
      } else {
        widen(dy[k][0], g);
      }
      if constexpr (SWIGLU) {
        float gate[8], up[8], du[8];
        widen(z[k], gate);
        widen(u[k], up);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float s = sigmoid(gate[i]);
          d[i] = g[i] * up[i] * s * (1.f + gate[i] * (1.f - s));
          du[i] = g[i] * (gate[i] * s);
          sg[i] += d[i];
          su[i] += du[i];
        }
        if (a.dz) *reinterpret_cast<v4u*>(a.dz + row * a.N + width + c) = narrow(du);
      } else {
        float x[8];
        if (ACT != kActNone) widen(z[k], x);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          d[i] = ACT == kActNone ? g[i] : g[i] * activate_slope(x[i], ACT);
          sg[i] += d[i];
        }
      }
      if (a.dz) *reinterpret_cast<v4u*>(a.dz + row * a.N + c) = narrow(d);
    }
  }
  if (!a.dbias) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    sums[wave][lane * 8 + i][0] = sg[i];
    if constexpr (SWIGLU) sums[wave][lane * 8 + i][1] = su[i];
  }
  __syncthreads();
  float* out = a.partial + static_cast<int64_t>(blockIdx.y) * a.N;
  for (int i = threadIdx.x; i < 512; i += 256) {
    const int col = blockIdx.x * 512 + i;
    if (col >= width) continue;
    out[col] = sums[0][i][0] + sums[1][i][0] + sums[2][i][0] + sums[3][i][0];
    if constexpr (SWIGLU) out[width + col] = sums[0][i][1] + sums[1][i][1] + sums[2][i][1] + sums[3][i][1];
  }
}

// The parts' sums, a wavefront 64 columns, the four of a workgroup every fourth part.
__global__ __launch_bounds__(256) void bias_sum_kernel(ActBackwardArgs a) {
  __shared__ float sums[4][64];
  const int lane = lane_id(), wave = threadIdx.x / kWave;
  const int c = blockIdx.x * 64 + lane;
  float s = 0.f;
  for (int p = wave; c < a.N && p < a.parts; p += 32) {               // eight loads under way together
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = p + 4 * k < a.parts ? a.partial[static_cast<int64_t>(p + 4 * k) * a.N + c] : 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) s += v[k];
  }
  sums[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < a.N) {
    s = sums[0][lane] + sums[1][lane] + sums[2][lane] + sums[3][lane];
    a.dbias[c] = a.accumulate ? a.dbias[c] + s : s;
  }
}

__global__ __launch_bounds__(256) void bias_zero_kernel(float* p, int n) {
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i < n) p[i] = 0.f;
}

template <int ACT>
void launch_act(const ActBackwardArgs& a, dim3 grid, hipStream_t st) {
  if (a.dy_f32) act_backward_kernel<true, ACT><<<grid, 256, 0, st>>>(a);
  else act_backward_kernel<false, ACT><<<grid, 256, 0, st>>>(a);
}

}  // namespace

hipError_t launch_linear(const LinearArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  if (a.rows <= kLinearFewRows) {
    // one workgroup a CU: tiles of 32 rows of the weight where 16 make more than
    // the GPU holds at a time
    const bool swiglu = a.epi.act == kActSwiglu, wide = (a.N + 15) / 16 > 256;
    if (swiglu && wide) launch_few<2, true>(a, st);
    else if (swiglu) launch_few<1, true>(a, st);
    else if (wide) launch_few<2, false>(a, st);
    else launch_few<1, false>(a, st);
    return hipGetLastError();
  }
  GemmRowsArgs g{};
  g.g.G = 1;
  g.g.limit = a.rows;
  g.q = a.x;
  g.p = a.w;
  g.q_rows = a.rows;
  g.C = a.K;
  g.NO = a.N;
  g.out = static_cast<uint16_t*>(a.out);
  g.type = kGemmBf16;
  g.expected = static_cast<int>(a.rows);
  g.epi = a.epi;
  return launch_gemm_linear(g, st);
}

hipError_t launch_act_backward(const ActBackwardArgs& args, hipStream_t st) {
  ActBackwardArgs a = args;
  if (a.rows == 0) {
    if (a.dbias && !a.accumulate) bias_zero_kernel<<<(a.N + 255) / 256, 256, 0, st>>>(a.dbias, a.N);
    return hipGetLastError();
  }
  const int width = a.act == kActSwiglu ? a.N / 2 : a.N;
  const unsigned cols = (width + 511) / 512;
  // as many parts as fill the GPU a few times over, of at least 16 rows; with a
  // bias no more than the caller's workspace has rows
  int64_t parts = (a.rows + 15) / 16, most = 4096 / cols + 1;
  if (a.dbias && most > a.parts) most = a.parts;
  if (parts > most) parts = most;
  if (parts > 65535) parts = 65535;
  const int64_t per = (a.rows + parts - 1) / parts;
  a.rows_per_part = static_cast<int>(per);
  a.parts = static_cast<int>((a.rows + per - 1) / per);
  const dim3 grid(cols, a.parts);
  switch (a.act) {
    case kActNone: launch_act<kActNone>(a, grid, st); break;
    case kActRelu: launch_act<kActRelu>(a, grid, st); break;
    case kActSilu: launch_act<kActSilu>(a, grid, st); break;
    case kActGelu: launch_act<kActGelu>(a, grid, st); break;
    case kActGeluTanh: launch_act<kActGeluTanh>(a, grid, st); break;
    default: launch_act<kActSwiglu>(a, grid, st); break;
  }
  if (a.dbias) bias_sum_kernel<<<(a.N + 63) / 64, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace miep
