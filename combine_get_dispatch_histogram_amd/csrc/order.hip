// order.hip -- between a normal dispatch and its experts: received rows to
// slots in expert order, and expert outputs back to received rows.
//
// expert_order is a stable counting sort of the (row, k) entries by expert.
// A rank's rows name only its own L experts, so the work is cut by rank and,
// inside a rank, into parts: one kernel counts each part's entries per expert;
// the second starts every counter at its expert's first slot plus the entries
// of the parts (and, in the part, of the wavefronts) before it, and gives out
// slots 64 entries at a time, equal experts in lane order.  No counter is
// shared between wavefronts then, so the order never depends on timing.  A few
// entries are counted by every workgroup of the placing kernel for itself: one
// launch instead of two.  16384
// tokens' top-8 over 64 ranks (12 MB to move) take 12.2 us, of which two launches
// are about 7: bound by those and a memory latency each.
#include "device.h"
#include "kernels.h"

namespace miep {

constexpr int kOrderWaves = 8;                 // wavefronts of a part in the placing kernel
constexpr int kOrderThreads = kOrderWaves * kWave;
// A lane keeps this many entries in registers: their loads are in flight
// together, and a wavefront whose share fits reads it only once (one load at a
// time, twice, the placing of 16384 tokens' top-8 over 64 ranks took 15.6 us).
constexpr int kOrderHold = 8;

// Rows [first, last) of part p of rank r, inside the allocated rows whatever
// the offsets hold.
__device__ __forceinline__ void part_rows(const OrderArgs& a, int r, int p, int64_t* first, int64_t* last) {
  int64_t lo = a.off[r], hi = a.off[r + 1];
  lo = lo < 0 ? 0 : lo > a.rows ? a.rows : lo;
  hi = hi < lo ? lo : hi > a.rows ? a.rows : hi;
  *first = lo + (hi - lo) * p / a.parts;
  *last = lo + (hi - lo) * (p + 1) / a.parts;
}

// Entries i0 + lane, + 64, ...: the lane's local experts of kOrderHold of them, -1
// where there is none.
__device__ __forceinline__ void hold(const OrderArgs& a, int64_t i0, int64_t i1, int step, int (&e)[kOrderHold]) {
  int64_t v[kOrderHold];
#pragma unroll
  for (int k = 0; k < kOrderHold; ++k) {
    v[k] = -1;
    if (i0 + k * step < i1) v[k] = a.topk[i0 + k * step];
  }
#pragma unroll
  for (int k = 0; k < kOrderHold; ++k) e[k] = v[k] >= 0 && v[k] < a.L ? static_cast<int>(v[k]) : -1;
}

__global__ __launch_bounds__(kOrderThreads) void order_count_kernel(OrderArgs a) {
  __shared__ int count[kMaxLocalExperts];
  const int r = blockIdx.x / a.parts, p = blockIdx.x - r * a.parts;
  for (int l = threadIdx.x; l < a.L; l += kOrderThreads) count[l] = 0;
  __syncthreads();
  int64_t first, last;
  part_rows(a, r, p, &first, &last);
  for (int64_t i = first * a.K + threadIdx.x; i < last * a.K; i += kOrderHold * kOrderThreads) {
    int e[kOrderHold];
    hold(a, i, last * a.K, kOrderThreads, e);
#pragma unroll
    for (int k = 0; k < kOrderHold; ++k)
      if (e[k] >= 0) atomicAdd(&count[e[k]], 1);
  }
  __syncthreads();
  int32_t* out = a.counts + static_cast<int64_t>(p) * a.E + r * a.L;
  for (int l = threadIdx.x; l < a.L; l += kOrderThreads) out[l] = count[l];
}

// One launch, a part a rank, up to this many entries and experts (a call for 64
// tokens' top-8 over 8 ranks 7.3 us against 9.7, with 4096 entries 8.4 against
// 10.5; with 8192 the same, and over 64 ranks 14 against 10.6).
constexpr int kOneEntries = kOrderHold * kOrderThreads, kOneExperts = 2048;

template <bool ONE>
__global__ __launch_bounds__(kOrderThreads) void order_place_kernel(OrderArgs a) {
  __shared__ int next[kOrderWaves][kMaxLocalExperts];   // each wavefront's next slot per expert
  __shared__ int sums[512], waves[kOrderWaves];
  const int tid = threadIdx.x, lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int r = blockIdx.x / a.parts, p = blockIdx.x - r * a.parts;
  int64_t first, last;
  part_rows(a, r, p, &first, &last);
  // this wavefront's entries, in blocks of what its lanes hold
  constexpr int kBlock = kOrderHold * kWave;
  const int64_t entries = (last - first) * a.K;
  const int64_t i0 = first * a.K + entries * wave / kOrderWaves, i1 = first * a.K + entries * (wave + 1) / kOrderWaves;
  int held[kOrderHold];
  hold(a, i0 + lane, i1, kWave, held);

  for (int l = tid; l < kOrderWaves * a.L; l += kOrderThreads) next[l / a.L][l % a.L] = 0;
  __shared__ int total[ONE ? kOneExperts : 1], from[ONE ? kMaxRanks + 1 : 1];
  if constexpr (ONE) {
    for (int e = tid; e < a.E; e += kOrderThreads) total[e] = 0;
    for (int q = tid; q <= a.R; q += kOrderThreads)
      from[q] = static_cast<int>(min(max(static_cast<int64_t>(a.off[q]), static_cast<int64_t>(0)), a.rows));
  }
  __syncthreads();
  if constexpr (ONE) {
    const int end = from[a.R] * a.K;
    for (int i = tid; i < end; i += kBlock * kOrderWaves) {
      int e[kOrderHold];
      hold(a, i, end, kOrderThreads, e);
#pragma unroll
      for (int k = 0; k < kOrderHold; ++k) {
        if (e[k] < 0) continue;
        const int row = fdiv(i + k * kOrderThreads, a.Kdiv);
        int lo = 0, hi = a.R;                                         // the row's rank: the last that begins at or before it
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (from[mid] <= row) lo = mid;
          else hi = mid;
        }
        atomicAdd(&total[lo * a.L + e[k]], 1);
      }
    }
  }
  for (int64_t i = i0; i < i1; i += kBlock) {
    if (i != i0) hold(a, i + lane, i1, kWave, held);
#pragma unroll
    for (int k = 0; k < kOrderHold; ++k)
      if (held[k] >= 0) atomicAdd(&next[wave][held[k]], 1);
  }
  __syncthreads();

  // first slots: prefix of the experts' aligned totals, 512 experts at a time
  // (up to 256 experts: several threads add up the parts of one)
  int64_t slots = 0;
  int width = kOrderThreads;
  while (width / 2 >= a.E) width /= 2;
  for (int e0 = 0; e0 < a.E; e0 += kOrderThreads) {
    const int e = e0 + (tid & (width - 1));
    int all = 0, before = 0;
    if (e < a.E)
      for (int q = tid / width; q < a.parts; q += kOrderThreads / width) {
        int c;
        if constexpr (ONE) c = total[e];
        else c = a.counts[static_cast<int64_t>(q) * a.E + e];
        all += c;
        before += q < p ? c : 0;
      }
    if (width < kOrderThreads) {
      sums[tid] = 0;
      __syncthreads();
      atomicAdd(&sums[tid & (width - 1)], all);
      atomicAdd(&sums[256 + (tid & (width - 1))], before);
      __syncthreads();
      all = tid < width ? sums[tid] : 0;
      before = tid < width ? sums[256 + tid] : 0;
    }
    const bool mine = e < a.E && tid < width;
    const int padded = mine ? (all + a.align - 1) / a.align * a.align : 0;
    const int inc = wave_inclusive_scan(padded);
    __syncthreads();
    if (lane == kWave - 1) waves[wave] = inc;
    __syncthreads();
    int64_t at = slots + inc - padded;
    for (int w = 0; w < kOrderWaves; ++w) {
      if (w < wave) at += waves[w];
      slots += waves[w];
    }
    if (mine) {
      if (blockIdx.x == 0) {
        a.begin[e] = static_cast<int>(at);
        a.group_rows[e] = all;
      }
      if (e / a.L == r) {
        int s = static_cast<int>(at) + before;
        for (int w = 0; w < kOrderWaves; ++w) {
          const int c = next[w][e - r * a.L];
          next[w][e - r * a.L] = s;
          s += c;
        }
        if (p == 0)
          for (int64_t q = at + all; q < at + padded; ++q)
            if (q >= 0 && q < a.slots) a.slot_row[q] = -1;
      }
    }
  }
  __syncthreads();

  int bits = 0;
  while ((1 << bits) < a.L) ++bits;
  for (int64_t i = i0; i < i1; i += kBlock) {
    if (i1 - i0 > kBlock) hold(a, i + lane, i1, kWave, held);         // longer shares: read again
#pragma unroll
    for (int k = 0; k < kOrderHold; ++k) {
      const int64_t n = i + k * kWave + lane;
      if (n - lane >= i1) break;
      const int e = max(held[k], 0);
      uint64_t same = ballot(held[k] >= 0);
      for (int b = 0; b < bits; ++b) {
        const uint64_t set = ballot((e >> b) & 1);
        same &= ((e >> b) & 1) ? set : ~set;
      }
      int slot = -1;
      if (held[k] >= 0) {
        slot = next[wave][e] + __popcll(same & lanemask_lt());
        if ((same >> lane) == 1) next[wave][e] = slot + 1;            // the last of the equal ones
        if (slot >= 0 && slot < a.slots) a.slot_row[slot] = fdiv(static_cast<int>(n), a.Kdiv);
        else slot = -1;
      }
      if (n < i1) a.row_slot[n] = slot;
    }
  }

  // slots behind the last expert's, and rows behind the last received one
  const int64_t step = static_cast<int64_t>(gridDim.x) * kOrderThreads, own = blockIdx.x * static_cast<int64_t>(kOrderThreads) + tid;
  for (int64_t s = max(slots, static_cast<int64_t>(0)) + own; s < a.slots; s += step) a.slot_row[s] = -1;
  int64_t end = a.off[a.R];
  end = end < 0 ? 0 : end > a.rows ? a.rows : end;
  for (int64_t i = end * a.K + own; i < a.rows * a.K; i += step) a.row_slot[i] = -1;
  if (a.status && blockIdx.x == 0 && tid == 0) *a.status = slots > a.slots ? kStatusCapacity : 0;
}

hipError_t launch_order(const OrderArgs& args, hipStream_t st) {
  OrderArgs a = args;
  a.Kdiv = make_fastdiv(a.K);                                        // entries stay below 2^31
  // a part is worth the entries that its lanes hold: fewer leave more to sum up than to sort
  constexpr int kPart = kOrderHold * kOrderThreads;
  const int64_t want = (a.rows * a.K / a.R + kPart - 1) / kPart;
  if (want < a.parts) a.parts = want < 1 ? 1 : static_cast<int>(want);
  const int64_t grid = static_cast<int64_t>(a.parts) * a.R;
  if (grid > max_blocks(kOrderThreads)) return hipErrorInvalidConfiguration;
  if (a.parts == 1 && a.rows * a.K <= kOneEntries && a.E <= kOneExperts) {
    order_place_kernel<true><<<static_cast<unsigned>(grid), kOrderThreads, 0, st>>>(a);
    return hipGetLastError();
  }
  order_count_kernel<<<static_cast<unsigned>(grid), kOrderThreads, 0, st>>>(a);
  order_place_kernel<false><<<static_cast<unsigned>(grid), kOrderThreads, 0, st>>>(a);
  return hipGetLastError();
}

// ---- reduce
__device__ __forceinline__ void widen(const v4u& v, float (&f)[8]) {
  f[0] = bf16_lo(v.x); f[1] = bf16_hi(v.x); f[2] = bf16_lo(v.y); f[3] = bf16_hi(v.y);
  f[4] = bf16_lo(v.z); f[5] = bf16_hi(v.z); f[6] = bf16_lo(v.w); f[7] = bf16_hi(v.w);
}
__device__ __forceinline__ v4u narrow(const float (&f)[8]) {
  return v4u{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])};
}

// One workgroup a row; a thread owns 8 channels at a time.  The row's slots
// and weights are read by the lanes k of every wavefront and broadcast.
// Terms are added in ascending k in fp32, one rounding to bf16.  Bound by
// memory: 4096 slots of 7168 to 2,700 rows (97 MB) take 18 us, 5.4 TB/s;
// four slots' loads are in flight at a time.
__global__ __launch_bounds__(256) void reduce_kernel(ReduceArgs a) {
  const int lane = lane_id();
  int64_t rows = a.rows;
  if (a.num_rows) rows = min(rows, static_cast<int64_t>(max(*a.num_rows, 0)));
  const int nv = a.H / 8;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    int slot = -1;
    float w = 1.f;
    if (lane < a.K) {
      slot = a.row_slot[row * a.K + lane];
      if (a.w) w = a.w[row * a.K + lane];
    }
    const uint64_t live = ballot(slot >= 0 && slot < a.slots);
    for (int v = threadIdx.x; v < nv; v += 256) {
      float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      uint64_t left = live;
      while (left) {
        v4u d[4];
        float g[4];
        int n = 0;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          g[q] = 0.f;
          if (left) {
            const int b = __builtin_ctzll(left);
            left &= left - 1;
            g[q] = __int_as_float(readlane(__float_as_int(w), b));
            d[q] = ld16(a.z + static_cast<int64_t>(readlane(slot, b)) * a.H + v * 8);
            n = q + 1;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          if (q < n) {
            float f[8];
            widen(d[q], f);
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fmaf(g[q], f[k], acc[k]);
          }
      }
      *reinterpret_cast<v4u*>(a.out + row * a.H + v * 8) = narrow(acc);
    }
  }
}

// 16 bytes of rows that are used once.
__device__ __forceinline__ v4u ld16_once(const void* p) {
  const u32x4 t = __builtin_nontemporal_load(static_cast<const u32x4*>(p));
  return v4u{t.x, t.y, t.z, t.w};
}
__device__ __forceinline__ void st16_once(void* p, const v4u& v) {
  const u32x4 t = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(t, static_cast<u32x4*>(p));
}

// Gradient: dz[slot(row, k)] = w[row][k] * dy[row], dw[row][k] = <dy[row],
// z[slot(row, k)]>.  Eight entries at a time share one read of dy's row; the
// dot products are summed over lanes, then wavefronts, in a fixed order.  Bound
// by memory: 32768 slots of 7168 (1 GB) 185 us, 5.4 TB/s.
template <bool STREAM>
__global__ __launch_bounds__(256) void reduce_backward_kernel(ReduceArgs a) {
  constexpr int NB = 8;
  __shared__ float part[4][NB];
  const int lane = lane_id();
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / kWave);
  int64_t rows = a.rows;
  if (a.num_rows) rows = min(rows, static_cast<int64_t>(max(*a.num_rows, 0)));
  const int nv = a.H / 8;
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    int slot = -1;
    float w = 1.f;
    if (lane < a.K) {
      slot = a.row_slot[row * a.K + lane];
      if (a.w) w = a.w[row * a.K + lane];
    }
    const bool ok = slot >= 0 && slot < a.slots;
    uint64_t left = ballot(ok);
    if (a.dw && wave == 0 && lane < a.K && !ok) a.dw[row * a.K + lane] = 0.f;
    while (left) {
      int64_t at[NB];
      int which[NB];
      float g[NB], dot[NB];
      int n = 0;
#pragma unroll
      for (int q = 0; q < NB; ++q) {
        dot[q] = 0.f;
        g[q] = 0.f;
        at[q] = 0;
        which[q] = 0;
        if (left) {
          const int b = __builtin_ctzll(left);
          left &= left - 1;
          which[q] = b;
          g[q] = __int_as_float(readlane(__float_as_int(w), b));
          at[q] = static_cast<int64_t>(readlane(slot, b)) * a.H;
          n = q + 1;
        }
      }
      for (int v = threadIdx.x; v < nv; v += 256) {
        float dy[8];
        widen(ld16(a.dy + row * a.H + v * 8), dy);
        v4u d[NB];
        if (a.dw) {
#pragma unroll
          for (int q = 0; q < NB; ++q)
            if (q < n) d[q] = STREAM ? ld16_once(a.z + at[q] + v * 8) : ld16(a.z + at[q] + v * 8);
        }
#pragma unroll
        for (int q = 0; q < NB; ++q)
          if (q < n) {
            float o[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) o[k] = g[q] * dy[k];
            if constexpr (STREAM) st16_once(a.out + at[q] + v * 8, narrow(o));
            else *reinterpret_cast<v4u*>(a.out + at[q] + v * 8) = narrow(o);
            if (a.dw) {
              float f[8];
              widen(d[q], f);
#pragma unroll
              for (int k = 0; k < 8; ++k) dot[q] = fmaf(dy[k], f[k], dot[q]);
            }
          }
      }
      if (a.dw) {
#pragma unroll
        for (int q = 0; q < NB; ++q) {
#pragma unroll
          for (int s = 32; s > 0; s >>= 1) dot[q] += __shfl_xor(dot[q], s);
          if (lane == 0) part[wave][q] = dot[q];
        }
        __syncthreads();
        if (threadIdx.x == 0) {
#pragma unroll
          for (int q = 0; q < NB; ++q)
            if (q < n) a.dw[row * a.K + which[q]] = ((part[0][q] + part[1][q]) + part[2][q]) + part[3][q];
        }
        __syncthreads();
      }
    }
  }
}

hipError_t launch_reduce(const ReduceArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>(a.rows < 65536 ? a.rows : 65536);
  reduce_kernel<<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

hipError_t launch_reduce_backward(const ReduceArgs& a, hipStream_t st) {
  if (a.rows == 0) return hipSuccess;
  const unsigned grid = static_cast<unsigned>(a.rows < 65536 ? a.rows : 65536);
  // Slots of half the 256 MiB last-level cache or more pass it by (32768 slots
  // of 7168: 203 -> 187 us).
  if (2 * a.slots * a.H >= (128ll << 20)) reduce_backward_kernel<true><<<grid, 256, 0, st>>>(a);
  else reduce_backward_kernel<false><<<grid, 256, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace miep
