// kernels.h -- internal launch interface between the C ABI (api.cpp) and the
// gfx950 kernels.  Host code only sees these argument structs and launchers;
// every launcher enqueues on the given stream and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace miep {

constexpr int kWave = 64;          // CDNA wavefront width
// A grid dimension counts its work-items in 32 bits: the largest number of
// workgroups of `threads` threads one 1-D launch may ask for.  Launches past
// it return hipErrorInvalidConfiguration instead of a truncated grid.
constexpr int64_t max_blocks(int64_t threads) { return ((int64_t(1) << 32) - 1) / threads; }
constexpr int kFp8Group = 128;     // channels per FP8 scale
constexpr int kMaxRanks = 256;     // logical ranks supported by one call
constexpr int kMaxExperts = 8192;  // experts (LDS histogram bound)
constexpr int kStatusCapacity = 4; // device status word value of MIEP_ECAPACITY

// Division by a launch constant without the ~30-instruction integer divide:
// floor(n / d) = (n * m) >> shift with shift = 31 + ceil(log2 d) and m =
// ceil(2^shift / d), which is at least 2^31 and below 2^32.  Writing m =
// (2^shift + e) / d with 0 <= e < d, the product overshoots n / d by n * e /
// (d * 2^shift), below the 1 / d gap to the next integer because n * e < 2^31
// * d <= 2^shift; and n * m < 2^63.  So it is exact for every 0 <= n < 2^31
// and 1 <= d < 2^31.
struct FastDiv {
  uint32_t m;
  int shift;
  int d;
};
inline FastDiv make_fastdiv(int d) {
  FastDiv f;
  f.d = d > 0 ? d : 1;
  f.shift = 31;
  while ((1ll << (f.shift - 31)) < f.d) ++f.shift;
  f.m = static_cast<uint32_t>(((1ull << f.shift) + static_cast<uint64_t>(f.d) - 1) / static_cast<uint64_t>(f.d));
  return f;
}

// ---- layout histogram (one workgroup per source partition)
struct LayoutArgs {
  int S, T, K, E, R, L;
  FastDiv Ldiv;             // experts per rank
  const int64_t* topk_idx;  // [S*T][K]
  int32_t* ntpr;            // [S][R]
  int32_t* ntp_rdma;        // [S][R/8] or null
  int32_t* ntpe;            // [S][E]
  uint8_t* in_rank;         // [S*T][R]
};
hipError_t launch_layout(const LayoutArgs& a, hipStream_t st);

// ---- notify: prefix matrices, receive offsets, send_head (one workgroup per
// group of channels of a source, or per source where that kernel's conditions
// do not hold)
// group_w == 0: the destinations are the R ranks of in_rank's rows.
// group_w == 8: the destinations are R groups of 8 ranks (rows of R*8
// bytes); a token goes to a group when it goes to any of its ranks.
struct NotifyArgs {
  int S, T, R, C, E, L, align;
  int group_w;
  FastDiv tcdiv;            // tokens per channel, ceil(T / C)
  int nonempty;             // channels holding tokens, ceil(T / tcdiv.d)
  const uint8_t* in_rank;   // [S*T][R] (or [S*T][R*group_w])
  const int32_t* ntpr;      // [S][R]
  const int32_t* ntpe;      // [S][E] or null
  int32_t* rpm;             // [S][R]
  int32_t* cpm;             // [S][R][C]
  int32_t* rcpm;            // [R][S][C]
  int32_t* off;             // [R+1]
  int32_t* send_head;       // [S*T][R]
  int32_t* nrte;            // [R][L] or null
  // Device status word (null: none): workgroup 0 writes kStatusCapacity when
  // the receive rows exceed `capacity`, else 0 -- or, with status_or, writes
  // only on an overflow (a second notify of the same call keeps the first's).
  int32_t* status = nullptr;
  int64_t capacity = 0;
  int status_or = 0;
};
hipError_t launch_notify(const NotifyArgs& a, hipStream_t st);
// Zero-fill of an int32 array by a kernel (no memset node in captured graphs).
hipError_t launch_fill_zero(int32_t* p, int64_t n, hipStream_t st);

// ---- pack: send_head-driven copy of every token to each receiving rank
enum PackKind { kPackBf16 = 0, kPackFp8 = 1, kPackCastFp8 = 2 };
struct PackArgs {
  int64_t N;      // tokens
  int T, H, K, E, L, R;
  int kind;       // PackKind
  int round_scale;
  int meta;       // write recv_src_idx / recv_topk_* (fresh dispatch)
  int64_t capacity;
  const void* x;
  const float* x_scales;
  const int64_t* topk_idx;
  const float* topk_weights;
  const int32_t* send_head;
  const int32_t* off;
  void* recv_x;
  float* recv_x_scales;
  uint8_t* recv_ue = nullptr;  // [cap][H/128] exponent bytes of power-of-two scales (fused cast), or null
  int64_t* recv_topk_idx;
  float* recv_topk_weights;
  int32_t* recv_src_idx;
  // Forwarding from group rows (all null / 0 for a direct dispatch):
  const int32_t* count;      // device row count; rows n >= *count are skipped
  const int32_t* group_off;  // [groups+1] first row of each group; lane j of row n's group g is rank g*group_w + j
  int groups, group_w;
  const int32_t* src_tok;    // [N] source token of row n (top-k metadata, recv_src_idx)
  int cpol = -1;             // cache-policy code of this launch (-1: the default)
  // Receive records of a fresh direct dispatch in their own wavefronts (one
  // per (source, rank)): needs the rank prefix matrix and the membership.
  int S = 0;
  const int32_t* rpm = nullptr;       // [S][R] inclusive rows per rank from sources 0..s
  const uint8_t* in_rank = nullptr;   // [S*T][R]
  int rec_waves = 0, rec_blocks = 0;  // set by launch_pack
  int rec_parts = 1;                  // record wavefronts per (source, rank), each taking every rec_parts-th part
  int rec_last = 0;                   // record workgroups at the end of the grid instead of the front
};
hipError_t launch_pack(const PackArgs& a, hipStream_t st);

// ---- combine: send_head-driven gather and fp32 sum back to token order
struct CombineArgs {
  int64_t N;
  int H, K, R;
  int64_t capacity;
  const uint16_t* y;
  const float* w;            // [cap][K] or null
  const uint16_t* bias0;     // [N][H] or null
  const uint16_t* bias1;     // [N][H] or null
  const int32_t* send_head;
  const int32_t* off;
  uint16_t* out;             // [N][H]
  float* out_w;              // [N][K] or null
  // Group-level reduction (all null / 0 for a direct combine): rows n >=
  // *count are skipped; lane j of row n's group g reads rank g*group_w + j.
  const int32_t* count;
  const int32_t* group_off;  // [groups+1]
  int groups, group_w;
  int cpol = -1;             // cache-policy code of this launch (-1: the default)
  // Row element types (the two-level combine's fp32 partials): y is fp32
  // [cap][H] when in_f32, out is fp32 [N][H] when out_f32 (no rounding).
  int in_f32 = 0, out_f32 = 0;
  int bias_nt = 0;           // bias rows loaded non-temporally (set by launch_combine)
};
hipError_t launch_combine(const CombineArgs& a, hipStream_t st);

// ---- relay: per group row, its source token and its rows in the group's ranks
struct RelayMetaArgs {
  int64_t N;                  // source tokens
  int G, R;                   // groups of 8, ranks
  int64_t rdma_capacity;
  const int32_t* send_rdma_head;  // [N][G]
  const int32_t* rdma_off;        // [G+1]
  const int32_t* send_head;       // [N][R]
  int32_t* rdma_src_idx;          // [rdma_capacity]
  int32_t* send_nvl_head;         // [rdma_capacity][8]
};
hipError_t launch_relay_meta(const RelayMetaArgs& a, hipStream_t st);

// ---- low-latency: per-block message counts, then messages and packed rows in one pass
struct LLArgs {
  int R, T, M, H, K, E, L, d;
  int use_fp8, round_scale, use_ue8m0;
  int64_t msg_bytes;
  const uint16_t* x;
  const int64_t* topk_idx;
  uint8_t* msg;              // [L][R][M] messages, or null: not materialised
  int32_t* msg_count;        // [L][R]
  void* prx;                 // [L][R*M][H] codes or bf16
  float* prs;                // [L][R*M][H/128]
  uint8_t* prue;             // [L][R*M][H/128] or null
  int32_t* src_info;         // [L][R*M]
  int64_t* layout_range;     // [L][R]
  int32_t* count;            // [L]
  int32_t* cumulative;       // [L] or null
  const int32_t* mask;       // [R] nonzero = masked rank, or null
};
hipError_t launch_ll(const LLArgs& a, hipStream_t st);
// The allocation-free variant's count buffer: a file-scope device array of
// kLLScratchCounts int32 (one copy per device); its device address for the
// current device, looked up once per device.
constexpr int kLLScratchCounts = 65536;
constexpr int kMaxDevices = 64;
hipError_t ll_scratch_counts(int32_t** out);

// ---- low-latency combine: rank d's expert outputs back to source-token order
struct LLCombineArgs {
  int R, T, M, H, K, E, L, d;
  const uint16_t* y;             // [L][R*M][H]
  const int32_t* src_info;       // [L][R*M]
  const int64_t* layout_range;   // [L][R]
  const int64_t* topk_idx;       // [R*T][K]
  const float* w;                // [R*T][K] or null
  uint16_t* out;                 // [R*T][H]
};
hipError_t launch_ll_combine(const LLCombineArgs& a, hipStream_t st);

// ---- rank mask helpers: set one entry (launch_mask_set), clear all
// (launch_fill_zero), copy out (launch_copy_i32); tiny kernels
hipError_t launch_mask_set(int32_t* mask, int rank, int value, hipStream_t st);
hipError_t launch_copy_i32(const int32_t* src, int32_t* dst, int n, hipStream_t st);

// ---- groups of rows of one layout: group i holds rows[i] rows from begin[i]
// (null: from i * stride, at most stride of them).  Device data, never
// trusted: kernels read each group as its part inside [0, limit).  Layouts have
// at most kMostRows rows and walks at most as many tiles, which leaves room for
// the 32-bit sums of rows and tiles with a tile, a step or a grid.
constexpr int kMostRows = 0x7fff0000, kMostTiles = kMostRows;
struct GroupArgs {
  int G;
  int stride;
  const int32_t* begin;
  const int32_t* rows;       // null (dense products): one group, the whole layout
  int64_t limit;             // rows of the layout
};

// ---- grouped products, rows side: out[i][p] = sum_c Q[src(i)][c] * P_g[p][c]
// for the rows i of every group g (P_g transposed for the rows' gradient)
enum GemmType { kGemmBf16 = 0, kGemmFp8 = 1, kGemmFp8Ue8m0 = 2 };

// What happens to a product z before it is stored:
//   out = f(z + bias) + residual, z + bias kept aside where asked
// kActSwiglu: the product's columns are [gate | up], out = silu(gate) * up has half of them.
enum Activation { kActNone = 0, kActRelu = 1, kActSilu = 2, kActGelu = 3, kActGeluTanh = 4, kActSwiglu = 5 };
struct Epilogue {
  const float* bias;           // [NO] or null
  const uint16_t* residual;    // [rows][NO or NO/2] bf16 or null
  uint16_t* z;                 // [rows][NO] bf16 or null
  int act;
  int out_f32;
};

struct GemmRowsArgs {
  GroupArgs g;
  const void* q;               // [q_rows][C]
  const void* p;               // [G][NO][C], or [G][C][NO] (bf16, transposed)
  const void* q_scales;        // FP8: [q_rows][C/128]
  const void* p_scales;        // FP8: [G][ceil(NO/128)][C/128]
  const int32_t* row_index;    // [limit] source row of each layout row, or null (itself)
  int64_t q_rows;
  int C, NO;                   // contraction and output width, elements
  uint16_t* out;               // [limit][NO]
  int type, transposed;
  int expected;                // rows a group is expected to hold (0: limit / G)
  Epilogue epi;                // of the linear product
};
hipError_t launch_gemm_rows(const GemmRowsArgs& a, hipStream_t st);

// ---- grouped products, weight gradient: out_g[n][k] (+)= sum over the rows i
// of group g of Q[i][n] * P[src(i)][k]
struct GemmWeightArgs {
  GroupArgs g;
  const uint16_t* q;           // [limit][N] output gradients
  const uint16_t* p;           // [p_rows][K] the product's rows
  const int32_t* row_index;    // [limit] or null
  int64_t p_rows;
  int N, K;
  void* out;                   // [G][N][K] fp32 or bf16
  int out_f32, accumulate;
};
hipError_t launch_gemm_weight(const GemmWeightArgs& a, hipStream_t st);

// ---- activation between the two products: rows of [gate | up], 2 * I wide
struct SwigluArgs {
  GroupArgs g;
  int I;
  int round_scale;
  const uint16_t* h;         // [limit][2 * I]
  const uint16_t* da;        // backward: [limit][I]
  void* out;                 // [limit][I] bf16 or E4M3; backward: [limit][2 * I] bf16
  float* scales;             // FP8: [limit][I/128]
  uint8_t* scales_ue8m0;     // FP8: [limit][I/128] or null
  int rows_per_tile;         // set by the launcher
};
enum SwigluKind { kSwigluBf16 = 0, kSwigluFp8 = 1, kSwigluBackward = 2 };
hipError_t launch_swiglu(const SwigluArgs& a, int kind, hipStream_t st);

// ---- expert order: stable counting sort of the received rows' (row, k)
// entries by expert, in `parts` workgroups a rank
constexpr int kMaxLocalExperts = 2048;   // LDS counters of one rank
struct OrderArgs {
  int64_t rows;              // receive rows allocated
  int K, E, R, L, align, parts;
  FastDiv Kdiv;              // set by the launcher
  int64_t slots;             // slots allocated
  const int64_t* topk;       // [rows][K] local expert of each entry, or -1
  const int32_t* off;        // [R+1]
  int32_t* counts;           // [parts][E] workspace
  int32_t* begin;            // [E]
  int32_t* group_rows;       // [E]
  int32_t* slot_row;         // [slots]
  int32_t* row_slot;         // [rows][K]
  int32_t* status;           // or null
};
hipError_t launch_order(const OrderArgs& a, hipStream_t st);

// ---- expert reduce: y[row] = sum over k of w[row][k] * z[slot(row, k)], and its gradient
struct ReduceArgs {
  int64_t rows, slots;
  int H, K;
  const int32_t* row_slot;   // [rows][K]
  const int32_t* num_rows;   // device: rows in use, or null (all)
  const float* w;            // [rows][K] or null (1)
  const uint16_t* z;         // [slots][H]
  const uint16_t* dy;        // backward: [rows][H]
  uint16_t* out;             // y [rows][H]; backward: dz [slots][H]
  float* dw;                 // backward: [rows][K] or null
};
hipError_t launch_reduce(const ReduceArgs& a, hipStream_t st);
hipError_t launch_reduce_backward(const ReduceArgs& a, hipStream_t st);

// ---- dense product with an epilogue: out = epilogue(x w^T), one weight for all rows
struct LinearArgs {
  int64_t rows;
  int N, K;                    // the product's columns and contraction
  const uint16_t* x;           // [rows][K]
  const uint16_t* w;           // [N][K]
  void* out;                   // [rows][N], or [rows][N/2] (kActSwiglu); bf16 or fp32
  Epilogue epi;
};
hipError_t launch_linear(const LinearArgs& a, hipStream_t st);
hipError_t launch_gemm_linear(const GemmRowsArgs& a, hipStream_t st);   // more than a few rows
constexpr int kLinearFewRows = 64;

// ---- gradient through bias and activation: dz = dy * f'(z), dbias = its sum over the rows
struct ActBackwardArgs {
  int64_t rows;
  int N, act;
  int dy_f32;
  int parts, rows_per_part;    // the rows each workgroup of a column sums
  const void* dy;              // [rows][N or N/2] bf16 or fp32
  const uint16_t* z;           // [rows][N] or null (kActNone)
  uint16_t* dz;                // [rows][N] or null
  float* partial;              // [parts][N]
  float* dbias;                // [N] or null
  int accumulate;              // dbias is added to
};
hipError_t launch_act_backward(const ActBackwardArgs& a, hipStream_t st);

// ---- a few tokens through their experts
constexpr int kLayerTokens = 128, kLayerListBytes = 49024;
// Where a workgroup keeps its lists of experts and their tokens in LDS (bytes).
struct ListsLayout {
  int words, shares, entries;  // 64-bit words of an expert's token mask; shares (16 tokens of an expert) and positions at most
  int start, share, token, weight;
  int64_t end;
};
__host__ __device__ inline ListsLayout lists_layout(int N, int K, int E) {
  ListsLayout l;
  l.words = (N + 63) / 64;
  l.entries = N * K;
  l.shares = (E < l.entries ? E : l.entries) + l.entries / 16;
  l.end = (static_cast<int64_t>(E) * (l.words * 8 + 2) + l.shares * 8ll + l.entries * 6ll + 40) / 16 * 16;
  l.start = E * l.words * 8;
  l.share = (l.start + E * 2 + 7) / 8 * 8;
  l.token = l.share + l.shares * 8;
  l.weight = (l.token + l.entries * 2 + 3) / 4 * 4;
  return l;
}
struct LayerArgs {
  int N, K, E, H, I;
  int tile;                    // output channels a workgroup; set by the launcher
  int64_t first;               // the first expert that is here
  int type;                    // GemmType of the weights
  const uint16_t* x;           // [N][H]
  const int64_t* idx;          // [N][K]
  const float* wts;            // [N][K]
  const void* w1;              // [E][2I][H]
  const void* w2;              // [E][H][I]
  const void* s1;              // E4M3: [E][2I/128][H/128]
  const void* s2;              // E4M3: [E][H/128][I/128]
  const uint16_t* residual;    // [N][H] or null
  uint16_t* a;                 // [N*K][I] between the two products
  uint16_t* y;                 // [N][H]
};
hipError_t launch_layer(const LayerArgs& a, hipStream_t st);

// ---- the router's choice and its gradient
enum GateScore { kGateSoftmax = 0, kGateSigmoid = 1 };
constexpr int kGateExperts = 2048, kGateTopk = 64, kGateGroups = 64;
struct GateArgs {
  int64_t N;
  int E, K;
  int score, renorm;
  int groups, top_groups, group_best;
  float scale;
  int f32;                     // logits (and their gradient): fp32, or bf16
  int per_group, lanes, each;  // set by the launcher
  FastDiv per_div;             // set by the launcher
  const void* logits;          // [N][E]
  const float* bias;           // [E] or null
  int64_t* idx;                // [N][K]
  float* w;                    // [N][K]
  const float* d_w;            // backward: [N][K]
  void* d_logits;              // backward: [N][E]
};
hipError_t launch_gate(const GateArgs& a, bool backward, hipStream_t st);

// Optional launch-geometry overrides read once from the environment
// (MIEP_PACK_VPL, MIEP_PACK_SLICES, MIEP_COMBINE_VPL, MIEP_COMBINE_SLICES,
// MIEP_COMBINE_MAXR, MIEP_PACK_NT, MIEP_COMBINE_NT, MIEP_LL_SPLIT,
// MIEP_LL_VPL, MIEP_CAST_TPB, MIEP_LLC_VPL, MIEP_LLC_SLICES, MIEP_LLC_NT,
// MIEP_LL_NT, MIEP_PACK_RECORDS, MIEP_LL_TPB, MIEP_LL_COUNT_SRC,
// MIEP_NOTIFY_CHAN, MIEP_BIAS_NT):
// used by geometry sweeps, never required.
// combine_maxr: source rows whose loads are issued together.
// pack_nt / combine_nt: cache policy of the row traffic, bit 0 =
// non-temporal loads, bit 1 = non-temporal stores, bit 2 = device-scope
// (sc1) stores; -1 (unset) leaves it to the launch.  Defaults, measured on
// MI355X: over the whole normal step (layout, dispatch, combine back to
// back) pack 6 (plain loads of x, non-temporal device-scope stores) and
// combine 5 (non-temporal loads of the expert outputs, device-scope
// stores); setting both or neither of the non-temporal bits costs ~20% in
// either kernel.  The relay's forwarding pack and group-level combine take 7
// (its group rows are written once and read once more right after); its
// first hop and token-level combine keep the direct path's 6 and 5.  ll_split: workgroups per
// low-latency (expert, source) block.  cast_tpb: fused FP8 cast with one
// token per workgroup (1), or 1 KiB slices (0 or -1, the default).
// llc_vpl / llc_slices / llc_nt: low-latency combine vectors per lane,
// slices per token and cache-policy code (as pack_nt); ll_nt: the
// low-latency send's cache-policy code.  pack_records: 0 writes a fresh
// dispatch's receive records from the payload wavefronts instead of the
// record wavefronts (-1, the default: record wavefronts where supported).
// ll_tpb: threads per low-latency send workgroup (256, 512 or 1024; 0 =
// chosen per call); ll_count_src: 0 counts messages with one workgroup per
// (l, s) block instead of one per source (-1, the default).  notify_chan: 0
// runs the per-source notify everywhere, n > 0 caps the channels per
// workgroup of the channel-group notify (-1, the default: as many whole
// channels as fit in one wavefront, where supported).  bias_nt: 1 loads the
// combine's bias rows non-temporally, 0 with the default policy (-1, the
// default: non-temporally when a bias is larger than half the 256 MiB
// last-level cache, which it then could not hold anyway).
struct Tuning {
  int pack_vpl, pack_slices, combine_vpl, combine_slices, combine_maxr, pack_nt, combine_nt, ll_split, ll_vpl,
      cast_tpb, llc_vpl, llc_slices, llc_nt, ll_nt, pack_records, ll_tpb, ll_count_src, notify_chan, bias_nt;
};
const Tuning& tuning();

}  // namespace miep
