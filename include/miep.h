/*
 * miep.h -- C ABI of the MI355X (gfx950) MoE expert-parallel core:
 * layout histogram, normal-mode dispatch with its handle, cached dispatch,
 * combine (with optional bias rows), the two-level relay (dispatch through
 * one buffer per group of 8 ranks and the two-level combine), low-latency
 * (expert-major, optionally FP8) dispatch and combine, the low-latency
 * rank mask, and what the experts compute between dispatch and combine:
 * expert order, grouped matrix products (bf16 with their gradients, E4M3),
 * the activation between them, and the weighted sum back to received rows;
 * and the block around them: the router's choice, dense products with their
 * epilogue, and the whole expert layer for a few tokens.
 *
 * One GPU plays every rank: the R logical ranks are partitions of one
 * device's HBM, and the S source partitions are the token blocks that the
 * R ranks would each send.  No inter-GPU transport is involved.
 *
 * Pages the calls follow (titles as published):
 *   [Ch4]  "Chapter 4  V1: layout, dispatch and combine", sections 4.1-4.5
 *   [NvLL] "DeepEP Normal vs Low-Latency dual-mode analysis"
 *   [Phil] "Normal vs Low-Latency: two communication philosophies in
 *          DeepEP V1 / V2 / DeepGEMM"
 *
 * Conventions for every call
 *   - Pointers are DEVICE pointers unless a parameter says "host", owned by
 *     the caller; the library keeps no pointer after the call returns and
 *     allocates no device memory.
 *   - `stream` is a hipStream_t (NULL = the null stream).  Every call only
 *     enqueues work on it and returns; the caller orders and synchronises.
 *   - Integer matrices are row-major int32 unless noted; booleans are one
 *     byte, 0 or 1.  bf16 data is passed as its 16-bit patterns.
 *   - Every call returns miep_status and miep_last_error() describes a
 *     failure (thread-local, host memory owned by the library).  Argument
 *     errors (EINVAL, EUNSUPPORTED) are found before anything is enqueued;
 *     an EHIP from a call that launches several kernels may leave its
 *     earlier kernels enqueued.  No call aborts, traps or prints.
 *   - Device-side bounds: rows at or past `recv_capacity` are never
 *     written; top-k entries outside [0, num_experts) are treated as masked.
 *   - Errors the host cannot see at call time (a receive side larger than
 *     its fixed capacity) are reported through a caller-owned device status
 *     word: the call writes 0 or the miep_status code, and
 *     miep_check_status() reads it back synchronously.
 */
#ifndef MIEP_H
#define MIEP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum miep_status {
  MIEP_OK = 0,
  MIEP_EINVAL = 1,       /* a bad argument: null pointer, size or flag */
  MIEP_EUNSUPPORTED = 2, /* valid, but outside what the kernels handle (e.g. R > 256, misaligned x) */
  MIEP_EHIP = 3,         /* the HIP runtime refused a launch */
  MIEP_ECAPACITY = 4     /* device status: the receive rows exceeded a fixed capacity (rows past it were dropped) */
} miep_status;

/* Payload kinds of a normal-mode dispatch. */
typedef enum miep_xkind {
  MIEP_X_BF16 = 0,          /* x: [N][H] bf16; rows travel as 2H bytes                         */
  MIEP_X_FP8 = 1,           /* x: [N][H] E4M3 codes + x_scales [N][H/128] fp32 (pre-quantised)  */
  MIEP_X_BF16_CAST_FP8 = 2  /* x: [N][H] bf16, cast per 128 channels to E4M3 + fp32 scales      */
} miep_xkind;

/* Sizes of one normal-mode problem.  N = num_src * num_tokens tokens. */
typedef struct miep_problem {
  int32_t num_src;          /* S: source partitions (the sending ranks), <= 2^20         */
  int32_t num_tokens;       /* T: tokens per source partition                             */
  int32_t hidden;           /* H: channels per token, <= 2^24                             */
  int32_t num_topk;         /* K: experts per token, <= 64; a dispatch needs
                               N * min(K, R) <= 2^31-1 (int32 receive rows)                */
  int32_t num_experts;      /* E: experts; expert e lives on rank e / (E / R)              */
  int32_t num_ranks;        /* R: receiving ranks, 1..256; R > 8 needs R % 8 == 0          */
  int32_t num_channels;     /* C: channels splitting each source's tokens (ceil(T/C) each), <= 1024 */
  int32_t expert_alignment; /* a >= 1: per-expert receive counts rounded up to a multiple  */
} miep_problem;

/* The normal-mode handle ([Ch4] 4.2: a reverse-routing record, reused by
 * cached dispatch and combine).  All arrays are caller-owned device memory;
 * miep_dispatch fills every non-const member, is_token_in_rank is its input.
 *   rank_prefix_matrix[s][r]            inclusive over sources: rows rank r receives from sources 0..s
 *   channel_prefix_matrix[s][r][c]      inclusive over channels: tokens of source s, channels 0..c, sent to r
 *   recv_channel_prefix_matrix[r][s][c] rank r's row count before source s plus channel_prefix_matrix[s][r][c]
 *   recv_rank_offset[r]                 first receive row of rank r; [R] = total rows (may exceed capacity)
 *   recv_src_idx[row]                   token index t (within its source) of each receive row
 *   is_token_in_rank[n][r]              layout membership, n = s*T + t
 *   send_head[n][r]                     row of token n inside rank r's block, or -1
 * Rank r's rows are recv rows [recv_rank_offset[r], recv_rank_offset[r+1]),
 * ordered by (source, token).  The handle stays valid while the arrays live
 * and the routing is unchanged. */
typedef struct miep_handle {
  int32_t* rank_prefix_matrix;         /* [S][R]    */
  int32_t* channel_prefix_matrix;      /* [S][R][C] */
  int32_t* recv_channel_prefix_matrix; /* [R][S][C] */
  int32_t* recv_rank_offset;           /* [R + 1]   */
  int32_t* recv_src_idx;               /* [recv_capacity] */
  const uint8_t* is_token_in_rank;     /* [N][R]    */
  int32_t* send_head;                  /* [N][R]    */
  int64_t recv_capacity;               /* rows allocated in every receive-side array */
} miep_handle;

/* get_dispatch_layout -- [Ch4] 4.1: from the top-k routing compute the
 * tokens per rank, per RDMA rank (groups of 8 ranks, [NvLL] RDMA rank
 * translation), per expert, and the token-in-rank membership.
 *   topk_idx                 [N][K] int64, negative = masked
 *   num_tokens_per_rank      [S][R]   out
 *   num_tokens_per_rdma_rank [S][R/8] out; must be NULL when R <= 8, non-NULL when R > 8
 *   num_tokens_per_expert    [S][E]   out (counts top-k entries)
 *   is_token_in_rank         [N][R]   out (0/1 bytes)
 * Errors: EINVAL for a null required pointer or bad sizes (E % R != 0,
 * R > 8 with R % 8 != 0); EUNSUPPORTED for R > 256 or E > 8192. */
miep_status miep_get_dispatch_layout(const miep_problem* p, const int64_t* topk_idx,
                                     int32_t* num_tokens_per_rank, int32_t* num_tokens_per_rdma_rank,
                                     int32_t* num_tokens_per_expert, uint8_t* is_token_in_rank, void* stream);

/* dispatch -- [Ch4] 4.1 fresh branch: notify (the prefix matrices) then
 * pack every token into each rank that receives it, rank-major.
 *   x                  [N][H] per x_kind (16-byte aligned; H % 8 == 0, FP8 kinds H % 128 == 0)
 *   x_scales           [N][H/128] fp32 for MIEP_X_FP8, else ignored
 *   round_scale        for MIEP_X_BF16_CAST_FP8: power-of-two scales
 *   use_ue8m0          ([Ch4] 4.3 flag) also emit each power-of-two scale 2^e as
 *                      its exponent byte e + 127; needs MIEP_X_BF16_CAST_FP8 with
 *                      round_scale (else EINVAL).  The fp32 scales are written too.
 *   topk_idx           [N][K] int64, nullable (then no recv_topk_* output)
 *   topk_weights       [N][K] fp32, nullable
 *   num_tokens_per_rank   [S][R] from get_dispatch_layout (source of the rank prefixes)
 *   num_tokens_per_expert [S][E] from get_dispatch_layout, nullable
 *   recv_x             [cap][H] bf16, or [cap][H] E4M3 codes for the FP8 kinds
 *   recv_x_scales      [cap][H/128] fp32 for the FP8 kinds
 *   recv_x_scales_ue8m0 [cap][H/128] uint8, required with use_ue8m0, else ignored
 *   recv_topk_idx      [cap][K] int64: local expert id (e - r*E/R) where expert e is on the row's rank, else -1
 *   recv_topk_weights  [cap][K] fp32: the weight there, else 0
 *   num_recv_tokens_per_expert [R][E/R] out, nullable: per-expert receive count rounded up to expert_alignment
 *   status             one int32 of device memory, nullable: set to 0, or to
 *                      MIEP_ECAPACITY when the receive rows exceed recv_capacity
 *   h                  the handle (all members required; cap = h->recv_capacity)
 * Size the receive side exactly with sum(num_tokens_per_rank) (never
 * overflows), or with a worst case (the num_worst_tokens mode of [Ch4] 4.1):
 * recv_rank_offset[R] reports the true total either way, and rows at or past
 * the capacity are neither written nor, later, combined -- a token whose row
 * fell past it loses that contribution in miep_combine.  A dispatch whose
 * status reads MIEP_ECAPACITY must be redone with a larger capacity before
 * its handle is used. */
miep_status miep_dispatch(const miep_problem* p, const void* x, int32_t x_kind, const float* x_scales,
                          int32_t round_scale, int32_t use_ue8m0, const int64_t* topk_idx, const float* topk_weights,
                          const int32_t* num_tokens_per_rank, const int32_t* num_tokens_per_expert, void* recv_x,
                          float* recv_x_scales, uint8_t* recv_x_scales_ue8m0, int64_t* recv_topk_idx,
                          float* recv_topk_weights, int32_t* num_recv_tokens_per_expert, int32_t* status,
                          const miep_handle* h, void* stream);

/* cached_dispatch -- [Ch4] 4.1 cached branch: with a handle from an earlier
 * dispatch of the same routing, move only x (and its scales); there are no
 * top-k arguments.  Arguments as in miep_dispatch (use_ue8m0 and
 * recv_x_scales_ue8m0 likewise); only h->send_head, h->recv_rank_offset and
 * h->recv_capacity are read. */
miep_status miep_cached_dispatch(const miep_problem* p, const void* x, int32_t x_kind, const float* x_scales,
                                 int32_t round_scale, int32_t use_ue8m0, const miep_handle* h, void* recv_x,
                                 float* recv_x_scales, uint8_t* recv_x_scales_ue8m0, void* stream);

/* check_status -- host-side read of a status word written by miep_dispatch
 * or miep_relay_dispatch: waits for `stream` (synchronous), copies the word
 * and returns it (MIEP_OK or MIEP_ECAPACITY).  EINVAL for a null pointer,
 * EHIP if the copy fails. */
miep_status miep_check_status(const int32_t* status, void* stream);

/* combine -- [Ch4] 4.2 and 4.4: send expert outputs back through the handle
 * and add them per source token in fp32 (no gate weights applied), and
 * separately add the received top-k weights.  Contributions are added in
 * ascending rank order; a token no rank received combines to zero.  Only
 * rows below h->recv_capacity are read (after an overflowed dispatch the
 * rows past it are missing from the sums).
 * [Ch4] 4.2 also unpacks a bias into two rows for the combine without a
 * formula; here each given bias row is added to its token's fp32 sum after
 * the received contributions, bias_0 first (a token no rank received then
 * combines to its bias).
 *   y                     [cap][H] bf16 expert outputs in the receive layout
 *   recv_topk_weights     [cap][K] fp32, nullable
 *   bias_0, bias_1        [N][H] bf16 each, nullable, 16-byte aligned
 *   combined_x            [N][H] bf16 out (round to nearest even)
 *   combined_topk_weights [N][K] fp32 out, nullable (required if recv_topk_weights is given)
 * Reads h->send_head, h->recv_rank_offset, h->recv_capacity. */
miep_status miep_combine(const miep_problem* p, const uint16_t* y, const float* recv_topk_weights,
                         const uint16_t* bias_0, const uint16_t* bias_1, const miep_handle* h,
                         uint16_t* combined_x, float* combined_topk_weights, void* stream);

/* The two-level relay's handle ([NvLL] normal-mode internode dispatch:
 * RDMA to the destination node, then forwarding over NVLink inside it;
 * [Ch4] 4.2: the internode handle adds RDMA prefixes and source metadata).
 * Groups g = 0..G-1 of 8 ranks (ranks 8g..8g+7, the RDMA rank translation)
 * stand for the nodes.  All arrays are caller-owned device memory filled by
 * miep_relay_dispatch:
 *   rdma_rank_prefix_matrix[s][g]            inclusive over sources: group rows group g receives from sources 0..s
 *   rdma_channel_prefix_matrix[s][g][c]      inclusive over channels: tokens of source s, channels 0..c, sent to group g
 *   recv_rdma_channel_prefix_matrix[g][s][c] group g's row count before source s plus rdma_channel_prefix_matrix[s][g][c]
 *   recv_rdma_offset[g]                      first group row of group g; [G] = total group rows
 *   send_rdma_head[n][g]                     row of token n inside group g's block, or -1
 *   rdma_src_idx[row]                        source token n = s*T + t of each group row
 *   send_nvl_head[row][j]                    row of the group row inside rank 8g+j's receive block, or -1
 * A token goes to group g when it goes to any of the group's ranks; group
 * g's rows are [recv_rdma_offset[g], recv_rdma_offset[g+1]), in (source,
 * token) order.  send_head, send_rdma_head and send_nvl_head must be
 * 16-byte aligned, is_token_in_rank 8-byte aligned. */
typedef struct miep_relay_handle {
  int32_t* rdma_rank_prefix_matrix;         /* [S][G]    */
  int32_t* rdma_channel_prefix_matrix;      /* [S][G][C] */
  int32_t* recv_rdma_channel_prefix_matrix; /* [G][S][C] */
  int32_t* recv_rdma_offset;                /* [G + 1]   */
  int32_t* send_rdma_head;                  /* [N][G]    */
  int32_t* rdma_src_idx;                    /* [rdma_capacity] */
  int32_t* send_nvl_head;                   /* [rdma_capacity][8] */
  int64_t rdma_capacity;                    /* group rows allocated in rdma_x, rdma_src_idx, send_nvl_head */
} miep_relay_handle;

/* relay_dispatch -- the normal dispatch through the two-level relay: each
 * token is written once per destination group into the group rows (rdma_x;
 * the FP8 cast of MIEP_X_BF16_CAST_FP8 happens once, before this first hop),
 * then every group row is forwarded to each of the group's ranks that
 * receive the token.  The receive side (recv_x, recv_x_scales,
 * recv_topk_*, num_recv_tokens_per_expert and the handle h) is exactly that
 * of miep_dispatch with the same arguments; rh describes the group rows.
 *   num_tokens_per_rdma_rank [S][G] from get_dispatch_layout (required)
 *   rdma_x        [rdma_capacity][H] bf16, or E4M3 codes for the FP8 kinds (16-byte aligned)
 *   rdma_x_scales [rdma_capacity][H/128] fp32 for the FP8 kinds
 * Other arguments as in miep_dispatch.  Needs R % 8 == 0 and R > 8.  Group
 * rows at or past rh->rdma_capacity are neither written nor forwarded;
 * recv_rdma_offset[G] reports the true total.  `status` (nullable) reads
 * MIEP_ECAPACITY when either the group rows or the receive rows exceed
 * their capacity, else 0. */
miep_status miep_relay_dispatch(const miep_problem* p, const void* x, int32_t x_kind, const float* x_scales,
                                int32_t round_scale, const int64_t* topk_idx, const float* topk_weights,
                                const int32_t* num_tokens_per_rank, const int32_t* num_tokens_per_rdma_rank,
                                const int32_t* num_tokens_per_expert, void* rdma_x, float* rdma_x_scales,
                                void* recv_x, float* recv_x_scales, int64_t* recv_topk_idx,
                                float* recv_topk_weights, int32_t* num_recv_tokens_per_expert, int32_t* status,
                                const miep_handle* h, const miep_relay_handle* rh, void* stream);

/* relay_cached_dispatch -- [Ch4] 4.1 cached branch through the relay: with
 * the handles of an earlier miep_relay_dispatch of the same routing, move
 * only x (and its scales) through the group rows to the ranks' rows; no
 * top-k arguments.  Reads h->send_head's placement only through rh
 * (send_rdma_head, recv_rdma_offset, send_nvl_head) and h->recv_rank_offset;
 * arguments as in miep_relay_dispatch. */
miep_status miep_relay_cached_dispatch(const miep_problem* p, const void* x, int32_t x_kind, const float* x_scales,
                                       int32_t round_scale, const miep_handle* h, const miep_relay_handle* rh,
                                       void* rdma_x, float* rdma_x_scales, void* recv_x, float* recv_x_scales,
                                       void* stream);

/* relay_combine -- the two-level combine, the reverse of miep_relay_dispatch
 * ([NvLL] normal mode reduces inside the node first, then once more across
 * nodes; [Ch4] 4.4: additions only, weights reduced separately).  First
 * level: each group row sums, in fp32 from its first term, the rows of the
 * group's ranks j ascending that hold it, into rdma_y: rounded to bf16 (the
 * type a partial travels in), or kept fp32 when partial_f32 is set (twice
 * the partial bytes; the result is then one fp32 sum rounded once, which
 * stays within bf16 rounding of the fp32 reference even where partials
 * cancel); the received top-k weights likewise in fp32 into rdma_w.
 * Second level: each source token sums its groups' partials g ascending in
 * fp32, then bias_0 and bias_1 as in miep_combine, rounded once more to
 * bf16.  A token no rank received combines to zero (or its bias).
 *   y                     [cap][H] bf16 expert outputs in the receive layout
 *   recv_topk_weights     [cap][K] fp32, nullable
 *   bias_0, bias_1        [N][H] bf16, nullable
 *   partial_f32           0: bf16 partials, 1: fp32 partials
 *   rdma_y                [rdma_capacity][H] bf16 (or fp32) scratch (out: the partials), 16-byte aligned
 *   rdma_w                [rdma_capacity][K] fp32 scratch, required if recv_topk_weights is given
 *   combined_x            [N][H] bf16 out
 *   combined_topk_weights [N][K] fp32 out, nullable (required if recv_topk_weights is given)
 * Reads h->recv_rank_offset, h->recv_capacity and rh's heads and offsets. */
miep_status miep_relay_combine(const miep_problem* p, const uint16_t* y, const float* recv_topk_weights,
                               const uint16_t* bias_0, const uint16_t* bias_1, const miep_handle* h,
                               const miep_relay_handle* rh, int32_t partial_f32, void* rdma_y, float* rdma_w,
                               uint16_t* combined_x, float* combined_topk_weights, void* stream);

/* Sizes of one low-latency problem, seen from the receiving rank dest_rank. */
typedef struct miep_ll_problem {
  int32_t num_ranks;   /* R: source ranks (all ranks send), 1..1024          */
  int32_t num_tokens;  /* T: tokens per source rank, T <= max_tokens          */
  int32_t max_tokens;  /* M: num_max_dispatch_tokens_per_rank (slot capacity) */
  int32_t hidden;      /* H: H % 8 == 0; with FP8, H % 128 == 0               */
  int32_t num_topk;    /* K */
  int32_t num_experts; /* E: E % R == 0; L = E / R local experts per rank     */
  int32_t dest_rank;   /* d: the receiving rank modelled                      */
} miep_ll_problem;

/* Bytes of one low-latency message ([Phil] message format): a 16-byte
 * header (int32 source token index + 3 reserved int32, zero here), then
 * either H E4M3 bytes and H/128 fp32 scales, or 2H bf16 bytes, rounded up
 * to a multiple of 16 bytes (FP8 with H % 512 != 0: up to 12 padding bytes,
 * left unwritten).  Host-only; -1 for hidden <= 0. */
int64_t miep_ll_msg_bytes(int32_t hidden, int32_t use_fp8);

/* low_latency_dispatch -- [NvLL] low-latency dispatch (send loop, receive
 * layout) and [Ch4] 4.3 outputs.  Send side: every top-k entry of a source
 * token that names one of rank d's local experts becomes one message,
 * written expert-major to slot (l, s, j) of msg_buf; j counts such entries
 * of source s in (token, k) order.  Receive side: for each local expert l
 * the (l, s) blocks are packed in ascending s.
 *   x              [R*T][H] bf16;  topk_idx [R*T][K] int64 (negative = masked)
 *   use_fp8        cast per 128 channels (round_scale: power-of-two scales;
 *                  use_ue8m0 additionally emits exponent bytes, requires round_scale)
 *   msg_buf        [L][R][M] messages of miep_ll_msg_bytes() (16-byte aligned) -- scratch standing in for the transport
 *   msg_count      [L][R] int32 out: messages per (local expert, source), capped at M
 *   packed_recv_x  [L][R*M][H] E4M3 codes, or bf16 without FP8 (rows past the count untouched)
 *   packed_recv_x_scales [L][R*M][H/128] fp32 (FP8 only)
 *   packed_recv_x_scales_ue8m0 [L][R*M][H/128] uint8 exponent + 127, nullable (FP8 + use_ue8m0 only)
 *   packed_recv_src_info [L][R*M] int32: source token index of each row
 *   packed_recv_layout_range [L][R] int64: (first row << 32) | count
 *   packed_recv_count [L] int32: rows per local expert
 *   cumulative_local_expert_recv_stats [L] int32, nullable: += packed_recv_count
 *   mask_buffer    [R] int32, nullable: rank masking ([NvLL] low-latency
 *                  send loop and receive wait), nonzero = masked.  If rank d
 *                  or source s is masked, no message travels from s to d:
 *                  the (l, s) blocks hold 0 rows.
 * Errors: EINVAL for bad sizes or flags, FP8 with H % 128 != 0, or a null
 * required pointer; EUNSUPPORTED for R > 1024, M > 4096, K > 64,
 * H % 8 != 0, or misaligned x / msg_buf / packed_recv_x. */
miep_status miep_ll_dispatch(const miep_ll_problem* q, const uint16_t* x, const int64_t* topk_idx, int32_t use_fp8,
                             int32_t round_scale, int32_t use_ue8m0, void* msg_buf, int32_t* msg_count,
                             void* packed_recv_x, float* packed_recv_x_scales, uint8_t* packed_recv_x_scales_ue8m0,
                             int32_t* packed_recv_src_info, int64_t* packed_recv_layout_range,
                             int32_t* packed_recv_count, int32_t* cumulative_local_expert_recv_stats,
                             const int32_t* mask_buffer, void* stream);

/* low_latency_dispatch_noalloc -- for callers that cannot allocate device
 * memory (code under HIP graph capture, tight serving loops, harnesses that
 * forbid hipMalloc): miep_ll_dispatch without the message buffer and counts.
 * Same arguments and the same receive side (packed_recv_*, cumulative stats,
 * rank mask) as miep_ll_dispatch; the messages, which only stand in for the
 * transport, are not materialised, and the per-(local expert, source)
 * message counts that its two kernels share live in a device array of the
 * library (65536 int32 per device, held until the process ends).
 * It allocates nothing (no hipMalloc, no hipFree, no allocating library call).
 * Every call on one device shares that array: calls that overlap on one
 * device (concurrent streams) race and must be ordered by the caller; each
 * call overwrites every count it reads, so nothing needs clearing.
 * Errors: as miep_ll_dispatch; EUNSUPPORTED when num_experts (L * R counts)
 * exceeds 65536; EHIP if the device address of the array cannot be found. */
miep_status miep_ll_dispatch_noalloc(const miep_ll_problem* q, const uint16_t* x, const int64_t* topk_idx,
                                     int32_t use_fp8, int32_t round_scale, int32_t use_ue8m0, void* packed_recv_x,
                                     float* packed_recv_x_scales, uint8_t* packed_recv_x_scales_ue8m0,
                                     int32_t* packed_recv_src_info, int64_t* packed_recv_layout_range,
                                     int32_t* packed_recv_count, int32_t* cumulative_local_expert_recv_stats,
                                     const int32_t* mask_buffer, void* stream);

/* low_latency_combine -- [Ch4] 4.3 and [NvLL] name it beside the
 * low-latency dispatch without its arithmetic.  Here it is the reverse of
 * miep_ll_dispatch seen from rank d: each source token (s, t) gets back the
 * rows of d's local experts that its top-k entries were sent to (the slot
 * rule of the dispatch: the j-th entry of source s naming expert d*L + l,
 * in (token, k) order, is row l*R*M + begin(l, s) + j), each multiplied by
 * the entry's gate weight when topk_weights is given, summed in fp32 in
 * ascending k and rounded once to bf16.  Entries dropped at the slot cap or
 * by rank masking (slot >= count) contribute nothing; a token without a row
 * combines to +0.0.
 *   y                       [L][R*M][H] bf16 expert outputs, packed like packed_recv_x (16-byte aligned)
 *   packed_recv_src_info    [L][R*M] int32 from miep_ll_dispatch
 *   packed_recv_layout_range [L][R] int64 from miep_ll_dispatch
 *   topk_idx                [R*T][K] int64, the routing given to miep_ll_dispatch
 *   topk_weights            [R*T][K] fp32, nullable (then rows are summed unweighted)
 *   combined_x              [R*T][H] bf16 out (16-byte aligned)
 * A handle from another routing is not detected: a row whose src_info does
 * not name the token is skipped, and every access stays inside y.
 * Errors: as miep_ll_dispatch for sizes; EINVAL for a null required pointer. */
miep_status miep_ll_combine(const miep_ll_problem* q, const uint16_t* y, const int32_t* packed_recv_src_info,
                            const int64_t* packed_recv_layout_range, const int64_t* topk_idx,
                            const float* topk_weights, uint16_t* combined_x, void* stream);

/* Rank mask buffer helpers ([NvLL]: the low-latency buffer's mask can be
 * queried, updated and cleaned; a rank is masked when it stops answering).
 * mask_buffer is [num_ranks] int32 device memory owned by the caller.
 *   update: mask_buffer[rank] = value (nonzero = masked)
 *   clean:  every entry = 0
 *   query:  out[r] = mask_buffer[r] for every r (out: [num_ranks] int32 device)
 * Small kernels (no memset or copy nodes), enqueued on `stream`.
 * Errors: EINVAL for a null pointer, num_ranks <= 0 or rank out of range. */
miep_status miep_mask_update(int32_t* mask_buffer, int32_t num_ranks, int32_t rank, int32_t value, void* stream);
miep_status miep_mask_clean(int32_t* mask_buffer, int32_t num_ranks, void* stream);
miep_status miep_mask_query(const int32_t* mask_buffer, int32_t num_ranks, int32_t* out, void* stream);

/* ------------------------------------------------------------------ experts
 * Between dispatch and combine.  A set of row groups names, for each expert
 * g, the rows of one layout that are its own: rows [begin[g], begin[g] +
 * rows[g]) -- the slots of miep_expert_order, or any ragged layout -- or,
 * with begin NULL, rows [g*stride, g*stride + min(rows[g], stride)), the
 * packed blocks of the low-latency dispatch (rows = packed_recv_count, stride
 * = R*M).  Both arrays are device data, read when the kernels run; whatever
 * they hold, only rows in [0, num_rows) are touched.  Groups may be empty and
 * need no alignment; groups that overlap leave either one's result in the
 * shared rows (num_rows in the limits below then counts them in each).  Rows
 * of an output that lie in no group are left as they were, and rows of an
 * input that lie in no group are never read into a result. */
typedef struct miep_row_groups {
  const int32_t* begin;  /* [num_groups] first row, or NULL (g * stride)        */
  const int32_t* rows;   /* [num_groups] rows                                   */
  int64_t num_rows;      /* rows of the layout, 0..2^31-2^16                    */
  int32_t num_groups;    /* 0..8192                                             */
  int32_t stride;        /* rows between group starts where begin is NULL (> 0) */
} miep_row_groups;

/* expert_order -- the received rows of a normal dispatch in expert order: a
 * slot for every (row, k) whose recv_topk_idx names a local expert.  Slots
 * are expert-major (global expert e = rank * E/R + local), each expert's from
 * a multiple of expert_alignment on, and inside an expert in (row, k) order.
 *   recv_topk_idx    [num_rows][K] int64 from miep_dispatch (entries outside [0, E/R) have no slot)
 *   recv_rank_offset [R + 1] int32 from the handle
 *   workspace        [parts][E] int32, parts >= 1: the parts a rank's rows may be sorted in
 *                    (256 / R is enough to fill the GPU); of one call at a time
 *   group_begin      [E] int32 out: first slot of each expert
 *   group_rows       [E] int32 out: its slots (num_recv_tokens_per_expert with expert_alignment 1)
 *   slot_row         [num_slots] int32 out: received row of each slot, -1 where there is none
 *   row_slot         [num_rows][K] int32 out: slot of each entry, or -1 (and for every row behind the last)
 *   status           one int32, nullable: 0, or MIEP_ECAPACITY when the experts need more than num_slots
 *                    (entries past it get no slot)
 * num_rows * K + (expert_alignment - 1) * E slots are always enough.
 * Errors: EINVAL for bad sizes or null pointers; EUNSUPPORTED for R > 256, E > 8192, E/R > 2048,
 * K > 64, or num_rows * K + expert_alignment * E > 2^31-1. */
miep_status miep_expert_order(const int64_t* recv_topk_idx, const int32_t* recv_rank_offset, int64_t num_rows,
                              int32_t num_topk, int32_t num_experts, int32_t num_ranks, int32_t expert_alignment,
                              int32_t* workspace, int32_t parts, int32_t* group_begin, int32_t* group_rows,
                              int32_t* slot_row, int64_t num_slots, int32_t* row_slot, int32_t* status, void* stream);

/* expert_reduce -- expert outputs in slot order back to received rows:
 * y[row] = sum over k of topk_weights[row][k] * z[row_slot[row][k]], added in
 * ascending k in fp32 and rounded once; entries without a slot add nothing, a
 * row without any is zero.  With topk_weights NULL every weight is 1, which
 * also turns the slots' input gradients into the rows'.
 *   z          [num_slots][H] bf16, 16-byte aligned; H % 8 == 0
 *   row_slot   [num_rows][K] int32
 *   total_rows one int32 of device memory, nullable: rows at or past it (recv_rank_offset + R) are left as they were
 *   y          [num_rows][H] bf16 out */
miep_status miep_expert_reduce(const uint16_t* z, int64_t num_slots, int32_t hidden, const int32_t* row_slot,
                               int64_t num_rows, int32_t num_topk, const int32_t* total_rows,
                               const float* topk_weights, uint16_t* y, void* stream);

/* expert_reduce_backward -- its gradients: dz[row_slot[row][k]] =
 * topk_weights[row][k] * dy[row] (bf16; slots that no entry names are left as
 * they were) and, when d_topk_weights is given, d_topk_weights[row][k] =
 * <dy[row], z[row_slot[row][k]]> in fp32 (0 without a slot).  z may be NULL
 * when d_topk_weights is. */
miep_status miep_expert_reduce_backward(const uint16_t* dy, const uint16_t* z, int64_t num_slots, int32_t hidden,
                                        const int32_t* row_slot, int64_t num_rows, int32_t num_topk,
                                        const int32_t* total_rows, const float* topk_weights, uint16_t* dz,
                                        float* d_topk_weights, void* stream);

/* grouped_gemm -- every group's rows times its expert's weights:
 *   y[i][n] = sum over k of x[src(i)][k] * w[g][n][k]     for the rows i of group g
 * in fp32, rounded once to bf16.
 *   x         [x_rows][K] bf16.  src(i) = i (x_rows == num_rows), or row_index[i]
 *   row_index [num_rows] int32, nullable: source row of each layout row (slot_row of
 *             miep_expert_order), any of them any number of times; a row whose index is
 *             outside [0, x_rows) gives zeros.  A gathered x is at most 64 GiB.
 *   w         [num_groups][N][K] bf16;  y [num_rows][N] bf16 out
 *   expected_rows  rows a group is expected to hold, 0 = num_rows / num_groups: chooses the tile,
 *             never the result's meaning.  Give it where the layout is mostly empty (low latency, or slots
 *             for the worst case): 29 rows in 8 blocks of 256 take 79 us with it and 108 without.
 * x, w, y 16-byte aligned; N % 8 == 0, K % 8 == 0, both at most 2^21, and
 * (num_rows / 32 + 1 + num_groups) * (max(N, K) / 128 + 1) at most 2^31-2^16.
 * Errors: EINVAL for null pointers or sizes, EUNSUPPORTED for the limits above. */
miep_status miep_grouped_gemm(const miep_row_groups* g, const uint16_t* x, int64_t x_rows, const uint16_t* w,
                              int32_t n, int32_t k, const int32_t* row_index, int32_t expected_rows, uint16_t* y,
                              void* stream);

/* grouped_gemm_dgrad -- gradient of the rows: dx[i][k] = sum over n of
 * dy[i][n] * w[g][n][k].  dy [num_rows][N] bf16, dx [num_rows][K] bf16 out (in
 * layout rows: expert_reduce without weights adds gathered rows up). */
miep_status miep_grouped_gemm_dgrad(const miep_row_groups* g, const uint16_t* dy, const uint16_t* w, int32_t n,
                                    int32_t k, int32_t expected_rows, uint16_t* dx, void* stream);

/* grouped_gemm_wgrad -- gradient of the weights: dw[g][n][k] = sum over the
 * rows i of group g of dy[i][n] * x[src(i)][k], summed in fp32.
 *   dw_f32      1: dw is fp32; 0: bf16, rounded once
 *   accumulate  1 (fp32 only): added to what dw holds.  0: dw is overwritten, with zeros for an empty group.
 * Rows whose row_index is outside [0, x_rows) contribute nothing, whatever dy holds there. */
miep_status miep_grouped_gemm_wgrad(const miep_row_groups* g, const uint16_t* dy, const uint16_t* x, int64_t x_rows,
                                    const int32_t* row_index, int32_t n, int32_t k, int32_t dw_f32,
                                    int32_t accumulate, void* dw, void* stream);

/* grouped_gemm_fp8 -- miep_grouped_gemm on E4M3 codes with the scales that an
 * FP8 dispatch or the fused cast writes:
 *   y[i][n] = sum over blocks b of x_scales[src(i)][b] * w_scales[g][n/128][b] *
 *             (sum over k in block b of x[src(i)][k] * w[g][n][k])
 * rounded once to bf16.  The matrix instruction cuts the products of each 8
 * consecutive channels toward zero to multiples of 2^(e - 13), e the largest
 * sum of the two operands' exponents in a nonzero one of them, and adds the
 * rest in fp32: a group loses less than 7 * 2^(e - 13), times its scales.
 *   x [x_rows][K], w [num_groups][N][K] E4M3; K % 128 == 0, N % 8 == 0
 *   x_scales [x_rows][K/128], w_scales [num_groups][ceil(N/128)][K/128]: fp32, or with
 *   scales_ue8m0 the exponent bytes e + 127 of power-of-two scales 2^e */
miep_status miep_grouped_gemm_fp8(const miep_row_groups* g, const uint8_t* x, const void* x_scales, int64_t x_rows,
                                  const uint8_t* w, const void* w_scales, int32_t scales_ue8m0, int32_t n, int32_t k,
                                  const int32_t* row_index, int32_t expected_rows, uint16_t* y, void* stream);

/* swiglu -- a = silu(gate) * up over the groups' rows of h [num_rows][2*I] =
 * [gate | up], in fp32, rounded once.  a [num_rows][I] bf16; I % 8 == 0.
 * swiglu_fp8 casts the fp32 value per 128 channels (I % 128 == 0) by the rule
 * of the FP8 dispatch: a E4M3, a_scales [num_rows][I/128] fp32 (powers of two
 * with round_scale), a_scales_ue8m0 their exponent bytes (nullable, needs
 * round_scale).  swiglu_backward: dh [num_rows][2*I] from da [num_rows][I]; dh
 * may be h itself.  Otherwise no output of these calls overlaps an input. */
miep_status miep_swiglu(const miep_row_groups* g, const uint16_t* h, int32_t inner, uint16_t* a, void* stream);
miep_status miep_swiglu_fp8(const miep_row_groups* g, const uint16_t* h, int32_t inner, int32_t round_scale,
                            uint8_t* a, float* a_scales, uint8_t* a_scales_ue8m0, void* stream);
miep_status miep_swiglu_backward(const miep_row_groups* g, const uint16_t* da, const uint16_t* h, int32_t inner,
                                 uint16_t* dh, void* stream);

/* ------------------------------------------------------------------ the block around them
 * gate_topk -- the router's choice: the K experts of each token and their
 * weights, as dispatch and the expert layer take them.
 *   s = softmax(logits) over the experts, or sigmoid(logits) of each;
 *   chosen: the K largest s + bias, equal ones by the lower index, among the experts of the topk_groups best
 *   groups (num_groups equal ranges of experts; a group's score is the sum of its largest group_best s + bias);
 *   topk_weights = scale * s, or with renormalize scale * s / (sum of the chosen s).
 * bias enters the choice alone.  Without bias and groups the logits themselves are compared, otherwise s + bias in
 * 64 bits, so that the choice is the formula's.  A logit of -inf or NaN is a masked expert: never chosen, score 0;
 * +inf counts as the type's largest number.  A bias of -inf or NaN leaves its expert out of the choice, +inf counts as
 * fp32's largest number.  A group of one expert scores what that does; one that has fewer than group_best of its
 * experts left comes behind all others.  Where fewer than K experts are left, the last topk_idx are -1, weight 0.
 *   logits [num_tokens][E] fp32 (logits_f32) or bf16;  bias [E] fp32, nullable;  both 16-byte aligned
 *   topk_idx [num_tokens][K] int64 out, descending;  topk_weights [num_tokens][K] fp32 out
 * Errors: EINVAL for sizes, flags or null pointers; EUNSUPPORTED for E > 2048, K > 64, num_groups > 64. */
typedef struct miep_gate {
  int64_t num_tokens;    /* N >= 0                                     */
  int32_t num_experts;   /* E                                          */
  int32_t num_topk;      /* K <= E                                     */
  int32_t sigmoid;       /* 0: softmax, 1: sigmoid                     */
  int32_t renormalize;   /* weights of a token add up to scale         */
  int32_t num_groups;    /* >= 1, divides E                            */
  int32_t topk_groups;   /* 1..num_groups                              */
  int32_t group_best;    /* 1 or 2                                     */
  int32_t logits_f32;    /* logits and d_logits: 1 fp32, 0 bf16        */
  float scale;
} miep_gate;
miep_status miep_gate_topk(const miep_gate* g, const void* logits, const float* bias, int64_t* topk_idx,
                           float* topk_weights, void* stream);

/* gate_topk_backward -- gradient of the logits, [N][E] in the logits' type,
 * from the weights' (the choice itself has none; entries outside [0, E) and
 * those of masked experts add nothing, whatever d_topk_weights holds there; an
 * expert named twice adds both). */
miep_status miep_gate_topk_backward(const miep_gate* g, const float* d_topk_weights, const void* logits,
                                    const int64_t* topk_idx, void* d_logits, void* stream);

/* linear -- one weight for all rows (router, shared expert):
 *   z = x w^T + bias,  y = f(z) + residual
 * in fp32, rounded once.  f: the identity, relu, silu, gelu (by the error
 * function, to 1e-7) or its tanh form; or SwiGLU, with z = [gate | up] and y =
 * silu(gate) * up + residual of half the columns.
 *   x [rows][K], w [N][K] bf16;  bias [N] fp32, nullable
 *   residual [rows][N or N/2] bf16, nullable; may be y itself
 *   z [rows][N] bf16 out, nullable: kept for the backward pass
 *   y [rows][N or N/2] out, bf16 or fp32 (y_f32)
 * Everything 16-byte aligned, rows at most 2^31-2^16; N, K % 8 == 0 (SwiGLU: N % 16 == 0), at most 2^21; SwiGLU's w
 * under 4 GiB less 1024 rows; (rows / 32 + 2) * (max(N, K) / 128 + 1), in whole numbers, at most 2^31-2^16 (tiles).
 * Errors: EINVAL for null pointers, sizes, flags; EUNSUPPORTED for the limits above. */
enum { MIEP_ACT_NONE = 0, MIEP_ACT_RELU = 1, MIEP_ACT_SILU = 2, MIEP_ACT_GELU = 3, MIEP_ACT_GELU_TANH = 4, MIEP_ACT_SWIGLU = 5 };
miep_status miep_linear(const uint16_t* x, int64_t rows, const uint16_t* w, int32_t n, int32_t k, const float* bias,
                        int32_t activation, const uint16_t* residual, uint16_t* z, void* y, int32_t y_f32,
                        void* stream);

/* linear_act_backward -- dz = dy * f'(z) (bf16, rounded once; nullable) and
 * dbias[n] = sum of dz's unrounded column over the rows, in fp32 (nullable;
 * accumulate: added to what dbias holds).
 *   dy [rows][N or N/2] bf16 or fp32 (dy_f32);  z [rows][N] bf16 from miep_linear (MIEP_ACT_NONE: ignored)
 *   workspace [parts][N] fp32, parts >= 1, where dbias is given: the parts the rows may be summed in (one for
 *   every 16 rows, up to 256, is enough to fill the GPU); of one call at a time
 * relu's f' is 1 for z > 0 and 0 elsewhere, also where z is no number.
 * linear_dgrad -- dx = dy w.  linear_wgrad -- dw = dy^T x, fp32 (dw_f32; accumulate: added) or bf16.
 * Alignment, limits and errors of all three: as linear's (linear_act_backward: without K), and for linear_wgrad at most
 * 2^24 tiles of 128 x 128 of dw. */
miep_status miep_linear_act_backward(const void* dy, int32_t dy_f32, const uint16_t* z, int64_t rows, int32_t n,
                                     int32_t activation, uint16_t* dz, float* dbias, int32_t accumulate,
                                     float* workspace, int32_t parts, void* stream);
miep_status miep_linear_dgrad(const uint16_t* dy, int64_t rows, const uint16_t* w, int32_t n, int32_t k, uint16_t* dx,
                              void* stream);
miep_status miep_linear_wgrad(const uint16_t* dy, const uint16_t* x, int64_t rows, int32_t n, int32_t k,
                              int32_t dw_f32, int32_t accumulate, void* dw, void* stream);

/* expert_layer -- a few tokens through their experts and back, in place of
 * dispatch, the experts' products and combine (decoding):
 *   y[t] = residual[t] + sum over k of topk_weights[t][k] * W2_e (silu(g) * u),  [g | u] = W1_e x[t]
 * for the entries e = topk_idx[t][k] in [first_expert, first_expert + num_experts); others (masked, or another
 * rank's) add nothing.  Every chosen expert's weights are read once.  Sums are fp32, silu(g) * u is rounded to bf16
 * between the products, y once; a token's experts are added in ascending order, an expert named twice with the sum
 * of its weights.
 *   x [N][H] bf16;  w1 [E][2I][H] = [gate | up], w2 [E][H][I], all bf16, or all E4M3 codes with a scale for each 128 x
 *   128 block: w1_scales [E][2I/128][H/128], w2_scales [E][H/128][I/128], fp32 or (scales_ue8m0) exponent bytes
 *   (2^(byte-127); 255 is NaN).  Codes are multiplied as bf16 numbers, which they are exactly: x is not cast.
 *   residual [N][H] bf16, nullable; may be y itself
 *   workspace [N*K][I] bf16, of one call at a time
 * N at most 128; H, I % 8 == 0 (E4M3: % 128 == 0); weights of one expert under 4 GiB, workspace too; E * (8 *
 * ceil(N/64) + 2) + 8 * min(E, N*K) + 6.5 * N*K under 49,000 bytes.  Larger batches: dispatch.
 * Errors: EINVAL for null pointers, sizes, flags; EUNSUPPORTED for the limits above. */
typedef struct miep_layer {
  int32_t num_tokens;    /* N >= 0                        */
  int32_t num_topk;      /* K <= 64                       */
  int32_t num_experts;   /* E, those that are here        */
  int32_t hidden;        /* H                             */
  int32_t inner;         /* I                             */
  int32_t scales_ue8m0;  /* E4M3: scales are exponent bytes */
  int64_t first_expert;  /* >= 0                          */
} miep_layer;
miep_status miep_expert_layer(const miep_layer* q, const uint16_t* x, const int64_t* topk_idx,
                              const float* topk_weights, const uint16_t* w1, const uint16_t* w2,
                              const uint16_t* residual, uint16_t* workspace, uint16_t* y, void* stream);
miep_status miep_expert_layer_fp8(const miep_layer* q, const uint16_t* x, const int64_t* topk_idx,
                                  const float* topk_weights, const uint8_t* w1, const void* w1_scales,
                                  const uint8_t* w2, const void* w2_scales, const uint16_t* residual,
                                  uint16_t* workspace, uint16_t* y, void* stream);

/* Description of the last failure on this thread ("" if none). Host-only. */
const char* miep_last_error(void);

/* Library version string. Host-only. */
const char* miep_version(void);

#ifdef __cplusplus
}
#endif

#endif /* MIEP_H */
