/*
 * moe_int4.h — C ABI of the MI355X (gfx950) int4 mixture-of-experts layer.
 *
 * The layer: a router scores E experts per token and keeps the top k, a
 * shared expert sees every token, and each expert is a SwiGLU MLP whose three
 * matrices are stored as affine 4-bit integers in groups of 64 with a bf16
 * scale and bias per group. The routing metadata (histogram, prefix scan,
 * scatter, block map) is built on the GPU on the caller's stream with no host
 * synchronisation, and the expert GEMMs read the packed weights and expand
 * them tile by tile on chip with fp32 accumulation.
 *   Sources: diariobitcoin.com, "Perplexity libera Lily, un motor de IA que
 *   supera a MLX-LM en Apple Silicon", sections "Qwen3.6 combina tres cargas de
 *   trabajo" (256 experts, eight per token, shared expert; 4-bit affine g64
 *   format), "Las optimizaciones en el prefill" (dequant fused in the grouped
 *   GEMM, fp32 accumulation; routing histogram, prefix scan, scatter and block
 *   map kept on the GPU; 32-row blocks; bounded prefill chunks) and "El decode
 *   busca mover menos datos" (batch-1 decode is bandwidth bound).
 *
 * Conventions for every entry point:
 *  - Pointers marked "device" are HIP device pointers; "host" are host memory.
 *    bf16 values are passed as uint16_t bit patterns.
 *  - The caller owns every buffer. The library never allocates, frees or keeps
 *    pointers after a call returns; device buffers must stay valid until the
 *    work enqueued on `stream` completes.
 *  - `stream` is a hipStream_t (NULL = the default stream). Work is enqueued
 *    asynchronously; no entry point synchronises the host. Device faults
 *    surface at the caller's next synchronisation.
 *  - Return value: MOE_OK (0) or a negative MOE_E* code. Arguments are checked
 *    before anything is enqueued, so on error nothing has been launched.
 *  - Alignment: x, y, the workspace, the unfused weight buffer, router_w and
 *    the packed blobs must be 16-byte aligned (the kernels move them in
 *    16-byte vectors); logits, logits_out, router_bias and the route_out
 *    arrays 4-byte aligned. Misaligned pointers give MOE_EINVAL. (Fresh
 *    torch / hipMalloc allocations are 256-byte aligned.)
 *  - Supported dims: E <= 256 and E % 64 == 0, top_k == 8, gemm one of
 *    MOE_GEMM_*, block_m 32 or 16
 *    (the routing block size, which is also the row count of the exact
 *    grouped GEMMs' work items; diariobitcoin.com, "Perplexity libera Lily...",
 *    section "Las optimizaciones en el prefill": 32-row blocks replaced
 *    16-row ones), H % 256 == 0 (H <= 4096), I % 128 == 0
 *    (I <= 4096), and T * top_k < 2^30 tokens x slots per call (pair
 *    indices are 32-bit).
 */
#ifndef MOE_INT4_H
#define MOE_INT4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_OK 0
#define MOE_EINVAL (-1)       /* null or misaligned pointer, negative size, bad enum */
#define MOE_EUNSUPPORTED (-2) /* dims outside the supported set above         */
#define MOE_EWORKSPACE (-3)   /* workspace smaller than moe_workspace_bytes   */
#define MOE_EHIP (-4)         /* a HIP launch reported an error               */
#define MOE_EBUFFER (-5)      /* host output buffer too small (packers)       */
#define MOE_EFORMAT (-6)      /* int4 code outside 0..15                      */
#define MOE_ESCRATCH (-7)     /* request exceeds the library's static scratch  */

/* Layer dimensions: hidden size H, expert intermediate size I, routed experts
 * E, experts per token top_k, rows per routing block block_m, and which
 * grouped-GEMM kernels the prefill uses (gemm, one of MOE_GEMM_*):
 *   MOE_GEMM_EXACT  work items of block_m rows; the int4 codes enter the
 *                   matrix cores as exact bf16 values 128 + q and scale and
 *                   bias are applied per output and group in fp32 (weights
 *                   used exactly); suited to short chunks, where few rows
 *                   share an expert and the layer streams weights from HBM;
 *   MOE_GEMM_WIDE   work items of up to 144 rows of one expert; each weight
 *                   is expanded once per item to bf16 w = q*scale + bias
 *                   (fp32 value rounded once to bf16) and the matrix cores
 *                   accumulate x.w in fp32; suited to long chunks, where many
 *                   rows share each expanded weight;
 *   MOE_GEMM_AUTO   (0) WIDE for chunks whose pairs average at least 36 rows
 *                   per expert (top_k * T_chunk >= 36 * E), else EXACT.
 * (diariobitcoin.com, "Perplexity libera Lily...", section "Las
 * optimizaciones en el prefill": the grouped GEMM reconstructs the 4-bit
 * weights block by block on chip with fp32 accumulation.) Decode ignores
 * gemm. */
#define MOE_GEMM_AUTO 0
#define MOE_GEMM_EXACT 1
#define MOE_GEMM_WIDE 2
typedef struct {
  int32_t H, I, E, top_k, block_m, gemm;
} moe_dims;

/* Device weights of one layer. Every pointer is a device pointer. The blobs
 * must have been packed for the dims passed with them (E, H, I): their
 * headers are not read at call time, since that would need a device read
 * and a host synchronisation, so blobs of another shape give wrong results,
 * not an error code. The caller keeps them alive until the stream work that
 * uses them completes. */
typedef struct {
  const void* router_w3;       /* pack_router_bf16x3 blob of Wr (prefill router)     */
  const float* router_w;       /* [E][H] fp32 Wr, row-major (decode router)           */
  const float* router_bias;    /* [E] fp32 added to the logits, or NULL                */
  const void* experts_gate_up; /* pack_int4_g64 blob: E experts, gate and up paired   */
  const void* experts_down;    /* pack_int4_g64 blob: E experts, down                  */
  const void* shared_gate_up;  /* pack_int4_g64 blob: 1 expert, gate and up paired    */
  const void* shared_down;     /* pack_int4_g64 blob: 1 expert, down                   */
} moe_layer_weights;

/* Routing metadata (device buffers the caller provides). For T tokens:
 *   topk_idx [T][k] int32  selected experts, larger logit first, ties to the
 *                          lower expert index; slot j of token t is pair t*k+j
 *   topk_w   [T][k] fp32   softmax over all E logits restricted to the k
 *                          selected experts and renormalised to sum to one
 *   hist     [E]    int32  pairs routed to each expert (sums to k*T)
 *   offsets  [E+1]  int32  exclusive prefix sum of hist; offsets[E] = k*T
 *   perm     [k*T]  int32  perm[pos] = pair placed at row pos; the pairs of one
 *                          expert are contiguous, in ascending pair order
 *   inv_perm [k*T]  int32  inv_perm[pair] = pos
 *   block_map [moe_max_blocks(T)][3] int32  for each expert in ascending order,
 *                          ceil(hist[e]/block_m) entries (expert, first row,
 *                          rows in 1..block_m); entries past num_blocks are
 *                          not written
 *   num_blocks [1] int32
 * (diariobitcoin.com, "Perplexity libera Lily...", section "Las optimizaciones
 * en el prefill": histogram, prefix scan, scatter and block map; 32-row blocks.)
 */
typedef struct {
  int32_t* topk_idx;
  float* topk_w;
  int32_t* hist;
  int32_t* offsets;
  int32_t* perm;
  int32_t* inv_perm;
  int32_t* block_map;
  int32_t* num_blocks;
} moe_route_out;

/* Upper bound on the routing blocks of T tokens: ceil(k*T/block_m) + E.
 * Returns a negative code for invalid dims. */
int64_t moe_max_blocks(const moe_dims* dims, int32_t T);

/* Bytes of a pack_int4_g64 blob holding `count` experts of [N][K] matrices
 * (paired != 0: two matrices, gate and up, per expert). 0 if unsupported. */
size_t moe_packed_bytes(int32_t count, int32_t N, int32_t K, int32_t paired);

/* Pack affine int4 weights (host -> host) into the device layout the kernels
 * read. Logical input per matrix, row-major: q [count][N][K] uint8 in 0..15,
 * scale and bias [count][N][K/64] bf16 bits; weight w[n][c] =
 * q[n][c]*scale[n][c/64] + bias[n][c/64] (diariobitcoin.com, "Perplexity
 * libera Lily...", section "Qwen3.6 combina tres cargas de trabajo": 4-bit
 * affine, groups of 64, bf16 scale and bias). With q1/s1/b1 non-null the
 * expert holds two matrices of the same shape (gate = 0, up = 1) interleaved
 * in 32-row slices; with them null, one matrix. The blob is a 256-byte header
 * (magic "MI4G", version 1, count, N, K, paired) followed by one region per
 * expert; the layout is internal to this library and only read by it.
 * K % 64 == 0; N % 32 == 0 (paired) or N % 64 == 0. Returns MOE_EBUFFER if
 * out_bytes < moe_packed_bytes(...), MOE_EFORMAT if a code exceeds 15. */
int pack_int4_g64(const uint8_t* q0, const uint16_t* s0, const uint16_t* b0,
                  const uint8_t* q1, const uint16_t* s1, const uint16_t* b1,
                  int32_t count, int32_t N, int32_t K, void* out, size_t out_bytes);

/* Bytes of a pack_router_bf16x3 blob for an [E][H] router matrix. */
size_t moe_router_packed_bytes(int32_t E, int32_t H);

/* Pack the fp32 router matrix Wr [E][H] (host) into three bf16 planes with
 * Wr = hi + mid + lo exactly (each plane the next 8 significant bits), laid
 * out for the matrix cores (host -> host). E % 64 == 0, H % 64 == 0. */
int pack_router_bf16x3(const float* wr, int32_t E, int32_t H, void* out, size_t out_bytes);

/* Workspace bytes for a call. mode 0: moe_prefill_layer with chunks of at
 * most T_chunk tokens; mode 1: moe_decode_layer with up to T_chunk (<= 4)
 * tokens; mode 2: moe_route of up to T_chunk tokens. */
int moe_workspace_bytes(const moe_dims* dims, int32_t T_chunk, int32_t mode, size_t* bytes);

/* Routing only: from fp32 logits [T][E] (device) fill every field of `out`
 * (device buffers sized for T) on `stream`. T = 0 is a no-op. */
int moe_route(const moe_dims* dims, const float* logits, int32_t T, const moe_route_out* out,
              void* ws, size_t ws_bytes, void* stream);

/* The prefill MoE layer: y [T][H] bf16 = shared(x) + sum_j topk_w * expert(x)
 * for x [T][H] bf16 (both device). Tokens are processed in consecutive chunks
 * of at most chunk_T tokens (chunk_T <= 0: one chunk) reusing one workspace
 * (diariobitcoin.com, "Perplexity libera Lily...", section "Las optimizaciones
 * en el prefill": long prompts run in bounded chunks). logits_out (device
 * [T][E] fp32) receives the router logits when non-null. route_out, when
 * non-null, receives the routing metadata of the LAST chunk (sized for that
 * chunk's token count). Numerics: fp32 router logits; int4 weights expanded
 * on chip as dims->gemm states (exact codes with fp32 scale and bias, or
 * bf16 weights rounded once); fp32 accumulation;
 * the SwiGLU product h is rounded to bf16 before the down projection; each
 * of the k routed down outputs is rounded to bf16 (it enters with a routing
 * weight of about 1/k), the shared expert's stays fp32, and they are summed
 * in fp32 in a fixed order; y is rounded once to bf16. T = 0 is a no-op. */
int moe_prefill_layer(const moe_dims* dims, const moe_layer_weights* w, const uint16_t* x,
                      uint16_t* y, int32_t T, int32_t chunk_T, float* logits_out,
                      const moe_route_out* route_out, void* ws, size_t ws_bytes, void* stream);

/* The same layer for 1 <= T <= 4 tokens (decode), organised as matrix-vector
 * passes over only the selected experts' packed weights (diariobitcoin.com,
 * "Perplexity libera Lily...", section "El decode busca mover menos datos":
 * batch-1 decode is bandwidth bound). logits_out / route_out as above
 * (route_out: topk_idx, topk_w, hist, offsets, perm, inv_perm, block_map and
 * num_blocks are all filled). */
int moe_decode_layer(const moe_dims* dims, const moe_layer_weights* w, const uint16_t* x,
                     uint16_t* y, int32_t T, float* logits_out, const moe_route_out* route_out,
                     void* ws, size_t ws_bytes, void* stream);

/* moe_decode_layer for callers that cannot allocate: code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc. Same
 * arguments and results as moe_decode_layer without the workspace: the
 * decode kernels' scratch (router logits, top-k, SwiGLU rows) lives in a
 * static device array of MOE_NOALLOC_SCRATCH_BYTES bytes inside the library,
 * one copy per GPU, held until the process ends. The call allocates and
 * frees nothing (its first call on a device resolves that device's array
 * address once with hipGetSymbolAddress; make that first call outside graph
 * capture). Nothing in the array needs to start at zero: every call writes
 * what it reads. Calls that overlap on one GPU (several streams, or several
 * host threads) share the array and race: serialise them. Returns
 * MOE_ESCRATCH if the request needs more scratch than the array holds (the
 * supported dims with T <= 4 need at most 299,520 bytes), otherwise the
 * codes of moe_decode_layer (MOE_EHIP also if the array's address cannot be
 * resolved). */
#define MOE_NOALLOC_SCRATCH_BYTES (320 * 1024)
int moe_decode_layer_noalloc(const moe_dims* dims, const moe_layer_weights* w, const uint16_t* x,
                             uint16_t* y, int32_t T, float* logits_out,
                             const moe_route_out* route_out, void* stream);

/* The prefill layer with host-synchronised routing, for measuring what
 * GPU-resident routing saves (diariobitcoin.com, "Perplexity libera Lily...",
 * section "Las optimizaciones en el prefill": keeping histogram, scan,
 * scatter and block map on the GPU, with no CPU round trip, sped prefill
 * up). Same arguments and results as moe_prefill_layer (no logits or
 * metadata outputs), but per chunk the calling thread waits for the routing
 * kernels, reads the work-item count back (4 bytes, device -> host) and
 * launches the grouped GEMMs with grids of exactly one block per work unit
 * instead of the persistent grids. It synchronises the host once per chunk,
 * so it cannot be captured in a graph. */
int moe_prefill_layer_host_routed(const moe_dims* dims, const moe_layer_weights* w,
                                  const uint16_t* x, uint16_t* y, int32_t T, int32_t chunk_T,
                                  void* ws, size_t ws_bytes, void* stream);

/* The prefill layer without fused dequantisation, for measuring what the
 * fusion saves (diariobitcoin.com, "Perplexity libera Lily...", section "Las
 * optimizaciones en el prefill": reconstructing the weights inside the
 * grouped GEMM, never writing them back, sped prefill up). Per chunk, after
 * the routing, every expert with rows and the shared expert are expanded to
 * bf16 w = q*s + b (one rounding) into wbuf (device, caller-owned,
 * moe_unfused_weight_bytes bytes), then the grouped GEMMs read those bf16
 * weights. Same results as moe_prefill_layer up to the bf16 rounding of the
 * weights (no logits or metadata outputs). MOE_EBUFFER if wbuf is too
 * small. */
int moe_unfused_weight_bytes(const moe_dims* dims, size_t* bytes);
int moe_prefill_layer_unfused(const moe_dims* dims, const moe_layer_weights* w, const uint16_t* x,
                              uint16_t* y, int32_t T, int32_t chunk_T, void* wbuf, size_t wbuf_bytes,
                              void* ws, size_t ws_bytes, void* stream);

/* Timing variants for benchmarks: identical to moe_prefill_layer /
 * moe_decode_layer, and in addition record the caller's events (hipEvent_t
 * handles created by the caller) on `stream`: events[i] just before the i-th
 * kernel launch and one more after the last launch, so consecutive events
 * bracket one kernel each. Prefill launches 6 kernels per chunk (router,
 * top-k, scan/scatter, gate/up, down, combine) and needs
 * n_events >= 6 * chunks + 1; decode launches 3 (router, top-k + gate/up,
 * down + combine) and needs n_events >= 4. MOE_EINVAL if too few events. */
int moe_prefill_layer_profiled(const moe_dims* dims, const moe_layer_weights* w,
                               const uint16_t* x, uint16_t* y, int32_t T, int32_t chunk_T,
                               float* logits_out, const moe_route_out* route_out, void* ws,
                               size_t ws_bytes, void* stream, void* const* events,
                               int32_t n_events);
int moe_decode_layer_profiled(const moe_dims* dims, const moe_layer_weights* w, const uint16_t* x,
                              uint16_t* y, int32_t T, float* logits_out,
                              const moe_route_out* route_out, void* ws, size_t ws_bytes,
                              void* stream, void* const* events, int32_t n_events);

/* ---------------------------------------------------------------- around the layer
 *
 * The operators next to the layer in a transformer block: the residual add
 * and RMS norm that make its input, routing rules other than the softmax
 * top-8 of moe_route, and projections of packed int4 weights with low-rank
 * adapters. They follow the conventions at the top of this file. */

/* Element types of moe_add_rmsnorm. */
#define MOE_BF16 0
#define MOE_F16 1
#define MOE_F32 2
/* 8-bit outputs of moe_add_rmsnorm: none, signed integers -127..127, or
 * e4m3 floating point (OCP: no infinities, largest value 448). */
#define MOE_OUT8_NONE 0
#define MOE_OUT8_INT8 1
#define MOE_OUT8_E4M3 2

/* Row length H (1..16384), element type of the rows (x, residual, h, y) and
 * of the weight (the rows' type or MOE_F32), 8-bit output and the number of
 * consecutive values that share one of its scales (group: 0 = the whole row,
 * or 32, 64, 128 or 256, dividing H), eps > 0, and a constant added to every
 * weight (1 for weights stored as their distance from one, else 0). */
typedef struct {
  int32_t H, dtype, weight_dtype, out8, group;
  float eps, weight_offset;
} moe_norm;

/* Residual add and RMS norm of T rows, per row:
 *   h = x + residual, rounded to the rows' type (h = x without a residual)
 *   r = 1 / sqrt(mean(h^2) + eps)
 *   v = h * r * (weight + weight_offset)
 *   y = v, rounded to the rows' type
 *   s = max |v| over a group / 127 (int8) or / 448 (e4m3)
 *   q = v / s, rounded to the nearest 8-bit value (ties to even), limited to
 *       +-127 / +-448; 0 where s = 0
 * with sums and v in fp32 (q is formed from v, not from y). x [T][H] with row
 * stride ldx; residual, h_out, y [T][H] and q [T][H] (one byte a value) with
 * row strides ld_residual, ld_h, ld_y, ld_q, all in elements, from H to 2^20
 * (those of null pointers are not looked at); scales
 * [T][H / group] (one per row for group 0) contiguous. residual, h_out, y may
 * each be null; q and scales are both given with an 8-bit output and both
 * null without; h_out, y or q has to be given. h_out may be x or residual
 * and y may be x, residual or h_out, with the same row stride (each row is
 * read whole before it is written; y over h_out leaves y); any other overlap
 * of an output with another argument is not allowed. Pointers need their
 * element's alignment only; 16-byte aligned rows are faster. A NaN or
 * infinity in a row makes its y NaN or 0 as the formulas do in fp32 and the
 * scales of the groups it reaches NaN or infinite (q: 0, or e4m3's NaN). The
 * sum of squares has fp32's range: rows of values beyond about 1e19 / sqrt(H)
 * overflow to r = 0. T = 0 is a no-op. */
int moe_add_rmsnorm(const moe_norm* norm, const void* x, int64_t ldx, const void* residual,
                    int64_t ld_residual, const void* weight, void* h_out, int64_t ld_h, void* y,
                    int64_t ld_y, void* q, int64_t ld_q, float* scales, int32_t T, void* stream);

/* Scores of a gate. */
#define MOE_SCORE_SOFTMAX 0 /* softmax over the E logits            */
#define MOE_SCORE_SIGMOID 1 /* 1 / (1 + exp(-logit)) of each logit  */
/* How a group of experts is ranked. */
#define MOE_GROUP_MAX 0  /* by its largest key                  */
#define MOE_GROUP_TOP2 1 /* by the sum of its two largest keys  */

/* A routing rule. For one token, over E logits:
 *   score_e = softmax or sigmoid of the logits
 *   key_e   = score_e + balance_bias_e (null: 0)
 *   the n_groups groups of E / n_groups consecutive experts are ranked as
 *   group_score says, and the topk_groups best (ties: the lower group) keep
 *   their experts;
 *   the top_k largest keys among those are selected, larger first, ties to
 *   the lower expert;
 *   weight_j = score_j, divided by the sum over the selected experts if
 *   renorm (0 if that sum is 0), times scale.
 * Ranks are those of the scores and keys evaluated in 64 bits. An expert
 * whose logit is -inf or NaN, or whose key is -inf or NaN, is masked: it
 * ranks after every other, has weight 0, and does not count towards its
 * group's rank (a group of masked experts ranks last). A logit of +inf takes
 * the softmax's mass (shared equally among several). Where masking leaves
 * fewer than top_k experts, the lowest masked ones fill the remaining slots,
 * with weight 0. Supported: E 1..256, top_k 1..16 and <= E, block_m 32 or 16,
 * n_groups 1..64 dividing E, topk_groups 1..n_groups with at least top_k
 * experts in them, scale finite. balance_bias is a device pointer. */
typedef struct {
  int32_t E, top_k, block_m, score, n_groups, topk_groups, group_score, renorm;
  float scale;
  const float* balance_bias; /* [E] fp32, or NULL */
} moe_gate;

/* moe_max_blocks for a gate, and the workspace of moe_route_gated for up to T
 * tokens. */
int64_t moe_gate_max_blocks(const moe_gate* gate, int32_t T);
int moe_gate_workspace_bytes(const moe_gate* gate, int32_t T, size_t* bytes);

/* moe_route with a gate: from fp32 logits [T][E] (device) every field of
 * `out` (k = gate->top_k, E = gate->E, block_m = gate->block_m). T * top_k <
 * 2^30 and T <= 2^28 - 64 (MOE_EUNSUPPORTED otherwise). Results do not depend
 * on the workspace's contents. T = 0 is a no-op. */
int moe_route_gated(const moe_gate* gate, const float* logits, int32_t T, const moe_route_out* out,
                    void* ws, size_t ws_bytes, void* stream);

/* moe_prefill_layer and moe_decode_layer with a gate in the place of the
 * softmax top-8: the same arguments, workspaces (moe_workspace_bytes) and
 * results, with topk_idx and topk_w from the gate. gate->E, top_k and block_m
 * have to be the dims' (MOE_EINVAL otherwise). */
int moe_prefill_layer_gated(const moe_dims* dims, const moe_gate* gate, const moe_layer_weights* w,
                            const uint16_t* x, uint16_t* y, int32_t T, int32_t chunk_T,
                            float* logits_out, const moe_route_out* route_out, void* ws,
                            size_t ws_bytes, void* stream);
int moe_decode_layer_gated(const moe_dims* dims, const moe_gate* gate, const moe_layer_weights* w,
                           const uint16_t* x, uint16_t* y, int32_t T, float* logits_out,
                           const moe_route_out* route_out, void* ws, size_t ws_bytes, void* stream);

/* Low-rank adapters of one projection [N][K]: n adapters with space for R
 * ranks each (R % 8 == 0, 8..128). Adapter a adds
 * scales[a] * B_a (A_a x) with the first ranks[a] rows of A_a and columns of
 * B_a (ranks[a] is limited to 0..R); what lies behind them is not used. A, B
 * 16-byte aligned, ranks and scales 4-byte aligned; all device pointers. */
typedef struct {
  int32_t n, R;
  const uint16_t* A;    /* [n][R][K] bf16                */
  const uint16_t* B;    /* [n][N][R] bf16                */
  const int32_t* ranks; /* [n], or NULL: R for each      */
  const float* scales;  /* [n], or NULL: 1 for each      */
} moe_adapters;

/* Workspace of moe_project for up to T tokens (R: the adapters' R, 0 without
 * adapters). */
int moe_project_workspace_bytes(int32_t N, int32_t K, int32_t R, int32_t T, size_t* bytes);

/* A projection by packed int4 weights beside the adapters of many requests:
 *   y[t] = W x[t] + scales[a] * B_a (A_a x[t]),  a = adapter_of[t]
 * for x [T][K] and y [T][N] bf16 with row strides ldx >= K, ldy >= N
 * (elements, multiples of 8, at most 2^20). blob: a pack_int4_g64 blob
 * (device) of one matrix [N][K] (count 1, not paired); N % 64 == 0, K % 128 == 0, K <= 16384,
 * N <= 65536, T <= 2^30. adapter_of [T] (device, int32) names each token's
 * adapter, in any order; -1, and any other value outside 0..n-1, means none.
 * ad and adapter_of are both given or both null. An adapter's NaN or infinity
 * reaches its own tokens only. gemm is a MOE_GEMM_* value: how W enters the
 * matrix cores, as in moe_dims (EXACT: used exactly, WIDE: rounded once to
 * bf16, AUTO: whichever takes less time for T and N). fp32 accumulation; A_a x
 * is kept to at least 16 significant bits between the two products; y is
 * rounded once.
 * x and y must not overlap. ws 16-byte aligned. T = 0 is a no-op. */
int moe_project(const void* blob, int32_t N, int32_t K, const uint16_t* x, int64_t ldx, uint16_t* y,
                int64_t ldy, int32_t T, const moe_adapters* ad, const int32_t* adapter_of,
                int32_t gemm, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------- the mixer half of a block
 *
 * What stands between moe_add_rmsnorm and the layer in a block: a projection
 * of 8-bit rows, rotary positions, linear attention with a decay for each
 * head, and the norm after a block with its gate, its residual scale and the
 * norm of the next block. They follow the conventions at the top of this
 * file; none has a backward pass (the library trains nothing). */

/* A projection by 8-bit integers with a scale for each token and each output:
 *   y[t][n] = x_scales[t] * w_scales[n] * sum_k x[t][k] w[n][k] + bias[n]
 * for x [T][K] with row stride ldx (bytes, a multiple of 16, from K to 2^20),
 * as moe_add_rmsnorm and moe_gated_norm leave int8 rows with one scale a row
 * (their e4m3 rows and rows with a scale for each group are not read here),
 * and w [N][K] row-major, contiguous; both 16-byte aligned, any value
 * -128..127. x_scales [T], w_scales [N] and bias [N] (or null) fp32. y [T][N]
 * of type dtype (MOE_BF16, MOE_F16 or MOE_F32), aligned to its element, with
 * row stride ldy (elements, from N to 2^20). K % 64 == 0, 64..65536; N
 * 1..2^18; T <= 2^30. Sums are exact (32-bit integers); the scales and the
 * bias are applied in fp32 and the result is rounded once. x and y must not
 * overlap. It needs no workspace: moe_project_int8_workspace_bytes gives 0 for
 * every size, and ws (null or 16-byte aligned) and ws_bytes are reserved, never
 * read or written. T = 0 is a no-op. */
int moe_project_int8_workspace_bytes(int32_t N, int32_t K, int32_t T, size_t* bytes);
int moe_project_int8(const int8_t* w, const float* w_scales, const float* bias, int32_t N, int32_t K,
                     const int8_t* x, int64_t ldx, const float* x_scales, void* y, int64_t ldy,
                     int32_t dtype, int32_t T, void* ws, size_t ws_bytes, void* stream);

/* Frequencies of rotary positions (for any others, such as a YaRN whose ramp
 * runs over the pairs' index between two rounded bounds, as many checkpoints
 * have it, moe_rope_turns takes a model's own radians): pair i of a turned part of rot_dim values
 * turns by radians[i] = base^(-2i / rot_dim) per position, and for long
 * contexts by less (factor >= 1):
 *   MOE_ROPE_LINEAR  radians / factor
 *   MOE_ROPE_NTK     the base times factor^(rot_dim / (rot_dim - 2))
 *   MOE_ROPE_YARN    ("YaRN: Efficient Context Window Extension of Large
 *                    Language Models", Peng et al., section 3) with r the
 *                    turns of a pair over `context` positions and
 *                    c = clamp((r - slow) / (fast - slow), 0, 1):
 *                    radians (c + (1 - c) / factor), and the magnitude
 *                    0.1 ln(factor) + 1 on cosine and sine (else 1)
 * base > 0 and finite; context > 0 and fast > slow for YARN; rot_dim even, 2 to
 * 1024 (more than 2 for NTK). radians [rot_dim / 2] and magnitude on the host. */
#define MOE_ROPE_PLAIN 0
#define MOE_ROPE_LINEAR 1
#define MOE_ROPE_NTK 2
#define MOE_ROPE_YARN 3
typedef struct {
  int32_t kind;
  double base, factor, context, slow, fast;
} moe_rope_scaling;
int moe_rope_radians(const moe_rope_scaling* scaling, int32_t rot_dim, double* radians,
                     float* magnitude);

/* radians[n] per position (at most 2^61 either way) as whole numbers of 2^-64
 * turns, modulo one turn, each the nearest or its neighbour (host -> host): the
 * product of one and a position is exact. */
int moe_rope_turns(const double* radians, int32_t n, uint64_t* turns);

/* Heads of head_dim values (2..1024), whose first rot_dim (even, 2..head_dim)
 * are turned: pairs (i, i + rot_dim / 2), or (2i, 2i + 1) if interleaved;
 * inverse != 0 turns by the opposite angles. magnitude is a factor on cosine
 * and sine (finite). turns: device, [rot_dim / 2], 8-byte aligned. */
typedef struct {
  int32_t head_dim, rot_dim, dtype, interleaved, inverse;
  float magnitude;
  const uint64_t* turns;
} moe_rotary;

/* Rotary positions of T tokens: with f the turns of a pair (a, b) per position
 *   a' = m (a cos(2 pi f p) - b sin(2 pi f p)), b' = m (a sin(..) + b cos(..))
 * p = positions[t] (device, int32, any value). q [T][q_heads][head_dim] and,
 * unless null, k [T][k_heads][head_dim], heads contiguous within rows of
 * strides ldq and ldk (elements, from heads * head_dim to 2^20), aligned to
 * their element; q_out and k_out the same with ldqo and ldko. q_out may be q
 * and k_out k, with the same stride; the values behind rot_dim are copied to
 * another buffer and left alone in place. Any other overlap of an output with
 * another argument is not allowed (q and k may be parts of one row, and so may
 * the outputs). 1..1024 heads each. However far the position, an angle modulo
 * one turn is off by less than 1.4 * 2^-32 turns (what 2^31 positions make of a
 * frequency's rounding, and the lower 32 bits, which are dropped); from there on
 * cosine and sine are formed in fp32 and err by at most 4 * 2^-24 more. Sums in
 * fp32, one rounding. T <= 2^30; T = 0 is a no-op. */
int moe_rope(const moe_rotary* rope, const void* q, int64_t ldq, void* q_out, int64_t ldqo,
             int32_t q_heads, const void* k, int64_t ldk, void* k_out, int64_t ldko,
             int32_t k_heads, const int32_t* positions, int32_t T, void* stream);

/* Linear attention: v_heads states of [qk_dim][v_dim], v_heads a multiple of
 * qk_heads (1..1024), qk_dim and v_dim multiples of 8, 8..256. Value head h
 * uses the queries and keys of head h / (v_heads / qk_heads). scale finite. */
typedef struct {
  int32_t qk_heads, v_heads, qk_dim, v_dim;
  float scale;
} moe_linear;

/* Linear attention over sequences, per value head:
 *   S_t = exp(g_t) S_(t-1) + k_t v_t^T,   o_t = scale * q_t S_t
 * q, k [T][qk_heads][qk_dim], v, o [T][v_heads][v_dim] bf16, 16-byte aligned,
 * heads contiguous within rows of strides ldq, ldk, ldv, ldo (elements,
 * multiples of 8, at most 2^20). g = log_decay, fp32: [T][v_heads] with row
 * stride ld_decay (v_heads..2^20), or [v_heads] for all tokens with ld_decay
 * 0. A g of -inf forgets everything finite before the token (a NaN or infinity
 * in a state stays, as its product with 0); where g is above 0, exp of its sum
 * over a sequence has to be finite.
 * Sequence i holds the tokens cu_seqlens[i] .. cu_seqlens[i + 1] - 1
 * (device, int32 [n_seqs + 1], not decreasing, from 0; values are limited to
 * 0..T); rows of o behind the last are left as they were. Its state starts as
 * state_in[slots_in[i]] and ends as state_out[slots_out[i]]: fp32
 * [n][v_heads][qk_dim][v_dim], 16-byte aligned, n = n_in and n_out. Null
 * slots stand for i; a slot outside 0..n-1 (-1) starts from zeros or is not
 * kept, and so is every one of a null state. An empty sequence's state is
 * copied (a zero may lose its sign). state_in may be state_out; a slot that
 * one sequence writes must not be read or written by another (any number may
 * read the same one).
 * n_seqs <= 65536, T <= 2^30. States, sums and decays are fp32 or more; the
 * state's update keeps 24 significant bits of v's decayed rows, and for o the
 * state and the decayed products of q and k are rounded to bf16 as operands
 * of the matrix cores (o's own type). How a sequence is cut, and so the last
 * bits of its o and state, depends on the call: on T, and on whether a
 * sequence of up to 8 tokens is one of 8 or more (then o's operands are not
 * rounded, as in moe_linear_attention_step); one call gives the same bits
 * each time. |v| is below 2^120. A NaN or infinity in a token's row reaches
 * that token's o and, from k, v or g, the later ones of its sequence and its
 * state (as NaN or infinity; from v in its own column only), nothing else. ws
 * 16-byte aligned, of moe_linear_workspace_bytes (null where that is 0); its
 * contents do not matter, and a workspace for T tokens and n_seqs serves fewer.
 * o must not overlap any input. n_seqs = 0 is a no-op. */
int moe_linear_workspace_bytes(const moe_linear* linear, int32_t n_seqs, int32_t T, size_t* bytes);
int moe_linear_attention(const moe_linear* linear, const uint16_t* q, int64_t ldq, const uint16_t* k,
                         int64_t ldk, const uint16_t* v, int64_t ldv, const float* log_decay,
                         int64_t ld_decay, const int32_t* cu_seqlens, int32_t n_seqs,
                         const float* state_in, const int32_t* slots_in, int32_t n_in,
                         float* state_out, const int32_t* slots_out, int32_t n_out, uint16_t* o,
                         int64_t ldo, int32_t T, void* ws, size_t ws_bytes, void* stream);

/* The same for T sequences of one token each (decode): token t is sequence t.
 * No operand is rounded on the way to o. T <= 65536; T = 0 is a no-op. */
int moe_linear_attention_step(const moe_linear* linear, const uint16_t* q, int64_t ldq,
                              const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                              const float* log_decay, int64_t ld_decay, const float* state_in,
                              const int32_t* slots_in, int32_t n_in, float* state_out,
                              const int32_t* slots_out, int32_t n_out, uint16_t* o, int64_t ldo,
                              int32_t T, void* stream);

/* Gates of moe_gated_norm: none, z / (1 + exp(-z)), 1 / (1 + exp(-z)). */
#define MOE_GATE_NONE 0
#define MOE_GATE_SILU 1
#define MOE_GATE_SIGMOID 2

/* Rows of H values (1..16384) of type dtype; the type of weight, next_weight
 * and channel_scale (the rows' or MOE_F32). normalize: whether the first norm
 * is taken, over `group` consecutive values (0: the row, or 32, 64, 128 or
 * 256, dividing H). gate: a MOE_GATE_*; gate_per_row: one gate value a row
 * instead of H. next: whether the second norm is taken. out8 and out8_group as
 * out8 and group of moe_norm. eps and next_eps at least 2^-126, all others
 * finite. */
typedef struct {
  int32_t H, dtype, weight_dtype, normalize, group, gate, gate_per_row, next, out8, out8_group;
  float eps, weight_offset, scale, next_eps, next_offset;
} moe_block_norm;

/* The norm after a block (or of its heads) with its gate, the residual add
 * with a scale, and the norm before the next block, per row of T:
 *   u = x / sqrt(mean_group(x^2) + eps) * (weight + weight_offset)   normalize
 *   v = scale * channel_scale * u * act(gate) + residual
 *   h = v, rounded to the rows' type
 *   v = v / sqrt(mean_row(v^2) + next_eps) * (next_weight + next_offset)  next
 *   y = v, rounded to the rows' type
 *   q, scales: v in 8 bits, as moe_add_rmsnorm forms them
 * in fp32, each output rounded once (the second norm takes the sum before it
 * is rounded to h). x, residual, gate [T][H] ([T] for gate_per_row), h_out, y
 * and q with row strides ldx, ld_residual, ld_gate (from 1 for gate_per_row),
 * ld_h, ld_y, ld_q in elements, up to 2^20. weight [group] ([H] for group 0)
 * or null (the first norm without a weight; always null without a norm),
 * channel_scale [H] or null, next_weight [H] with next. gate is given unless
 * MOE_GATE_NONE. residual may be null, and so may h_out and y (y only with
 * next); q and scales are both given with an 8-bit output; one output at least.
 * h_out and y may each be x, residual or a gate [T][H], with the same row
 * stride (each row is read whole before it is written; y over h_out leaves
 * y); any other overlap of an output with another argument is not allowed.
 * Pointers need their element's alignment only. T = 0 is a no-op. */
int moe_gated_norm(const moe_block_norm* norm, const void* x, int64_t ldx, const void* weight,
                   const void* gate, int64_t ld_gate, const void* channel_scale,
                   const void* residual, int64_t ld_residual, const void* next_weight, void* h_out,
                   int64_t ld_h, void* y, int64_t ld_y, void* q, int64_t ld_q, float* scales,
                   int32_t T, void* stream);

/* Static description of an error code. */
const char* moe_strerror(int code);

/* Test hook: expand expert `expert` of a pack_int4_g64 blob (device) on the
 * GPU with the same load-and-convert code the GEMM kernels use, writing fp32
 * w[n][c] = q*scale + bias to out (device) as [N][K] (paired: [2][N][K], gate
 * then up). */
int moe_test_dequant(const void* blob, int32_t count, int32_t N, int32_t K, int32_t paired,
                     int32_t expert, float* out, void* stream);

/* Measurement helpers, not part of the layer: achievable ceilings of the
 * device, for roofline fractions against measured as well as published peaks.
 *
 * moe_ceiling_read enqueues one streaming read of `bytes` (a multiple of 16,
 * >= 16) of device memory at `buf` by 2048 blocks of 256 threads, each block
 * one contiguous 1/2048 of the buffer (16-byte vector loads, eight in flight
 * per thread). `sink` (device, 4 bytes) is
 * written only if the XOR of a thread's data equals a fixed constant, which
 * keeps the loads live; callers ignore its value. Time it with events; for
 * HBM bandwidth use a buffer much larger than the 256 MB last-level cache.
 *
 * moe_ceiling_mfma enqueues 1024 blocks of four waves, each wave running
 * eight independent chains of 4 * `iters` (iters > 0) 16x16x32 bf16
 * matrix-core operations on register operands, and stores the flop count of
 * the launch in *flops (host). `random` nonzero: the operands are random bf16
 * values (magnitude in [0.5, 1), random sign) that change from one operation
 * to the next, as layer data does; zero: nearly constant operands. The
 * device sustains a lower clock on the first. `clocks` (device, may be null):
 * 2048 unsigned 64-bit values that receive, per block, the real-time ticks
 * (100 MHz) and the shader-clock ticks over its loop; their sums give the
 * clock the launch ran at. `sink` as above.
 *
 * Both return MOE_EINVAL for null pointers or bad sizes, MOE_EHIP if the
 * launch fails; they allocate nothing and do not synchronise. */
int moe_ceiling_read(const void* buf, size_t bytes, uint32_t* sink, void* stream);
int moe_ceiling_mfma(int32_t iters, int32_t random, float* sink, unsigned long long* clocks,
                     double* flops, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_INT4_H */
