// Internal kernel interfaces of the int4 MoE library (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "device.h"
#include "layout.h"

namespace moe {

constexpr int kChunkPairs = 1024;  // (token, slot) pairs per scatter block
constexpr int kItemRows = 32;      // most rows of one expert per GEMM work item (one routing block)
constexpr int kWideRows = 144;     // rows per work item of the wide GEMMs
constexpr int kMaxGroups = 64;     // K / 64 upper bound of the expert GEMMs
constexpr int kDecodeMaxT = 4;
constexpr int kMaxSplits = 8;      // router K splits summed by the top-k kernel

struct TopkArgs {
  const float* partial;   // [splits][T][E]
  int splits;
  const float* rbias;     // [E] or null
  float* logits_out;      // [T][E] or null
  int32_t* topk_idx;      // [T][k]
  float* topk_w;          // [T][k]
  int32_t* chunk_hist;    // [chunks][E] (zeroed beforehand) or null
  int T, E, k;
};

struct ScatterArgs {
  const int32_t* topk_idx;
  const int32_t* chunk_hist;
  int32_t *hist, *offsets, *perm, *inv_perm, *block_map, *num_blocks;
  int32_t *items, *num_items;  // GEMM work list or null
  int T, E, k, block_m;
  int item_rows;               // rows per GEMM work item
  int longest_first;           // 1: the work list holds every expert's full items
                               // (expert order), then the experts' last partial
                               // items, larger first (ties: lower expert)
};

// Which GEMM: gate/up with SwiGLU, or down (routed and shared items) writing
// per-(token, slot) fp32 rows that the combine kernel sums into y.
enum GemmMode { kGateUp = 0, kDown = 1 };

struct GemmArgs {
  const int32_t* items;      // routed work list [max][3] (expert, first row, rows)
  const int32_t* num_items;  // device scalar
  int shared_slots;          // shared-expert items (item_rows tokens each)
  int item_rows;             // rows per work item, <= kItemRows (the routing block size)
  const uint8_t* blob;       // routed experts (past the header)
  const uint8_t* shared_blob;
  int64_t expert_bytes;
  int N, K, paired;          // packed geometry of this matrix set
  int bf16_weights;          // 1: blob / shared_blob hold bf16-expanded weights (no header)
  int T;                     // tokens in this chunk
  int k;                     // experts per token
  // activations
  const uint16_t* act;       // gate/up: x [T][K]; down: h [(k+1)T][K]
  const int32_t* perm;       // [kT]
  // outputs
  uint16_t* h_out;           // gate/up: h [(k+1)T][N] bf16
  uint16_t* partial_r;       // down, routed rows: [T*k][N] bf16 at pair p = t*k + j
  float* partial_s;          // down, shared-expert rows: [T][N] fp32
  int cus;                   // wide GEMMs: compute units (set by the launcher)
};

// Compute units of the current device, rounded down to a multiple of 8 (the
// XCD count); cached per device.
int compute_units();

hipError_t launch_router(const uint16_t* x, const uint16_t* planes, float* partial, int T, int H,
                         int E, int splits, int* zero_buf, int zero_count, hipStream_t s);
hipError_t launch_topk(const TopkArgs& a, hipStream_t s);
hipError_t launch_scan_scatter(const ScatterArgs& a, hipStream_t s);
hipError_t launch_fill_zero(int* p, int n, hipStream_t s);
// grid_blocks > 0: that many blocks (rounded up to a multiple of 8) instead
// of the persistent grid (used when the host knows the exact unit count).
hipError_t launch_gemm(GemmMode mode, const GemmArgs& a, hipStream_t s, int grid_blocks = 0);
// The wide GEMMs (items of up to kWideRows rows, weights expanded to bf16
// once per item): a.items / a.num_items hold kWideRows-row items and
// a.shared_slots counts kWideRows-token shared items; max_slots bounds
// items + shared items (the grid is sized from it, extra blocks exit).
hipError_t launch_gemm_wide(GemmMode mode, const GemmArgs& a, int max_slots, hipStream_t s);
// y[t][n] = bf16(shared[t][n] + sum_{j<k} topk_w[t][j] * routed[t*k + j][n]) (j ascending).
hipError_t launch_combine(const uint16_t* routed, const float* shared, const float* topk_w, uint16_t* y,
                          int T, int N, int k, hipStream_t s);
// The unfused comparison path: every expert of a packed blob with rows (hist
// null or hist[e] > 0), and the shared expert, expanded to bf16 w = q s + b
// (one rounding) into `out` / `out_shared` in the kBf16GroupBytes layout.
hipError_t launch_expand_bf16(const uint8_t* blob, int64_t expert_bytes, const uint8_t* shared_blob,
                              int count, const int32_t* hist, int N, int K, int paired, uint8_t* out,
                              uint8_t* out_shared, hipStream_t s);
hipError_t launch_test_dequant(const uint8_t* expert_base, int N, int K, int paired, float* out,
                               hipStream_t s);

struct DecodeArgs {
  const uint16_t* x;          // [T][H]
  const float* router_w;      // [E][H]
  const float* rbias;         // [E] or null
  float* logits;              // [T][E]
  float* logits_out;          // [T][E] or null
  int32_t* topk_idx;          // [T][k]
  float* topk_w;              // [T][k]
  int32_t *hist, *offsets, *perm, *inv_perm, *block_map, *num_blocks;  // optional route_out
  const uint8_t* gu_blob;     // routed gate/up experts (past header)
  const uint8_t* gu_shared;
  int64_t gu_expert_bytes;
  const uint8_t* dn_blob;
  const uint8_t* dn_shared;
  int64_t dn_expert_bytes;
  uint16_t* h;                // [k*T + T][I] bf16 (slot order: pairs, then shared)
  uint16_t* y;                // [T][H]
  int T, H, I, E, k, block_m;
};

// ---- around the layer

constexpr int kNormBf16 = 0, kNormF16 = 1, kNormF32 = 2;  // MOE_BF16, MOE_F16, MOE_F32
constexpr int kOut8None = 0, kOut8Int8 = 1, kOut8E4m3 = 2;
constexpr int kNormMaxH = 16384;

struct NormArgs {
  const void *x, *residual, *weight;  // residual: or null
  void *h_out, *y, *q;                // each or null
  float* scales;
  int64_t ldx, ld_residual, ld_h, ld_y, ld_q;
  int T, H, dtype, weight_f32, out8, group;
  float eps, weight_offset;
};
hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s);

constexpr int kMaxGateK = 16;       // experts per token of a gate
constexpr int kMaxGateGroups = 64;

struct GateArgs {
  const float* partial;   // [splits][T][E]
  int splits;
  const float* rbias;     // [E] or null: added to the logits
  float* logits_out;      // [T][E] or null
  const float* balance;   // [E] or null: added to the scores for selection
  int32_t* topk_idx;      // [T][k]
  float* topk_w;          // [T][k]
  int32_t* chunk_hist;    // [chunks][E] (zeroed beforehand) or null
  uint8_t* counts;        // gate_counts_bytes (launch_gate_route)
  int T, E, k, sigmoid, n_groups, topk_groups, group_top2, renorm;
  float scale;
  // set by the launchers
  int group_size, group_lanes_log2, vectors;
  uint32_t group_magic;
};
// topk_idx, topk_w and chunk_hist.
hipError_t launch_gate_topk(const GateArgs& a, hipStream_t s);

struct GateScatter {
  const int32_t* topk_idx;
  const uint8_t* counts;
  int32_t *hist, *offsets, *perm, *inv_perm, *block_map, *num_blocks;
  int T, E, k, block_m;
  int count_tokens, pieces;  // tokens per row of counts, pieces per block; set by the launcher
};
// Everything moe_route gives, in one launch for few tokens, two otherwise.
size_t gate_counts_bytes(int T);
hipError_t launch_gate_route(const GateArgs& a, const GateScatter& sc, hipStream_t s);

constexpr int kMaxRank = 128;

struct ProjectArgs {
  const uint8_t* blob;       // one matrix [N][K] (past the header)
  const uint16_t* x;         // [T], row stride ldx
  uint16_t* y;               // [T], row stride ldy
  const int32_t* adapter_of; // [T] or null: no adapters
  const uint16_t *A, *B;     // [n][R][K], [n][N][R]
  const int32_t* ranks;      // [n] or null
  const float* scales;       // [n] or null
  void* ws;                  // project_ws_bytes
  int64_t ldx, ldy;
  int N, K, T, n, R, gemm;
};
size_t project_ws_bytes(int N, int K, int R, int T);
hipError_t launch_project(const ProjectArgs& a, hipStream_t s);

// ---- the mixer half of a block

constexpr int kInt8MaxK = 65536, kInt8MaxN = 1 << 18;

struct Int8Args {
  const int8_t *w, *x;       // [N][K], [T] with row stride ldx
  const float *w_scales, *x_scales, *bias;  // [N], [T], [N] or null
  void* y;                   // [T], row stride ldy
  int64_t ldx, ldy;
  int N, K, T, dtype;
  int wide;                  // rows of y are 16-byte aligned; set by the launcher
};
hipError_t launch_project_int8(const Int8Args& a, hipStream_t s);

struct RopeArgs {
  const void* x[2];          // queries, keys: [T][heads][D], row stride ldx
  void* y[2];
  const int32_t* positions;  // [T]
  const uint64_t* turns;     // [rot / 2]
  int64_t ldx[2], ldy[2];
  int heads[2], copy[2];     // copy: the values behind the turned part go to another buffer
  int T, D, rot, dtype, interleaved;
  uint32_t flip;             // sign bit of the sine's factor
  float magnitude;
  // set by the launcher
  uint32_t items, per_token, per_token_magic, units, units_magic;
  int turn_units;
};
hipError_t launch_rope(const RopeArgs& a, hipStream_t s);

constexpr int kLinearMaxDim = 256;

struct LinearArgs {
  const uint16_t *q, *k, *v;  // [T][heads][dim], row strides ldq, ldk, ldv
  const float* decay;         // [v_heads], or [T] with row stride ld_decay
  const int32_t* cu_seqlens;  // [n_seqs + 1], or null: a token a sequence
  const float* state_in;      // [n_in][v_heads][qk_dim][v_dim] or null
  float* state_out;           // [n_out][v_heads][qk_dim][v_dim] or null
  const int32_t *slots_in, *slots_out;  // [n_seqs], or null: the sequence's index
  uint16_t* o;                // [T][v_heads][v_dim], row stride ldo
  void* ws;                   // linear_ws_bytes
  int64_t ldq, ldk, ldv, ldo, ld_decay;
  int n_seqs, n_in, n_out, T, qk_heads, v_heads, qk_dim, v_dim;
  float scale;
  // set by the launcher: tokens of a window, how many windows, and over how many
  // blocks the sequences of a single one are spread; whether the states that
  // sequences over several windows start from are copied
  int window, windows, strands, copied;
  int short_tokens;  // sequences of at most so many tokens are walked through
};
size_t linear_ws_bytes(const LinearArgs& a);
hipError_t launch_linear_attention(const LinearArgs& a, hipStream_t s);
hipError_t launch_linear_step(const LinearArgs& a, hipStream_t s);

constexpr int kGateNone = 0, kGateSilu = 1, kGateSigmoid = 2;

struct GatedArgs {
  const void *x, *weight, *gate, *channel, *residual, *next_weight;  // all but x: or null
  void *h_out, *y, *q;
  float* scales;
  int64_t ldx, ld_gate, ld_residual, ld_h, ld_y, ld_q;
  int T, H, dtype, weight_f32, normalize, group, gate_kind, gate_per_row, next, out8, out8_group;
  float eps, weight_offset, scale, next_eps, next_offset;
};
hipError_t launch_gated_norm(const GatedArgs& a, hipStream_t s);

// ev (optional): four events recorded before each of the three launches and after the last.
// gate (optional): a routing rule in the place of the softmax top-k (its sizes
// are a's; no events then). Requires k == 8.
hipError_t launch_decode(const DecodeArgs& a, hipStream_t s, hipEvent_t* ev = nullptr,
                         const GateArgs* gate = nullptr);

}  // namespace moe
