// C ABI of the operators of a block's mixer half: argument checks and the
// launches on the caller's stream (include/moe_int4.h).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include "../../include/moe_int4.h"
#include "checks.h"
#include "kernels.h"

using namespace moe;

namespace {

constexpr int32_t kMaxTokens = 1 << 30;  // token indices and their tiles stay 32-bit
constexpr int32_t kMaxSeqs = 65536;
constexpr int32_t kMaxHeads = 1024;
constexpr int32_t kMaxRopeDim = 1024;

constexpr double kMaxRadians = 0x1p61;

// r / (2 pi) modulo 1, in steps of 2^-64 to the nearest (but for the 2^-67 turns
// that 128 bits of 1 / (2 pi) leave at the largest r): the whole number m of
// r = m 2^e times those bits, of which the bits that weigh 2^-64 to 2^-1 remain.
uint64_t turns_of(double r) {
  constexpr uint64_t kHigh = 0x28be60db9391054a, kLow = 0x7f09d5f47d4d3770;  // 2^128 / (2 pi)
  int e;
  const uint64_t m = (uint64_t)std::ldexp(std::frexp(std::fabs(r), &e), 53);
  const int drop = 64 - (e - 53);  // 55 or more, as r is at most 2^61
  const unsigned __int128 low = (unsigned __int128)m * kLow, high = (unsigned __int128)m * kHigh + (uint64_t)(low >> 64);
  const uint64_t bottom = (uint64_t)low;  // the product is high 2^64 + bottom
  uint64_t u = 0;
  if (drop < 64)
    u = (uint64_t)(high << (64 - drop)) + (bottom >> drop) + (bottom >> (drop - 1) & 1);
  else if (drop == 64)
    u = (uint64_t)high + (bottom >> 63);
  else if (drop < 192)
    u = (uint64_t)(high >> (drop - 64)) + (uint64_t)(high >> (drop - 65) & 1);
  return r < 0 ? 0 - u : u;
}

bool type_ok(int t) { return t >= MOE_BF16 && t <= MOE_F32; }
int type_bytes(int t) { return t == MOE_F32 ? 4 : 2; }
bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool stride_ok(int64_t ld, int64_t least) { return ld >= least && ld <= kMaxRowStride; }
bool group_ok(int group, int H) {
  return group == 0 || ((group == 32 || group == 64 || group == 128 || group == 256) && H % group == 0);
}

int check_int8(int N, int K, int T) {
  if (T < 0) return MOE_EINVAL;
  return N >= 1 && N <= kInt8MaxN && K >= 64 && K <= kInt8MaxK && K % 64 == 0 && T <= kMaxTokens ? MOE_OK
                                                                                              : MOE_EUNSUPPORTED;
}

int check_linear(const moe_linear* l) {
  if (!l || !std::isfinite(l->scale)) return MOE_EINVAL;
  const auto dim = [](int d) { return d >= 8 && d <= kLinearMaxDim && d % 8 == 0; };
  return l->qk_heads >= 1 && l->v_heads >= 1 && l->v_heads <= kMaxHeads && l->v_heads % l->qk_heads == 0 &&
                 dim(l->qk_dim) && dim(l->v_dim)
             ? MOE_OK
             : MOE_EUNSUPPORTED;
}

LinearArgs linear_args(const moe_linear* l, int n_seqs, int T) {
  LinearArgs a{};
  a.qk_heads = l->qk_heads;
  a.v_heads = l->v_heads;
  a.qk_dim = l->qk_dim;
  a.v_dim = l->v_dim;
  a.scale = l->scale;
  a.n_seqs = n_seqs;
  a.T = T;
  return a;
}

// The arguments that both forms of linear attention take.
int linear_rows(const moe_linear* l, LinearArgs& a, const uint16_t* q, int64_t ldq, const uint16_t* k, int64_t ldk,
                const uint16_t* v, int64_t ldv, const float* log_decay, int64_t ld_decay, const float* state_in,
                const int32_t* slots_in, int32_t n_in, float* state_out, const int32_t* slots_out, int32_t n_out,
                uint16_t* o, int64_t ldo) {
  if ((state_in && n_in < 1) || (state_out && n_out < 1) || (slots_in && !state_in) || (slots_out && !state_out) ||
      !al16(state_in) || !al16(state_out) || !al4(slots_in) || !al4(slots_out))
    return MOE_EINVAL;
  if (a.T) {  // (no token: no row is read or written)
    const int64_t qk = (int64_t)l->qk_heads * l->qk_dim, vo = (int64_t)l->v_heads * l->v_dim;
    const void* rows[] = {q, k, v, o};
    const int64_t lds[] = {ldq, ldk, ldv, ldo}, least[] = {qk, qk, vo, vo};
    for (int i = 0; i < 4; ++i)
      if (!rows[i] || !al16(rows[i]) || lds[i] % 8 || !stride_ok(lds[i], least[i])) return MOE_EINVAL;
    if (!log_decay || !al4(log_decay) || (ld_decay != 0 && !stride_ok(ld_decay, l->v_heads))) return MOE_EINVAL;
  }
  a.q = q;
  a.k = k;
  a.v = v;
  a.o = o;
  a.decay = log_decay;
  a.ldq = ldq;
  a.ldk = ldk;
  a.ldv = ldv;
  a.ldo = ldo;
  a.ld_decay = ld_decay;
  a.state_in = state_in;
  a.slots_in = slots_in;
  a.n_in = n_in;
  a.state_out = state_out;
  a.slots_out = slots_out;
  a.n_out = n_out;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_project_int8_workspace_bytes(int32_t N, int32_t K, int32_t T, size_t* bytes) {
  if (!bytes) return MOE_EINVAL;
  const int rc = check_int8(N, K, T);
  if (rc == MOE_OK) *bytes = 0;  // (each of the kernels joins its parts within a block)
  return rc;
}

int moe_project_int8(const int8_t* w, const float* w_scales, const float* bias, int32_t N, int32_t K,
                     const int8_t* x, int64_t ldx, const float* x_scales, void* y, int64_t ldy,
                     int32_t dtype, int32_t T, void* ws, size_t /*ws_bytes*/, void* stream) {
  if (!type_ok(dtype)) return MOE_EINVAL;
  const int rc = check_int8(N, K, T);
  if (rc != MOE_OK || T == 0) return rc;
  if (!w || !w_scales || !x || !x_scales || !y || !al16(w) || !al16(x) || !al4(w_scales) || !al4(x_scales) ||
      !al4(bias) || !aligned(y, type_bytes(dtype)) || ldx % 16 || !stride_ok(ldx, K) || !stride_ok(ldy, N) ||
      !al16(ws))
    return MOE_EINVAL;
  Int8Args a{};
  a.w = w;
  a.x = x;
  a.w_scales = w_scales;
  a.x_scales = x_scales;
  a.bias = bias;
  a.y = y;
  a.ldx = ldx;
  a.ldy = ldy;
  a.N = N;
  a.K = K;
  a.T = T;
  a.dtype = dtype;
  return hip_status(launch_project_int8(a, static_cast<hipStream_t>(stream)));
}

int moe_rope_radians(const moe_rope_scaling* s, int32_t rot_dim, double* radians, float* magnitude) {
  if (!s || !radians || !magnitude || s->kind < MOE_ROPE_PLAIN || s->kind > MOE_ROPE_YARN ||
      !std::isfinite(s->base) || s->base <= 0)
    return MOE_EINVAL;
  if (rot_dim < 2 || rot_dim > kMaxRopeDim || rot_dim % 2 || (s->kind == MOE_ROPE_NTK && rot_dim == 2))
    return MOE_EUNSUPPORTED;
  if (s->kind != MOE_ROPE_PLAIN && (!std::isfinite(s->factor) || s->factor < 1)) return MOE_EINVAL;
  if (s->kind == MOE_ROPE_YARN && (!std::isfinite(s->context) || s->context <= 0 || !std::isfinite(s->slow) ||
                                   !std::isfinite(s->fast) || s->fast <= s->slow))
    return MOE_EINVAL;
  const double base = s->kind == MOE_ROPE_NTK ? s->base * std::pow(s->factor, rot_dim / (rot_dim - 2.0)) : s->base;
  for (int i = 0; i < rot_dim / 2; ++i) {
    double r = std::pow(base, -2.0 * i / rot_dim);
    if (s->kind == MOE_ROPE_LINEAR) r /= s->factor;
    if (s->kind == MOE_ROPE_YARN) {
      const double turns = s->context * r / 6.283185307179586476925;
      const double kept = std::min(1.0, std::max(0.0, (turns - s->slow) / (s->fast - s->slow)));
      r *= kept + (1 - kept) / s->factor;
    }
    radians[i] = r;
  }
  *magnitude = s->kind == MOE_ROPE_YARN ? (float)(0.1 * std::log(s->factor) + 1) : 1.f;
  return MOE_OK;
}

int moe_rope_turns(const double* radians, int32_t n, uint64_t* turns) {
  if (!radians || !turns || n < 0) return MOE_EINVAL;
  for (int i = 0; i < n; ++i)
    if (!std::isfinite(radians[i])) return MOE_EINVAL;
  for (int i = 0; i < n; ++i)
    if (std::fabs(radians[i]) > kMaxRadians) return MOE_EUNSUPPORTED;
  for (int i = 0; i < n; ++i) turns[i] = turns_of(radians[i]);
  return MOE_OK;
}

int moe_rope(const moe_rotary* r, const void* q, int64_t ldq, void* q_out, int64_t ldqo,
             int32_t q_heads, const void* k, int64_t ldk, void* k_out, int64_t ldko,
             int32_t k_heads, const int32_t* positions, int32_t T, void* stream) {
  if (!r || T < 0 || !type_ok(r->dtype) || (r->interleaved != 0 && r->interleaved != 1) ||
      (r->inverse != 0 && r->inverse != 1) || !std::isfinite(r->magnitude))
    return MOE_EINVAL;
  if (r->head_dim < 2 || r->head_dim > kMaxRopeDim || r->rot_dim < 2 || r->rot_dim > r->head_dim || r->rot_dim % 2 ||
      q_heads < 1 || q_heads > kMaxHeads || (k && (k_heads < 1 || k_heads > kMaxHeads)) || T > kMaxTokens)
    return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  const int eb = type_bytes(r->dtype);
  if (!q || !q_out || (k != nullptr) != (k_out != nullptr) || !positions || !al4(positions) || !r->turns ||
      !aligned(r->turns, 8))
    return MOE_EINVAL;
  const int64_t wq = (int64_t)q_heads * r->head_dim, wk = (int64_t)k_heads * r->head_dim;
  if (!aligned(q, eb) || !aligned(q_out, eb) || !stride_ok(ldq, wq) || !stride_ok(ldqo, wq) || (q == q_out && ldq != ldqo))
    return MOE_EINVAL;
  if (k && (!aligned(k, eb) || !aligned(k_out, eb) || !stride_ok(ldk, wk) || !stride_ok(ldko, wk) ||
            (k == k_out && ldk != ldko)))
    return MOE_EINVAL;
  RopeArgs a{};
  a.x[0] = q;
  a.y[0] = q_out;
  a.ldx[0] = ldq;
  a.ldy[0] = ldqo;
  a.heads[0] = q_heads;
  a.copy[0] = q != q_out;
  if (k) {
    a.x[1] = k;
    a.y[1] = k_out;
    a.ldx[1] = ldk;
    a.ldy[1] = ldko;
    a.heads[1] = k_heads;
    a.copy[1] = k != k_out;
  }
  a.positions = positions;
  a.turns = r->turns;
  a.T = T;
  a.D = r->head_dim;
  a.rot = r->rot_dim;
  a.dtype = r->dtype;
  a.interleaved = r->interleaved;
  a.flip = r->inverse ? 0x80000000u : 0u;
  a.magnitude = r->magnitude;
  return hip_status(launch_rope(a, static_cast<hipStream_t>(stream)));
}

int moe_linear_workspace_bytes(const moe_linear* l, int32_t n_seqs, int32_t T, size_t* bytes) {
  const int rc = check_linear(l);
  if (rc != MOE_OK) return rc;
  if (!bytes || n_seqs < 0 || T < 0) return MOE_EINVAL;
  if (n_seqs > kMaxSeqs || T > kMaxTokens) return MOE_EUNSUPPORTED;
  *bytes = linear_ws_bytes(linear_args(l, n_seqs, T));
  return MOE_OK;
}

int moe_linear_attention(const moe_linear* l, const uint16_t* q, int64_t ldq, const uint16_t* k,
                         int64_t ldk, const uint16_t* v, int64_t ldv, const float* log_decay,
                         int64_t ld_decay, const int32_t* cu_seqlens, int32_t n_seqs,
                         const float* state_in, const int32_t* slots_in, int32_t n_in,
                         float* state_out, const int32_t* slots_out, int32_t n_out, uint16_t* o,
                         int64_t ldo, int32_t T, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_linear(l);
  if (rc != MOE_OK) return rc;
  if (n_seqs < 0 || T < 0) return MOE_EINVAL;
  if (n_seqs > kMaxSeqs || T > kMaxTokens) return MOE_EUNSUPPORTED;
  if (n_seqs == 0) return MOE_OK;
  LinearArgs a = linear_args(l, n_seqs, T);
  rc = linear_rows(l, a, q, ldq, k, ldk, v, ldv, log_decay, ld_decay, state_in, slots_in, n_in, state_out, slots_out,
                   n_out, o, ldo);
  if (rc != MOE_OK) return rc;
  const size_t need = linear_ws_bytes(a);
  if (!cu_seqlens || !al4(cu_seqlens) || (need && !ws) || !al16(ws)) return MOE_EINVAL;
  if (ws_bytes < need) return MOE_EWORKSPACE;
  a.cu_seqlens = cu_seqlens;
  a.ws = ws;
  return hip_status(launch_linear_attention(a, static_cast<hipStream_t>(stream)));
}

int moe_linear_attention_step(const moe_linear* l, const uint16_t* q, int64_t ldq,
                              const uint16_t* k, int64_t ldk, const uint16_t* v, int64_t ldv,
                              const float* log_decay, int64_t ld_decay, const float* state_in,
                              const int32_t* slots_in, int32_t n_in, float* state_out,
                              const int32_t* slots_out, int32_t n_out, uint16_t* o, int64_t ldo,
                              int32_t T, void* stream) {
  int rc = check_linear(l);
  if (rc != MOE_OK) return rc;
  if (T < 0) return MOE_EINVAL;
  if (T > kMaxSeqs) return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  LinearArgs a = linear_args(l, T, T);
  rc = linear_rows(l, a, q, ldq, k, ldk, v, ldv, log_decay, ld_decay, state_in, slots_in, n_in, state_out, slots_out,
                   n_out, o, ldo);
  if (rc != MOE_OK) return rc;
  return hip_status(launch_linear_step(a, static_cast<hipStream_t>(stream)));
}

int moe_gated_norm(const moe_block_norm* n, const void* x, int64_t ldx, const void* weight,
                   const void* gate, int64_t ld_gate, const void* channel_scale,
                   const void* residual, int64_t ld_residual, const void* next_weight, void* h_out,
                   int64_t ld_h, void* y, int64_t ld_y, void* q, int64_t ld_q, float* scales,
                   int32_t T, void* stream) {
  const auto flag = [](int f) { return f == 0 || f == 1; };
  const auto eps_ok = [](float e) { return std::isfinite(e) && e >= 0x1p-126f; };
  if (!n || T < 0 || !type_ok(n->dtype) || (n->weight_dtype != n->dtype && n->weight_dtype != MOE_F32) ||
      !flag(n->normalize) || !flag(n->gate_per_row) || !flag(n->next) || n->gate < MOE_GATE_NONE ||
      n->gate > MOE_GATE_SIGMOID || n->out8 < MOE_OUT8_NONE || n->out8 > MOE_OUT8_E4M3 || !eps_ok(n->eps) ||
      !eps_ok(n->next_eps) || !std::isfinite(n->weight_offset) || !std::isfinite(n->scale) ||
      !std::isfinite(n->next_offset))
    return MOE_EINVAL;
  if (n->H < 1 || n->H > kNormMaxH || !group_ok(n->group, n->H) || !group_ok(n->out8_group, n->H))
    return MOE_EUNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || (!h_out && !y && !q) || (y && !n->next) || (weight && !n->normalize) ||
      (next_weight != nullptr) != (n->next != 0) || (gate != nullptr) != (n->gate != MOE_GATE_NONE) ||
      (q != nullptr) != (n->out8 != MOE_OUT8_NONE) || (scales != nullptr) != (q != nullptr))
    return MOE_EINVAL;
  const int eb = type_bytes(n->dtype), wb = type_bytes(n->weight_dtype), H = n->H;
  const bool wide_gate = gate && !n->gate_per_row;
  if (!aligned(weight, wb) || !aligned(channel_scale, wb) || !aligned(next_weight, wb) || !al4(scales) ||
      (q && !stride_ok(ld_q, H)) || (gate && !wide_gate && (!aligned(gate, eb) || !stride_ok(ld_gate, 1))))
    return MOE_EINVAL;
  const void* rows[] = {x, residual, wide_gate ? gate : nullptr, h_out, y};
  const int64_t lds[] = {ldx, ld_residual, ld_gate, ld_h, ld_y};
  for (int i = 0; i < 5; ++i)
    if (rows[i] && (!aligned(rows[i], eb) || !stride_ok(lds[i], H))) return MOE_EINVAL;
  // an output may replace a row that has been read only where both have one stride
  for (int out = 3; out < 5; ++out)
    for (int i = 0; i < out; ++i)
      if (rows[out] && rows[out] == rows[i] && lds[out] != lds[i]) return MOE_EINVAL;
  GatedArgs a{};
  a.x = x;
  a.weight = weight;
  a.gate = gate;
  a.channel = channel_scale;
  a.residual = residual;
  a.next_weight = next_weight;
  a.h_out = h_out;
  a.y = y;
  a.q = q;
  a.scales = scales;
  a.ldx = ldx;
  a.ld_gate = ld_gate;
  a.ld_residual = ld_residual;
  a.ld_h = ld_h;
  a.ld_y = ld_y;
  a.ld_q = ld_q;
  a.T = T;
  a.H = H;
  a.dtype = n->dtype;
  a.weight_f32 = n->weight_dtype == MOE_F32;
  a.normalize = n->normalize;
  a.group = n->group;
  a.gate_kind = n->gate;
  a.gate_per_row = n->gate_per_row;
  a.next = n->next;
  a.out8 = n->out8;
  a.out8_group = n->out8_group;
  a.eps = n->eps;
  a.weight_offset = n->weight_offset;
  a.scale = n->scale;
  a.next_eps = n->next_eps;
  a.next_offset = n->next_offset;
  return hip_status(launch_gated_norm(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
