// Linear attention with a decay for each head (gfx950).
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
//
// for each value head, whose queries and keys are those of the key head
// v_head * qk_heads / v_heads. States are fp32 [qk_dim][v_dim].
#include "kernels.h"

namespace moe {

namespace {

constexpr int kStepCols = 32;  // columns of the state a block holds

// Bounds of sequence i, in range whatever the device array holds.
__device__ inline void bounds(const LinearArgs& a, int i, int& begin, int& end) {
  begin = min(max(a.cu_seqlens ? a.cu_seqlens[i] : i, 0), a.T);
  end = min(max(a.cu_seqlens ? a.cu_seqlens[i + 1] : i + 1, begin), a.T);
}
__device__ inline int slot_of(const int32_t* slots, int i, int n) {
  const int s = slots ? slots[i] : i;
  return s >= 0 && s < n ? s : -1;
}

}  // namespace

// Block: one sequence, one value head, 32 columns of its state in registers:
// thread (r, c) holds rows r + 32 p, columns 4 c .. 4 c + 3. Token after token.
template <int NP>
__global__ __launch_bounds__(256) void linear_walk_kernel(LinearArgs a) {
  __shared__ float part[4][kStepCols];
  const int tid = threadIdx.x, wave = tid >> 6, c = tid & 7, r = tid >> 3;
  const int col = blockIdx.z * kStepCols + 4 * c;
  const int head = blockIdx.y, seq = blockIdx.x, kh = head / (a.v_heads / a.qk_heads);
  const bool in = col < a.v_dim;
  int begin, end;
  bounds(a, seq, begin, end);
  const int64_t state = (int64_t)a.qk_dim * a.v_dim;
  float S[NP][4] = {};
  const int si = a.state_in ? slot_of(a.slots_in, seq, a.n_in) : -1;
  if (si >= 0 && in) {
    const float* p = a.state_in + ((int64_t)si * a.v_heads + head) * state + col;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (r + 32 * i < a.qk_dim) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(p + (int64_t)(r + 32 * i) * a.v_dim);
#pragma unroll
        for (int j = 0; j < 4; ++j) S[i][j] = v[j];
      }
  }
  for (int t = begin; t < end; ++t) {
    const uint16_t* q = a.q + (int64_t)t * a.ldq + (int64_t)kh * a.qk_dim;
    const uint16_t* k = a.k + (int64_t)t * a.ldk + (int64_t)kh * a.qk_dim;
    float v[4] = {}, o[4] = {};
    if (in) {
      const u32x2 w = *reinterpret_cast<const u32x2*>(a.v + (int64_t)t * a.ldv + (int64_t)head * a.v_dim + col);
      v[0] = bf16lo(w.x);
      v[1] = bf16hi(w.x);
      v[2] = bf16lo(w.y);
      v[3] = bf16hi(w.y);
    }
    const float d = expf(a.decay[a.ld_decay ? (int64_t)t * a.ld_decay + head : head]);
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      if (r + 32 * i >= a.qk_dim) continue;
      const float kv = bf16f(k[r + 32 * i]), qv = bf16f(q[r + 32 * i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] = __builtin_fmaf(kv, v[j], S[i][j] * d);
        o[j] = __builtin_fmaf(qv, S[i][j], o[j]);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] += __shfl_xor(o[j], 8);
      o[j] += __shfl_xor(o[j], 16);
      o[j] += __shfl_xor(o[j], 32);
    }
    if ((tid & 63) < 8)
#pragma unroll
      for (int j = 0; j < 4; ++j) part[wave][4 * c + j] = o[j];
    __syncthreads();
    if (tid < kStepCols && blockIdx.z * kStepCols + tid < a.v_dim)
      a.o[(int64_t)t * a.ldo + (int64_t)head * a.v_dim + blockIdx.z * kStepCols + tid] =
          f2bf(a.scale * ((part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid])));
    __syncthreads();
  }
  const int so = a.state_out ? slot_of(a.slots_out, seq, a.n_out) : -1;
  if (so >= 0 && in) {
    float* p = a.state_out + ((int64_t)so * a.v_heads + head) * state + col;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (r + 32 * i < a.qk_dim)
        *reinterpret_cast<f32x4*>(p + (int64_t)(r + 32 * i) * a.v_dim) = f32x4{S[i][0], S[i][1], S[i][2], S[i][3]};
  }
}

size_t linear_ws_bytes(const LinearArgs& /*a*/) { return 0; }

namespace {

hipError_t launch_walk(const LinearArgs& a, hipStream_t s) {
  const dim3 grid(a.n_seqs, a.v_heads, (a.v_dim + kStepCols - 1) / kStepCols), block(256);
  if (a.qk_dim <= 64)
    hipLaunchKernelGGL(linear_walk_kernel<2>, grid, block, 0, s, a);
  else if (a.qk_dim <= 128)
    hipLaunchKernelGGL(linear_walk_kernel<4>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(linear_walk_kernel<8>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_attention(const LinearArgs& a, hipStream_t s) { return launch_walk(a, s); }
hipError_t launch_linear_step(const LinearArgs& a, hipStream_t s) { return launch_walk(a, s); }

}  // namespace moe
