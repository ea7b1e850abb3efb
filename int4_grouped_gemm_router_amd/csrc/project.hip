// A projection by packed int4 weights beside the low-rank adapters of many
// requests (gfx950, bf16 matrix cores, fp32 accumulation).
//
//   z[t] = scales[a] * A_a x[t],  y[t] = W x[t] + B_a z[t],  a = adapter_of[t]
//
// Two launches: the adapters' first product into the workspace, then the
// projection, whose epilogue adds the second product.
#include "kernels.h"

namespace moe {

namespace {

__device__ inline int adapter_at(const ProjectArgs& a, int t) {
  const int i = a.adapter_of[t];
  return i >= 0 && i < a.n ? i : -1;
}

__device__ inline int rank_of(const ProjectArgs& a, int i) {
  return a.ranks ? min(max(a.ranks[i], 0), a.R) : a.R;
}

}  // namespace

// z [T][R] fp32. Grid: T blocks of four waves; wave w takes ranks w, w + 4, ...
__global__ __launch_bounds__(256) void adapter_down_kernel(ProjectArgs a) {
  const int t = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int i = adapter_at(a, t);
  const int rank = i >= 0 ? rank_of(a, i) : 0;
  const float scale = i >= 0 && a.scales ? a.scales[i] : 1.f;
  const uint16_t* x = a.x + (int64_t)t * a.ldx;
  for (int r = wave; r < a.R; r += 4) {
    float v = 0.f;
    if (r < rank) {
      const uint16_t* A = a.A + ((int64_t)i * a.R + r) * a.K;
      for (int c = 2 * lane; c < a.K; c += 128) {
        const uint32_t xv = *reinterpret_cast<const uint32_t*>(x + c);
        const uint32_t av = *reinterpret_cast<const uint32_t*>(A + c);
        v = __builtin_fmaf(bf16lo(xv), bf16lo(av), v);
        v = __builtin_fmaf(bf16hi(xv), bf16hi(av), v);
      }
      v = wave_sum(v) * scale;
    }
    if (lane == 0) static_cast<float*>(a.ws)[(int64_t)t * a.R + r] = v;
  }
}

// Grid: (N / 64, ceil(T / 16)); block: one wave, 16 tokens by 64 columns.
// Exact codes: acc += s * x.(128 + q) + (b - 128 s) * sum(x) per group.
__global__ __launch_bounds__(64) void project_kernel(ProjectArgs a) {
  const int lane = threadIdx.x, c16 = lane & 15, kb = lane >> 4;
  const int wt = blockIdx.x, t0 = blockIdx.y * 16;
  const PackGeom geom = pack_geom(a.N, a.K, 0);
  const int G = geom.G;
  const ExpandConsts xk = expand_consts();
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
  const uint16_t* x = a.x + (int64_t)min(t0 + c16, a.T - 1) * a.ldx + 8 * kb;
  const uint8_t* nib = a.blob + geom.nib_off + (int64_t)wt * G * kNibBytes + lane * 16;
  const uint8_t* sbp = a.blob + geom.sb_off + (int64_t)wt * G * kSbBytes + c16 * 16;
  f32x4 acc[4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) acc[ct] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int g = 0; g < G; ++g) {
    const u32x4 a0 = *reinterpret_cast<const u32x4*>(x + g * kGroup);
    const u32x4 a1 = *reinterpret_cast<const u32x4*>(x + g * kGroup + 32);
    const u32x4 w0 = *reinterpret_cast<const u32x4*>(nib + (int64_t)g * kNibBytes);
    const u32x4 w1 = *reinterpret_cast<const u32x4*>(nib + (int64_t)g * kNibBytes + 1024);
    const u32x4 sbv = *reinterpret_cast<const u32x4*>(sbp + (int64_t)g * kSbBytes);
    const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
    const float sc[4] = {bf16lo(sbv.x), bf16hi(sbv.x), bf16lo(sbv.y), bf16hi(sbv.y)};
    const float bi[4] = {bf16lo(sbv.z), bf16hi(sbv.z), bf16lo(sbv.w), bf16hi(sbv.w)};
    f32x4 xs = mfma16(a0, ones, f32x4{0.f, 0.f, 0.f, 0.f});
    xs = mfma16(a1, ones, xs);
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      f32x4 p = mfma16(a0, expand_codes(words[2 * ct], xk), f32x4{0.f, 0.f, 0.f, 0.f});
      p = mfma16(a1, expand_codes(words[2 * ct + 1], xk), p);
      const float bp = bi[ct] - 128.0f * sc[ct];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[ct][i] = __builtin_fmaf(bp, xs[i], __builtin_fmaf(sc[ct], p[i], acc[ct][i]));
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = t0 + 4 * kb + i;
    if (t >= a.T) continue;
    const int ad = a.adapter_of ? adapter_at(a, t) : -1;
    const int rank = ad >= 0 ? rank_of(a, ad) : 0;
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      const int n = 64 * wt + 16 * ct + c16;
      float v = acc[ct][i];
      if (ad >= 0) {
        const uint16_t* B = a.B + ((int64_t)ad * a.N + n) * a.R;
        for (int r = 0; r < rank; ++r) v = __builtin_fmaf(static_cast<float*>(a.ws)[(int64_t)t * a.R + r], bf16f(B[r]), v);
      }
      a.y[(int64_t)t * a.ldy + n] = f2bf(v);
    }
  }
}

size_t project_ws_bytes(int /*N*/, int /*K*/, int R, int T) {
  return ((size_t)T * R * 4 + 255) / 256 * 256;
}

hipError_t launch_project(const ProjectArgs& a, hipStream_t s) {
  if (a.adapter_of) hipLaunchKernelGGL(adapter_down_kernel, dim3(a.T), dim3(256), 0, s, a);
  hipLaunchKernelGGL(project_kernel, dim3(a.N / 64, (a.T + 15) / 16), dim3(64), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
