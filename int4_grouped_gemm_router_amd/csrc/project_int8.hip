// A projection by 8-bit integers (gfx950 integer matrix cores):
//   y[t][n] = x_scales[t] w_scales[n] sum_k x[t][k] w[n][k] + bias[n]
// Sums are exact in 32-bit integers (K <= 65536, so at most 2^30).
#include "kernels.h"

namespace moe {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// D = A(16x64) * B(64x16) + C of signed bytes; lane l holds row (A) or column
// (B) l%16 and sixteen consecutive k of block l/16; D as of mfma16.
__device__ inline i32x4 mfma16_i8(i32x4 a, i32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
}

__device__ inline void put_value(void* y, int dtype, int64_t at, float v) {
  if (dtype == kNormBf16)
    static_cast<uint16_t*>(y)[at] = f2bf(v);
  else if (dtype == kNormF16)
    static_cast<uint16_t*>(y)[at] = __builtin_bit_cast(uint16_t, (_Float16)v);
  else
    static_cast<float*>(y)[at] = v;
}

}  // namespace

// Block: 64 tokens x 64 outputs, a wave 16 outputs of them.
__global__ __launch_bounds__(256) void int8_simple_kernel(Int8Args a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c16 = lane & 15, kb = lane >> 4;
  const int64_t t0 = (int64_t)blockIdx.y * 64;
  const int n0 = blockIdx.x * 64 + wave * 16;
  const int8_t* w = a.w + (int64_t)min(n0 + c16, a.N - 1) * a.K + 16 * kb;
  i32x4 acc[4] = {};
  const int8_t* x[4];
  for (int m = 0; m < 4; ++m) {
    const int64_t t = t0 + 16 * m + c16;
    x[m] = a.x + (t < a.T ? t : a.T - 1) * a.ldx + 16 * kb;
  }
  for (int k = 0; k < a.K; k += 64) {
    const i32x4 wv = *reinterpret_cast<const i32x4*>(w + k);
#pragma unroll
    for (int m = 0; m < 4; ++m) acc[m] = mfma16_i8(wv, *reinterpret_cast<const i32x4*>(x[m] + k), acc[m]);
  }
  for (int m = 0; m < 4; ++m) {
    const int64_t t = t0 + 16 * m + c16;
    if (t >= a.T) continue;
    const float xs = a.x_scales[t];
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + 4 * kb + i;
      if (n >= a.N) continue;
      float v = (float)acc[m][i] * xs * a.w_scales[n];
      if (a.bias) v += a.bias[n];
      put_value(a.y, a.dtype, t * a.ldy + n, v);
    }
  }
}

size_t int8_ws_bytes(int /*N*/, int /*K*/, int /*T*/) { return 0; }

hipError_t launch_project_int8(const Int8Args& a, hipStream_t s) {
  constexpr int kLaunchTokens = 1 << 20;
  for (int64_t t0 = 0; t0 < a.T; t0 += kLaunchTokens) {
    Int8Args c = a;
    c.T = (int)(a.T - t0 < kLaunchTokens ? a.T - t0 : kLaunchTokens);
    c.x += t0 * a.ldx;
    c.x_scales += t0;
    c.y = static_cast<char*>(c.y) + t0 * a.ldy * (a.dtype == kNormF32 ? 4 : 2);
    hipLaunchKernelGGL(int8_simple_kernel, dim3((a.N + 63) / 64, (c.T + 63) / 64), dim3(256), 0, s, c);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
