// Residual add and RMS norm of rows, with an optional 8-bit output (gfx950).
//
//   h = x + residual (rounded to the rows' type), r = rsqrt(mean(h^2) + eps),
//   v = h r (w + offset), y = v, s = max |v| / Q per group, q = v / s
//
// One pass over memory: a block of 256 threads holds its row in registers
// (up to 16384 values), so x and residual are read once and every output is
// written once; the sum of squares and v are fp32. What bounds it is the
// memory traffic, and for a few rows the latency of one load, one block
// reduction and one store.
#include "kernels.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;

struct RowsBf16 {
  typedef uint16_t type;
  static __device__ float get(type v) { return bf16f(v); }
  static __device__ type put(float v) { return f2bf(v); }
};
struct RowsF16 {
  typedef uint16_t type;
  static __device__ float get(type v) { return (float)__builtin_bit_cast(_Float16, v); }
  static __device__ type put(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
};
struct RowsF32 {
  typedef float type;
  static __device__ float get(type v) { return v; }
  static __device__ type put(float v) { return v; }
};

template <class T, int N>
struct alignas(sizeof(T) * N) Vec {
  T v[N];
};

// Sum over the block's four waves, returned to every thread.
__device__ inline float block_sum(float v, float* s) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  v = (s[0] + s[1]) + (s[2] + s[3]);
  __syncthreads();
  return v;
}

// |v| as ordered bits: their integer maximum is the largest magnitude, with
// NaN above infinity.
__device__ inline uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// v / s rounded to 8 bits. Scales below fp32's normal range are coarse, so
// the quotient is limited to the format's largest value.
__device__ inline uint8_t to_int8(float v, float s) {
  float t = s > 0.f ? v / s : 0.f;  // s NaN: 0
  t = fminf(fmaxf(t, -127.f), 127.f);
  return v == v && s < INFINITY ? (uint8_t)(int8_t)(int)rintf(t) : 0;
}
__device__ inline uint8_t to_e4m3(float v, float s) {
  float t = s == 0.f ? 0.f : v / s;
  if (t > 448.f) t = 448.f;
  if (t < -448.f) t = -448.f;
  return (uint8_t)(__builtin_amdgcn_cvt_pk_fp8_f32(t, 0.f, 0, false) & 0xFF);
}

}  // namespace

// Grid: T blocks, one row each. Thread i owns the VEC consecutive values
// from (i + 256 j) VEC, j < NV. LW: values per load (VEC, or 1 where the
// addresses are not aligned).
template <class R, int VEC, int LW, int NV>
__global__ __launch_bounds__(kNormThreads) void add_rmsnorm_kernel(NormArgs a) {
  typedef typename R::type E;
  __shared__ float red[4];
  __shared__ uint32_t redm[4];
  const int tid = threadIdx.x, H = a.H;
  const int64_t row = blockIdx.x;
  const E* x = static_cast<const E*>(a.x) + row * a.ldx;
  const E* res = a.residual ? static_cast<const E*>(a.residual) + row * a.ld_residual : nullptr;
  float v[NV][VEC];
  float ss = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (tid + kNormThreads * j) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i) v[j][i] = 0.f;
    if constexpr (LW == VEC) {
      if (c + VEC <= H) {
        const Vec<E, VEC> xv = *reinterpret_cast<const Vec<E, VEC>*>(x + c);
#pragma unroll
        for (int i = 0; i < VEC; ++i) v[j][i] = R::get(xv.v[i]);
        if (res) {
          const Vec<E, VEC> rv = *reinterpret_cast<const Vec<E, VEC>*>(res + c);
#pragma unroll
          for (int i = 0; i < VEC; ++i) v[j][i] = R::get(R::put(v[j][i] + R::get(rv.v[i])));
        }
      }
    }
    if (LW != VEC || c + VEC > H) {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (c + i < H) {
          v[j][i] = R::get(x[c + i]);
          if (res) v[j][i] = R::get(R::put(v[j][i] + R::get(res[c + i])));
        }
    }
#pragma unroll
    for (int i = 0; i < VEC; ++i) ss = __builtin_fmaf(v[j][i], v[j][i], ss);
  }
  ss = block_sum(ss, red);
  const float r = 1.0f / sqrtf(ss / (float)H + a.eps);

  auto store = [&](E* dst, int j) {
    const int c = (tid + kNormThreads * j) * VEC;
    if (LW == VEC && c + VEC <= H) {
      Vec<E, VEC> o;
#pragma unroll
      for (int i = 0; i < VEC; ++i) o.v[i] = R::put(v[j][i]);
      *reinterpret_cast<Vec<E, VEC>*>(dst + c) = o;
    } else {
#pragma unroll
      for (int i = 0; i < VEC; ++i)
        if (c + i < H) dst[c + i] = R::put(v[j][i]);
    }
  };
  if (a.h_out) {
    E* h = static_cast<E*>(a.h_out) + row * a.ld_h;
#pragma unroll
    for (int j = 0; j < NV; ++j) store(h, j);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (tid + kNormThreads * j) * VEC;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i < H) {
        const float w = a.weight_f32 ? static_cast<const float*>(a.weight)[c + i]
                                     : R::get(static_cast<const E*>(a.weight)[c + i]);
        v[j][i] = v[j][i] * r * (w + a.weight_offset);
      }
  }
  if (a.y) {
    E* y = static_cast<E*>(a.y) + row * a.ld_y;
#pragma unroll
    for (int j = 0; j < NV; ++j) store(y, j);
  }
  if (!a.q) return;

  const float Q = a.out8 == kOut8Int8 ? 127.f : 448.f;
  uint32_t m[NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    m[j] = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) m[j] = max(m[j], abs_bits(v[j][i]));
  }
  if (a.group) {
    // group / VEC consecutive threads hold a group (VEC = 8 whenever there
    // are groups, so at most 32 lanes of one wave)
#pragma unroll
    for (int j = 0; j < NV; ++j)
      for (int o = 1; o < a.group / VEC; o <<= 1) m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], o));
  } else {
    uint32_t all = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) all = max(all, m[j]);
    for (int o = 1; o < 64; o <<= 1) all = max(all, (uint32_t)__shfl_xor((int)all, o));
    if ((tid & 63) == 0) redm[tid >> 6] = all;
    __syncthreads();
    all = max(max(redm[0], redm[1]), max(redm[2], redm[3]));
#pragma unroll
    for (int j = 0; j < NV; ++j) m[j] = all;
  }
  uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ld_q;
  const int groups = a.group ? H / a.group : 1;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (tid + kNormThreads * j) * VEC;
    const float s = __uint_as_float(m[j]) / Q;
    if (c < H && (a.group ? c % a.group == 0 : c == 0)) a.scales[row * groups + (a.group ? c / a.group : 0)] = s;
#pragma unroll
    for (int i = 0; i < VEC; ++i)
      if (c + i < H) q[c + i] = a.out8 == kOut8Int8 ? to_int8(v[j][i], s) : to_e4m3(v[j][i], s);
  }
}

namespace {

template <class R, int VEC, int LW>
void launch_vec(const NormArgs& a, hipStream_t s) {
  const dim3 grid(a.T), block(kNormThreads);
  const int per = kNormThreads * VEC;
  if (a.H <= per)
    hipLaunchKernelGGL((add_rmsnorm_kernel<R, VEC, LW, 1>), grid, block, 0, s, a);
  else if (a.H <= 4 * per)
    hipLaunchKernelGGL((add_rmsnorm_kernel<R, VEC, LW, 4>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((add_rmsnorm_kernel<R, VEC, LW, kNormMaxH / per>), grid, block, 0, s, a);
}

template <class R>
void launch_rows(const NormArgs& a, hipStream_t s) {
  if (a.aligned)
    launch_vec<R, 8, 8>(a, s);
  else
    launch_vec<R, 8, 1>(a, s);
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& a, hipStream_t s) {
  if (a.dtype == kNormBf16)
    launch_rows<RowsBf16>(a, s);
  else if (a.dtype == kNormF16)
    launch_rows<RowsF16>(a, s);
  else
    launch_rows<RowsF32>(a, s);
  return hipGetLastError();
}

}  // namespace moe
