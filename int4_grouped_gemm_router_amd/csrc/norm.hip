// Residual add and RMS norm of rows, with an optional 8-bit output (gfx950).
//
//   h = x + residual (rounded to the rows' type), r = rsqrt(mean(h^2) + eps),
//   v = h r (w + offset), y = v, s = max |v| / Q per group, q = v / s
//
// One pass over memory: a row is held in the registers of 16, 64 or 256
// threads (up to 16384 values), so x and residual are read once and every
// output is written once; the sum of squares and v are fp32. The memory
// traffic bounds it up to 4096 values, the waves that their registers leave
// room for in longer rows, and for a few rows the latency of one load, one
// reduction and one store. Threads keep their weights over the rows they take
// in turn.
#include <type_traits>

#include "kernels.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kNormThreads = 256;
constexpr int kVec = 8;  // consecutive values a thread owns

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

// Eight values at an address that only their own type aligns: global memory
// takes wide accesses at any address (a little slower off 16 bytes).
template <class E>
struct __attribute__((packed, aligned(sizeof(E)))) Eight {
  E v[kVec];
};
struct __attribute__((packed, aligned(1))) Bytes8 {
  uint32_t v[2];
};

// Reductions over the threads of a row (TPR of them, consecutive), returned
// to each: within sixteen lanes by DPP, the four sixteens of a wave by lane
// reads, the waves of a block through LDS.
template <int TPR, class F>
__device__ inline uint32_t row_all(uint32_t v, uint32_t* s, F f) {
  v = f(v, dpp<0xB1>(v));   // lane ^ 1
  v = f(v, dpp<0x4E>(v));   // lane ^ 2
  v = f(v, dpp<0x141>(v));  // mirror within 8
  v = f(v, dpp<0x140>(v));  // mirror within 16
  if constexpr (TPR >= 64) {
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
    const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    v = f(f(a, b), f(c, d));
  }
  if constexpr (TPR == 256) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = f(f(s[0], s[1]), f(s[2], s[3]));
    __syncthreads();
  }
  return v;
}

__device__ inline uint32_t add_bits(uint32_t a, uint32_t b) {
  return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
}
__device__ inline uint32_t max_bits(uint32_t a, uint32_t b) { return max(a, b); }

// A group's scale and what its quotients are formed with. The values t of a
// row are v up to the factor f (1 <= f < 2), which cancels in v / s = t Q / m
// with m the largest |t| of the group: that quotient of t and m, corrected
// once, is rounded correctly, where v / s from a rounded v and s is off by a
// few units (and more 8-bit values land on the wrong side of a tie). t itself
// is exact for 16-bit rows and weights without an offset, else rounded once
// or twice.
struct Group {
  float s, m, inv, f;
  bool plain;  // m is far from under- and overflow
};
template <int OUT8>
constexpr float kTop = OUT8 == kOut8Int8 ? 127.f : 448.f;

template <int OUT8>
__device__ inline Group group_of_max(float m, float f) {
  Group g;
  g.m = m;
  g.f = f;
  g.s = m * f / kTop<OUT8>;
  g.plain = m >= 0x1p-100f && m < 0x1p100f;
  g.inv = g.plain ? 1.0f / m : 0.f;
  return g;
}

// The quotient of t before rounding; otherwise than plain: 0 for s = 0,
// limited quotients for the coarse scales below the normal range, and NaN (or
// 0 for int8) where the scale is not finite.
template <int OUT8>
__device__ inline float quotient(float t, const Group& g) {
  constexpr float Q = kTop<OUT8>;
  if (g.plain) {
    // t Q = n + e exactly (products of fp16 have 22 bits, and Q up to seven
    // more), so that the remainder t Q - q m is rounded only once
    const float n = t * Q, e = __builtin_fmaf(t, Q, -n), q = n * g.inv;
    return __builtin_fmaf(__builtin_fmaf(-q, g.m, n) + e, g.inv, q);
  }
  float q = g.s == 0.f ? 0.f : t * g.f / g.s;
  if (OUT8 == kOut8Int8 && !(g.s < INFINITY)) q = 0.f;
  if (q > Q) q = Q;
  if (q < -Q) q = -Q;
  return OUT8 == kOut8Int8 && !(q == q) ? 0.f : q;
}

// Eight quotients rounded to int8 (the integer is in the low bits of
// q + 1.5 2^23, rounded to even by that addition) or e4m3.
template <int OUT8>
__device__ inline Bytes8 eight_bits(const float (&t)[kVec], const Group& g) {
  Bytes8 o;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = quotient<OUT8>(t[4 * h + i], g);
    if (OUT8 == kOut8Int8) {
      uint32_t b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(q[i] + 12582912.0f);
      const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0C);
      o.v[h] = lo | hi;
    } else {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      w = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], w, true);
      o.v[h] = (uint32_t)w;
    }
  }
  return o;
}

}  // namespace

// Block: 256 threads, 256 / TPR rows at a time; blocks take rows in turn.
// Thread i of a row owns the eight values from (i + TPR j) * 8, j < NV. RES:
// a residual is added. OUT8: the 8-bit output.
template <class R, int TPR, int NV, bool RES, int OUT8>
__global__ __launch_bounds__(kNormThreads) void add_rmsnorm_kernel(NormArgs a) {
  typedef typename R::type E;
  __shared__ uint32_t red[4];
  constexpr int kRows = kNormThreads / TPR;
  const int lt = threadIdx.x % TPR, H = a.H;
  float w[NV][kVec];
  auto weights = [&](const auto* p, auto get) {
    typedef typename std::remove_const<typename std::remove_pointer<decltype(p)>::type>::type W;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lt + TPR * j) * kVec;
      if (c + kVec <= H) {
        const Eight<W> e = *reinterpret_cast<const Eight<W>*>(p + c);
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[j][i] = get(e.v[i]) + a.weight_offset;
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) w[j][i] = c + i < H ? get(p[c + i]) + a.weight_offset : 0.f;
      }
    }
  };
  if (a.weight_f32)
    weights(static_cast<const float*>(a.weight), [](float v) { return v; });
  else
    weights(static_cast<const E*>(a.weight), [](E v) { return R::get(v); });
  // (every thread of a block takes the same number of turns: the reductions
  // of a row of 256 threads have barriers; the other rows end on their own)
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < a.T; row += (int64_t)gridDim.x * kRows) {
    const E* x = static_cast<const E*>(a.x) + row * a.ldx;
    const E* res = RES ? static_cast<const E*>(a.residual) + row * a.ld_residual : nullptr;
    Eight<E> xv[NV], rv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (lt + TPR * j) * kVec;
      if (c + kVec <= H) {
        xv[j] = *reinterpret_cast<const Eight<E>*>(x + c);
        if constexpr (RES) rv[j] = *reinterpret_cast<const Eight<E>*>(res + c);
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          xv[j].v[i] = c + i < H ? x[c + i] : E(0);
          if constexpr (RES) rv[j].v[i] = c + i < H ? res[c + i] : E(0);
        }
      }
    }
    float v[NV][kVec];
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float part = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[j][i] = R::get(xv[j].v[i]);
        if constexpr (RES) v[j][i] = R::get(R::put(v[j][i] + R::get(rv[j].v[i])));
        part = __builtin_fmaf(v[j][i], v[j][i], part);
      }
      ss += part;
    }
    ss = __uint_as_float(row_all<TPR>(__float_as_uint(ss), red, add_bits));
    const float r = 1.0f / sqrtf(ss / (float)H + a.eps);

    auto store = [&](E* dst, auto value) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        if (c + kVec <= H) {
          Eight<E> o;
#pragma unroll
          for (int i = 0; i < kVec; ++i) o.v[i] = R::put(value(j, i));
          *reinterpret_cast<Eight<E>*>(dst + c) = o;
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (c + i < H) dst[c + i] = R::put(value(j, i));
        }
      }
    };
    if (a.h_out) store(static_cast<E*>(a.h_out) + row * a.ld_h, [&](int j, int i) { return v[j][i]; });
    if (a.y) store(static_cast<E*>(a.y) + row * a.ld_y, [&](int j, int i) { return v[j][i] * r * w[j][i]; });
    if constexpr (OUT8 != kOut8None) {
      // v with the power of two in r only (both products are exact for 16-bit
      // rows and weights without an offset): the rest of r is the group scale's
      // factor
      const float p = __uint_as_float(__float_as_uint(r) & 0x7F800000u), f = p > 0.f ? r / p : r;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] = v[j][i] * p * w[j][i];
      // |v| as ordered bits: their integer maximum is the largest magnitude,
      // with NaN above infinity (values past the row are 0)
      uint32_t m[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        m[j] = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          m[j] = max(m[j], (lt + TPR * j) * kVec + i < H ? __float_as_uint(v[j][i]) & 0x7FFFFFFFu : 0u);
      }
      if (a.group) {
        // group / 8 consecutive lanes hold a group: 4, 8, 16 or 32
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          m[j] = max(m[j], dpp<0xB1>(m[j]));
          m[j] = max(m[j], dpp<0x4E>(m[j]));
          if (a.group >= 64) m[j] = max(m[j], dpp<0x141>(m[j]));
          if (a.group >= 128) m[j] = max(m[j], dpp<0x140>(m[j]));
          if (a.group >= 256) m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
        }
      } else {
        uint32_t all = m[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) all = max(all, m[j]);
        all = row_all<TPR>(all, red, max_bits);
#pragma unroll
        for (int j = 0; j < NV; ++j) m[j] = all;
      }
      uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ld_q;
      float* scales = a.scales + row * (a.group ? H / a.group : 1);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        if (c >= H) continue;
        const Group g = group_of_max<OUT8>(__uint_as_float(m[j]), f);
        if (a.group ? c % a.group == 0 : c == 0) scales[a.group ? c / a.group : 0] = g.s;
        const Bytes8 o = eight_bits<OUT8>(v[j], g);
        if (c + kVec <= H) {
          *reinterpret_cast<Bytes8*>(q + c) = o;
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (c + i < H) q[c + i] = (uint8_t)(o.v[i >> 2] >> (8 * (i & 3)));
        }
      }
    }
  }
}

namespace {

template <class R, int TPR, int NV>
void launch_shape(const NormArgs& a, hipStream_t s) {
  // enough blocks for eight waves on every SIMD, where their registers leave
  // room (for six to eight up to 4096 values, three to five from 4097 on, one or
  // two from 8193); each takes rows in turn
  constexpr int kRows = kNormThreads / TPR;
  const int64_t blocks = ((int64_t)a.T + kRows - 1) / kRows;
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048)), block(kNormThreads);
  if (a.residual) {
    if (a.out8 == kOut8Int8)
      hipLaunchKernelGGL((add_rmsnorm_kernel<R, TPR, NV, true, kOut8Int8>), grid, block, 0, s, a);
    else if (a.out8 == kOut8E4m3)
      hipLaunchKernelGGL((add_rmsnorm_kernel<R, TPR, NV, true, kOut8E4m3>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((add_rmsnorm_kernel<R, TPR, NV, true, kOut8None>), grid, block, 0, s, a);
  } else {
    if (a.out8 == kOut8Int8)
      hipLaunchKernelGGL((add_rmsnorm_kernel<R, TPR, NV, false, kOut8Int8>), grid, block, 0, s, a);
    else if (a.out8 == kOut8E4m3)
      hipLaunchKernelGGL((add_rmsnorm_kernel<R, TPR, NV, false, kOut8E4m3>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((add_rmsnorm_kernel<R, TPR, NV, false, kOut8None>), grid, block, 0, s, a);
  }
}

// One load of each input per thread where the threads of a block or of a wave
// allow it, more blocks rather than longer rows per thread: rows of 2048
// values by 256 threads take 2.4 us for one row, 4.8 for 1024, 51.5 for 16384
// (5.2 TB/s), by one wave with four loads a lane 3.9, 6.3 and 54.7. As many
// bytes in rows of 4096 values move at 5.0 TB/s, of 5120, 7168 and 8192 at 3.7,
// 4.0 and 4.4, of 16384 at 2.3 (with e4m3 4.9, 3.2, 3.5, 3.9 and 1.9).
template <class R>
void launch_rows(const NormArgs& a, hipStream_t s) {
  if (a.H <= 128)
    launch_shape<R, 16, 1>(a, s);
  else if (a.H <= 512)
    launch_shape<R, 64, 1>(a, s);
  else if (a.H <= 1024)
    launch_shape<R, 64, 2>(a, s);
  else if (a.H <= 2048)
    launch_shape<R, 256, 1>(a, s);
  else if (a.H <= 4096)
    launch_shape<R, 256, 2>(a, s);
  else if (a.H <= 8192)
    launch_shape<R, 256, 4>(a, s);
  else
    launch_shape<R, 256, kNormMaxH / (256 * kVec)>(a, s);
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs& in, hipStream_t s) {
  NormArgs a = in;
  if (a.group == a.H) a.group = 0;  // one scale a row either way
  if (a.dtype == kNormBf16)
    launch_rows<RowsBf16>(a, s);
  else if (a.dtype == kNormF16)
    launch_rows<RowsF16>(a, s);
  else
    launch_rows<RowsF32>(a, s);
  return hipGetLastError();
}

}  // namespace moe
