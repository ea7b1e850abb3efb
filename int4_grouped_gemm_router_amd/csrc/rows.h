// What the row operators share (gfx950): element types, wide accesses at any
// alignment, reductions over the threads of a row, and 8-bit outputs.
#pragma once

#include "device.h"
#include "kernels.h"
#include "topk.h"

namespace moe {

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
// reads, the waves of a block (256 threads a row or more) through LDS.
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
  if constexpr (TPR >= 256) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = f(f(s[0], s[1]), f(s[2], s[3]));
#pragma unroll
    for (int w = 4; w < TPR / 64; w += 4) v = f(v, f(f(s[w], s[w + 1]), f(s[w + 2], s[w + 3])));
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

}  // namespace moe
