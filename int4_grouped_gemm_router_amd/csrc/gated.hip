// The norm after a block (or of its heads) with a gate, the residual add with
// a scale, the norm before the next block, and an 8-bit output (gfx950).
//
//   u = x rsqrt(mean_group(x^2) + eps) (weight + offset)
//   v = residual + scale channel_scale u act(gate),  h = v
//   v = v rsqrt(mean_row(v^2) + next_eps) (next_weight + next_offset),  y = v
//   s = max |v| / Q per 8-bit group,  q = v / s
//
// One pass over memory, as the plain norm does it: a row in the registers of
// 16 to 1024 threads, eight consecutive values a thread and access (sixteen in
// the longest rows), every sum and v in fp32. A group of 32 to 256 values lies in
// 4 to 32 neighbouring lanes, so the first norm needs no LDS unless it spans the
// row. The weights of the first norm, the channels' scale and the scalar one are
// one factor a value, kept over the rows that a thread takes in turn. Memory
// bounds it, and with a gate per value the exponentials come near.
#include <type_traits>

#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

// threads of a block: 256, or those of a longer row
template <int TPR>
constexpr int kGatedThreads = TPR > 256 ? TPR : 256;

// Waves of a SIMD that the registers are for: eight (64 registers) for rows of 16
// bits, but six with a second norm and an 8-bit output at once, which spill at
// eight: 16384 x 512 70 against 19 us, 8192 x 4096 73, 69, 4096 x 8192 145, 92. At
// 256 threads a row the spills stay out of the way (16384 x 2048 65.7 at either).
template <class R, int TPR, int NV, int OUT8, bool NEXT>
constexpr int kGatedWaves = NV > 1 || sizeof(typename R::type) == 4 ? 4 : NEXT && OUT8 != kOut8None && TPR != 256 ? 6 : 8;

// e^z to about an ulp: the part of z log2(e) that its product loses is put
// back as a factor. Below -110 the result is 0 in every use here (1 + e^z).
__device__ inline float exp_full(float z) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500e-8f;  // log2(e) in two parts
  z = z < -110.f ? -110.f : z;
  const float t = z * kHi, e = __builtin_fmaf(z, kHi, -t) + z * kLo;
  const float p = __builtin_amdgcn_exp2f(t);
  return p < INFINITY ? __builtin_fmaf(p, e * 0.693147181f, p) : p;
}

// For rows of 16 bits without the part that the product loses: it errs by
// 2^-24 |z| log2(e), far below those rows' own 2^-9 or 2^-12.
template <class R>
__device__ inline float sigmoid(float z) {
  const float e = sizeof(typename R::type) == 4 ? exp_full(-z) : __builtin_amdgcn_exp2f(z * -1.44269504f);
  return __builtin_amdgcn_rcpf(1.0f + e);
}

// 1 / sqrt(x) for x >= 2^-126: the instruction's and one step of Newton's method.
__device__ inline float inverse_root(float x) {
  const float r = __builtin_amdgcn_rsqf(x);
  const float e = __builtin_fmaf(-x * r, r, 1.0f);
  return x < INFINITY ? __builtin_fmaf(0.5f * r, e, r) : r;
}

// The sum over the lanes that hold a group of `group` values (32, 64, 128 or
// 256: 4, 8, 16 or 32 lanes), in each.
__device__ inline float group_sum(float s, int group) {
  uint32_t v = __float_as_uint(s);
  v = add_bits(v, dpp<0xB1>(v));
  v = add_bits(v, dpp<0x4E>(v));
  if (group >= 64) v = add_bits(v, dpp<0x141>(v));
  if (group >= 128) v = add_bits(v, dpp<0x140>(v));
  if (group >= 256) v = add_bits(v, (uint32_t)__shfl_xor((int)v, 16));
  return __uint_as_float(v);
}

// row_all with one barrier: s is not used again before another barrier that
// every thread reaches after its reads here.
template <int TPR, class F>
__device__ inline uint32_t row_all_once(uint32_t v, uint32_t* s, F f) {
  v = row_all<(TPR < 64 ? TPR : 64)>(v, s, f);
  if constexpr (TPR >= 256) {
    if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
    __syncthreads();
    v = f(f(s[0], s[1]), f(s[2], s[3]));
#pragma unroll
    for (int w = 4; w < TPR / 64; w += 4) v = f(v, f(f(s[w], s[w + 1]), f(s[w + 2], s[w + 3])));
  }
  return v;
}

}  // namespace

// Block: 256 threads, 256 / TPR rows at a time, or TPR and one; blocks take
// rows in turn. Thread i of a row owns the eight values from (i + TPR j) * 8,
// j < NV. NEXT: the second norm. 64 registers for rows of 16 bits, so that eight
// waves fit a SIMD: 16384 x 2048 with residual, second norm and int8 takes 65 us
// (4.6 TB/s), with the 94 registers of a next row loaded ahead 73; 1500 x 4096
// fp16, gated by heads of 128, 16 and 20.
template <class R, int TPR, int NV, int OUT8, bool NEXT>
__global__ __launch_bounds__(kGatedThreads<TPR>, (kGatedWaves<R, TPR, NV, OUT8, NEXT>)) void gated_norm_kernel(GatedArgs a) {
  typedef typename R::type E;
  __shared__ uint32_t red[2][3][16];  // by turns: [turn % 2][which reduction][wave]
  constexpr int kRows = kGatedThreads<TPR> / TPR;
  const int lt = kRows > 1 ? threadIdx.x % TPR : threadIdx.x, H = a.H;
  const bool wide_gate = a.gate_kind && !a.gate_per_row;
  Eight<E> xv[NV], gv[NV], rv[NV];
  E row_gate = E(0);
  auto load_rows = [&](int64_t row) {
    auto load = [&](const void* p, int64_t ld, Eight<E> (&out)[NV]) {
      const E* x = static_cast<const E*>(p) + row * ld;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        if (c + kVec <= H) {
          out[j] = *reinterpret_cast<const Eight<E>*>(x + c);
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i) out[j].v[i] = c + i < H ? x[c + i] : E(0);
        }
      }
    };
    load(a.x, a.ldx, xv);
    if (wide_gate) load(a.gate, a.ld_gate, gv);
    if (a.gate_per_row) row_gate = static_cast<const E*>(a.gate)[row * a.ld_gate];
    if (a.residual) load(a.residual, a.ld_residual, rv);
  };
  // (one row a block: the same for all threads, and so are its addresses)
  const int64_t first = (int64_t)blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / TPR : 0), step = (int64_t)gridDim.x * kRows;

  // p's values at c .. c + 7 (index masked by `mask`; group weights repeat), 0 past the row
  auto eight = [&](const void* p, bool f32, int c, int mask, float add, float (&out)[kVec]) {
    if (f32) {
      const float* f = static_cast<const float*>(p) + (c & mask);
      if (c + kVec <= H) {
        const Eight<float> e = *reinterpret_cast<const Eight<float>*>(f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[i] = e.v[i] + add;
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[i] = c + i < H ? f[i] + add : 0.f;
      }
    } else {
      const E* f = static_cast<const E*>(p) + (c & mask);
      if (c + kVec <= H) {
        const Eight<E> e = *reinterpret_cast<const Eight<E>*>(f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[i] = R::get(e.v[i]) + add;
      } else {
#pragma unroll
        for (int i = 0; i < kVec; ++i) out[i] = c + i < H ? R::get(f[i]) + add : 0.f;
      }
    }
  };
  float w[NV][kVec], nw[NV][kVec];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = (lt + TPR * j) * kVec;
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[j][i] = a.scale;
    if (a.channel) {
      float f[kVec];
      eight(a.channel, a.weight_f32, c, -1, 0.f, f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[j][i] *= f[i];
    }
    if (a.weight) {
      float f[kVec];
      eight(a.weight, a.weight_f32, c, a.group ? a.group - 1 : -1, a.weight_offset, f);
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[j][i] *= f[i];
    }
    if constexpr (NEXT) eight(a.next_weight, a.weight_f32, c, -1, a.next_offset, nw[j]);
  }
  int turn = 0;
  for (int64_t row = first; row < a.T; row += step, turn ^= 1) {
    load_rows(row);
    float v[NV][kVec], g[NV][kVec], res[NV][kVec];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        v[j][i] = R::get(xv[j].v[i]);
        g[j][i] = R::get(gv[j].v[i]);
        res[j][i] = R::get(rv[j].v[i]);
      }
    const float zr = R::get(row_gate);
    auto squares = [&](int j) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) s = __builtin_fmaf(v[j][i], v[j][i], s);
      return s;
    };
    auto multiply = [&](int j, float f) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[j][i] *= f;
    };
    if (a.normalize) {
      if (a.group) {
        const float of = 1.0f / (float)a.group;
#pragma unroll
        for (int j = 0; j < NV; ++j) multiply(j, inverse_root(group_sum(squares(j), a.group) * of + a.eps));
      } else {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) ss += squares(j);
        ss = __uint_as_float(row_all_once<TPR>(__float_as_uint(ss), red[turn][0], add_bits));
        const float r = inverse_root(ss * (1.0f / (float)H) + a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j) multiply(j, r);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[j][i] *= w[j][i];
    const bool silu = a.gate_kind == kGateSilu;
    if (wide_gate) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] *= sigmoid<R>(g[j][i]) * (silu ? g[j][i] : 1.0f);
    } else if (a.gate_kind) {
      const float f = sigmoid<R>(zr) * (silu ? zr : 1.0f);
#pragma unroll
      for (int j = 0; j < NV; ++j) multiply(j, f);
    }
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] += res[j][i];
    }
    auto store = [&](void* p, int64_t ld) {
      E* dst = static_cast<E*>(p) + row * ld;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        if (c + kVec <= H) {
          Eight<E> o;
#pragma unroll
          for (int i = 0; i < kVec; ++i) o.v[i] = R::put(v[j][i]);
          *reinterpret_cast<Eight<E>*>(dst + c) = o;
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (c + i < H) dst[c + i] = R::put(v[j][i]);
        }
      }
    };
    if (a.h_out) store(a.h_out, a.ld_h);
    if constexpr (NEXT) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) ss += squares(j);
      ss = __uint_as_float(row_all_once<TPR>(__float_as_uint(ss), red[turn][1], add_bits));
      const float r = inverse_root(ss * (1.0f / (float)H) + a.next_eps);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] = v[j][i] * r * nw[j][i];
      if (a.y) store(a.y, a.ld_y);
    }
    if constexpr (OUT8 != kOut8None) {
      // |v| as ordered bits: their integer maximum is the largest magnitude,
      // with NaN above infinity (values past the row are left out: an infinite
      // gate of the row makes NaN of their zeros)
      uint32_t m[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        m[j] = 0;
        if (c + kVec <= H) {
#pragma unroll
          for (int i = 0; i < kVec; ++i) m[j] = max(m[j], __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
        } else {
#pragma unroll
          for (int i = 0; i < kVec; ++i)
            if (c + i < H) m[j] = max(m[j], __float_as_uint(v[j][i]) & 0x7FFFFFFFu);
        }
      }
      if (a.out8_group) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          m[j] = max(m[j], dpp<0xB1>(m[j]));
          m[j] = max(m[j], dpp<0x4E>(m[j]));
          if (a.out8_group >= 64) m[j] = max(m[j], dpp<0x141>(m[j]));
          if (a.out8_group >= 128) m[j] = max(m[j], dpp<0x140>(m[j]));
          if (a.out8_group >= 256) m[j] = max(m[j], (uint32_t)__shfl_xor((int)m[j], 16));
        }
      } else {
        uint32_t all = m[0];
#pragma unroll
        for (int j = 1; j < NV; ++j) all = max(all, m[j]);
        all = row_all_once<TPR>(all, red[turn][2], max_bits);
#pragma unroll
        for (int j = 0; j < NV; ++j) m[j] = all;
      }
      uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ld_q;
      float* scales = a.scales + row * (a.out8_group ? H / a.out8_group : 1);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        if (c >= H) continue;
        const Group gr = group_of_max<OUT8>(__uint_as_float(m[j]), 1.0f);
        if (a.out8_group ? c % a.out8_group == 0 : c == 0) scales[a.out8_group ? c / a.out8_group : 0] = gr.s;
        const Bytes8 o = eight_bits<OUT8>(v[j], gr);
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

template <class R, int TPR, int NV, int OUT8>
void launch_next(const GatedArgs& a, dim3 grid, hipStream_t s) {
  if (a.next)
    hipLaunchKernelGGL((gated_norm_kernel<R, TPR, NV, OUT8, true>), grid, dim3(kGatedThreads<TPR>), 0, s, a);
  else
    hipLaunchKernelGGL((gated_norm_kernel<R, TPR, NV, OUT8, false>), grid, dim3(kGatedThreads<TPR>), 0, s, a);
}

template <class R, int TPR, int NV>
void launch_shape(const GatedArgs& a, hipStream_t s) {
  // twice the blocks that fill every SIMD with eight waves (2048 blocks of 256
  // threads take 68 us where 4096 take 65 and 16384, a row each, 79)
  constexpr int kRows = kGatedThreads<TPR> / TPR;
  constexpr int64_t kMost = 4096 * 256 / kGatedThreads<TPR>;
  const int64_t blocks = ((int64_t)a.T + kRows - 1) / kRows;
  const dim3 grid((unsigned)(blocks < kMost ? blocks : kMost));
  if (a.out8 == kOut8Int8)
    launch_next<R, TPR, NV, kOut8Int8>(a, grid, s);
  else if (a.out8 == kOut8E4m3)
    launch_next<R, TPR, NV, kOut8E4m3>(a, grid, s);
  else
    launch_next<R, TPR, NV, kOut8None>(a, grid, s);
}

template <class R>
void launch_rows(const GatedArgs& a, hipStream_t s) {
  if (a.H <= 128)
    launch_shape<R, 16, 1>(a, s);
  else if (a.H <= 512)
    launch_shape<R, 64, 1>(a, s);
  else if (a.H <= 2048)
    launch_shape<R, 256, 1>(a, s);
  else if (a.H <= 4096)
    launch_shape<R, 512, 1>(a, s);
  else if (a.H <= 8192)
    launch_shape<R, 1024, 1>(a, s);
  else
    launch_shape<R, 1024, kNormMaxH / (1024 * kVec)>(a, s);
}

}  // namespace

hipError_t launch_gated_norm(const GatedArgs& in, hipStream_t s) {
  GatedArgs a = in;
  if (a.group == a.H) a.group = 0;
  if (a.out8_group == a.H) a.out8_group = 0;
  if (a.dtype == kNormBf16)
    launch_rows<RowsBf16>(a, s);
  else if (a.dtype == kNormF16)
    launch_rows<RowsF16>(a, s);
  else
    launch_rows<RowsF32>(a, s);
  return hipGetLastError();
}

}  // namespace moe
