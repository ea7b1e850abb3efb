// The norm after a block (or of its heads) with a gate, the residual add with
// a scale, the norm before the next block, and an 8-bit output (gfx950).
//
//   u = x rsqrt(mean_group(x^2) + eps) (weight + offset)
//   v = residual + scale channel_scale u act(gate),  h = v
//   v = v rsqrt(mean_row(v^2) + next_eps) (next_weight + next_offset),  y = v
//   s = max |v| / Q per 8-bit group,  q = v / s
//
// One pass over memory, as the plain norm does it: a row in the registers of
// 16 to 1024 threads, eight consecutive values a thread and access, every
// sum and v in fp32. A group of 32 to 256 values lies in 4 to 32 neighbouring
// lanes, so the first norm needs no LDS unless it spans the row. The weights
// of the first norm, the channels' scale and the scalar one are one factor a
// value, kept over the rows that a thread takes in turn.
#include <type_traits>

#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

// threads of a block: 256, or those of a longer row
template <int TPR>
constexpr int kGatedThreads = TPR > 256 ? TPR : 256;

// e^z to about an ulp: the part of z log2(e) that its product loses is put
// back as a factor. Below -110 the result is 0 in every use here (1 + e^z).
__device__ inline float exp_full(float z) {
  constexpr float kHi = 1.44269502162933349609375f, kLo = 1.925963033500e-8f;  // log2(e) in two parts
  z = z < -110.f ? -110.f : z;
  const float t = z * kHi, e = __builtin_fmaf(z, kHi, -t) + z * kLo;
  const float p = __builtin_amdgcn_exp2f(t);
  return p < INFINITY ? __builtin_fmaf(p, e * 0.693147181f, p) : p;
}

__device__ inline float sigmoid(float z) { return __builtin_amdgcn_rcpf(1.0f + exp_full(-z)); }

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

}  // namespace

// Block: 256 threads, 256 / TPR rows at a time, or TPR and one; blocks take rows in turn.
// Thread i of a row owns the eight values from (i + TPR j) * 8, j < NV.
template <class R, int TPR, int NV, int OUT8>
__global__ __launch_bounds__(kGatedThreads<TPR>) void gated_norm_kernel(GatedArgs a) {
  typedef typename R::type E;
  __shared__ uint32_t red[16];
  constexpr int kRows = kGatedThreads<TPR> / TPR;
  const int lt = threadIdx.x % TPR, H = a.H;
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
    for (int i = 0; i < kVec; ++i) {
      w[j][i] = a.scale;
      nw[j][i] = 0.f;
    }
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
    if (a.next) eight(a.next_weight, a.weight_f32, c, -1, a.next_offset, nw[j]);
  }
  for (int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TPR; row < a.T; row += (int64_t)gridDim.x * kRows) {
    Eight<E> xv[NV], gv[NV], rv[NV];
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
    E row_gate = E(0);
    if (a.gate_kind) {
      if (a.gate_per_row)
        row_gate = static_cast<const E*>(a.gate)[row * a.ld_gate];
      else
        load(a.gate, a.ld_gate, gv);
    }
    if (a.residual) load(a.residual, a.ld_residual, rv);

    float v[NV][kVec];
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[j][i] = R::get(xv[j].v[i]);
    auto squares = [&](int j) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kVec; ++i) s = __builtin_fmaf(v[j][i], v[j][i], s);
      return s;
    };
    if (a.normalize) {
      if (a.group) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          const float r = 1.0f / sqrtf(group_sum(squares(j), a.group) / (float)a.group + a.eps);
#pragma unroll
          for (int i = 0; i < kVec; ++i) v[j][i] *= r;
        }
      } else {
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j) ss += squares(j);
        ss = __uint_as_float(row_all<TPR>(__float_as_uint(ss), red, add_bits));
        const float r = 1.0f / sqrtf(ss / (float)H + a.eps);
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < kVec; ++i) v[j][i] *= r;
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[j][i] *= w[j][i];
    if (a.gate_kind) {
      const bool silu = a.gate_kind == kGateSilu;
      if (a.gate_per_row) {
        const float z = R::get(row_gate);
        float f = sigmoid(z);
        if (silu) f *= z;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < kVec; ++i) v[j][i] *= f;
      } else {
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
          for (int i = 0; i < kVec; ++i) {
            const float z = R::get(gv[j].v[i]);
            v[j][i] *= sigmoid(z) * (silu ? z : 1.0f);
          }
      }
    }
    if (a.residual) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] += R::get(rv[j].v[i]);
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
    if (a.next) {
      // the sum of squares first: its reduction does not wait for h's stores
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) ss += squares(j);
      if (a.h_out) store(a.h_out, a.ld_h);
      ss = __uint_as_float(row_all<TPR>(__float_as_uint(ss), red, add_bits));
      const float r = 1.0f / sqrtf(ss / (float)H + a.next_eps);
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[j][i] = v[j][i] * r * nw[j][i];
      if (a.y) store(a.y, a.ld_y);
    } else {
      if (a.h_out) store(a.h_out, a.ld_h);
    }
    if constexpr (OUT8 != kOut8None) {
      // |v| as ordered bits: their integer maximum is the largest magnitude,
      // with NaN above infinity (values past the row are left out)
      uint32_t m[NV];
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        m[j] = 0;
#pragma unroll
        for (int i = 0; i < kVec; ++i)
          m[j] = max(m[j], (lt + TPR * j) * kVec + i < H ? __float_as_uint(v[j][i]) & 0x7FFFFFFFu : 0u);
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
        all = row_all<TPR>(all, red, max_bits);
#pragma unroll
        for (int j = 0; j < NV; ++j) m[j] = all;
      }
      uint8_t* q = static_cast<uint8_t*>(a.q) + row * a.ld_q;
      float* scales = a.scales + row * (a.out8_group ? H / a.out8_group : 1);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const int c = (lt + TPR * j) * kVec;
        if (c >= H) continue;
        const Group g = group_of_max<OUT8>(__uint_as_float(m[j]), 1.0f);
        if (a.out8_group ? c % a.out8_group == 0 : c == 0) scales[a.out8_group ? c / a.out8_group : 0] = g.s;
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
void launch_shape(const GatedArgs& a, hipStream_t s) {
  constexpr int kRows = kGatedThreads<TPR> / TPR;
  const int64_t blocks = ((int64_t)a.T + kRows - 1) / kRows;
  const dim3 grid((unsigned)(blocks < 2048 ? blocks : 2048)), block(kGatedThreads<TPR>);
  if (a.out8 == kOut8Int8)
    hipLaunchKernelGGL((gated_norm_kernel<R, TPR, NV, kOut8Int8>), grid, block, 0, s, a);
  else if (a.out8 == kOut8E4m3)
    hipLaunchKernelGGL((gated_norm_kernel<R, TPR, NV, kOut8E4m3>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((gated_norm_kernel<R, TPR, NV, kOut8None>), grid, block, 0, s, a);
}

template <class R>
void launch_rows(const GatedArgs& a, hipStream_t s) {
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
    launch_shape<R, 512, 2>(a, s);
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
