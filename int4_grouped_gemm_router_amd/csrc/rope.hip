// Rotary positions for queries and keys (gfx950).
//
// A pair (a, b) of a head turns by position * frequency:
//   a' = m (a cos - b sin),  b' = m (a sin + b cos)
// Frequencies are whole numbers of 2^-64 turns, so the product with a position
// taken modulo 2^64 is the angle modulo one turn without any rounding, however
// far the position; its upper 32 bits (2^-32 turns) are split into a quarter
// and a rest of at most an eighth of a turn, where the Taylor series of sine
// and cosine to x^9 and x^10 err by less than 3e-9.
//
// Memory bounds long calls (16384 tokens of 40 heads of 128: 72 us, 4.6 TB/s),
// one load and one store's latency short ones (4.2 us for one token). A thread
// owns eight pairs of a token (eight values from each half, or sixteen
// neighbouring ones) and, in long calls, four heads, over which it uses the
// eight angles; the values behind the turned part are copied sixteen at a time
// where the output is another buffer.
#include "kernels.h"
#include "rows.h"

namespace moe {

namespace {

constexpr int kRopeThreads = 256;

struct Turn {
  float c, s;
};

__device__ inline Turn turn_of(uint64_t freq, int32_t position, float magnitude, uint32_t flip) {
  const uint32_t u = (uint32_t)((freq * (uint64_t)(int64_t)position) >> 32);
  const uint32_t quarter = (u + 0x20000000u) >> 30;
  const float x = (float)(int32_t)(u - (quarter << 30)) * 1.46291807926715968e-9f;  // 2 pi 2^-32
  const float x2 = x * x;
  float s = 2.75573192e-6f, c = -2.75573192e-7f;  // 1 / 9!, -1 / 10!
  s = __builtin_fmaf(s, x2, -1.98412698e-4f);
  c = __builtin_fmaf(c, x2, 2.48015873e-5f);
  s = __builtin_fmaf(s, x2, 8.33333333e-3f);
  c = __builtin_fmaf(c, x2, -1.38888889e-3f);
  s = __builtin_fmaf(s, x2, -1.66666667e-1f);
  c = __builtin_fmaf(c, x2, 4.16666667e-2f);
  s = __builtin_fmaf(s * x2, x, x);
  c = __builtin_fmaf(c, x2, -0.5f);
  c = __builtin_fmaf(c, x2, 1.0f);
  const bool odd = quarter & 1;
  float cs = odd ? s : c, sn = odd ? c : s;
  cs *= magnitude;
  sn *= magnitude;
  // quarters 1 and 2 have a negative cosine, 2 and 3 (the last two) a negative sine
  Turn t;
  t.c = __uint_as_float(__float_as_uint(cs) ^ ((quarter + 1) << 30 & 0x80000000u));
  t.s = __uint_as_float(__float_as_uint(sn) ^ ((quarter << 30 & 0x80000000u) ^ flip));
  return t;
}

}  // namespace

// Thread: unit `u` (eight pairs, or sixteen copied values) of heads hb * HPT ..
// of token t; the units of a head are neighbours.
template <class R, int HPT, bool INTER>
__global__ __launch_bounds__(kRopeThreads) void rope_kernel(RopeArgs a) {
  typedef typename R::type E;
  const uint32_t id = blockIdx.x * kRopeThreads + threadIdx.x;
  if (id >= a.items) return;
  // id / per_token and its rest / units, by a product that is short by one at most
  uint32_t t = __umulhi(id, a.per_token_magic), rest = id - t * a.per_token;
  if (rest >= a.per_token) {
    ++t;
    rest -= a.per_token;
  }
  uint32_t hb = __umulhi(rest, a.units_magic), u = rest - hb * a.units;
  if (u >= a.units) {
    ++hb;
    u -= a.units;
  }
  const int heads = a.heads[0] + a.heads[1], half = a.rot >> 1;
  const E* src[HPT];
  E* dst[HPT];
  bool on[HPT];
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    const int h = (int)hb * HPT + j;
    const int k = h >= a.heads[0];
    on[j] = h < heads;
    const int64_t at = (int64_t)(h - (k ? a.heads[0] : 0)) * a.D;
    src[j] = static_cast<const E*>(a.x[k]) + (int64_t)t * a.ldx[k] + at;
    dst[j] = static_cast<E*>(a.y[k]) + (int64_t)t * a.ldy[k] + at;
    if (u >= (uint32_t)a.turn_units && !a.copy[k]) on[j] = false;
  }
  if (u >= (uint32_t)a.turn_units) {
    const int c = a.rot + 16 * ((int)u - a.turn_units);
    if (c + 16 <= a.D) {
      Eight<E> lo[HPT], hi[HPT];
#pragma unroll
      for (int j = 0; j < HPT; ++j)
        if (on[j]) {
          lo[j] = *reinterpret_cast<const Eight<E>*>(src[j] + c);
          hi[j] = *reinterpret_cast<const Eight<E>*>(src[j] + c + 8);
        }
#pragma unroll
      for (int j = 0; j < HPT; ++j)
        if (on[j]) {
          *reinterpret_cast<Eight<E>*>(dst[j] + c) = lo[j];
          *reinterpret_cast<Eight<E>*>(dst[j] + c + 8) = hi[j];
        }
    } else {
#pragma unroll
      for (int j = 0; j < HPT; ++j)
        for (int i = c; on[j] && i < a.D; ++i) dst[j][i] = src[j][i];
    }
    return;
  }
  const int p0 = 8 * (int)u, n = min(8, half - p0);
  const int at0 = INTER ? 2 * p0 : p0, at1 = INTER ? at0 + 8 : half + p0;
  Eight<E> x0[HPT], x1[HPT];
  if (n == 8) {
#pragma unroll
    for (int j = 0; j < HPT; ++j)
      if (on[j]) {
        x0[j] = *reinterpret_cast<const Eight<E>*>(src[j] + at0);
        x1[j] = *reinterpret_cast<const Eight<E>*>(src[j] + at1);
      }
  } else {
    // value i of the sixteen belongs to the turned part
#pragma unroll
    for (int j = 0; j < HPT; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const bool in0 = INTER ? i < 2 * n : i < n, in1 = INTER ? i + 8 < 2 * n : i < n;
        x0[j].v[i] = on[j] && in0 ? src[j][at0 + i] : E(0);
        x1[j].v[i] = on[j] && in1 ? src[j][at1 + i] : E(0);
      }
  }
  const int32_t position = a.positions[t];
  Turn turn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) turn[i] = turn_of(a.turns[min(p0 + i, half - 1)], position, a.magnitude, a.flip);
#pragma unroll
  for (int j = 0; j < HPT; ++j) {
    if (!on[j]) continue;
    Eight<E> y0, y1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float p = R::get(INTER ? (i < 4 ? x0[j].v[2 * i & 7] : x1[j].v[2 * i & 7]) : x0[j].v[i]);
      const float q = R::get(INTER ? (i < 4 ? x0[j].v[(2 * i & 7) + 1] : x1[j].v[(2 * i & 7) + 1]) : x1[j].v[i]);
      const E r0 = R::put(__builtin_fmaf(p, turn[i].c, -(q * turn[i].s)));
      const E r1 = R::put(__builtin_fmaf(p, turn[i].s, q * turn[i].c));
      if (INTER) {
        (i < 4 ? y0 : y1).v[2 * i & 7] = r0;
        (i < 4 ? y0 : y1).v[(2 * i & 7) + 1] = r1;
      } else {
        y0.v[i] = r0;
        y1.v[i] = r1;
      }
    }
    if (n == 8) {
      *reinterpret_cast<Eight<E>*>(dst[j] + at0) = y0;
      *reinterpret_cast<Eight<E>*>(dst[j] + at1) = y1;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (INTER ? i < 2 * n : i < n) dst[j][at0 + i] = y0.v[i];
        if (INTER ? i + 8 < 2 * n : i < n) dst[j][at1 + i] = y1.v[i];
      }
    }
  }
}

namespace {

template <class R, int HPT>
void launch_heads(const RopeArgs& a, hipStream_t s) {
  const dim3 grid((a.items + kRopeThreads - 1) / kRopeThreads), block(kRopeThreads);
  if (a.interleaved)
    hipLaunchKernelGGL((rope_kernel<R, HPT, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((rope_kernel<R, HPT, false>), grid, block, 0, s, a);
}

template <class R>
void launch_type(const RopeArgs& a, int hpt, hipStream_t s) {
  if (hpt == 4)
    launch_heads<R, 4>(a, s);
  else
    launch_heads<R, 1>(a, s);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& in, hipStream_t s) {
  RopeArgs a = in;
  const int heads = a.heads[0] + a.heads[1];
  a.turn_units = (a.rot / 2 + 7) / 8;
  a.units = a.turn_units + (a.copy[0] || a.copy[1] ? (a.D - a.rot + 15) / 16 : 0);
  // four heads a thread once there are threads enough for every compute unit
  const int hpt = heads >= 4 && (int64_t)a.T * heads * a.units >= 4 * 256 * 256 ? 4 : 1;
  const int blocks = (heads + hpt - 1) / hpt;
  a.per_token = (uint32_t)blocks * a.units;
  a.per_token_magic = (uint32_t)(((uint64_t(1) << 32) - (a.per_token == 1)) / a.per_token);
  a.units_magic = (uint32_t)(((uint64_t(1) << 32) - (a.units == 1)) / a.units);
  const size_t eb = a.dtype == kNormF32 ? 4 : 2;
  const int64_t total = a.T, most = (int64_t(1) << 31) / a.per_token;  // tokens of a launch
  for (int64_t t0 = 0; t0 < total; t0 += most) {
    RopeArgs c = a;
    c.T = (int)(total - t0 < most ? total - t0 : most);
    c.items = (uint32_t)c.T * c.per_token;
    c.positions += t0;
    for (int i = 0; i < 2; ++i) {
      c.x[i] = static_cast<const char*>(c.x[i]) + t0 * c.ldx[i] * eb;
      c.y[i] = static_cast<char*>(c.y[i]) + t0 * c.ldy[i] * eb;
    }
    if (a.dtype == kNormBf16)
      launch_type<RowsBf16>(c, hpt, s);
    else if (a.dtype == kNormF16)
      launch_type<RowsF16>(c, hpt, s);
    else
      launch_type<RowsF32>(c, hpt, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
