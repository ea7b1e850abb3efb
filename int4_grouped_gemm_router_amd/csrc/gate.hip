// Routing rules beyond the softmax top-8: softmax or sigmoid scores, a bias
// for balance that only selection sees, groups of experts, any top-k up to
// 16, weights renormalised or not, scaled (gfx950).
//
//   score = softmax(l) or 1 / (1 + exp(-l)),  key = score + bias
//   groups ranked by their largest key or the sum of their two largest
//   top-k keys inside the best groups, weight = score (/ sum) * scale
//
// Ranks are decided on keys in 64 bits: with a bias, two keys whose logits
// are far apart can be closer than an fp32 exponential's error, and the
// selected experts must not depend on it.
//
// One wave per token, four experts a lane.
#include "kernels.h"
#include "topk.h"

namespace moe {

namespace {

// Order-preserving 64-bit image of a key (never 0, so 0 can mark an expert
// or group that is out of the running); NaN as -inf, -0 as +0.
__device__ inline uint64_t key_order(double v) {
  if (!(v == v)) v = -INFINITY;
  if (v == 0.0) v = 0.0;
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
constexpr uint64_t kMaskedKey = 0x000FFFFFFFFFFFFFull;  // key_order(-inf)

__device__ inline double key_value(uint64_t o) {
  return __longlong_as_double((long long)(o >> 63 ? o & 0x7FFFFFFFFFFFFFFFull : ~o));
}

// Largest key over the wave, ties to the lower index, returned to every lane.
__device__ inline void wave_best(uint64_t& k, int& i) {
  for (int o = 1; o < 64; o <<= 1) {
    const uint64_t ok = __shfl_xor((unsigned long long)k, o);
    const int oi = __shfl_xor(i, o);
    if (ok > k || (ok == k && oi < i)) {
      k = ok;
      i = oi;
    }
  }
}

__device__ inline double wave_sum_f64(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

}  // namespace

__global__ __launch_bounds__(256) void gate_topk_kernel(GateArgs a) {
  const int lane = threadIdx.x & 63;
  const int t = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.T) return;
  const int E = a.E, k = a.k;
  double score[4];
  uint64_t key[4];
  float l[4];
  float mx = -INFINITY;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    l[i] = -INFINITY;
    if (e < E) {
      float v = 0.f;
      for (int sp = 0; sp < a.splits; ++sp) v += a.partial[((int64_t)sp * a.T + t) * E + e];
      if (a.rbias) v += a.rbias[e];
      if (a.logits_out) a.logits_out[(int64_t)t * E + e] = v;
      l[i] = v == v ? v : -INFINITY;
    }
    mx = fmaxf(mx, l[i]);
  }
  for (int o = 1; o < 64; o <<= 1) mx = fmaxf(mx, __shfl_xor(mx, o));
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (l[i] == -INFINITY)
      score[i] = 0.0;
    else if (a.sigmoid)
      score[i] = 1.0 / (1.0 + exp(-(double)l[i]));
    else
      score[i] = l[i] == mx ? 1.0 : exp((double)l[i] - (double)mx);
    sum += score[i];
  }
  if (!a.sigmoid) {
    sum = wave_sum_f64(sum);
#pragma unroll
    for (int i = 0; i < 4; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int e = lane + 64 * i;
    key[i] = 0;
    if (e < E) {
      key[i] = l[i] == -INFINITY ? kMaskedKey : key_order(score[i] + (a.balance ? (double)a.balance[e] : 0.0));
      if (key[i] == kMaskedKey) score[i] = 0.0;
    }
  }
  if (a.n_groups > 1) {
    const int size = E / a.n_groups;
    uint64_t mine = 0;  // lane g: the rank key of group g
    for (int g = 0; g < a.n_groups; ++g) {
      auto best_but = [&](int skip, int& at) {
        uint64_t b = 0;
        at = E;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = lane + 64 * i;
          if (e < E && e / size == g && e != skip && key[i] > b) {
            b = key[i];
            at = e;
          }
        }
        wave_best(b, at);
        return b;
      };
      int at, at2;
      uint64_t b = best_but(-1, at);
      if (a.group_top2) {
        const uint64_t b2 = best_but(at, at2);
        if (b2 > kMaskedKey) b = key_order(key_value(b) + key_value(b2));
      }
      if (lane == g) mine = b;
    }
    uint64_t kept = 0;
    for (int r = 0; r < a.topk_groups; ++r) {
      uint64_t b = mine;
      int at = lane;
      wave_best(b, at);
      kept |= 1ull << at;
      if (lane == at) mine = 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = lane + 64 * i;
      if (e < E && !(kept >> (e / size) & 1)) key[i] = 0;
    }
  }
  int sel = 0;
  double sel_score = 0.0;
  for (int r = 0; r < k; ++r) {
    uint64_t b = 0;
    int at = E;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (key[i] > b) {
        b = key[i];
        at = lane + 64 * i;
      }
    wave_best(b, at);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at == lane + 64 * i) {
        s = score[i];
        key[i] = 0;
      }
    s = __shfl(s, at & 63);
    if (lane == r) {
      sel = at;
      sel_score = s;
    }
  }
  const double z = wave_sum_f64(lane < k ? sel_score : 0.0);
  if (lane < k) {
    const int64_t pair = (int64_t)t * k + lane;
    double w = sel_score;
    if (a.renorm) w = z > 0.0 ? w / z : 0.0;
    a.topk_idx[pair] = sel;
    a.topk_w[pair] = (float)(w * (double)a.scale);
    if (a.chunk_hist) atomicAdd(&a.chunk_hist[(pair / kChunkPairs) * E + sel], 1);
  }
}

hipError_t launch_gate_topk(const GateArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(gate_topk_kernel, dim3((a.T + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
