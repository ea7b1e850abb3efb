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
// selected experts must not depend on it. Nearly every token is settled in
// fp32 all the same: the fp32 keys carry a bound on their error, and only a
// token with two candidates closer than it at a rank that matters (well under
// one in a hundred) is decided again in 64 bits.
//
// Kernels:
//   gate_topk     sixteen lanes per token, four tokens a wave; for
//                 moe_route_gated also the expert counts of each block
//   gate_scatter  per piece of tokens: totals and bases per expert from those
//                 counts, a stable scatter, and a share of the block map
//   gate_small    both in one block, for up to kGateSmallT tokens
#include "kernels.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kGateWaves = 16;
constexpr int kGateThreads = 64 * kGateWaves;
constexpr int kScatterTokens = 128;  // tokens per scatter block
constexpr int kScatterBlocks = 512;
constexpr int kGateSmallT = 64;

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

// Largest key over the wave and its index, returned to every lane; ties to the
// lowest lane, whose index has to be the lowest too. (Two 32-bit maxima over
// the lanes; shuffles of the 64-bit keys took seven times as long, which a
// late wave in doubt adds to the whole launch.)
__device__ inline void wave_best(uint64_t& k, int& i) {
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  const uint32_t mh = wave_max_u32(hi), ml = wave_max_u32(hi == mh ? lo : 0u);
  const uint64_t best = (uint64_t)mh << 32 | ml;
  const int win = __builtin_ctzll(__ballot(k == best));
  i = __builtin_amdgcn_readlane(i, win);
  k = best;
}

__device__ inline double wave_sum_f64(double v) {
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// Reductions over the 16 lanes of a row, returned to each of them: lane ^ 1,
// lane ^ 2, mirror within 8, mirror within 16.
template <class F>
__device__ inline float row_reduce(float v, F f) {
  v = f(v, __uint_as_float(dpp<0xB1>(__float_as_uint(v))));
  v = f(v, __uint_as_float(dpp<0x4E>(__float_as_uint(v))));
  v = f(v, __uint_as_float(dpp<0x141>(__float_as_uint(v))));
  return f(v, __uint_as_float(dpp<0x140>(__float_as_uint(v))));
}
__device__ inline float row_max(float v) {
  return row_reduce(v, [](float x, float y) { return fmaxf(x, y); });
}
__device__ inline float row_min(float v) {
  return row_reduce(v, [](float x, float y) { return fminf(x, y); });
}
__device__ inline float row_sum(float v) {
  return row_reduce(v, [](float x, float y) { return x + y; });
}
__device__ inline uint32_t row_max_u32(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  return max(v, dpp<0x140>(v));
}
template <int CTRL>
__device__ inline double dpp_f64(double v) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = dpp<CTRL>((uint32_t)u), hi = dpp<CTRL>((uint32_t)(u >> 32));
  return __longlong_as_double((long long)(hi << 32 | lo));
}
__device__ inline double row_sum_f64(double v) {
  v += dpp_f64<0xB1>(v);
  v += dpp_f64<0x4E>(v);
  v += dpp_f64<0x141>(v);
  return v + dpp_f64<0x140>(v);
}

// Group of expert e: e / size as the high half of e * ceil(2^32 / size), exact
// for e < 256 (size 1 has no such factor).
__device__ inline int group_of(const GateArgs& a, int e) {
  return a.group_size == 1 ? e : (int)__umulhi((uint32_t)e, a.group_magic);
}

// One token's selection in 64 bits: lane j < k gets the expert of rank j and
// its weight. l: the lane's logits (-inf: masked), b: their biases; kept: per
// group whether it is kept, or null where that is to be decided too.
__device__ void gate_select_exact(const GateArgs& a, const float (&l)[4], const float (&b)[4], float mx,
                                  const uint8_t* kept_groups, int& sel, float& w) {
  const int lane = threadIdx.x & 63, E = a.E, k = a.k;
  double score[4];
  uint64_t key[4];
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
    key[i] = 0;
    if (4 * lane + i < E) {
      key[i] = l[i] == -INFINITY ? kMaskedKey : key_order(score[i] + (double)b[i]);
      if (key[i] == kMaskedKey) score[i] = 0.0;
    }
  }
  if (a.n_groups > 1 && kept_groups) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (e < E && !kept_groups[group_of(a, e)]) key[i] = 0;
    }
  } else if (a.n_groups > 1) {
    uint64_t mine = 0;  // lane g: the rank key of group g
    for (int g = 0; g < a.n_groups; ++g) {
      auto best_but = [&](int skip, int& at) {
        uint64_t best = 0;
        at = E;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * lane + i;
          if (e < E && group_of(a, e) == g && e != skip && key[i] > best) {
            best = key[i];
            at = e;
          }
        }
        wave_best(best, at);
        return best;
      };
      int at, at2;
      uint64_t best = best_but(-1, at);
      if (a.group_top2) {
        const uint64_t second = best_but(at, at2);
        if (second > kMaskedKey) best = key_order(key_value(best) + key_value(second));
      }
      if (lane == g) mine = best;
    }
    uint64_t kept = 0;
    for (int r = 0; r < a.topk_groups; ++r) {
      uint64_t best = mine;
      int at = lane;
      wave_best(best, at);
      kept |= 1ull << at;
      if (lane == at) mine = 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (e < E && !(kept >> group_of(a, e) & 1)) key[i] = 0;
    }
  }
  double sel_score = 0.0;
  sel = 0;
  for (int r = 0; r < k; ++r) {
    uint64_t best = 0;
    int at = E;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (key[i] > best) {
        best = key[i];
        at = 4 * lane + i;
      }
    wave_best(best, at);
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at == 4 * lane + i) {
        s = score[i];
        key[i] = 0;
      }
    s = __shfl(s, at >> 2);
    if (lane == r) {
      sel = at;
      sel_score = s;
    }
  }
  const double z = wave_sum_f64(lane < k ? sel_score : 0.0);
  double v = sel_score;
  if (a.renorm) v = z > 0.0 ? v / z : 0.0;
  w = (float)(v * (double)a.scale);
}

// The sum over the router's K splits plus the router's bias: logits of token
// t, four consecutive experts from e on (the last four, or the last one
// repeated, where e is past the end: no branch separates the loads).
__device__ inline void load_logits(const GateArgs& a, int64_t t, int e, float (&v)[4]) {
  const int E = a.E;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = 0.f;
  if (a.vectors) {
    for (int sp = 0; sp < a.splits; ++sp) {
      const f32x4 p = *reinterpret_cast<const f32x4*>(a.partial + ((int64_t)sp * a.T + t) * E + min(e, E - 4));
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += p[i];
    }
  } else {
    for (int sp = 0; sp < a.splits; ++sp)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += a.partial[((int64_t)sp * a.T + t) * E + min(e + i, E - 1)];
  }
  if (a.rbias) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += a.rbias[min(e + i, E - 1)];
  }
}

// A wave's own LDS, per token: the keys for the groups (one word of padding
// per sixteen spreads the groups over the banks), the groups' rank keys and
// whether they are kept; then the logits.
struct SelectLds {
  float v[4][256 + 16];
  float group[4][kMaxGateGroups];
  uint8_t kept[4][kMaxGateGroups];
};
__device__ inline int key_at(int e) { return e + (e >> 4); }

// Four tokens' selections, t0 + lane / 16 each: lane c = lane % 16 < k gets
// the expert of rank c and its weight. Lane c holds the experts
// 64 j + 4 c + u (j < NJ, u < 4) of its token. KD: at least min(k, 15) + 1.
template <int NJ, int KD>
__device__ void gate_select(const GateArgs& a, int t0, SelectLds& L, int& sel, float& w) {
  constexpr int NS = 4 * NJ;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int E = a.E, k = a.k;
  const int64_t t = min(t0 + q, a.T - 1);
  float l[NS], b[NS], lv[NJ][4];
#pragma unroll
  for (int j = 0; j < NJ; ++j) load_logits(a, t, 64 * j + 4 * c, lv[j]);
#pragma unroll
  for (int i = 0; i < NS; ++i) b[i] = 0.f;
  if (a.balance) {
#pragma unroll
    for (int i = 0; i < NS; ++i) b[i] = a.balance[min(64 * (i >> 2) + 4 * c + (i & 3), E - 1)];
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const float(&v)[4] = lv[j];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = 64 * j + 4 * c + u;
      l[4 * j + u] = (e < E) & (v[u] == v[u]) ? v[u] : -INFINITY;
    }
    if (a.logits_out && t0 + q < a.T) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (64 * j + 4 * c + u < E) a.logits_out[t * E + 64 * j + 4 * c + u] = v[u];
    }
  }
  float mx = l[0];
#pragma unroll
  for (int i = 1; i < NS; ++i) mx = fmaxf(mx, l[i]);
  mx = row_max(mx);
  // fp32 scores with the hardware exponential and reciprocal. Errors, with
  // u = 2^-24: the exponent's product and the difference to the maximum round
  // by u of their size, which moves e^-d by at most u d e^-d < u / 2; the
  // exponential, the reciprocal and the quotient add 2 u of the value each,
  // the softmax's sum, added in pairs, 8 u, and the bias's addition u of the
  // key. Of the range, largest score + largest bias, that is below 16 u with
  // a softmax and below 8 u with a sigmoid, whose derivative is at most 1/4.
  float s[NS], top = 1.0f;
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));  // (-inf: 1 / inf)
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float p = __expf(l[i] == mx ? 0.f : l[i] - mx);
      s[i] = l[i] == -INFINITY ? 0.f : p;
    }
    float z[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) z[i] = s[i];
#pragma unroll
    for (int n = NS / 2; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] += z[i + n];
    const float sum = row_sum(z[0]);
    top = sum > 0.f ? 1.0f / sum : 0.f;
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] *= top;
  }
  float bmax = 0.f;  // the largest |bias| (a NaN is the largest of all, and leaves every token in doubt)
  if (a.balance) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) m = max(m, __float_as_uint(b[i]) & 0x7FFFFFFFu);
    bmax = __uint_as_float(row_max_u32(m));
  }
  const float range = top + bmax;
  const float err = (a.sigmoid ? 0x1p-21f : 0x1p-20f) * range;
  // a decision the fp32 keys cannot settle, and whether it is one of groups
  bool near = !(range < 1e30f), near_groups = near;
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    s[i] = l[i] == -INFINITY ? -INFINITY : s[i] + b[i];
    if (!(s[i] == s[i])) s[i] = -INFINITY;
  }
  uint32_t in = ~0u;  // bit i: expert i's group is kept
  if (a.n_groups > 1) {
    // group g: 2^lg lanes (up to sixteen groups), or lane g % 16
    const int size = a.group_size, lg = a.group_lanes_log2, p = c & ((1 << lg) - 1);
#pragma unroll
    for (int i = 0; i < NS; ++i) L.v[q][key_at(64 * (i >> 2) + 4 * c + (i & 3))] = s[i];
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    float lo = INFINITY, hi = -INFINITY;
    for (int g = c >> lg; g < a.n_groups; g += 16) {
      float m1 = -INFINITY, m2 = -INFINITY;
      constexpr int kReads = 8;  // under way at once
      for (int i0 = p; i0 < size; i0 += kReads << lg) {
        float v[kReads];
#pragma unroll
        for (int j = 0; j < kReads; ++j) v[j] = L.v[q][key_at(g * size + min(i0 + (j << lg), size - 1))];
#pragma unroll
        for (int j = 0; j < kReads; ++j) {
          const float x = i0 + (j << lg) < size ? v[j] : -INFINITY;
          m2 = fmaxf(m2, fminf(m1, x));
          m1 = fmaxf(m1, x);
        }
      }
      // over the group's lanes (all that hold a part agree after each step)
      auto join = [&](uint32_t o1, uint32_t o2) {
        const float x1 = __uint_as_float(o1), x2 = __uint_as_float(o2);
        m2 = fmaxf(fmaxf(m2, x2), fminf(m1, x1));
        m1 = fmaxf(m1, x1);
      };
      const auto u = [](float f) { return __float_as_uint(f); };
      if (lg >= 1) join(dpp<0xB1>(u(m1)), dpp<0xB1>(u(m2)));
      if (lg >= 2) join(dpp<0x4E>(u(m1)), dpp<0x4E>(u(m2)));
      if (lg >= 3) join(dpp<0x141>(u(m1)), dpp<0x141>(u(m2)));
      if (lg >= 4) join(dpp<0x140>(u(m1)), dpp<0x140>(u(m2)));
      if (p == 0) L.group[q][g] = a.group_top2 && m2 > -INFINITY ? m1 + m2 : m1;
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    for (int g = c; g < a.n_groups; g += 16) {
      const float mine = L.group[q][g];
      int rank = 0;
      for (int o0 = 0; o0 < a.n_groups; o0 += 8) {
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = L.group[q][min(o0 + j, a.n_groups - 1)];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int o = o0 + j;
          rank += (o < a.n_groups) & ((v[j] > mine) | ((v[j] == mine) & (o < g)));
        }
      }
      const bool kept = rank < a.topk_groups;
      L.kept[q][g] = kept;
      if (kept)
        lo = fminf(lo, mine);
      else
        hi = fmaxf(hi, mine);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    lo = row_min(lo);
    hi = row_max(hi);
    near_groups |= hi > -INFINITY && !(lo - hi > 4.0f * err);
    near |= near_groups;
    in = 0u;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const int e = 64 * (i >> 2) + 4 * c + (i & 3);
      const uint32_t kept = L.kept[q][group_of(a, min(e, E - 1))];
      in |= (e < E ? kept : 0u) << i;
    }
  }
  // keys as 24-bit fixed point over the range (0: masked or out of the
  // running), then the lane's slot and the lane: all keys of a token differ
  const float scale = 16777000.0f / (range + bmax);
  uint32_t key[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const bool out = (s[i] == -INFINITY) | !(in >> i & 1);
    const uint32_t v = out ? 0u : 1u + (uint32_t)(fmaxf(s[i] + bmax, 0.f) * scale);
    key[i] = v << 8 | (uint32_t)(i << 4) | (uint32_t)c;
  }
  // the lane's keys in descending order
#pragma unroll
  for (int n = 2; n <= NS; n *= 2)
#pragma unroll
    for (int j = n / 2; j > 0; j /= 2)
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int o = i ^ j;
        if (o > i) {
          const uint32_t x = max(key[i], key[o]), y = min(key[i], key[o]);
          key[i] = (i & n) == 0 ? x : y;
          key[o] = (i & n) == 0 ? y : x;
        }
      }
  // k + 1 rounds: the row's largest head; its lane drops it
  constexpr int ND = NS < KD ? NS : KD;
  uint32_t mine = 0, next = 0;  // the keys of rank c and c + 1
  for (int r = 0; r <= k; ++r) {
    const uint32_t m = row_max_u32(key[0]);
    mine = c == r ? m : mine;
    next = c == r - 1 ? m : next;
    const bool own = key[0] == m;
#pragma unroll
    for (int i = 0; i + 1 < ND; ++i) key[i] = own ? key[i + 1] : key[i];
    if constexpr (ND == NS) key[NS - 1] = own ? 0u : key[NS - 1];
  }
  // twice the bound in steps of the fixed point (16 u of the range is at most
  // 16 of the 2^24 steps over range + bias), and what the steps cut off
  const uint32_t close = (a.sigmoid ? 16 : 32) + 4;
  const uint32_t vm = mine >> 8, vn = next >> 8;
  if (c < k) near |= vm == 0 || (vn > 0 && vm - vn <= close);
  sel = 64 * (int)(mine >> 6 & 3) + 4 * (int)(mine & 15) + (int)(mine >> 4 & 3);
  // the weights in 64 bits from the selected logits; where the fp32 sum over
  // the experts is used (softmax, not renormalised) it errs by a few 2^-24
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    *reinterpret_cast<f32x4*>(&L.v[q][64 * j + 4 * c]) = f32x4{l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]};
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  double v = 0.0;
  if (c < k) {
    const float x = L.v[q][sel];
    const double e = exp(a.sigmoid ? -(double)x : (x == mx ? 0.0 : (double)x - (double)mx));
    v = a.sigmoid ? 1.0 / (1.0 + e) : e;
  }
  if (a.renorm) {
    const double sum = row_sum_f64(v);
    v = sum > 0.0 ? v / sum : 0.0;
  } else if (!a.sigmoid) {
    v *= (double)top;
  }
  w = (float)(v * (double)a.scale);
  // in doubt: those tokens again, one at a time
  uint64_t doubt = __ballot(near && t0 + q < a.T);
  const uint64_t doubt_groups = __ballot(near_groups);
  while (doubt) {
    const int row = __builtin_ctzll(doubt) >> 4;
    doubt &= ~(0xFFFFull << (16 * row));
    float l4[4], b4[4], top4;
    load_logits(a, t0 + row, 4 * lane, l4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (!(e < E && l4[i] == l4[i])) l4[i] = -INFINITY;
      b4[i] = a.balance && e < E ? a.balance[e] : 0.f;
    }
    top4 = __shfl(mx, 16 * row);
    int se;
    float we;
    gate_select_exact(a, l4, b4, top4, doubt_groups >> (16 * row) & 0xFFFF ? nullptr : L.kept[row], se, we);
    se = __shfl(se, c);
    we = __shfl(we, c);
    if (q == row) {
      sel = se;
      w = we;
    }
  }
}

// Exclusive prefix sum of v over the first 256 threads of the block (total in
// every thread); every thread calls it.
__device__ inline int scan256(int v, int* scratch /* 4 ints */, int& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int inc = v;
  for (int o = 1; o < 64; o <<= 1) {
    const int n = __shfl_up(inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 63 && wave < 4) scratch[wave] = inc;
  __syncthreads();
  int base = 0;
  total = 0;
  for (int w = 0; w < 4; ++w) {
    if (w < wave) base += scratch[w];
    total += scratch[w];
  }
  __syncthreads();
  return base + inc - v;
}

struct PlaceLds {
  int at[kGateWaves][256];  // per wave and expert: pairs, then the next position
  int base[256];            // first position of each expert's pairs of this block
  int scratch[4];
};

// Stable scatter of n pairs (first pair p0, experts pe) of one block, in
// L.base order: wave w places a contiguous piece of them.
__device__ inline void place_pairs(const GateScatter& a, PlaceLds& L, const int32_t* pe, int p0, int n) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int piece = (n + 64 * kGateWaves - 1) / (64 * kGateWaves) * 64;
  const int f = min(wave * piece, n), end = min(f + piece, n);
  for (int i = tid; i < kGateWaves * 256; i += kGateThreads) (&L.at[0][0])[i] = 0;
  __syncthreads();
  for (int i = f + lane; i < end; i += 64) atomicAdd(&L.at[wave][pe[i]], 1);
  __syncthreads();
  if (tid < a.E) {
    int c[kGateWaves], run = L.base[tid];
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) c[w] = L.at[w][tid];
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) {
      L.at[w][tid] = run;
      run += c[w];
    }
  }
  __syncthreads();
  for (int i = f + lane; i < end; i += 64) {
    const int e = pe[i];
    const uint64_t peers = match_any((uint32_t)e, 8);
    const int rank = __popcll(peers & lanemask_lt());
    const int pos = L.at[wave][e] + rank;
    a.perm[pos] = p0 + i;
    a.inv_perm[p0 + i] = pos;
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    if (rank == 0) L.at[wave][e] += __popcll(peers);
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  }
}

// Histogram, offsets and block map from each expert's total (thread e < E:
// tot, and off, its first position); block b of nb writes the map entries of
// experts b, b + nb, ...; block 0 the rest. Every thread calls it.
__device__ inline void write_map(const GateScatter& a, PlaceLds& L, int tot, int off, int pairs, int b, int nb) {
  const int tid = threadIdx.x, E = a.E;
  int blocks_total;
  const int blocks = tid < E ? (tot + a.block_m - 1) / a.block_m : 0;
  const int first = scan256(blocks, L.scratch, blocks_total);
  if (b == 0) {
    if (tid < E) {
      a.hist[tid] = tot;
      a.offsets[tid] = off;
    }
    if (tid == 0) {
      a.offsets[E] = pairs;
      *a.num_blocks = blocks_total;
    }
  }
  if (tid < E && tid % nb == b)
    for (int i = 0; i < blocks; ++i) {
      int* m = a.block_map + 3 * (int64_t)(first + i);
      m[0] = tid;
      m[1] = off + i * a.block_m;
      m[2] = min(a.block_m, tot - i * a.block_m);
    }
}

}  // namespace

// Grid: ceil(T / (4 W)). Block: W waves, four tokens each. COUNTS: the block
// writes its row of expert counts [grid][256] bytes (at most 64 each);
// otherwise counts are added to chunk_hist (when given).
template <int NJ, int KD, int W, bool COUNTS>
__global__ __launch_bounds__(64 * W) void gate_topk_kernel(GateArgs a) {
  __shared__ SelectLds L[W];
  __shared__ int cnt[COUNTS ? 256 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15;
  if constexpr (COUNTS) {
    if (tid < 256) cnt[tid] = 0;
    __syncthreads();
  }
  const int t0 = (blockIdx.x * W + wave) * 4, t = t0 + (lane >> 4);
  if (t0 < a.T) {
    int sel;
    float w;
    gate_select<NJ, KD>(a, t0, L[wave], sel, w);
    if (t < a.T && c < a.k) {
      const int64_t pair = (int64_t)t * a.k + c;
      a.topk_idx[pair] = sel;
      a.topk_w[pair] = w;
      if constexpr (COUNTS)
        atomicAdd(&cnt[sel], 1);
      else if (a.chunk_hist)
        atomicAdd(&a.chunk_hist[(pair / kChunkPairs) * a.E + sel], 1);
    }
  }
  if constexpr (COUNTS) {
    __syncthreads();
    if (tid < 256) a.counts[(int64_t)blockIdx.x * 256 + tid] = (uint8_t)cnt[tid];
  }
}

// Block: 16 waves, `pieces` consecutive pieces of 128 tokens. Every block sums
// all rows of counts (256 rows of 256 bytes for 4096 and for 16384 tokens), a
// wave a row at a time, a lane four experts.
__global__ __launch_bounds__(kGateThreads) void gate_scatter_kernel(GateScatter a) {
  __shared__ PlaceLds L;
  __shared__ int32_t pe[kScatterTokens * kMaxGateK];
  __shared__ int part[2][kGateWaves][256];  // [total, before][wave]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, step = kScatterTokens * a.k;
  const int p0 = blockIdx.x * a.pieces * step, end = min(p0 + a.pieces * step, a.T * a.k);
  const int rows = (a.T + a.count_tokens - 1) / a.count_tokens;
  const int mine = blockIdx.x * a.pieces * (kScatterTokens / a.count_tokens);
  {
    int tot[4] = {0, 0, 0, 0}, bef[4] = {0, 0, 0, 0};
    constexpr int kRows = 8;  // loads under way
    for (int r0 = wave; r0 < rows; r0 += kRows * kGateWaves) {
      uint32_t v[kRows];
#pragma unroll
      for (int j = 0; j < kRows; ++j)
        v[j] = *reinterpret_cast<const uint32_t*>(a.counts + (int64_t)min(r0 + kGateWaves * j, rows - 1) * 256 + 4 * lane);
#pragma unroll
      for (int j = 0; j < kRows; ++j) {
        const int r = r0 + kGateWaves * j;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int x = r < rows ? (int)(v[j] >> (8 * h) & 0xFFu) : 0;
          tot[h] += x;
          bef[h] += r < mine ? x : 0;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      part[0][wave][4 * lane + h] = tot[h];
      part[1][wave][4 * lane + h] = bef[h];
    }
  }
  for (int i = tid; i < min(step, end - p0); i += kGateThreads) pe[i] = a.topk_idx[p0 + i];
  __syncthreads();
  int tot = 0, bef = 0;
  if (tid < E)
    for (int w = 0; w < kGateWaves; ++w) {
      tot += part[0][w][tid];
      bef += part[1][w][tid];
    }
  int pairs;
  const int off = scan256(tot, L.scratch, pairs);
  if (tid < E) L.base[tid] = off + bef;
  write_map(a, L, tot, off, pairs, blockIdx.x, gridDim.x);
  place_pairs(a, L, pe, p0, min(step, end - p0));
  for (int p = p0 + step; p < end; p += step) {
    __syncthreads();
    if (tid < E) L.base[tid] = L.at[kGateWaves - 1][tid];  // where the last piece ended
    for (int i = tid; i < min(step, end - p); i += kGateThreads) pe[i] = a.topk_idx[p + i];
    __syncthreads();
    place_pairs(a, L, pe, p, min(step, end - p));
  }
}

// One block of 16 waves: up to kGateSmallT = 64 tokens, four a wave.
template <int NJ, int KD>
__global__ __launch_bounds__(kGateThreads) void gate_small_kernel(GateArgs a, GateScatter sc) {
  __shared__ union {
    SelectLds select[kGateWaves];
    PlaceLds place;
  } L;
  __shared__ int32_t pe[kGateSmallT * kMaxGateK];
  __shared__ int cnt[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15;
  if (tid < 256) cnt[tid] = 0;
  __syncthreads();
  const int t0 = 4 * wave, t = t0 + (lane >> 4);
  if (t0 < a.T) {
    int sel;
    float w;
    gate_select<NJ, KD>(a, t0, L.select[wave], sel, w);
    if (t < a.T && c < a.k) {
      const int pair = t * a.k + c;
      a.topk_idx[pair] = sel;
      a.topk_w[pair] = w;
      pe[pair] = sel;
      atomicAdd(&cnt[sel], 1);
    }
  }
  __syncthreads();
  const int tot = tid < a.E ? cnt[tid] : 0;
  int pairs;
  const int off = scan256(tot, L.place.scratch, pairs);
  if (tid < a.E) L.place.base[tid] = off;
  write_map(sc, L.place, tot, off, pairs, 0, 1);
  place_pairs(sc, L.place, pe, 0, pairs);
}

// Selection blocks of 4 waves (16 tokens) up to 4096 tokens: they spread few
// tokens over the chip (512 tokens: 10.2 us in blocks of 32, 13.9 in blocks of
// 64). Blocks of 16 waves beyond: a quarter of the rows of counts, which every
// scatter block sums (16384 tokens: 12.8 us with 512 rows, 9.7 with 256).
static int count_tokens(int T) { return T <= 4096 ? 16 : 64; }

size_t gate_counts_bytes(int T) {
  return T <= kGateSmallT ? 0 : (size_t)((T + count_tokens(T) - 1) / count_tokens(T)) * 256;
}

namespace {

// What the kernels derive from the gate.
GateArgs prepared(const GateArgs& in) {
  GateArgs a = in;
  a.group_size = a.E / a.n_groups;
  a.group_magic = a.group_size > 1 ? (uint32_t)((0x100000000ull + a.group_size - 1) / a.group_size) : 0u;
  a.group_lanes_log2 = 0;
  while ((2 << a.group_lanes_log2) * a.n_groups <= 16) ++a.group_lanes_log2;
  a.vectors = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.partial) & 15) == 0;
  return a;
}

enum class GateLaunch { kTopk, kCounts, kSmall };

// Lanes hold four experts for E <= 64, eight for E <= 128, else sixteen; up
// to eight experts per token need nine heads of each.
template <GateLaunch L, int NJ, int KD>
void launch_gate(const GateArgs& a, const GateScatter* sc, hipStream_t s) {
  if constexpr (L == GateLaunch::kSmall)
    hipLaunchKernelGGL((gate_small_kernel<NJ, KD>), dim3(1), dim3(kGateThreads), 0, s, a, *sc);
  else if (L == GateLaunch::kCounts && count_tokens(a.T) == 64)
    hipLaunchKernelGGL((gate_topk_kernel<NJ, KD, 16, true>), dim3((a.T + 63) / 64), dim3(1024), 0, s, a);
  else
    hipLaunchKernelGGL((gate_topk_kernel<NJ, KD, 4, L == GateLaunch::kCounts>), dim3((a.T + 15) / 16), dim3(256), 0, s, a);
}
template <GateLaunch L>
hipError_t launch_gate(const GateArgs& a, const GateScatter* sc, hipStream_t s) {
  if (a.E <= 64)
    launch_gate<L, 1, 16>(a, sc, s);
  else if (a.E <= 128)
    launch_gate<L, 2, 16>(a, sc, s);
  else if (a.k <= 8)
    launch_gate<L, 4, 9>(a, sc, s);
  else
    launch_gate<L, 4, 16>(a, sc, s);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_topk(const GateArgs& in, hipStream_t s) {
  return launch_gate<GateLaunch::kTopk>(prepared(in), nullptr, s);
}

hipError_t launch_gate_route(const GateArgs& in, const GateScatter& scatter, hipStream_t s) {
  const GateArgs a = prepared(in);
  GateScatter sc = scatter;
  sc.count_tokens = count_tokens(a.T);
  if (a.T <= kGateSmallT) return launch_gate<GateLaunch::kSmall>(a, &sc, s);
  const hipError_t e = launch_gate<GateLaunch::kCounts>(a, nullptr, s);
  if (e != hipSuccess) return e;
  // One piece a block, and no more blocks than the chip holds at once, since
  // each sums all the counts (131072 tokens: 170 us with the selection in a
  // block per piece, 133 in 512 blocks; 1048576 tokens: 4898 and 1025).
  const int all = (a.T + kScatterTokens - 1) / kScatterTokens;
  sc.pieces = (all + kScatterBlocks - 1) / kScatterBlocks;
  hipLaunchKernelGGL(gate_scatter_kernel, dim3((all + sc.pieces - 1) / sc.pieces), dim3(kGateThreads), 0, s, sc);
  return hipGetLastError();
}

}  // namespace moe
