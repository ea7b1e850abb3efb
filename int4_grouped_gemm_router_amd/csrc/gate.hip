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
#include <cfloat>

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
// lowest lane, whose index has to be the lowest too. (A 32-bit maximum over
// the lanes, and a second one where the upper halves tie; shuffles of the
// 64-bit keys took seven times as long, which a late wave in doubt adds to
// the whole launch.)
__device__ inline void wave_best(uint64_t& k, int& i) {
  const uint32_t hi = (uint32_t)(k >> 32), lo = (uint32_t)k;
  const uint32_t mh = wave_max_u32(hi);
  uint64_t at = __ballot(hi == mh);
  if (at & (at - 1)) {
    const uint32_t ml = wave_max_u32(hi == mh ? lo : 0u);
    at = __ballot(hi == mh && lo == ml);
  }
  const int win = __builtin_ctzll(at);
  i = __builtin_amdgcn_readlane(i, win);
  k = (uint64_t)mh << 32 | (uint32_t)__builtin_amdgcn_readlane(lo, win);
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
__device__ inline double readlane_f64(double v, int lane) {
  const uint64_t u = (uint64_t)__double_as_longlong(v);
  const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((uint32_t)u, lane);
  const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((uint32_t)(u >> 32), lane);
  return __longlong_as_double((long long)(hi << 32 | lo));
}
__device__ inline double wave_sum_f64(double v) {
  v = row_sum_f64(v);
  return (readlane_f64(v, 0) + readlane_f64(v, 16)) + (readlane_f64(v, 32) + readlane_f64(v, 48));
}

// Group of expert e: e / size as the high half of e * ceil(2^32 / size), exact
// for e < 256 (size 1 has no such factor).
__device__ inline int group_of(const GateArgs& a, int e) {
  return a.group_size == 1 ? e : (int)__umulhi((uint32_t)e, a.group_magic);
}

// One token's selection in 64 bits: lane j < k gets the expert of rank j, with
// kMaskedSel added where it is masked. l: the lane's logits (-inf: masked), b:
// their biases; kept: bit g: group g is kept (decided here if !groups_known).
// least: no selected key is less (used if groups_known; NaN or -inf: not
// known). The few keys that are not less are ranked by comparing all pairs,
// from the wave's list in LDS; where there are too many, the largest is taken
// k times (which takes five times as long).
struct Candidate {
  uint64_t key;
  int e, pad;
};
constexpr int kCandidates = 64;
constexpr int kMaskedSel = 256;
__device__ int gate_select_exact(const GateArgs& a, const float (&l)[4], const float (&b)[4], float mx,
                                 bool groups_known, uint64_t kept, double least, Candidate* list) {
  const int lane = threadIdx.x & 63, E = a.E, k = a.k;
  double score[4];
  uint64_t key[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const double e = exp(a.sigmoid ? -(double)l[i] : (l[i] == mx ? 0.0 : (double)l[i] - (double)mx));
    score[i] = l[i] == -INFINITY ? 0.0 : e;
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < 4; ++i) score[i] = 1.0 / (1.0 + score[i]);
  } else {
    const double sum = wave_sum_f64((score[0] + score[1]) + (score[2] + score[3]));
#pragma unroll
    for (int i = 0; i < 4; ++i) score[i] = sum > 0.0 ? score[i] / sum : 0.0;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    key[i] = 0;
    if (4 * lane + i < E) key[i] = l[i] == -INFINITY ? kMaskedKey : key_order(score[i] + (double)b[i]);
  }
  if (a.n_groups > 1 && !groups_known) {
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
    kept = 0;
    for (int r = 0; r < a.topk_groups; ++r) {
      uint64_t best = mine;
      int at = lane;
      wave_best(best, at);
      kept |= 1ull << at;
      if (lane == at) mine = 0;
    }
  }
  if (a.n_groups > 1) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      if (e < E && !(kept >> group_of(a, e) & 1)) key[i] = 0;
    }
  }
  const uint64_t bound = groups_known && least > -INFINITY ? key_order(least) : 0;
  int n = 0, place[4];
  bool is[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    is[i] = bound > 0 && key[i] >= bound;
    const uint64_t lanes = __ballot(is[i]);
    place[i] = n + __popcll(lanes & lanemask_lt());
    n += __popcll(lanes);
  }
  if (n >= k && n <= kCandidates) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (is[i]) list[place[i]] = Candidate{key[i], 4 * lane + i, 0};
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    const Candidate mine = list[lane];
    int rank = 0;
    for (int o = 0; o < n; o += 4) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const Candidate x = list[o + j];  // (n <= 64: inside the list)
        rank += (o + j < n) & ((x.key > mine.key) | ((x.key == mine.key) & (x.e < mine.e)));
      }
    }
    // (the lanes past the candidates keep their own place, so all places differ; none is masked)
    return __builtin_amdgcn_ds_permute(4 * (lane < n ? rank : lane), mine.e);
  }
  int sel = 0;
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
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (at == 4 * lane + i) key[i] = 0;
    if (lane == r) sel = best == kMaskedKey ? at + kMaskedSel : at;
  }
  return sel;
}

// v[j][u] += row[64 j + e + u], four consecutive values each, all NJ loads
// under way at once (the last four, or the last one repeated, where they are
// past the end: no branch separates the loads).
template <int NJ>
__device__ inline void add_row(const GateArgs& a, const float* row, int e, float (&v)[NJ][4]) {
  const int E = a.E;
  f32x4 p[NJ];
  if (a.vectors) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) p[j] = *reinterpret_cast<const f32x4*>(row + min(64 * j + e, E - 4));
  } else {
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int u = 0; u < 4; ++u) p[j][u] = row[min(64 * j + e + u, E - 1)];
  }
#pragma unroll
  for (int j = 0; j < NJ; ++j)
#pragma unroll
    for (int u = 0; u < 4; ++u) v[j][u] += p[j][u];
}

// A wave's own LDS, per token: the keys for the groups (one word of padding
// per sixteen spreads the groups over the banks), or the two largest of every
// four consecutive keys; the groups' rank keys; then the logits, and
// the candidates of a token in doubt.
struct SelectLds {
  float v[4][256 + 16];
  union {
    float group[4][kMaxGateGroups];
    Candidate list[kCandidates];
  };
};
__device__ inline int key_at(int e) { return e + (e >> 4); }

// The two largest of values that are joined one or two at a time.
struct Top2 {
  float m1 = -INFINITY, m2 = -INFINITY;
  __device__ void add(float x) {
    m2 = fmaxf(m2, fminf(m1, x));
    m1 = fmaxf(m1, x);
  }
  __device__ void add(float x1, float x2) {  // x1 >= x2
    m2 = fmaxf(fmaxf(m2, x2), fminf(m1, x1));
    m1 = fmaxf(m1, x1);
  }
  template <int CTRL>
  __device__ void add_lane() {
    add(__uint_as_float(dpp<CTRL>(__float_as_uint(m1))), __uint_as_float(dpp<CTRL>(__float_as_uint(m2))));
  }
};

// Four tokens' selections, t0 + lane / 16 each: lane c = lane % 16 < k gets
// the expert of rank c and its weight. Lane c holds the experts
// 64 j + 4 c + u (j < NJ, u < 4) of its token. KD: at least min(k, 15) + 1.
template <int NJ, int KD>
__device__ void gate_select(const GateArgs& a, int t0, SelectLds& L, int& sel, float& w) {
  constexpr int NS = 4 * NJ;
  const int lane = threadIdx.x & 63, c = lane & 15, q = lane >> 4;
  const int E = a.E, k = a.k;
  const int64_t t = min(t0 + q, a.T - 1);
  // the sum over the router's K splits, the router's bias, the bias for balance
  float l[NS], lv[NJ][4], bv[NJ][4];
#pragma unroll
  for (int i = 0; i < NS; ++i) lv[i >> 2][i & 3] = bv[i >> 2][i & 3] = 0.f;
  if (a.balance) add_row<NJ>(a, a.balance, 4 * c, bv);
  for (int sp = 0; sp < a.splits; ++sp) add_row<NJ>(a, a.partial + ((int64_t)sp * a.T + t) * E, 4 * c, lv);
  if (a.rbias) add_row<NJ>(a, a.rbias, 4 * c, lv);
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int e = 64 * j + 4 * c + u;
      l[4 * j + u] = (e < E) & (lv[j][u] == lv[j][u]) ? lv[j][u] : -INFINITY;
    }
    if (a.logits_out && t0 + q < a.T) {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (64 * j + 4 * c + u < E) a.logits_out[t * E + 64 * j + 4 * c + u] = lv[j][u];
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
    for (int i = 0; i < NS; ++i) s[i] = __builtin_amdgcn_rcpf(1.0f + __expf(-l[i]));
  } else {
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] = __expf(fminf(l[i] - mx, 0.f));  // (infinity - infinity: 1)
    float z[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) z[i] = s[i];
#pragma unroll
    for (int n = NS / 2; n > 0; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) z[i] += z[i + n];
    top = 1.0f / row_sum(z[0]);
#pragma unroll
    for (int i = 0; i < NS; ++i) s[i] *= top;
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) s[i] = l[i] == -INFINITY ? -INFINITY : s[i];
  // What the fixed-point keys below span, [lowest, lowest + width], and the
  // largest magnitude in it. Biases up to 1: all that keys can be. Else (a
  // bias that masks an expert is -inf or NaN, or far below the others) the
  // token's own keys, down to eight scores' range below its best one: what lies
  // lower is selected only where little else is left, and then in 64 bits.
  float lowest = 0.f, width = top, range = top;
  if (a.balance) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < NS; ++i) {
      const float b = bv[i >> 2][i & 3];
      m = max(m, __float_as_uint(b) & 0x7FFFFFFFu);  // (NaN is the largest of all)
      s[i] += b;
      if (!(s[i] == s[i])) s[i] = -INFINITY;
    }
    const float bmax = __uint_as_float(row_max_u32(m));
    if (bmax <= 1.0f) {  // (the same in every lane)
      lowest = -bmax;
      range = top + bmax;
      width = range + bmax;
    } else {
      float hi = s[0];
#pragma unroll
      for (int i = 1; i < NS; ++i) hi = fmaxf(hi, s[i]);
      hi = row_max(hi);
      lowest = hi;
#pragma unroll
      for (int i = 0; i < NS; ++i) lowest = s[i] > hi - 8.0f ? fminf(lowest, s[i]) : lowest;
      lowest = row_min(lowest);
      range = fmaxf(top, fmaxf(fabsf(hi), fabsf(lowest)));
      width = hi - lowest + 0x1p-21f * range;  // (not 0 where all keys are equal)
    }
  }
  const float err = (a.sigmoid ? 0x1p-21f : 0x1p-20f) * range;
  // a decision the fp32 keys cannot settle, and whether it is one of groups
  // (all are where the best key is infinite or there is none)
  bool near = !(range < 1e30f), near_groups = near;
  uint64_t groups = 0;  // the token's kept groups
  if (a.n_groups > 1) {
    // group g: 2^lg lanes (up to sixteen groups), or lane g % 16
    const int size = a.group_size, lg = a.group_lanes_log2, p = c & ((1 << lg) - 1);
    const bool quads = size % 4 == 0;
    const int units = quads ? size / 4 : size;  // of a group
    if (quads) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const float x1 = fmaxf(s[4 * j], s[4 * j + 1]), n1 = fminf(s[4 * j], s[4 * j + 1]);
        const float x2 = fmaxf(s[4 * j + 2], s[4 * j + 3]), n2 = fminf(s[4 * j + 2], s[4 * j + 3]);
        *reinterpret_cast<f32x2*>(&L.v[q][2 * (16 * j + c)]) =
            f32x2{fmaxf(x1, x2), fmaxf(fminf(x1, x2), fmaxf(n1, n2))};
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS; ++i) L.v[q][key_at(64 * (i >> 2) + 4 * c + (i & 3))] = s[i];
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    float lo = INFINITY, hi = -INFINITY;
    for (int g = c >> lg; g < a.n_groups; g += 16) {
      Top2 m;
      constexpr int kReads = 4;  // under way at once
      for (int i0 = p; i0 < units; i0 += kReads << lg) {
        float v1[kReads], v2[kReads];
#pragma unroll
        for (int j = 0; j < kReads; ++j) {
          const int at = g * units + min(i0 + (j << lg), units - 1);
          if (quads) {
            const f32x2 v = *reinterpret_cast<const f32x2*>(&L.v[q][2 * at]);
            v1[j] = v.x;
            v2[j] = v.y;
          } else {
            v1[j] = L.v[q][key_at(at)];
            v2[j] = -INFINITY;
          }
        }
#pragma unroll
        for (int j = 0; j < kReads; ++j)
          if (i0 + (j << lg) < units) m.add(v1[j], v2[j]);
      }
      // over the group's lanes (all that hold a part agree after each step)
      if (lg >= 1) m.add_lane<0xB1>();
      if (lg >= 2) m.add_lane<0x4E>();
      if (lg >= 3) m.add_lane<0x141>();
      // (a sum of keys is above what groups of masked experts have)
      if (p == 0) L.group[q][g] = a.group_top2 && m.m2 > -INFINITY ? fmaxf(m.m1 + m.m2, -FLT_MAX) : m.m1;
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    for (int g0 = 0; g0 < a.n_groups; g0 += 16) {
      const int g = g0 + c;
      const float mine = L.group[q][g];
      int rank = 0;
      for (int o0 = 0; o0 < a.n_groups; o0 += 8) {
        const f32x4 va = *reinterpret_cast<const f32x4*>(&L.group[q][o0]);
        const f32x4 vb = *reinterpret_cast<const f32x4*>(&L.group[q][o0 + 4]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float v = j < 4 ? va[j & 3] : vb[j & 3];
          const int o = o0 + j;
          rank += (o < a.n_groups) & ((v > mine) | ((v == mine) & (o < g)));
        }
      }
      const bool is = g < a.n_groups, kept = is && rank < a.topk_groups;
      groups |= (__ballot(kept) >> (16 * q) & 0xFFFFull) << g0;
      lo = kept ? fminf(lo, mine) : lo;
      hi = is && !kept ? fmaxf(hi, mine) : hi;
    }
    lo = row_min(lo);
    hi = row_max(hi);
    // (groups whose keys are below `lowest` err by 2 u of what they are larger)
    const float larger = fmaxf(fabsf(lo) + fabsf(hi) - 4.0f * range, 0.f);
    near_groups |= hi > -INFINITY && !(lo - hi > 4.0f * err + 0x1p-22f * larger);
    near |= near_groups;
    if (quads) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        const bool kept = groups >> group_of(a, min(64 * j + 4 * c, E - 1)) & 1;
#pragma unroll
        for (int u = 0; u < 4; ++u) s[4 * j + u] = kept ? s[4 * j + u] : -INFINITY;
      }
    } else {
#pragma unroll
      for (int i = 0; i < NS; ++i) {
        const int e = 64 * (i >> 2) + 4 * c + (i & 3);
        s[i] = groups >> group_of(a, min(e, E - 1)) & 1 ? s[i] : -INFINITY;
      }
    }
  }
  // keys as 24-bit fixed point (0: masked, out of the running or below
  // `lowest`, at least 1 otherwise), then the lane's slot and the lane: all keys
  // of a token differ
  const float scale = 16777000.0f / width;
  uint32_t key[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    const uint32_t v = (uint32_t)fmaxf(__builtin_fmaf(s[i] - lowest, scale, 2.0f), 0.f);
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
  uint32_t mine = 0, m = 0;  // mine: the key of rank c
  for (int r = 0; r <= k; ++r) {
    m = row_max_u32(key[0]);
    mine = c == r ? m : mine;
    const bool own = key[0] == m;
#pragma unroll
    for (int i = 0; i + 1 < ND; ++i) key[i] = own ? key[i + 1] : key[i];
    if constexpr (ND == NS) key[NS - 1] = own ? 0u : key[NS - 1];
  }
  const uint32_t next = c == 15 ? m : dpp<0x101>(mine);  // of rank c + 1 (the lane above)
  // twice the bound in steps of the fixed point (all of them where it is more),
  // and what the steps cut off
  const uint32_t close = (uint32_t)fminf(2.0f * err * scale, 0x1p24f) + 5;
  const uint32_t vm = mine >> 8, vn = next >> 8;
  if (c < k) near |= vm == 0 || vm - vn <= close;
  sel = 64 * (int)(mine >> 6 & 3) + 4 * (int)(mine & 15) + (int)(mine >> 4 & 3);
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    *reinterpret_cast<f32x4*>(&L.v[q][64 * j + 4 * c]) = f32x4{l[4 * j], l[4 * j + 1], l[4 * j + 2], l[4 * j + 3]};
  __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
  // in doubt: those tokens again, one at a time, by the whole wave
  uint64_t doubt = __ballot(near && t0 + q < a.T);
  const uint64_t doubt_groups = __ballot(near_groups);
  while (doubt) {
    const int row = __builtin_ctzll(doubt) >> 4;
    doubt &= ~(0xFFFFull << (16 * row));
    float l4[4], b4[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = 4 * lane + i;
      b4[i] = a.balance && e < E ? a.balance[e] : 0.f;
      l4[i] = e < 64 * NJ ? L.v[row][e] : -INFINITY;
    }
    const float top4 = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(mx), 16 * row));
    const uint64_t kept = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(groups >> 32), 16 * row) << 32 |
                          (uint32_t)__builtin_amdgcn_readlane((uint32_t)groups, 16 * row);
    // the lowest selected fp32 key, less what it and a fixed-point step may err
    const uint32_t last = __builtin_amdgcn_readlane(vm, 16 * row + k - 1);
    const double step = 1.0 / (double)__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(scale), 16 * row));
    const uint32_t off = __builtin_amdgcn_readlane(close, 16 * row) + 4;
    const double from = (double)__uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(lowest), 16 * row));
    const double least = last > off ? (double)(last - off) * step + from : -(double)INFINITY;
    int se = gate_select_exact(a, l4, b4, top4, !(doubt_groups >> (16 * row) & 0xFFFF), kept, least, L.list);
    se = __shfl(se, c);
    if (q == row) sel = se;
  }
  // the weights in 64 bits from the selected logits; where the fp32 sum over
  // the experts is used (softmax, not renormalised) it errs by a few 2^-24: the
  // sum in 64 bits would need every expert's exponential in them (errors are
  // 5.6e-8 of the weights, 2.6e-8 of a rounding's own)
  double v = 0.0;
  if (c < k && sel < kMaskedSel) {
    const float x = L.v[q][sel];
    const double e = exp(a.sigmoid ? -(double)x : (x == mx ? 0.0 : (double)x - (double)mx));
    v = a.sigmoid ? 1.0 / (1.0 + e) : e;
  }
  sel &= kMaskedSel - 1;
  if (a.renorm) {
    const double sum = row_sum_f64(v);
    v = sum > 0.0 ? v / sum : 0.0;
  } else if (!a.sigmoid) {
    v *= (double)top;
  }
  w = (float)(v * (double)a.scale);
}

// Inclusive prefix sum over the wave: within rows of sixteen lanes, then the
// earlier rows' totals.
__device__ inline int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);  // the lane 1 below, 0 outside the row
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);  // 2
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);  // 4
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);  // 8
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // rows 1, 3: the last lane of the row below
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // rows 2, 3: lane 31
  return v;
}

// The block map's entry that begins at a pair, if one does: its position, its
// place among the expert's pairs, their number and their first block.
__device__ inline void write_block(const GateScatter& a, int e, int pos, int rank, int total, int first) {
  const int lg = a.block_m == 32 ? 5 : 4;
  if (rank & (a.block_m - 1)) return;
  int* m = a.block_map + 3 * (int64_t)(first + (rank >> lg));
  m[0] = e;
  m[1] = pos;
  m[2] = min(a.block_m, total - rank);
}

}  // namespace

// Grid: ceil(T / (4 W)). Block: W waves, four tokens each. COUNTS: the block
// writes its row of expert counts [grid][256] bytes (at most 64 each);
// otherwise counts are added to chunk_hist (when given). 256 experts, eight
// groups, sigmoid and bias: 6 us for 512 tokens (the chain of one wave, about
// 1300 vector instructions), 17 for 16384 (waves, four a SIMD, wait 0.52 of
// their time, and vector instructions issue in 0.36 of the SIMDs'); 60 experts,
// softmax, 2049 tokens: 4.
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
// wave a row at a time, a lane four experts. A token selects an expert at
// most once, so the tokens of a piece that selected an expert are a 128-bit
// mask, and a pair's place among them the bits below its token's. Latency
// bounds it: 5 us for 512 tokens, 5.8 for 16384 (131072 pairs).
__global__ __launch_bounds__(kGateThreads) void gate_scatter_kernel(GateScatter a) {
  __shared__ int part[2][kGateWaves][256];  // [total, before][wave]
  __shared__ int base[256];                 // first position of each expert's pairs of the piece
  __shared__ int total[256], first[256], first_block[256];
  __shared__ int sums[2][4];
  __shared__ u32x4 mask[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, step = kScatterTokens * a.k;
  const int p0 = blockIdx.x * a.pieces * step, end = min(p0 + a.pieces * step, a.T * a.k);
  const int rows = (a.T + a.count_tokens - 1) / a.count_tokens;
  const int mine = blockIdx.x * a.pieces * (kScatterTokens / a.count_tokens);
  constexpr int kPairs = kScatterTokens * kMaxGateK / kGateThreads;  // per thread and piece
  int e[kPairs];
  auto load = [&](int p) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int i = tid + kGateThreads * j;
      e[j] = i < step && p + i < end ? a.topk_idx[p + i] : -1;
    }
  };
  load(p0);
  {
    int tot[4] = {0, 0, 0, 0}, bef[4] = {0, 0, 0, 0};
    constexpr int kRows = 16;  // loads under way
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
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    *reinterpret_cast<i32x4*>(&part[0][wave][4 * lane]) = i32x4{tot[0], tot[1], tot[2], tot[3]};
    *reinterpret_cast<i32x4*>(&part[1][wave][4 * lane]) = i32x4{bef[0], bef[1], bef[2], bef[3]};
  }
  if (tid < 256) mask[tid] = u32x4{0u, 0u, 0u, 0u};
  __syncthreads();
  // thread e: expert e's pairs, and its blocks of the map
  int tot = 0, blocks = 0, scan = 0, scan_blocks = 0;
  if (tid < 256) {
    int bef = 0;
#pragma unroll
    for (int w = 0; w < kGateWaves; ++w) {
      tot += part[0][w][tid];
      bef += part[1][w][tid];
    }
    blocks = (tot + a.block_m - 1) / a.block_m;
    scan = wave_scan(tot);
    scan_blocks = wave_scan(blocks);
    if (lane == 63) {
      sums[0][wave] = scan;
      sums[1][wave] = scan_blocks;
    }
    base[tid] = bef;
    total[tid] = tot;
  }
  const int magic = (65536 + a.k - 1) / a.k;  // i / k is i * magic / 2^16 for i < 2048
  auto mark = [&] {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      const int t = (tid + kGateThreads * j) * magic >> 16;
      if (e[j] >= 0) atomicOr(reinterpret_cast<uint32_t*>(&mask[e[j]]) + (t >> 5), 1u << (t & 31));
    }
  };
  mark();
  __syncthreads();
  if (tid < 256) {
    for (int w = 0; w < wave; ++w) {
      scan += sums[0][w];
      scan_blocks += sums[1][w];
    }
    const int off = scan - tot;
    base[tid] += off;
    first[tid] = off;
    first_block[tid] = scan_blocks - blocks;
    if (blockIdx.x == 0) {
      if (tid < E) {
        a.hist[tid] = tot;
        a.offsets[tid] = off;
      }
      if (tid == 255) {
        a.offsets[E] = scan;
        *a.num_blocks = scan_blocks;
      }
    }
  }
  __syncthreads();
  for (int p = p0; p < end; p += step) {
    if (p > p0) {
      __syncthreads();
      if (tid < 256) {
        const u32x4 m = mask[tid];
        base[tid] += __popc(m.x) + __popc(m.y) + __popc(m.z) + __popc(m.w);
        mask[tid] = u32x4{0u, 0u, 0u, 0u};
      }
      load(p);
      __syncthreads();
      mark();
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      if (e[j] < 0) continue;
      const int i = tid + kGateThreads * j, t = i * magic >> 16;
      const u32x4 m = mask[e[j]];
      int pos = base[e[j]];
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t below = t >= 32 * (w + 1) ? ~0u : (t >= 32 * w ? (1u << (t & 31)) - 1u : 0u);
        pos += __popc(m[w] & below);
      }
      a.perm[pos] = p + i;
      a.inv_perm[p + i] = pos;
      write_block(a, e[j], pos, pos - first[e[j]], total[e[j]], first_block[e[j]]);
    }
  }
}

// One block, a wave for every four tokens, up to kGateSmallT = 64: the
// tokens that selected an expert are one 64-bit mask. 256 experts: 4.7 us for
// one token, 8.1 for 64 (6.2 for one with a sigmoid, a bias and eight groups);
// from there on two launches take no longer.
template <int NJ, int KD>
__global__ __launch_bounds__(kGateThreads) void gate_small_kernel(GateArgs a, GateScatter sc) {
  __shared__ SelectLds L[kGateWaves];
  __shared__ uint64_t mask[256];
  __shared__ int first[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, c = lane & 15, E = a.E;
  for (int i = tid; i < 256; i += blockDim.x) mask[i] = 0;
  const int t0 = 4 * wave, t = t0 + (lane >> 4), pair = t * a.k + c;
  const bool is = t < a.T && c < a.k;
  int sel;
  float w;
  gate_select<NJ, KD>(a, t0, L[wave], sel, w);
  __syncthreads();
  if (is) {
    a.topk_idx[pair] = sel;
    a.topk_w[pair] = w;
    atomicOr(reinterpret_cast<unsigned long long*>(&mask[sel]), 1ull << t);
  }
  __syncthreads();
  if (wave == 0) {  // lane: experts 4 lane + i; pairs and blocks (both at most 1024) are added up in one word
    const int up = sc.block_m - 1, lg = sc.block_m == 32 ? 5 : 4;
    int n[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      n[i] = __popcll(mask[4 * lane + i]);
      sum += n[i] + ((n[i] + up) >> lg << 16);
    }
    const int scan = wave_scan(sum);
    int at = scan - sum;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int x = 4 * lane + i;
      first[x] = at;
      if (x < E) {
        sc.hist[x] = n[i];
        sc.offsets[x] = at & 0xFFFF;
      }
      at += n[i] + ((n[i] + up) >> lg << 16);
    }
    if (lane == 63) {
      sc.offsets[E] = scan & 0xFFFF;
      *sc.num_blocks = scan >> 16;
    }
  }
  __syncthreads();
  if (is) {
    const uint64_t tokens = mask[sel];
    const int rank = __popcll(tokens & ((1ull << t) - 1)), pos = (first[sel] & 0xFFFF) + rank;
    sc.perm[pos] = pair;
    sc.inv_perm[pair] = pos;
    write_block(sc, sel, pos, rank, __popcll(tokens), first[sel] >> 16);
  }
}

// Tokens of a selection block, four a wave: as few as leave a block for each
// of the 256 compute units, so that a unit's waves do not share its SIMDs
// while others idle (2048 tokens: 10.3 us with the scatter in blocks of 16,
// 13.4 in blocks of 64; 8192: 14.3 us in blocks of 32, 16.3 in blocks of
// 64). More rows of counts than that cost every scatter block their sum (16384
// tokens: 23.2 us in blocks of 16, 17.1 in blocks of 64).
static int count_tokens(int T) { return T <= 4096 ? 16 : T <= 8192 ? 32 : 64; }

// Enough for every smaller T too: 4096 tokens have as many rows as 16384.
size_t gate_counts_bytes(int T) {
  if (T <= kGateSmallT) return 0;
  const int rows = (T + count_tokens(T) - 1) / count_tokens(T);
  return (size_t)(T > 4096 && rows < 256 ? 256 : rows) * 256;
}

namespace {

// What the kernels derive from the gate.
GateArgs prepared(const GateArgs& in) {
  GateArgs a = in;
  a.group_size = a.E / a.n_groups;
  a.group_magic = a.group_size > 1 ? (uint32_t)((0x100000000ull + a.group_size - 1) / a.group_size) : 0u;
  a.group_lanes_log2 = 0;
  while ((2 << a.group_lanes_log2) * a.n_groups <= 16) ++a.group_lanes_log2;
  const auto bits = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  a.vectors = a.E % 4 == 0 && ((bits(a.partial) | bits(a.rbias) | bits(a.balance)) & 15) == 0;
  return a;
}

enum class GateLaunch { kTopk, kCounts, kSmall };

// Lanes hold four experts for E <= 64, eight for E <= 128, else sixteen; up
// to eight experts per token need nine heads of each.
template <GateLaunch L, int NJ, int KD>
void launch_gate(const GateArgs& a, const GateScatter* sc, hipStream_t s) {
  if constexpr (L == GateLaunch::kSmall)
    hipLaunchKernelGGL((gate_small_kernel<NJ, KD>), dim3(1), dim3(64 * ((a.T + 3) / 4)), 0, s, a, *sc);
  else if (L == GateLaunch::kCounts && count_tokens(a.T) == 64)
    hipLaunchKernelGGL((gate_topk_kernel<NJ, KD, 16, true>), dim3((a.T + 63) / 64), dim3(1024), 0, s, a);
  else if (L == GateLaunch::kCounts && count_tokens(a.T) == 32)
    hipLaunchKernelGGL((gate_topk_kernel<NJ, KD, 8, true>), dim3((a.T + 31) / 32), dim3(512), 0, s, a);
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
  // block per piece, 133 in 512 blocks; 1048576 tokens: 4898 and 1025; both, with
  // a sigmoid and eight groups, 125 and 926 since).
  const int all = (a.T + kScatterTokens - 1) / kScatterTokens;
  sc.pieces = (all + kScatterBlocks - 1) / kScatterBlocks;
  hipLaunchKernelGGL(gate_scatter_kernel, dim3((all + sc.pieces - 1) / sc.pieces), dim3(kGateThreads), 0, s, sc);
  return hipGetLastError();
}

}  // namespace moe
