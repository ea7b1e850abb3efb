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
//   gate_topk     one wave per token, four consecutive experts a lane; for
//                 moe_route_gated also the expert counts of each 32 tokens
//   gate_scatter  per 128 tokens: totals and bases per expert from those
//                 counts, a stable scatter, and a share of the block map
//   gate_small    both in one block, for up to kGateSmallT tokens
#include "kernels.h"
#include "topk.h"

namespace moe {

namespace {

constexpr int kGateWaves = 16;
constexpr int kGateThreads = 64 * kGateWaves;
constexpr int kCountTokens = 32;                  // tokens per row of counts
constexpr int kScatterTokens = 4 * kCountTokens;  // tokens per scatter block
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

__device__ inline float wave_max_f32(float v) {  // v no NaN
  const uint32_t k = wave_max_u32(logit_key(v));
  return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}
__device__ inline float wave_min_f32(float v) { return -wave_max_f32(-v); }

// Group of expert e: e / size as the high half of e * ceil(2^32 / size), exact
// for e < 256 (size 1 has no such factor).
__device__ inline int group_of(const GateArgs& a, int e) {
  return a.group_size == 1 ? e : (int)__umulhi((uint32_t)e, a.group_magic);
}

// One token's selection in 64 bits: lane j < k gets the expert of rank j and
// its weight. l: the lane's logits (-inf: masked), b: their biases.
__device__ void gate_select_exact(const GateArgs& a, const float (&l)[4], const float (&b)[4], float mx, int& sel,
                                  float& w) {
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
  if (a.n_groups > 1) {
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

// One token's selection (lane j < k: the expert of rank j and its weight).
// gl: 256 floats of LDS of this wave's own. bmax: the largest |bias|.
__device__ void gate_select(const GateArgs& a, const float (&l)[4], const float (&b)[4], float bmax, float* gl,
                            int& sel, float& w) {
  const int lane = threadIdx.x & 63, E = a.E, k = a.k;
  const float mx = wave_max_f32(fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3])));
  // fp32 scores with the hardware exponential and reciprocal. Errors: the
  // exponent's product and the difference to the maximum round by 2^-24 of
  // their size, which moves e^-d by at most 2^-24 d e^-d < 2^-25 absolute;
  // the exponential, the reciprocal and the sum of up to 256 terms add a few
  // 2^-24 of the value, and adding the bias 2^-24 of the key. All together
  // stay below 2^-20 of (largest score + largest bias), the bound `err`.
  float s[4], top = 1.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float d = a.sigmoid ? -l[i] : (l[i] == mx ? 0.f : l[i] - mx);
    const float p = __expf(d);
    s[i] = l[i] == -INFINITY ? 0.f : (a.sigmoid ? __builtin_amdgcn_rcpf(1.0f + p) : p);
  }
  if (!a.sigmoid) {
    const float z = wave_sum((s[0] + s[1]) + (s[2] + s[3]));
    top = z > 0.f ? 1.0f / z : 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] *= top;
  }
  const float err = 0x1p-20f * (top + bmax);
  float hv[4];     // keys, larger first after the sort
  uint32_t hk[4], he[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    hv[i] = l[i] == -INFINITY ? -INFINITY : s[i] + b[i];
    if (!(hv[i] == hv[i])) hv[i] = -INFINITY;
    he[i] = 4 * lane + i;
    hk[i] = (int)he[i] < E ? logit_key(hv[i]) : 0u;
  }
  bool near = false;  // a decision the fp32 keys cannot settle
  if (a.n_groups > 1) {
    // 2^lg lanes per group, each over every 2^lg-th expert of it
    const int size = a.group_size, lg = a.group_lanes_log2, g = lane >> lg, p = lane & ((1 << lg) - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((int)he[i] < E) gl[he[i]] = hv[i];
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    float m1 = -INFINITY, m2 = -INFINITY;
    if (g < a.n_groups)
      for (int i = p; i < size; i += 1 << lg) {
        const float v = gl[g * size + i];
        m2 = fmaxf(m2, fminf(m1, v));
        m1 = fmaxf(m1, v);
      }
    for (int o = 1; o < 1 << lg; o <<= 1) {
      const float o1 = __shfl_xor(m1, o), o2 = __shfl_xor(m2, o);
      m2 = fmaxf(fmaxf(m2, o2), fminf(m1, o1));
      m1 = fmaxf(m1, o1);
    }
    __builtin_amdgcn_fence(__ATOMIC_SEQ_CST, "wavefront");
    const float gs = a.group_top2 && m2 > -INFINITY ? m1 + m2 : m1;
    int rank = 0;
    for (int q = 0; q < a.n_groups; ++q) {
      const float v = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(gs), q << lg));
      rank += v > gs || (v == gs && q < g);
    }
    const bool in = g < a.n_groups && rank < a.topk_groups, out = g < a.n_groups && rank >= a.topk_groups;
    if (a.topk_groups < a.n_groups) {
      const float lo = wave_min_f32(in ? gs : INFINITY), hi = wave_max_f32(out ? gs : -INFINITY);
      near = hi > -INFINITY && !(lo - hi > 4.0f * err);
    }
    const uint64_t kept = __ballot(in);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if ((int)he[i] < E && !(kept >> (group_of(a, (int)he[i]) << lg) & 1)) hk[i] = 0u;
  }
  // the lane's four in order: larger key first, equal keys by expert
  auto order = [&](int x, int y) {
    const bool sw = hk[y] > hk[x] || (hk[y] == hk[x] && he[y] < he[x]);
    const uint32_t k0 = hk[x], e0 = he[x];
    const float v0 = hv[x];
    hk[x] = sw ? hk[y] : k0;
    he[x] = sw ? he[y] : e0;
    hv[x] = sw ? hv[y] : v0;
    hk[y] = sw ? k0 : hk[y];
    he[y] = sw ? e0 : he[y];
    hv[y] = sw ? v0 : hv[y];
  };
  float sl[4] = {l[0], l[1], l[2], l[3]};
  order(0, 1);
  order(2, 3);
  order(0, 2);
  order(1, 3);
  order(1, 2);
  sel = 0;
  float sel_k = -INFINITY;
  uint32_t last = 0;  // the order key of rank k, 0: none
  for (int r = 0; r <= k; ++r) {
    const uint32_t m = wave_max_u32(hk[0]);
    if (r == k) {
      last = m;
      break;
    }
    const bool at_max = hk[0] == m;
    uint64_t cand = __ballot(at_max);
    // (equal keys: lanes hold consecutive experts, so the lowest lane has the lowest)
    const int win = __builtin_ctzll(cand);
    const int we = __builtin_amdgcn_readlane((int)he[0], win);
    const float wv = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(hv[0]), win));
    if (lane == r) {
      sel = we;
      sel_k = wv;
    }
    if (lane == win) {
      hk[0] = hk[1];
      hk[1] = hk[2];
      hk[2] = hk[3];
      hk[3] = 0u;
      he[0] = he[1];
      he[1] = he[2];
      he[2] = he[3];
      hv[0] = hv[1];
      hv[1] = hv[2];
      hv[2] = hv[3];
    }
  }
  const float last_v = last ? __uint_as_float(last & 0x80000000u ? last & 0x7FFFFFFFu : ~last) : -INFINITY;
  const float next_v = lane + 1 < k ? __shfl_down(sel_k, 1) : last_v;
  near |= lane < k && next_v > -INFINITY && !(sel_k - next_v > 2.0f * err);
  // the weights in 64 bits from the selected logits; where the fp32 sum over
  // the experts is used (softmax, not renormalised) it errs by a few 2^-24
  const int src = sel >> 2, sub = sel & 3;
  const float c0 = __shfl(sl[0], src), c1 = __shfl(sl[1], src), c2 = __shfl(sl[2], src), c3 = __shfl(sl[3], src);
  const float lsel = sub == 0 ? c0 : sub == 1 ? c1 : sub == 2 ? c2 : c3;
  if (__ballot(near)) {
    gate_select_exact(a, l, b, mx, sel, w);
    return;
  }
  double v = 0.0;
  if (lane < k && sel_k > -INFINITY) {
    const double e = exp(a.sigmoid ? -(double)lsel : (lsel == mx ? 0.0 : (double)lsel - (double)mx));
    v = a.sigmoid ? 1.0 / (1.0 + e) : e;
  }
  if (a.renorm) {
    double z = v;
    for (int o = 1; o < 16; o <<= 1) z += __shfl_xor(z, o);  // k <= 16: the first row of lanes
    v = z > 0.0 ? v / z : 0.0;
  } else if (!a.sigmoid) {
    v *= (double)top;
  }
  w = (float)(v * (double)a.scale);
}

// The lane's four logits of token t (masked: -inf) and, once, its biases.
__device__ inline void load_logits(const GateArgs& a, int64_t t, float (&l)[4]) {
  const int lane = threadIdx.x & 63, e = 4 * lane, E = a.E;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (a.vectors) {
    if (e < E)
      for (int sp = 0; sp < a.splits; ++sp) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(a.partial + ((int64_t)sp * a.T + t) * E + e);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += p[i];
      }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (e + i < E)
        for (int sp = 0; sp < a.splits; ++sp) v[i] += a.partial[((int64_t)sp * a.T + t) * E + e + i];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (e + i < E) {
      if (a.rbias) v[i] += a.rbias[e + i];
      if (a.logits_out) a.logits_out[t * E + e + i] = v[i];
      l[i] = v[i] == v[i] ? v[i] : -INFINITY;
    } else {
      l[i] = -INFINITY;
    }
  }
}

__device__ inline float load_biases(const GateArgs& a, float (&b)[4]) {
  const int e = 4 * (threadIdx.x & 63);
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    b[i] = a.balance && e + i < a.E ? a.balance[e + i] : 0.f;
    m = max(m, __float_as_uint(b[i]) & 0x7FFFFFFFu);  // (a NaN bias is the largest, and leaves every token near)
  }
  return a.balance ? __uint_as_float(wave_max_u32(m)) : 0.f;
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
    int run = L.base[tid];
    for (int w = 0; w < kGateWaves; ++w) {
      const int c = L.at[w][tid];
      L.at[w][tid] = run;
      run += c;
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

// Grid: ceil(T / 32). Block: 16 waves, two tokens each. COUNTS: the block
// writes its row of expert counts [ceil(T / 32)][E rounded up to 8] uint16;
// otherwise counts are added to chunk_hist (when given).
template <bool COUNTS>
__global__ __launch_bounds__(kGateThreads) void gate_topk_kernel(GateArgs a) {
  __shared__ float gl[kGateWaves][256];
  __shared__ int cnt[COUNTS ? 256 : 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if constexpr (COUNTS) {
    if (tid < 256) cnt[tid] = 0;
    __syncthreads();
  }
  float b[4];
  const float bmax = load_biases(a, b);
#pragma unroll 1
  for (int q = 0; q < kCountTokens / kGateWaves; ++q) {
    const int t = blockIdx.x * kCountTokens + q * kGateWaves + wave;
    if (t >= a.T) break;
    float l[4], w;
    int sel;
    load_logits(a, t, l);
    gate_select(a, l, b, bmax, gl[wave], sel, w);
    if (lane < a.k) {
      const int64_t pair = (int64_t)t * a.k + lane;
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
    const int Ep = round_up(a.E, 8);
    if (tid < Ep) a.counts[(int64_t)blockIdx.x * Ep + tid] = (uint16_t)cnt[tid];
  }
}

// Grid: ceil(T / 128). Block: 16 waves. Every block sums all rows of counts
// (512 rows of 512 bytes for 16384 tokens: 16-byte loads, 32 row groups).
__global__ __launch_bounds__(kGateThreads) void gate_scatter_kernel(GateScatter a) {
  __shared__ PlaceLds L;
  __shared__ int32_t pe[kScatterTokens * kMaxGateK];
  __shared__ int part[2][kGateWaves][256];  // [total, before][wave]
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int E = a.E, Ep = round_up(E, 8), cols = Ep / 8;
  const int p0 = blockIdx.x * kScatterTokens * a.k, n = min(kScatterTokens * a.k, a.T * a.k - p0);
  for (int i = tid; i < n; i += kGateThreads) pe[i] = a.topk_idx[p0 + i];
  const int rows = (a.T + kCountTokens - 1) / kCountTokens, mine = blockIdx.x * (kScatterTokens / kCountTokens);
  {
    const int c = lane & 31, rg = 2 * wave + (lane >> 5);
    int tot[8] = {0, 0, 0, 0, 0, 0, 0, 0}, bef[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    for (int r0 = 0; r0 < rows; r0 += 32 * 4) {
      u32x4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = min(r0 + 32 * j + rg, rows - 1);
        v[j] = *reinterpret_cast<const u32x4*>(a.counts + (int64_t)r * Ep + 8 * min(c, cols - 1));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int r = r0 + 32 * j + rg;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          const int lo = r < rows ? (int)(v[j][h] & 0xFFFFu) : 0, hi = r < rows ? (int)(v[j][h] >> 16) : 0;
          tot[2 * h] += lo;
          tot[2 * h + 1] += hi;
          bef[2 * h] += r < mine ? lo : 0;
          bef[2 * h + 1] += r < mine ? hi : 0;
        }
      }
    }
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      tot[h] += __shfl_xor(tot[h], 32);
      bef[h] += __shfl_xor(bef[h], 32);
      if (lane < 32) {
        part[0][wave][8 * c + h] = c < cols ? tot[h] : 0;
        part[1][wave][8 * c + h] = c < cols ? bef[h] : 0;
      }
    }
  }
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
  place_pairs(a, L, pe, p0, n);
}

// One block: up to kGateSmallT tokens, four a wave.
__global__ __launch_bounds__(kGateThreads) void gate_small_kernel(GateArgs a, GateScatter sc) {
  __shared__ PlaceLds L;
  __shared__ int32_t pe[kGateSmallT * kMaxGateK];
  __shared__ int cnt[256];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < 256) cnt[tid] = 0;
  __syncthreads();
  float b[4];
  const float bmax = load_biases(a, b);
#pragma unroll 1
  for (int t = wave; t < a.T; t += kGateWaves) {
    float l[4], w;
    int sel;
    load_logits(a, t, l);
    gate_select(a, l, b, bmax, reinterpret_cast<float*>(L.at[wave]), sel, w);
    if (lane < a.k) {
      const int pair = t * a.k + lane;
      a.topk_idx[pair] = sel;
      a.topk_w[pair] = w;
      pe[pair] = sel;
      atomicAdd(&cnt[sel], 1);
    }
  }
  __syncthreads();
  const int tot = tid < a.E ? cnt[tid] : 0;
  int pairs;
  const int off = scan256(tot, L.scratch, pairs);
  if (tid < a.E) L.base[tid] = off;
  write_map(sc, L, tot, off, pairs, 0, 1);
  place_pairs(sc, L, pe, 0, pairs);
}

size_t gate_counts_bytes(int E, int T) {
  return T <= kGateSmallT ? 0 : (size_t)((T + kCountTokens - 1) / kCountTokens) * round_up(E, 8) * 2;
}

namespace {

// What the kernels derive from the gate.
GateArgs prepared(const GateArgs& in) {
  GateArgs a = in;
  a.group_size = a.E / a.n_groups;
  a.group_magic = a.group_size > 1 ? (uint32_t)((0x100000000ull + a.group_size - 1) / a.group_size) : 0u;
  a.group_lanes_log2 = 0;
  while ((2 << a.group_lanes_log2) * a.n_groups <= 64) ++a.group_lanes_log2;
  a.vectors = a.E % 4 == 0 && (reinterpret_cast<uintptr_t>(a.partial) & 15) == 0;
  return a;
}

}  // namespace

hipError_t launch_gate_topk(const GateArgs& in, hipStream_t s) {
  const GateArgs a = prepared(in);
  const dim3 grid((a.T + kCountTokens - 1) / kCountTokens);
  hipLaunchKernelGGL(gate_topk_kernel<false>, grid, dim3(kGateThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_gate_route(const GateArgs& in, const GateScatter& sc, hipStream_t s) {
  const GateArgs a = prepared(in);
  if (a.T <= kGateSmallT) {
    hipLaunchKernelGGL(gate_small_kernel, dim3(1), dim3(kGateThreads), 0, s, a, sc);
    return hipGetLastError();
  }
  hipLaunchKernelGGL(gate_topk_kernel<true>, dim3((a.T + kCountTokens - 1) / kCountTokens), dim3(kGateThreads), 0, s, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(gate_scatter_kernel, dim3((a.T + kScatterTokens - 1) / kScatterTokens), dim3(kGateThreads), 0, s, sc);
  return hipGetLastError();
}

}  // namespace moe
