// Linear attention with a decay for each head (gfx950).
//
//   S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t
//
// for each value head, whose queries and keys are those of the key head
// v_head * qk_heads / v_heads. States are fp32 [qk_dim][v_dim].
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "topk.h"
#include "wide_expand.h"

namespace moe {

namespace {

constexpr int kStepCols = 32;  // columns of the state a block holds

// Bounds of sequence i, in range whatever the device array holds.
__device__ inline void bounds(const LinearArgs& a, int i, int& begin, int& end) {
  begin = min(max(a.cu_seqlens ? a.cu_seqlens[i] : i, 0), a.T);
  end = min(max(a.cu_seqlens ? a.cu_seqlens[i + 1] : i + 1, begin), a.T);
}
__device__ inline int slot_of(const int32_t* slots, int i, int n) {
  const int s = slots ? slots[i] : i;
  return s >= 0 && s < n ? s : -1;
}

}  // namespace

// Block: one sequence, one value head, 32 columns of its state in registers:
// thread (r, c) holds rows r + 32 p, columns 4 c .. 4 c + 3. Token after token,
// the next token's rows under way. The states' bytes bound it: 48 sequences of a
// token of 32 heads of 128 x 128 move 202 MB in 41 us (4.9 TB/s; with states
// loaded through the caches 47).
template <int NP>
__global__ __launch_bounds__(256) void linear_walk_kernel(LinearArgs a) {
  __shared__ float part[2][4][kStepCols];
  const int tid = threadIdx.x, wave = tid >> 6, c = tid & 7, r = tid >> 3;
  const int col = blockIdx.z * kStepCols + 4 * c;
  const int head = blockIdx.y, seq = blockIdx.x, kh = head / (a.v_heads / a.qk_heads);
  const bool in = col < a.v_dim;
  int begin, end;
  bounds(a, seq, begin, end);
  const int si = a.state_in ? slot_of(a.slots_in, seq, a.n_in) : -1, so = a.state_out ? slot_of(a.slots_out, seq, a.n_out) : -1;
  if (end - begin > a.short_tokens) return;
  if (begin == end && (so < 0 || (a.state_in == a.state_out && si == so))) return;
  const int64_t state = (int64_t)a.qk_dim * a.v_dim;
  f32x4 S[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) S[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (si >= 0 && in) {
    const float* p = a.state_in + ((int64_t)si * a.v_heads + head) * state + col;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (r + 32 * i < a.qk_dim) S[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + (int64_t)(r + 32 * i) * a.v_dim));
  }
  uint16_t kn[NP], qn[NP];
  u32x2 vn = {0u, 0u};
  float gn = 0.f;
  auto load = [&](int t) {
    const uint16_t* q = a.q + (int64_t)t * a.ldq + (int64_t)kh * a.qk_dim;
    const uint16_t* k = a.k + (int64_t)t * a.ldk + (int64_t)kh * a.qk_dim;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int row = min(r + 32 * i, a.qk_dim - 1);
      kn[i] = k[row];
      qn[i] = q[row];
    }
    if (in) vn = *reinterpret_cast<const u32x2*>(a.v + (int64_t)t * a.ldv + (int64_t)head * a.v_dim + col);
    gn = a.decay[a.ld_decay ? (int64_t)t * a.ld_decay + head : head];
  };
  if (begin < end) load(begin);
  for (int t = begin; t < end; ++t) {
    const float v[4] = {bf16lo(vn.x), bf16hi(vn.x), bf16lo(vn.y), bf16hi(vn.y)}, d = expf(gn);
    float kv[NP], qv[NP], o[4] = {};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      kv[i] = r + 32 * i < a.qk_dim ? bf16f(kn[i]) : 0.f;
      qv[i] = r + 32 * i < a.qk_dim ? bf16f(qn[i]) : 0.f;
    }
    if (t + 1 < end) load(t + 1);
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        S[i][j] = __builtin_fmaf(kv[i], v[j], S[i][j] * d);
        o[j] = __builtin_fmaf(qv[i], S[i][j], o[j]);
      }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o[j] += __shfl_xor(o[j], 8);
      o[j] += __shfl_xor(o[j], 16);
      o[j] += __shfl_xor(o[j], 32);
    }
    // (two sets of sums: a token's are read while the next one's are written)
    auto& sums = part[t & 1];
    if ((tid & 63) < 8)
#pragma unroll
      for (int j = 0; j < 4; ++j) sums[wave][4 * c + j] = o[j];
    __syncthreads();
    if (tid < kStepCols && (int)blockIdx.z * kStepCols + tid < a.v_dim)
      a.o[(int64_t)t * a.ldo + (int64_t)head * a.v_dim + blockIdx.z * kStepCols + tid] =
          f2bf(a.scale * ((sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid])));
  }
  if (so >= 0 && in) {
    float* p = a.state_out + ((int64_t)so * a.v_heads + head) * state + col;
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (r + 32 * i < a.qk_dim) *reinterpret_cast<f32x4*>(p + (int64_t)(r + 32 * i) * a.v_dim) = S[i];
  }
}

// ------------------------------------------------------------------ prompts: chunks of 32 tokens

namespace {

constexpr int kChunk = 32;
constexpr int kChunkThreads = 320;  // four waves that compute, one that fetches for them
constexpr int kMaxWindows = 512;
constexpr int kNowhere = INT32_MIN;  // a buffer offset past every end: such loads give zeros
constexpr float kLog2e = 1.44269504f;

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// 16 or 4 bytes a lane straight to LDS (from dst on, lane after lane), as
// assembly: before a transposing read of LDS the compiler waits for every copy
// it knows of, also those into other tiles. The kernel's own waits count them.
__device__ inline u32x4 words_of(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  return u32x4{(uint32_t)p, (uint32_t)(p >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
__device__ inline uint32_t lds_offset(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const void*)p;
}
__device__ inline void copy16_to_lds(u32x4 r, uint32_t dst, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(dst), "v"(voff), "s"(r) : "m0", "memory");
}
__device__ inline void copy4_to_lds(u32x4 r, uint32_t dst, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(dst), "v"(voff), "s"(r) : "m0", "memory");
}

// Four values of one column from four rows of LDS: the sixteen lanes of a group
// read four rows of sixteen values (lane l row l / 4, values 4 (l % 4) ..) and
// lane l gets column l of the four.
__device__ inline u32x2 column4(const void* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p));
}

// Rows of R 16-byte pieces lie in LDS without gaps, piece c of row r at
// c ^ swizzle(r): sixteen rows' same piece, and eight rows' same pair of
// pieces, are then in different banks. (The output launch of 16384 tokens of 32
// heads still counts 1.9 conflict cycles an LDS instruction; which of its
// accesses has them is not known.)
template <int R>
__device__ inline int swizzle(int r) {
  return R >= 16 ? 2 * (r & 7) | (r >> 3 & 1) : 2 * (r >> 1 & 3) | (r >> 3 & 1);
}

// A tensor's 32 rows as the lanes of one wave copy them to LDS, 64 pieces an
// instruction.
template <int R>
struct RowCopy {
  static constexpr int kN = kChunk * R / 64;  // instructions
  int off[kN];
  __device__ void init(int lane, int dim, int64_t ld) {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const int slot = 64 * i + lane, row = slot / R, c = (slot % R) ^ swizzle<R>(row);
      off[i] = 8 * c < dim ? row * (int)(ld * 2) + 16 * c : kNowhere;
    }
  }
  // base: the first row's values; records: bytes up to the end of the last row's
  __device__ void issue(u32x4* dst, const uint16_t* base, uint32_t records) const {
    const u32x4 r = words_of(base, records);
    const uint32_t to = lds_offset(dst);
#pragma unroll
    for (int i = 0; i < kN; ++i) copy16_to_lds(r, to + 1024 * i, (uint32_t)off[i]);
  }
};

// v from a lane of the same row of sixteen, as dpp; 0 past the row.
template <int CTRL>
__device__ inline float shifted(float v) {
  return __uint_as_float(dpp<CTRL>(__float_as_uint(v)));
}

// A state is 2^f times what the registers hold, so that a chunk's decay mostly
// costs one sum instead of a product per element: f takes the decays until it
// is far from 0, then the elements take it over.
__device__ inline bool keeps(float f) { return f >= -4.f && f <= 4.f; }
__device__ inline float factor_after(float f, float decay) { return keeps(f + decay) ? f + decay : 0.f; }

__device__ inline int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ inline float uniform_f(float v) { return __builtin_bit_cast(float, uniform(__builtin_bit_cast(int, v))); }

// A chunk: up to 32 tokens of one sequence, and the slots of its states (-1: none).
struct Item {
  int t0, count, in, out, flags;
};
constexpr int kItem = 1;     // there is one
constexpr int kFirst = 2;    // the first of its sequence in the window: the state is loaded
constexpr int kMiddle = 4;   // its sequence began in an earlier window
constexpr int kLast = 8;     // the last of its sequence: the state is kept
constexpr int kGoesOn = 16;  // its sequence goes on behind the window

// Sequences as a wave holds them: lane l has the beginning of sequence base + l
// (which is also the end of the one before) and its slots, so that a walk over
// up to 63 sequences waits for memory once. Whatever the arrays hold, bounds
// are in 0..T and ends not before their beginnings.
struct Sequences {
  int base, begins, in, out;
  __device__ void load(const LinearArgs& a, int first) {
    base = first;
    const int i = first + (int)(threadIdx.x & 63), n = min(i, a.n_seqs - 1);
    begins = min(max(a.cu_seqlens[min(i, a.n_seqs)], 0), a.T);
    const int si = a.state_in ? (a.slots_in ? a.slots_in[n] : n) : -1, so = a.state_out ? (a.slots_out ? a.slots_out[n] : n) : -1;
    in = si >= 0 && si < a.n_in ? si : -1;
    out = so >= 0 && so < a.n_out ? so : -1;
  }
  __device__ void hold(const LinearArgs& a, int i) {
    if (i < base || i > base + 62) load(a, i);
  }
  __device__ int begin(int i) const { return __builtin_amdgcn_readlane(begins, i - base); }
  __device__ int end(int i) const { return max(__builtin_amdgcn_readlane(begins, i + 1 - base), begin(i)); }
  __device__ int slot_in(int i) const { return __builtin_amdgcn_readlane(in, i - base); }
  __device__ int slot_out(int i) const { return __builtin_amdgcn_readlane(out, i - base); }
  // The last sequence that begins before token v > 0, or the first of all; held.
  __device__ int before(const LinearArgs& a, int v) {
    const int lane = threadIdx.x & 63;
    if (a.n_seqs <= 63) return max(__popcll(__ballot(lane < a.n_seqs && begins < v)) - 1, 0);  // (all of them are held)
    int lo = 0, len = a.n_seqs;  // the first that does not is in lo .. lo + len; 64 steps at a time
    while (len > 0) {
      const int step = (len + 63) / 64, at = lo + min((lane + 1) * step, len) - 1;
      const int below = __popcll(__ballot(a.cu_seqlens[at] < v));  // whole steps below v
      if (below == 64) {
        lo += len;
        break;
      }
      lo += min(below * step, len);
      len = min(step - 1, a.n_seqs - lo);
    }
    const int i = max(uniform(lo) - 1, 0);
    hold(a, i);
    return i;
  }
};

// The chunks of window w, one after the other; of one window, those of every
// a.strands-th sequence.
struct Walk {
  Sequences s;
  int begin, end, seq, of, pos, stop, flags;  // of: the chunks' sequence, seq: the next one
  bool last_window, open;
  __device__ Walk(const LinearArgs& a, int w, int strand) {
    begin = w * a.window;
    last_window = w == a.windows - 1;
    end = min(begin + a.window, a.T);
    s.load(a, 0);
    seq = begin > 0 ? s.before(a, begin) : strand;
    open = false;
    of = pos = stop = flags = 0;
  }
  __device__ __forceinline__ Item next(const LinearArgs& a) {
    while (!open) {
      if (seq >= a.n_seqs) return Item{0, 0, -1, -1, 0};
      s.hold(a, seq);
      const int b = s.begin(seq), e = s.end(seq);
      if (b >= end && !last_window) return Item{0, 0, -1, -1, 0};
      of = seq;
      seq += a.strands;
      if (b < begin && e <= begin) continue;      // before the window
      if (e - b <= a.short_tokens) continue;      // the other kernel's
      if (b == e) {
        // no token: its state only moves, if it does
        const int si = s.slot_in(of), so = s.slot_out(of);
        if (so < 0 || (a.state_in == a.state_out && si == so)) continue;
        return Item{0, 0, si, so, kItem | kFirst | kLast};
      }
      open = true;
      pos = max(b, begin);
      stop = min(e, end);
      flags = kItem | kFirst | (b < begin ? kMiddle : 0) | (e <= end ? kLast : kGoesOn);
    }
    Item it{pos, min(kChunk, stop - pos), s.slot_in(of), s.slot_out(of), flags & ~kLast};
    pos += it.count;
    if (pos >= stop) {
      it.flags |= flags & kLast;
      open = false;
    }
    flags &= ~kFirst;
    return it;
  }
};

// Where windows keep what they pass on (LinearArgs::ws): per window, whether
// its last sequence goes on behind it, whether that sequence began in it, and
// the slot of the state it began with; the sequence's decay over the window for each head; its
// state: first what the window adds to a state of zeros, then the state at the
// window's end; and a copy of the state it starts from.
struct Passed {
  int32_t* meta;  // [windows][4]
  float *decay, *state, *start;
};
__host__ __device__ inline int64_t state_values(const LinearArgs& a) { return (int64_t)a.v_heads * a.qk_dim * a.v_dim; }
__host__ __device__ inline Passed passed(const LinearArgs& a) {
  Passed p;
  p.meta = static_cast<int32_t*>(a.ws);
  p.decay = reinterpret_cast<float*>(p.meta) + 4 * (int64_t)a.windows;
  p.state = p.decay + ((int64_t)a.windows * a.v_heads + 3) / 4 * 4;
  p.start = p.state + a.windows * state_values(a);
  return p;
}

}  // namespace

// Block: one window of tokens, one value head, 64 NT columns of its state, of
// which each of the four waves holds 16 NT in registers as accumulators of the
// matrix cores. With G the running sum of g in a chunk, G_n its last,
//   O = scale (diag(e^G) Q S + (Q K^T .* e^(G_i - G_j), i >= j) V)
//   S = e^(G_n) S + K^T diag(e^(G_n - G_j)) V
// O is formed as its transpose. S is a matrix operand as it lies in the
// accumulators: of each 32 rows lane group g holds rows 8 g .. 8 g + 7, the ones
// that a matrix operand wants of it, because the keys enter the update with
// their columns in that order. So are the decayed products of queries and keys,
// which every wave forms for itself (12 of its 80 matrix operations a chunk), so
// that nothing but the rows goes through LDS. A fifth wave walks over the
// sequences, copies rows two chunks ahead and forms the decays of the next
// chunk; the four wait for nothing but it, once a chunk. (With that work spread
// over the four, a chunk of a lone block took 1.7 us instead of 1.1; 16 heads of
// 300 tokens 21.7, 15.8 us, 32 heads of 16384 tokens alike.) STATE: only S, from
// zeros, of the sequence that goes on behind the window.
//
// Latency bounds it: 16384 tokens of 32 heads of 128 x 128 in 16 windows take 59
// to 64, 14 and 138 to 157 us for the states, their passing and the outputs where
// each launch is waited for (the call, where they follow each other, takes 197);
// they move 0.18, 0.05 and 0.46 GB (2.8 to 3.6 TB/s); matrix cores are busy 0.31
// (the states) and 0.26 (the outputs) of the time, vector instructions issue in
// 0.37, LDS is read in 0.17.
template <int DK, int NT, int ST, bool STATE>
__global__ __launch_bounds__(kChunkThreads, DK == 128 ? 3 : 2) void linear_chunk_kernel(LinearArgs a) {
  constexpr int RQ = DK / 8, RV = 8 * NT, kCols = 64 * NT;
  __shared__ struct {
    struct {
      u32x4 q[STATE ? 1 : kChunk * RQ], k[kChunk * RQ], v[kChunk * RV];
    } tile[ST];
    float g[4][64];
    struct {
      float G[kChunk], Gs[kChunk];  // the sums of g in base 2, and with log2 |scale| added
      float w[kChunk];              // e^(G_n - G_j) over the state's factor after the chunk
      float total;                  // G_n
    } dec[2];
    Item item[4];
  } L;
  // (three waves a SIMD leave 168 registers each)
  constexpr bool kTight = DK == 128 && NT == 2 && !STATE;
  static_assert(ST == 3, "tile c + 2 goes where tile c - 1 was");
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int c16 = lane & 15, g4 = lane >> 4;
  const int slices = (a.v_dim + kCols - 1) / kCols;
  // heads that share queries and keys, and slices of a head, follow each other in one XCD
  const int units = (STATE ? a.windows - 1 : a.windows * a.strands) * a.v_heads * slices;
  const int per = (units + 7) / 8, u = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if ((int)(blockIdx.x >> 3) >= per || u >= units) return;
  const int slice = u % slices, head = u / slices % a.v_heads, part_of = u / slices / a.v_heads;
  const int w = a.strands > 1 ? 0 : part_of, strand = a.strands > 1 ? part_of : 0;
  const int kh = head / (a.v_heads / a.qk_heads), col0 = slice * kCols, cols = min(kCols, a.v_dim - col0);
  const Passed ps = passed(a);

  auto records = [](const Item& it, int64_t ld, int dim) {
    return it.count ? (uint32_t)(((it.count - 1) * ld + dim) * 2) : 0u;
  };
  if (wave == 4) {
    // The wave that fetches: turn c is between the barriers c and c + 1, in which
    // the others compute chunk c; in it this one has the copies of chunk c + 2 set
    // out and forms the decays of chunk c + 1.
    Walk walk(a, w, strand);
    bool any = true;
    if constexpr (STATE) {
      // the sequence with tokens on both sides of the window's end
      const int i = walk.s.before(a, walk.end), b = walk.s.begin(i);
      any = b < walk.end && walk.s.end(i) > walk.end && walk.s.end(i) - b > a.short_tokens;
      const int si = walk.s.slot_in(i);
      if (head == 0 && slice == 0 && lane == 0) {
        ps.meta[4 * w] = any;
        ps.meta[4 * w + 1] = b >= walk.begin;
        ps.meta[4 * w + 2] = si;
      }
      walk.seq = i;
    }
    if (!any) walk.seq = a.n_seqs;  // (no chunk)
    Item q0 = walk.next(a), q1 = walk.next(a), q2 = walk.next(a), q3;
    auto pass_on = [&](const Item& it, int slot) {
      if (lane == 0) L.item[slot] = it;
    };
    pass_on(q0, 0);
    pass_on(q1, 1);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (!(q0.flags & kItem)) return;
    const uint16_t* qb = a.q + (int64_t)kh * a.qk_dim;
    const uint16_t* kb = a.k + (int64_t)kh * a.qk_dim;
    const uint16_t* vb = a.v + (int64_t)head * a.v_dim + col0;
    RowCopy<RQ> cq, ck;
    RowCopy<RV> cv;
    if constexpr (!STATE) cq.init(lane, a.qk_dim, a.ldq);
    ck.init(lane, a.qk_dim, a.ldk);
    cv.init(lane, cols, a.ldv);
    // (every item, also one that is not there, has the same number of copies: the waits count on it)
    constexpr int kLoads = (STATE ? 1 : 2) * RowCopy<RQ>::kN + RowCopy<RV>::kN;
    static_assert(kLoads + 1 < 64, "what a wait can count");
    auto load_tile = [&](const Item& it, int st) {
      const int64_t t = it.t0;
      if constexpr (!STATE) cq.issue(L.tile[st].q, qb + t * a.ldq, records(it, a.ldq, a.qk_dim));
      ck.issue(L.tile[st].k, kb + t * a.ldk, records(it, a.ldk, a.qk_dim));
      cv.issue(L.tile[st].v, vb + t * a.ldv, records(it, a.ldv, cols));
    };
    auto load_g = [&](const Item& it, int slot) {
      const u32x4 r = words_of(a.decay + it.t0 * a.ld_decay + head, it.count ? (uint32_t)((it.count - 1) * a.ld_decay + 1) * 4u : 0u);
      copy4_to_lds(r, lds_offset(L.g[slot]), lane < it.count ? (uint32_t)(lane * a.ld_decay) * 4u : (uint32_t)kNowhere);
    };
    // The chunk's sums in base 2. A weight's exponent is a sum from its own token
    // on, so that small ones are precise beside large ones; the sums from the
    // front weigh products that are rounded to bf16. 2^-288 and less is 0 here.
    const float log_scale = __log2f(fabsf(a.scale));
    auto decays = [&](int slot, int to, float lf) -> float {
      float g = L.g[slot][lane] * kLog2e;
      g = g < -288.f ? -288.f : g;
      const float front = g + shifted<0x111>(g);  // of this lane and up to 1, 3, 7, 15 before it, in rows of sixteen
      float G = front + shifted<0x112>(front);
      G += shifted<0x114>(G);
      G += shifted<0x118>(G);
      float R = g + shifted<0x101>(g);  // of this lane and up to 1, 3, 7, 15 behind it, then without this lane
      R += shifted<0x102>(R);
      R += shifted<0x104>(R);
      R += shifted<0x108>(R);
      R = shifted<0x101>(R);
      const float first = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, G), 15));
      const float second = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, G), 31));
      if (lane >= 16) G += first;
      if (lane < 16) R += second;
      const float total = first + second;
      if (lane < kChunk) {
        L.dec[to].G[lane] = G;
        L.dec[to].Gs[lane] = G + log_scale;
        L.dec[to].w[lane] = __builtin_amdgcn_exp2f(R - factor_after(lf, total));
        if (lane == 0) L.dec[to].total = total;
      }
      return total;
    };

    load_g(q0, 0);
    load_g(q1, 1);
    load_g(q2, 2);
    load_tile(q0, 0);
    load_tile(q1, 1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLoads > 63 ? 63 : 2 * kLoads) : "memory");
    float total = decays(0, 0, 0.f), f = 0.f;
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
    int st = 2;
    for (int c = 0;; ++c) {
      // Chunk c is in LDS (what was issued after its rows: the decays of chunk
      // c + 2 and the rows of chunk c + 1).
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kLoads + 1) : "memory");
      if (!(q1.flags & kItem)) break;
      pass_on(q2, (c + 2) & 3);
      q3 = walk.next(a);
      load_g(q3, (c + 3) & 3);
      load_tile(q2, st);
      if (!STATE && (q0.flags & kFirst)) f = 0.f;
      f = factor_after(f, total);
      total = decays((c + 1) & 3, (c + 1) & 1, !STATE && (q1.flags & kFirst) ? 0.f : f);
      q0 = q1;
      q1 = q2;
      q2 = q3;
      st = st == 2 ? 0 : st + 1;
    }
    // (the copies into LDS that are under way end before the block does)
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    return;
  }

  // The waves that compute, before the one that fetches where they share a SIMD
  // (16384 tokens of 32 heads 202 -> 199 us).
  __builtin_amdgcn_s_setprio(2);
  auto item_of = [&](int slot) {
    const Item& it = L.item[slot];
    return Item{uniform(it.t0), uniform(it.count), uniform(it.in), uniform(it.out), uniform(it.flags)};
  };
  asm volatile("s_barrier" ::: "memory");
  Item q0 = item_of(0), q1;
  if (!(q0.flags & kItem)) return;
  const uint32_t sign = __float_as_uint(a.scale) & 0x80000000u;
  float sum = 0.f;  // of the window's logarithms (STATE)

  f32x4 S[DK / 16][NT];
#pragma unroll
  for (int i = 0; i < DK / 16; ++i)
#pragma unroll
    for (int n = 0; n < NT; ++n) S[i][n] = f32x4{0.f, 0.f, 0.f, 0.f};
  // where this lane's part of a state is: rows 32 (i / 2) + 8 g4 + 4 (i % 2) + r, column col + 16 n
  const int col = col0 + (wave * NT) * 16 + c16;
  // (by buffer accesses: rows past the state are past its end, columns are sent
  // there; loads give zeros and stores are dropped, without a branch between)
  const uint32_t head_bytes = (uint32_t)(a.qk_dim * a.v_dim * 4);
  auto each_of_state = [&](auto f) {
    // (hidden from the optimiser, which otherwise keeps every element's place in registers over the loop)
    int row0 = 8 * g4, step = uniform(a.v_dim * 4);
    asm volatile("" : "+v"(row0), "+s"(step));
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint32_t at = col + 16 * n < a.v_dim ? (uint32_t)(row0 * step + (col + 16 * n) * 4) : (uint32_t)kNowhere;
#pragma unroll
      for (int i = 0; i < DK / 16; ++i)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[i][n][r] = f(S[i][n][r], at + (uint32_t)((32 * (i >> 1) + 4 * (i & 1) + r) * step));
    }
  };
  auto load_state = [&](const float* p) {
    const rsrc_t r = make_rsrc(p, head_bytes);
    each_of_state([&](float, uint32_t at) { return __uint_as_float(bload1(r, at, 0)); });
  };
  auto store_state = [&](float* p, float f) {
    const rsrc_t r = make_rsrc(p, head_bytes);
    each_of_state([&](float s, uint32_t at) {
      __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(s * f), r, (int)at, 0, 0);
      return s;
    });
  };
  const int64_t head_state = (int64_t)a.qk_dim * a.v_dim;
  auto state_operand = [&](int s, int n) {
    const f32x4 x = S[2 * s][n], y = S[2 * s + 1][n];
    return u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3])};
  };

  // (the copy, where a later window's block may have written the state by now)
  auto first_state = [&](const Item& it) {
    const float* from = nullptr;
    if (it.flags & kMiddle)
      from = ps.state + (w - 1) * state_values(a);
    else if (it.in >= 0)
      from = a.copied && (it.flags & kGoesOn) ? ps.start + w * state_values(a) : a.state_in + it.in * state_values(a);
    if (from)
      load_state(from + head * head_state);
    else
      each_of_state([](float, uint32_t) { return 0.f; });
  };
  if constexpr (!STATE) first_state(q0);
  // A lane has four columns of two tiles (of columns, or of tokens where there is
  // one tile of columns); by exchanging the odd rows of sixteen lanes of the one
  // with the even rows of the other it has eight neighbouring columns of one, and
  // stores 16 bytes: 4 x 8 bytes a lane instead took 50 us more for 16384 tokens
  // of 32 heads of 128.
  auto side_by_side = [](u32x2 x, u32x2 y) {
    u32x4 r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const auto s = __builtin_amdgcn_permlane16_swap(x[i], y[i], false, false);
      r[i] = s[0];
      r[2 + i] = s[1];
    }
    return r;
  };
  uint32_t store_at;
  {
    const int row = NT == 2 ? c16 : 16 * (g4 & 1) + c16;
    const int c = wave * NT * 16 + (NT == 2 ? 16 * (g4 & 1) : 0) + 8 * (g4 >> 1);
    store_at = c < cols ? (uint32_t)(row * (int)(a.ldo * 2) + c * 2) : (uint32_t)kNowhere;
  }
  auto store_out = [&](const f32x4 (&y)[2][NT]) {
    auto packed = [](const f32x4& v) { return u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])}; };
    uint16_t* o = a.o + q0.t0 * a.ldo + (int64_t)head * a.v_dim + col0;
    Item rows = q0;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const u32x4 out = NT == 2 ? side_by_side(packed(y[i][0]), packed(y[i][NT - 1])) : side_by_side(packed(y[0][0]), packed(y[1][0]));
      __builtin_amdgcn_raw_buffer_store_b128(out, make_rsrc(o, records(rows, a.ldo, cols)), (int)store_at, 0, 0);
      o += 16 * a.ldo;
      rows.count = max(rows.count - 16, 0);
    }
  };

  // Where a lane reads in a tile, in bytes: the keys' columns (row krow, pieces 4 s
  // + c16 % 4) and the values' (the same row, pieces of this wave's tiles); its
  // query and key are row c16, pieces 4 s + g4. Steps of s and of tiles change
  // bits that nothing else sets, also under the swizzle.
  const int krow = 4 * g4 + (c16 >> 2);
  const int key_at = 16 * (krow * RQ + ((c16 & 3) ^ swizzle<RQ>(krow)));
  const int value_at = 16 * (krow * RV + ((2 * NT * wave + (c16 >> 1 & 1)) ^ swizzle<RV>(krow))) + 8 * (c16 & 1);
  auto piece = [](const u32x4* tile, int at) { return *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint8_t*>(tile) + at); };

  int st = 0;
  float f = 0.f;
  for (int c = 0;; ++c) {
    // Tile c and its decays are in LDS, and no wave reads tile c - 1 any more.
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    if (!STATE && c > 0 && (q0.flags & kFirst)) {
      f = 0.f;
      first_state(q0);
      // (a wait the compiler sees: it has none to add in every turn, which would be for the stores too)
      __builtin_amdgcn_s_waitcnt(0);
    }
    const auto& T = L.tile[st];
    const auto& D = L.dec[c & 1];
    const float f_before = f, decayed = f + uniform_f(D.total);
    f = keeps(decayed) ? decayed : 0.f;
    q1 = item_of((c + 1) & 3);

    // (hidden, so that places are formed again in each turn instead of filling registers over the loop)
    int ka = key_at, va = value_at, row = c16;
    if constexpr (kTight) asm volatile("" : "+v"(row), "+v"(ka), "+v"(va));
    int ra = 16 * (row * RQ + (g4 ^ swizzle<RQ>(row)));
    // values: this lane's column, tokens 4 g4 + r and 16 + 4 g4 + r
    auto values = [&](int n, int at) {
      const uint8_t* p = reinterpret_cast<const uint8_t*>(T.v) + (at ^ 32 * n);
      const u32x2 lo = column4(p), hi = column4(p + 16 * RV * 16);
      return u32x4{lo.x, lo.y, hi.x, hi.y};
    };
    // products of the keys (rows) and queries (columns; lane c has two) with their decays, as operands
    auto decayed_products = [&](const f32x4 (&p)[3], int c, u32x4 (&pa)[2]) {
      const float Gi0 = D.Gs[c], Gi1 = D.Gs[16 + c];
      const f32x4 Gj0 = *reinterpret_cast<const f32x4*>(&D.G[4 * g4]), Gj1 = *reinterpret_cast<const f32x4*>(&D.G[16 + 4 * g4]);
      float w00[4], w01[4], w11[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        w00[r] = 4 * g4 + r <= c ? p[0][r] * __builtin_amdgcn_exp2f(Gi0 - Gj0[r]) : 0.f;
        w01[r] = p[1][r] * __builtin_amdgcn_exp2f(Gi1 - Gj0[r]);
        w11[r] = 4 * g4 + r <= c ? p[2][r] * __builtin_amdgcn_exp2f(Gi1 - Gj1[r]) : 0.f;
      }
      // (the scale's sign, in both halves)
      const uint32_t flip = sign | sign >> 16;
      pa[0] = u32x4{pack_bf16x2(w00[0], w00[1]) ^ flip, pack_bf16x2(w00[2], w00[3]) ^ flip, 0u, 0u};
      pa[1] = u32x4{pack_bf16x2(w01[0], w01[1]) ^ flip, pack_bf16x2(w01[2], w01[3]) ^ flip,
                    pack_bf16x2(w11[0], w11[1]) ^ flip, pack_bf16x2(w11[2], w11[3]) ^ flip};
    };
    // the state's part of the output, by the decays and the scale
    auto scaled = [&](f32x4 (&o)[2][NT], int c) {
      const float fs = __uint_as_float(__float_as_uint(__builtin_amdgcn_exp2f(f_before)) ^ sign);
      const float e0 = __builtin_amdgcn_exp2f(D.Gs[c]) * fs, e1 = __builtin_amdgcn_exp2f(D.Gs[16 + c]) * fs;
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[0][n] = o[0][n] * e0;
        o[1][n] = o[1][n] * e1;
      }
    };
    // The state's part of the output (rows: columns of the state, columns: queries),
    // before this chunk enters the state, and the decayed products as operands.
    auto products = [&](int at0, int c, f32x4 (&oa)[2][NT], u32x4 (&pa)[2]) {
      f32x4 p[3];
      p[0] = p[1] = p[2] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int n = 0; n < NT; ++n) oa[0][n] = oa[1][n] = f32x4{0.f, 0.f, 0.f, 0.f};
      u32x4 qf[kTight ? 1 : DK / 32][2];
      auto of_state = [&](int s, const u32x4 (&q)[2]) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const u32x4 sb = state_operand(s, n);
          oa[0][n] = mfma16(sb, q[0], oa[0][n]);
          oa[1][n] = mfma16(sb, q[1], oa[1][n]);
        }
      };
#pragma unroll
      for (int s = 0; s < DK / 32; ++s) {
        const int at = at0 ^ 64 * s;
        u32x4 q[2], k[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          q[h] = piece(T.q + h * (16 * RQ), at);
          k[h] = piece(T.k + h * (16 * RQ), at);
        }
        p[0] = mfma16(k[0], q[0], p[0]);
        p[1] = mfma16(k[0], q[1], p[1]);
        p[2] = mfma16(k[1], q[1], p[2]);
        if constexpr (kTight) {
          of_state(s, q);
        } else {
          qf[s][0] = q[0];
          qf[s][1] = q[1];
        }
      }
      if constexpr (!kTight) {
#pragma unroll
        for (int s = 0; s < DK / 32; ++s) of_state(s, qf[s]);
      }
      decayed_products(p, c, pa);
      scaled(oa, c);
    };
    u32x4 vf[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) vf[n] = values(n, va);
    if constexpr (!STATE) {
      f32x4 oa[2][NT];
      u32x4 pa[2];
      products(ra, c16, oa, pa);
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        oa[0][n] = mfma16(vf[n], pa[0], oa[0][n]);
        oa[1][n] = mfma16(vf[n], pa[1], oa[1][n]);
      }
      store_out(oa);
    }
    // the chunk enters the state: the decayed values in three bf16 parts, which
    // hold all 24 bits of them
    u32x4 part[NT][3];
    auto make_parts = [&] {
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(&D.w[4 * g4]), w1 = *reinterpret_cast<const f32x4*>(&D.w[16 + 4 * g4]);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          const f32x4 ww = p < 2 ? w0 : w1;
          float x[2] = {bf16lo(vf[n][p]) * ww[2 * (p & 1)], bf16hi(vf[n][p]) * ww[2 * (p & 1) + 1]};
#pragma unroll
          for (int k = 0; k < 3; ++k) {
            part[n][k][p] = __builtin_amdgcn_perm(__float_as_uint(x[1]), __float_as_uint(x[0]), 0x07060302);
#pragma unroll
            for (int e = 0; e < 2 && k < 2; ++e) x[e] -= __uint_as_float(__float_as_uint(x[e]) & 0xFFFF0000u);
          }
        }
    };
    if constexpr (!kTight) make_parts();
    if constexpr (STATE) sum += D.total;
    // An infinity or NaN among the values met products of zero, which carried it
    // to earlier tokens: the output is formed again, token after token.
    bool again = false;
    if constexpr (!STATE) {
      u16x2 top = {0, 0};
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int p = 0; p < 4; ++p) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, vf[n][p] & 0x7FFF7FFFu));
      again = __ballot(max(top.x, top.y) >= 0x7F80) != 0;
    }
    if (again || !keeps(decayed)) {
      if (!STATE && again) {
        int q = c16;
        asm volatile("" : "+v"(q));  // (nothing of this is prepared or kept outside)
        asm volatile("" : "+v"(ra), "+v"(va));
        f32x4 oa[2][NT];
        u32x4 pa[2];
        products(ra, q, oa, pa);
#pragma unroll
        for (int n = 0; n < NT; ++n) vf[n] = values(n, va);
#pragma unroll 1
        for (int j = 0; j < kChunk; ++j) {
          // token j in an operand: word 2 (j / 16) + j / 2 % 2 of lane group j / 4 % 4
          const uint32_t half = g4 == (j >> 2 & 3) ? (j & 1 ? 0xFFFF0000u : 0xFFFFu) : 0u;
          const int word = 2 * (j >> 4) + (j >> 1 & 1);
          auto only = [&](const u32x4& x) {
            return u32x4{word == 0 ? x.x & half : 0u, word == 1 ? x.y & half : 0u, word == 2 ? x.z & half : 0u, word == 3 ? x.w & half : 0u};
          };
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const f32x4 y0 = mfma16(only(vf[n]), only(pa[0]), oa[0][n]), y1 = mfma16(only(vf[n]), only(pa[1]), oa[1][n]);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              oa[0][n][r] = q >= j ? y0[r] : oa[0][n][r];
              oa[1][n][r] = 16 + q >= j ? y1[r] : oa[1][n][r];
            }
          }
        }
        store_out(oa);
      }
      asm volatile("");  // (keeps the products in the branch)
      const float by = keeps(decayed) ? 1.f : __builtin_amdgcn_exp2f(decayed);
#pragma unroll
      for (int i = 0; i < DK / 16; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n) S[i][n] = S[i][n] * by;
    }
    if constexpr (kTight) make_parts();
    u32x4 kt[2][2];
    auto columns = [&](int s) {
      const uint8_t* p = reinterpret_cast<const uint8_t*>(T.k) + (ka ^ 64 * s);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const u32x2 lo = column4(p + 8 * e), hi = column4(p + 8 * e + 16 * RQ * 16);
        kt[s & 1][e] = u32x4{lo.x, lo.y, hi.x, hi.y};
      }
    };
    columns(0);
#pragma unroll
    for (int s = 0; s < DK / 32; ++s) {
      if (s + 1 < DK / 32) columns(s + 1);
      // (the small parts first)
#pragma unroll
      for (int k = 2; k >= 0; --k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int n = 0; n < NT; ++n) S[2 * s + e][n] = mfma16(kt[s & 1][e], part[n][k], S[2 * s + e][n]);
      __builtin_amdgcn_sched_barrier(0);  // (else the reads sink to their uses)
    }
    if (!STATE && (q0.flags & kLast)) {
      if (q0.out >= 0) store_state(a.state_out + q0.out * state_values(a) + head * head_state, __builtin_amdgcn_exp2f(f));
    }
    if (!(q1.flags & kItem)) break;
    q0 = q1;
    st = st == 2 ? 0 : st + 1;
  }
  if constexpr (STATE) {
    store_state(ps.state + w * state_values(a) + head * head_state, __builtin_amdgcn_exp2f(f));
    if (slice == 0 && tid == 0) ps.decay[w * a.v_heads + head] = __builtin_amdgcn_exp2f(sum);
  }
}

// What windows pass on: S at the end of each, from what each adds. Thread: four
// values of one head's state, window after window; what the next eight windows
// add is under way meanwhile. Latency bounds it: 15 windows of 32 heads 13 us.
__global__ __launch_bounds__(256) void linear_pass_kernel(LinearArgs a) {
  __shared__ struct {
    int on, begins, slot;
    float decay;
  } meta[kMaxWindows];
  const Passed ps = passed(a);
  const int head = blockIdx.y, n = a.windows - 1;
  for (int w = threadIdx.x; w < n; w += 256) {
    meta[w].on = ps.meta[4 * w];
    meta[w].begins = ps.meta[4 * w + 1];
    meta[w].slot = ps.meta[4 * w + 2];
    meta[w].decay = ps.decay[w * a.v_heads + head];
  }
  const int64_t head_state = (int64_t)a.qk_dim * a.v_dim;
  const int64_t at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  const int64_t stride = state_values(a), off = head * head_state + at;
  constexpr int kAhead = 8;
  f32x4 add[2][kAhead], start[2][kAhead];
  auto load = [&](auto s_, int w0) {
    constexpr int s = decltype(s_)::value;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int w = min(w0 + j, n - 1);
      add[s][j] = *reinterpret_cast<const f32x4*>(ps.state + w * stride + off);
      start[s][j] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (meta[w].on && meta[w].begins && meta[w].slot >= 0)
        start[s][j] = *reinterpret_cast<const f32x4*>(a.state_in + meta[w].slot * stride + off);
    }
  };
  f32x4 S = {0.f, 0.f, 0.f, 0.f};
  auto pass = [&](auto s_, int w0) {
    constexpr int s = decltype(s_)::value;
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int w = w0 + j;
      if (w >= n || !meta[w].on) continue;
      if (meta[w].begins) {
        S = start[s][j];
        if (a.copied) *reinterpret_cast<f32x4*>(ps.start + w * stride + off) = S;
      }
      S = S * meta[w].decay + add[s][j];
      *reinterpret_cast<f32x4*>(ps.state + w * stride + off) = S;
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  __syncthreads();
  if (at >= head_state) return;
  load(I0{}, 0);
  for (int w0 = 0; w0 < n; w0 += 2 * kAhead) {
    load(I1{}, w0 + kAhead);
    pass(I0{}, w0);
    load(I0{}, w0 + 2 * kAhead);
    pass(I1{}, w0 + kAhead);
  }
}

namespace {

// In a call of kManySeqs sequences or more, those of up to kShortTokens tokens are
// walked through by linear_walk_kernel, a block a sequence, head and 32 columns; in
// chunks they follow each other within a window, at 2.5 us each with 4 heads of
// 128 x 128 and 10 with 32. Chunks alone against the walk for short ones: 256
// single tokens and a prompt of 2000, 32 heads, 1393 and 325 us, 4 heads 344 and
// 69; 16 sequences of 4 tokens and two of 300, 4 heads, 52 and 29 (32 heads: 46
// and 53); 64 of 8 tokens and one of 500, 32 heads, 127 and 117. Where all are
// short enough for one window, chunks lose nothing: 8 sequences of a token, 32
// heads, 11.5 and 12.6, 64 of 8 tokens 62 and 88; with 4 heads, in several
// windows, 30 and 28. Limits of 1, 4, 8, 16 and 32 tokens: 64 of 8 and one of 500,
// 32 heads, 133, 133, 117, 115, 116; 64 of 16 and one of 500, 111, 112, 111, 172,
// 168 (a walk takes a token at a time). Below 8 sequences a launch more costs about
// what it saves: 4 sequences of a token 7.4 and 8.0, of 8 tokens 7.4 and 13.4.
constexpr int kManySeqs = 8, kShortTokens = 8;

// Columns of a state a block holds. Half of them where that fills the chip
// better than it costs in keys and queries read again: turns, states and their
// passing take less time. Heads of 128 x 128, 128 columns against 64: 16 heads of
// 4096 tokens 58, 50 us, of 8192 82, 77; 32 heads of 1777 tokens 54, 47, of 4096
// 81, 77, of 8192 120, 128; 64 heads of 1777 tokens 75.5, 73.4, of 2500 90.1,
// 90.7, of 4096 124, 131. The rule is that of 128 x 128; 16 heads of other sizes,
// 128 columns against 64: 96 x 80, 300 tokens 21.7, 16.0 us, 1777 34.2, 37.1, 4096
// 49.4, 47.2, 8192 68.3, 70.5; 64 x 128, 300 tokens 16.3, 13.3, 4096 45.2, 37.7,
// 8192 60.1, 56.2. (More than 128 rows leave no registers for 128 columns.)
int chunk_cols(const LinearArgs& a, int64_t T) {
  return a.qk_dim > 128 || a.v_dim <= 64 || T * a.v_heads <= 144 * 1024 ? 64 : 128;
}
// Windows for T tokens: enough for two blocks on each compute unit, of 64 tokens
// at least, of 128 from 1024 tokens on; one for few tokens, where two launches
// more cost more than they save, the more so the more heads the windows' states
// are passed for. One sequence of heads of 128 x 128, one window against
// windows: 4 heads of 384 tokens 17.8, 18.7 us, of 448 20.0, 19.4; 16 heads of
// 512 tokens 22.6, 23.2, of 768 31.7, 29.2; 32 heads of 768 tokens 32.4, 34.8, of
// 1024 41.3, 38.2; 64 heads of 1024 tokens 41.9, 54.5. Windows of at least 64
// and 128 tokens: 12 heads of 1024 tokens 29.3, 25.3, of 1777 35.8, 34.4. Other
// sizes, one window against windows: 16 heads of 64 x 64, 300 tokens 13.2, 17.8, 768
// 25.9, 20.8; of 200 x 200, 512 tokens 34.2, 50.7, 1024 61.5, 57.4; of 256 x 256, 768
// tokens 48.6, 58.8, 1024 62.0, 64.9, 1777 103, 78; 4 heads of 256 x 256, 300 tokens
// 22.6, 26.0, 512 33.0, 30.2; 64 heads of 64 x 64, 768 tokens 26.8, 30.9, 1024 34.0,
// 31.4.
int most_windows(const LinearArgs& a, int64_t T) {
  const int per = a.v_heads * ((a.v_dim + chunk_cols(a, T) - 1) / chunk_cols(a, T));
  const int64_t least = T < 1024 ? 64 : 128;
  if (T <= 384 + 6 * std::min(per, 128)) return 1;
  return (int)std::max<int64_t>(1, std::min<int64_t>(std::max(1, kMaxWindows / per), (T + least - 1) / least));
}
void set_windows(LinearArgs& a) {
  const int most = most_windows(a, a.T);
  a.window = (int)((((int64_t)a.T + most - 1) / most + kChunk - 1) / kChunk * kChunk);
  a.windows = std::max(1, (a.T + a.window - 1) / std::max(a.window, 1));
  // one window's sequences need not follow each other
  const int per = a.v_heads * ((a.v_dim + chunk_cols(a, a.T) - 1) / chunk_cols(a, a.T));
  a.strands = a.windows > 1 ? 1 : std::max(1, std::min(a.n_seqs, kMaxWindows / per));
}

template <int DK, int NT>
hipError_t launch_chunks(const LinearArgs& a, hipStream_t s) {
  const int slices = (a.v_dim + 64 * NT - 1) / (64 * NT), per = a.v_heads * slices;
  const auto grid = [](int units) { return dim3((units + 7) / 8 * 8); };
  if (a.windows > 1) {
    hipLaunchKernelGGL((linear_chunk_kernel<DK, NT, 3, true>), grid((a.windows - 1) * per), dim3(kChunkThreads), 0, s, a);
    hipLaunchKernelGGL(linear_pass_kernel, dim3((a.qk_dim * a.v_dim + 1023) / 1024, a.v_heads), dim3(256), 0, s, a);
  }
  hipLaunchKernelGGL((linear_chunk_kernel<DK, NT, 3, false>), grid(a.windows * a.strands * per), dim3(kChunkThreads), 0, s, a);
  return hipGetLastError();
}

// Sequences of at most a.short_tokens.
hipError_t launch_walk(const LinearArgs& a, hipStream_t s) {
  const dim3 grid(a.n_seqs, a.v_heads, (a.v_dim + kStepCols - 1) / kStepCols), block(256);
  if (a.qk_dim <= 64)
    hipLaunchKernelGGL(linear_walk_kernel<2>, grid, block, 0, s, a);
  else if (a.qk_dim <= 128)
    hipLaunchKernelGGL(linear_walk_kernel<4>, grid, block, 0, s, a);
  else
    hipLaunchKernelGGL(linear_walk_kernel<8>, grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace

size_t linear_ws_bytes(const LinearArgs& a) {
  // (a workspace for T tokens serves fewer)
  const int64_t n = std::max(most_windows(a, a.T), most_windows(a, std::min(a.T, 1023)));
  if (n <= 1) return 0;
  return (size_t)(n * (16 + 4 * (int64_t)a.v_heads + 8 * state_values(a)) + 16);
}

hipError_t launch_linear_attention(const LinearArgs& in, hipStream_t s) {
  LinearArgs a = in;
  a.short_tokens = a.n_seqs >= kManySeqs ? kShortTokens : -1;
  if (a.short_tokens >= 0) {
    const hipError_t e = launch_walk(a, s);
    if (e != hipSuccess || a.T <= 0) return e;
  }
  set_windows(a);
  // states written where others are read: sequences that go over several windows start from a copy
  const uintptr_t ib = reinterpret_cast<uintptr_t>(a.state_in), ob = reinterpret_cast<uintptr_t>(a.state_out);
  const uintptr_t bytes = 4 * (uintptr_t)state_values(a);
  a.copied = a.windows > 1 && a.state_in && a.state_out && ib < ob + a.n_out * bytes && ob < ib + a.n_in * bytes;
  if (a.qk_dim > 128) return launch_chunks<256, 1>(a, s);
  if (chunk_cols(a, a.T) == 64) return a.qk_dim <= 64 ? launch_chunks<64, 1>(a, s) : launch_chunks<128, 1>(a, s);
  return a.qk_dim <= 64 ? launch_chunks<64, 2>(a, s) : launch_chunks<128, 2>(a, s);
}

hipError_t launch_linear_step(const LinearArgs& in, hipStream_t s) {
  LinearArgs a = in;
  a.short_tokens = 1;
  return launch_walk(a, s);
}

}  // namespace moe
