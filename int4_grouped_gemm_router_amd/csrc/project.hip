// A projection by packed int4 weights beside the low-rank adapters of many
// requests (gfx950, bf16 matrix cores, fp32 accumulation).
//
//   z[t] = scales[a] * A_a x[t],  y[t] = W x[t] + B_a z[t],  a = adapter_of[t]
//
// Two launches: the adapters' first product z into the workspace (fp32 sums,
// kept as two bf16 halves: 16 significant bits), then the projection, in
// whose epilogue B_a z is a few more matrix-core operations per tile. One
// launch for one or two tokens of low rank.
//
// Tokens are never sorted by adapter: a 16-token tile walks over the distinct
// adapters of its tokens (one in a prompt, up to 16 in a batch of single
// tokens, where every adapter's bytes have to be read anyway), and a token
// takes the results of its own adapter by selection, so that another
// adapter's NaN or infinity never reaches it.
//
// The projection has two kernels:
//   project_split_kernel  exact codes; a block's eight waves split K and join
//                         through LDS: few rows, where the weights' bytes and
//                         the latency of one pass count
//   project_tile_kernel   256 x 256 tiles; each weight is expanded once per
//                         tile to bf16 and shared through LDS by its 256
//                         rows: many rows, where the matrix cores count
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "topk.h"
#include "wide_expand.h"

namespace moe {

namespace {

constexpr int kPWaves = 8;
constexpr int kPThreads = 64 * kPWaves;
// T R up to which the projection's blocks form z themselves, each reading all
// of the adapters' rows, and the launch before them is spared: two rows a wave,
// one pass. N 512 to 12288 and K 512 to 16384, in a graph: 0.82 to 0.98 of the
// two launches' time (4096 x 16384: 1.04); 32 rows, two passes, 1.04 to 1.5.
constexpr int kFusedRows = 2 * kPWaves;

// The adapter of token t, or -1.
__device__ inline int adapter_at(const ProjectArgs& a, int t) {
  const int i = t < a.T ? a.adapter_of[t] : -1;
  return i >= 0 && i < a.n ? i : -1;
}

// As the load and what is made of it, where other loads go in between.
__device__ inline int rank_load(const ProjectArgs& a, int i) { return a.ranks ? a.ranks[i] : a.R; }
__device__ inline int rank_value(const ProjectArgs& a, int v) { return min(max(v, 0), a.R); }
__device__ inline int rank_of(const ProjectArgs& a, int i) { return rank_value(a, rank_load(a, i)); }

// The distinct adapters of a wave's rows (lane r: row r's, or -1), in row
// order, found for all rows at once from one ballot per bit of the adapters'
// indices.
struct Distinct {
  int mine, n;      // n: how many
  uint64_t same;    // the lane's: rows of its adapter
  int place;        // of the lane's adapter, if its row is the first with it, else -1
  __device__ Distinct(int adapter, int adapters) : mine(adapter) {
    same = __ballot(mine >= 0);
    for (int b = 0; b < 31 && (adapters - 1) >> b; ++b) {
      const uint64_t bit = __ballot(mine >> b & 1);
      same &= mine >> b & 1 ? bit : ~bit;
    }
    const bool is = mine >= 0 && !(same & lanemask_lt());
    const uint64_t firsts = __ballot(is);
    n = __popcll(firsts);
    place = is ? __popcll(firsts & lanemask_lt()) : -1;
  }
  // The j-th (j < n) and its rows.
  __device__ int at(int j, uint64_t& rows) const {
    const int lane = __builtin_ctzll(__ballot(place == j));
    rows = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((uint32_t)(same >> 32), lane) << 32 |
           (uint32_t)__builtin_amdgcn_readlane((uint32_t)same, lane);
    return __builtin_amdgcn_readlane(mine, lane);
  }
};

// z's two halves [T][R]: the bf16 value nearest to z, and that of the rest. They
// enter the matrix cores as they are, and their 16 bits miss at most 2^-16 of z,
// far below y's own rounding (2^-8).
__device__ inline uint16_t* z_hi(const ProjectArgs& a) { return static_cast<uint16_t*>(a.ws); }
__device__ inline uint16_t* z_lo(const ProjectArgs& a) { return z_hi(a) + (int64_t)a.T * a.R; }

// A fragment (16 rows x 32 inputs, 16 bytes a lane) is copied from rows in
// memory to LDS by a wave: lane l copies chunk frag_chunk(l) (8 inputs) of row
// frag_row(l) to slot l. Four lanes cover a row's 64 bytes: sixteen lanes in a
// row that each read another row cost the address unit a cycle each, four
// times as long. Lane (c16, kb) of the matrix cores finds row c16, chunk kb in
// frag_slot(c16, kb); the chunks are swizzled so that the sixteen rows of one
// chunk lie in different LDS banks.
__device__ inline int frag_row(int l) { return l >> 2; }
__device__ inline int frag_chunk(int l) { return (l & 3) ^ (l >> 4); }
__device__ inline int frag_slot(int c16, int kb) { return 4 * c16 + (kb ^ (c16 >> 2)); }

// Waits until all but the newest N vector memory operations are done.
template <int N>
__device__ inline void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// The first `left` of eight ranks, the others zero.
__device__ inline u32x4 rank_mask(u32x4 v, int left) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = left >= 2 * j + 2 ? v[j] : (left == 2 * j + 1 ? v[j] & 0xFFFFu : 0u);
  return v;
}

// Sum over the wave, in every lane.
__device__ inline float sum_lanes(float v) {
  const auto at = [](uint32_t u) { return __uint_as_float(u); };
  v += at(dpp<0xB1>(__float_as_uint(v)));
  v += at(dpp<0x4E>(__float_as_uint(v)));
  v += at(dpp<0x141>(__float_as_uint(v)));
  v += at(dpp<0x140>(__float_as_uint(v)));
  const auto row = [&](int l) { return at(__builtin_amdgcn_readlane(__float_as_uint(v), l)); };
  return (row(0) + row(16)) + (row(32) + row(48));
}

// Eight consecutive ranks from r0 of row `row` of a [rows][R] array, zero
// from rank `have` (<= R) on.
__device__ inline u32x4 rank_chunk(const uint16_t* base, int64_t row, int R, int r0, int have) {
  u32x4 v = {0u, 0u, 0u, 0u};
  const int left = have - r0;
  if (left > 0) {
    v = *reinterpret_cast<const u32x4*>(base + row * R + r0);
    if (left < 8) v = rank_mask(v, left);
  }
  return v;
}

}  // namespace

// The adapters' first product. Block: one tile of 16 tokens, every
// `entries`-th distinct adapter of the tile and every `parts`-th 16 ranks of
// it; the eight waves split K in chunks of 128 inputs, kHeld of them at a time
// in the wave's own part of LDS (no barrier: the wave waits for its copies).
// Grid: token tiles x parts x entries (entries fastest). What counts is
// latency: the activations are under way before the adapters are known and
// serve every entry while they are held, and an entry's part of A is under way
// before its rank is known. K = 2048, rank 16: 4.3 us for 32 tokens of 32
// adapters (2.1 MB of them), 7.2 for 4096 tokens.
struct DownLds {
  static constexpr int kHeld = 2;
  u32x4 x[kPWaves][kHeld][4][64], a[kPWaves][kHeld][4][64];  // [wave][chunk][32 inputs][frag_slot]
  float red[kPWaves][16][17];
};

__global__ __launch_bounds__(kPThreads) void adapter_down_kernel(ProjectArgs a, int entries, int parts) {
  __shared__ DownLds L;
  constexpr int kHeld = DownLds::kHeld;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kb = lane >> 4;
  const int n_rt = (a.R + 15) / 16;
  const int entry = blockIdx.x % entries, part = blockIdx.x / entries % parts;
  const int t0 = blockIdx.x / entries / parts * 16;
  const int id = a.adapter_of[min(t0 + c16, a.T - 1)];
  const int chunks = a.K / 128, batches = (chunks + kPWaves * kHeld - 1) / (kPWaves * kHeld);
  const int slot = frag_slot(c16, kb);
  // wave w's chunks of a batch: w, w + 8 (chunks past the last repeat it and are not used)
  auto chunk = [&](int batch, int h) { return batch * kPWaves * kHeld + kPWaves * h + wave; };
  auto copy = [&](rsrc_t r, uint32_t off, int batch, u32x4 (&dst)[kHeld][4][64]) {
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        bload_lds(r, &dst[h][s][0], off + 64 * s, (uint32_t)min(chunk(batch, h), chunks - 1) * 256);
  };
  const int rows = min(16, a.T - t0);
  const rsrc_t xres = make_rsrc(a.x + (int64_t)t0 * a.ldx, (uint32_t)(((int64_t)(rows - 1) * a.ldx + a.K) * 2));
  const uint32_t xoff = (uint32_t)min(frag_row(lane), rows - 1) * (uint32_t)(a.ldx * 2) + 16 * frag_chunk(lane);
  int held = 0;
  copy(xres, xoff, 0, L.x[wave]);
  const Distinct adapters(lane < rows && id >= 0 && id < a.n ? id : -1, a.n);
  for (int j = entry; j < adapters.n; j += entries) {
    uint64_t same;
    const int ad = adapters.at(j, same);
    for (int rt = part; rt < n_rt; rt += parts) {
      const int ranks = min(16, a.R - 16 * rt);
      const rsrc_t ares = make_rsrc(a.A + ((int64_t)ad * a.R + 16 * rt) * a.K, (uint32_t)ranks * (uint32_t)a.K * 2);
      const uint32_t aoff = (uint32_t)min(frag_row(lane), ranks - 1) * (uint32_t)(a.K * 2) + 16 * frag_chunk(lane);
      f32x4 acc = {0.f, 0.f, 0.f, 0.f};
      const int rank_read = rank_load(a, ad);
      const float scale = a.scales ? a.scales[ad] : 1.f;
      for (int b = 0; b < batches; ++b) {
        if (held != b) copy(xres, xoff, b, L.x[wave]);
        held = b;
        copy(ares, aoff, b, L.a[wave]);
        wait_loads<0>();
#pragma unroll
        for (int h = 0; h < kHeld; ++h)
          if (chunk(b, h) < chunks) {
#pragma unroll
            for (int s = 0; s < 4; ++s) acc = mfma16(L.x[wave][h][s][slot], L.a[wave][h][s][slot], acc);
          }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next copies
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) L.red[wave][4 * kb + i][c16] = acc[i];
      __syncthreads();
      if (tid < 256) {
        const int row = tid >> 4, r = 16 * rt + (tid & 15);
        if ((same >> row & 1) && r < a.R) {
          float v = 0.f;
#pragma unroll
          for (int w = 0; w < kPWaves; ++w) v += L.red[w][row][tid & 15];
          v *= scale;
          if (r >= rank_value(a, rank_read)) v = 0.f;
          const uint16_t hi = f2bf(v);
          const int64_t at = (int64_t)(t0 + row) * a.R + r;
          z_hi(a)[at] = hi;
          z_lo(a)[at] = f2bf(v - bf16f(hi));
        }
      }
      __syncthreads();
    }
  }
  wait_loads<0>();  // no copy outlives its block
}

// Few rows: a block owns 16 MS tokens and 16 CT columns; wave w takes the
// 64-input groups w, w + 8, ... on its own: D groups ahead, the codes go to
// registers and the activations to the wave's own ring in LDS (no barrier:
// the wave waits for its copies), and the eight partial tiles are added in
// LDS in a fixed order. With the codes expanded to the exact bf16 values
// 128 + q, per group and column
//   acc += s * x.(128 + q) + (b - 128 s) * sum(x)
// which is x . (q s + b) with the weights used exactly. The distinct adapters
// of the tokens are dealt out over the waves too; their operands are loaded
// before the groups' products (NE adapters a wave, the first 32 ranks; the wait
// for an adapter's rank, the same in every lane, stands before its operands and
// drains the first groups' loads as well), and their B_a z goes to a tile of its
// own, added last, so a token's result does not depend on the others. 4096 x
// 2048: 7.4 us for one token with an adapter of rank 16 (latency of one pass,
// FUSED), 7.4 for 32 tokens with 32 adapters; 2048 x 2048 for 500 tokens: 13.6
// (one round of blocks, two waves a SIMD: waves wait 0.42 of their time, vector
// instructions issue in 0.24 of the SIMDs' and matrix cores are busy in 0.11).
template <int MS, int CT, int D>
struct SplitLds {
  static constexpr int kStride = 16 * CT + 4;  // floats; the pad spreads the rows over the banks
  static constexpr int kPlanes = MS * CT >= 16 ? 4 : 8;  // partial tiles held at once
  union {
    u32x4 x[kPWaves][D][MS][2][64];           // [wave][slot][16-token subtile][k half][frag_slot]
    float red[kPlanes + 1][16 * MS][kStride]; // the waves' tiles, then the adapters'
  };
};

// FUSED (T R <= kFusedRows): every block forms z itself, a wave one or two of
// the adapters' rows.
template <int MS, int CT, int D, int NE, bool FUSED>
__global__ __launch_bounds__(kPThreads, 2) void project_split_kernel(ProjectArgs a) {
  typedef SplitLds<MS, CT, D> Lds;
  __shared__ Lds L;
  __shared__ float zs[FUSED ? kFusedRows : 1];  // [T][R]
  static_assert(!FUSED || MS == 1, "the tokens are in one tile");
  constexpr int kSub = 4 / CT;  // blocks per 64-column wave tile
  constexpr int NW = CT == 4 ? 2 : 1;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kb = lane >> 4;
  const PackGeom geom = pack_geom(a.N, a.K, 0);
  const int G = geom.G;
  const int row_tiles = (a.T + 16 * MS - 1) / (16 * MS);
  // XCD x (blocks go to XCD b % 8 in turn) takes a contiguous range of units,
  // row tiles fastest, so the row tiles of one column tile share its weights
  // in that XCD's L2
  const int units = row_tiles * geom.n_wt * kSub;
  const int xcd = blockIdx.x & 7;
  const int u0 = (int)((int64_t)units * xcd / 8), u1 = (int)((int64_t)units * (xcd + 1) / 8);
  const int u = u0 + (blockIdx.x >> 3);
  if (u >= u1) return;
  const int t0 = u % row_tiles * (16 * MS), cb = u / row_tiles;
  const int wt = cb / kSub, ct0 = CT * (cb % kSub);
  const ExpandConsts xk = expand_consts();
  const u32x4 ones = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};

  const int id = a.adapter_of ? a.adapter_of[min(t0 + lane, a.T - 1)] : -1;
  const int rows = min(16 * MS, a.T - t0);
  const rsrc_t xres = make_rsrc(a.x + (int64_t)t0 * a.ldx, (uint32_t)(((int64_t)(rows - 1) * a.ldx + a.K) * 2));
  uint32_t xoff[MS];
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
    xoff[ms] = (uint32_t)min(16 * ms + frag_row(lane), rows - 1) * (uint32_t)(a.ldx * 2) + 16 * frag_chunk(lane);
  const int xl = frag_slot(c16, kb);
  const rsrc_t wres = make_rsrc(a.blob, (uint32_t)geom.expert_bytes);
  const uint32_t nbase = (uint32_t)(geom.nib_off + (int64_t)wt * G * kNibBytes + (ct0 >> 1) * 1024 + (ct0 & 1) * 8);
  const uint32_t sbase = (uint32_t)(geom.sb_off + (int64_t)wt * G * kSbBytes);

  // this wave's groups: wave, wave + 8, ... (loads past the last repeat it
  // and are not used)
  const int ng = wave < G ? (G - wave + kPWaves - 1) / kPWaves : 0;
  int next = wave;
  u32x4 w[D][NW], sb[D];
  auto load = [&](int s) {
    const uint32_t g = (uint32_t)min(next, G - 1);
    next += kPWaves;
#pragma unroll
    for (int ms = 0; ms < MS; ++ms) {
      bload_lds(xres, &L.x[wave][s][ms][0][0], xoff[ms], g * (2 * kGroup));
      bload_lds(xres, &L.x[wave][s][ms][1][0], xoff[ms] + 64, g * (2 * kGroup));
    }
    if constexpr (CT == 1) {
      const u32x2 v = bload2(wres, lane * 16, nbase + g * kNibBytes);
      w[s][0] = u32x4{v.x, v.y, 0u, 0u};
    } else {
#pragma unroll
      for (int h = 0; h < NW; ++h) w[s][h] = bload(wres, lane * 16, nbase + g * kNibBytes + 1024 * h);
    }
    sb[s] = bload(wres, c16 * 16, sbase + g * kSbBytes);
  };
#pragma unroll
  for (int s = 0; s < D; ++s) {
    load(s);
    __builtin_amdgcn_sched_barrier(0);  // the waits below count on the slots' order
  }

  // ---- the wave's adapters: the distinct ones of the rows, in row order,
  // every eighth; the first NE's operands are loaded here
  struct Entry {
    int ad;
    uint64_t same;  // its rows
  };
  const int mine = lane < rows && id >= 0 && id < a.n ? id : -1;  // lane r: the adapter of row r
  const uint64_t with = __ballot(mine >= 0);  // rows with an adapter
  auto entry = [&](const Distinct& d, int j) {
    Entry e;
    e.ad = d.at(j, e.same);
    return e;
  };
  struct Operands {
    u32x4 b[CT], zh[MS], zl[MS];
  };
  auto load_operands = [&](const Entry& e, int s, Operands& o) {
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
      o.b[ct] = rank_chunk(a.B, (int64_t)e.ad * a.N + 64 * wt + 16 * (ct0 + ct) + c16, a.R, s + 8 * kb, a.R);
#pragma unroll
    for (int ms = 0; ms < MS; ++ms) {
      if constexpr (FUSED) break;  // (from LDS, by fused_z)
      const int64_t t = min(t0 + 16 * ms + c16, a.T - 1);
      o.zh[ms] = rank_chunk(z_hi(a), t, a.R, s + 8 * kb, a.R);
      o.zl[ms] = rank_chunk(z_lo(a), t, a.R, s + 8 * kb, a.R);
    }
  };
  // z's halves in the place of the workspace's
  auto fused_z = [&](int s, Operands& o) {
    o.zh[0] = o.zl[0] = u32x4{0u, 0u, 0u, 0u};
    const int r0 = s + 8 * kb;
    if (c16 < a.T && r0 < a.R) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v0 = zs[c16 * a.R + r0 + 2 * j], v1 = zs[c16 * a.R + r0 + 2 * j + 1];
        o.zh[0][j] = pack_bf16x2(v0, v1);
        o.zl[0][j] = pack_bf16x2(v0 - bf16lo(o.zh[0][j]), v1 - bf16hi(o.zh[0][j]));
      }
    }
  };
  Entry first[NE];
  Operands ops[NE];
  int rank_first[NE];  // (not yet limited)
  int distinct = 0;
  if (with) {
    const Distinct d(mine, a.n);
    distinct = d.n;
#pragma unroll
    for (int k = 0; k < NE; ++k) {
      first[k].same = 0;
      if (wave + kPWaves * k < distinct) {
        first[k] = entry(d, wave + kPWaves * k);
        rank_first[k] = rank_load(a, first[k].ad);
        load_operands(first[k], 0, ops[k]);
      }
    }
  }
  if constexpr (FUSED) {
    constexpr int kRows = 2, kChunks = 4;  // rows at a time; 512 inputs each
    static_assert(kRows * kPWaves == kFusedRows, "one pass");
    const int n = a.T * a.R;  // (at least 8: one row a wave)
    float sum[kRows] = {0.f, 0.f};
    int ad[kRows], r[kRows];
    const uint16_t *ap[kRows], *xp[kRows];
#pragma unroll
    for (int h = 0; h < kRows; ++h) {
      const int i = min(wave + kPWaves * h, n - 1), t = i / a.R;
      r[h] = i - t * a.R;
      ad[h] = __builtin_amdgcn_readlane(mine, t);
      ap[h] = a.A + ((int64_t)max(ad[h], 0) * a.R + r[h]) * a.K;
      xp[h] = a.x + t * a.ldx;
    }
    for (int k0 = 0; k0 < a.K; k0 += 512 * kChunks) {
      u32x4 av[kRows][kChunks], xv[kRows][kChunks];
#pragma unroll
      for (int j = 0; j < kChunks; ++j) {
        const int k = k0 + 512 * j + 8 * lane;
#pragma unroll
        for (int h = 0; h < kRows; ++h) {
          av[h][j] = xv[h][j] = u32x4{0u, 0u, 0u, 0u};
          if (k < a.K) {
            av[h][j] = *reinterpret_cast<const u32x4*>(ap[h] + k);
            xv[h][j] = *reinterpret_cast<const u32x4*>(xp[h] + k);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kChunks; ++j)
#pragma unroll
        for (int h = 0; h < kRows; ++h)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            sum[h] = __builtin_fmaf(bf16lo(av[h][j][u]), bf16lo(xv[h][j][u]), sum[h]);
            sum[h] = __builtin_fmaf(bf16hi(av[h][j][u]), bf16hi(xv[h][j][u]), sum[h]);
          }
    }
#pragma unroll
    for (int h = 0; h < kRows; ++h) {
      const float v = sum_lanes(sum[h]);
      const bool is = ad[h] >= 0 && r[h] < rank_of(a, max(ad[h], 0));
      if (lane == 0 && wave + kPWaves * h < n)
        zs[wave + kPWaves * h] = is ? v * (a.scales ? a.scales[ad[h]] : 1.f) : 0.f;
    }
  }

  // ---- W x
  f32x4 acc[MS][CT];
#pragma unroll
  for (int ms = 0; ms < MS; ++ms)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) acc[ms][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto step = [&](int s) {
    u32x4 xa[MS][2];
#pragma unroll
    for (int ms = 0; ms < MS; ++ms) {
      xa[ms][0] = L.x[wave][s][ms][0][xl];
      xa[ms][1] = L.x[wave][s][ms][1][xl];
    }
    const uint32_t words[8] = {w[s][0].x, w[s][0].y, w[s][0].z, w[s][0].w, w[s][NW - 1].x, w[s][NW - 1].y,
                               w[s][NW - 1].z, w[s][NW - 1].w};
    f32x4 xs[MS];
#pragma unroll
    for (int ms = 0; ms < MS; ++ms)
      xs[ms] = mfma16(xa[ms][1], ones, mfma16(xa[ms][0], ones, f32x4{0.f, 0.f, 0.f, 0.f}));
    // this block's scales and biases: pairs of column tiles per word
    const uint32_t sw0 = CT == 4 || ct0 < 2 ? sb[s].x : sb[s].y, bw0 = CT == 4 || ct0 < 2 ? sb[s].z : sb[s].w;
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
      const uint32_t sw = ct < 2 ? sw0 : sb[s].y, bw = ct < 2 ? bw0 : sb[s].w;
      const bool hi = CT == 1 ? (ct0 & 1) : (ct & 1);
      const float sc = hi ? bf16hi(sw) : bf16lo(sw), bi = hi ? bf16hi(bw) : bf16lo(bw);
      const float bp = bi - 128.0f * sc;
      const u32x4 b0 = expand_codes(words[2 * ct], xk), b1 = expand_codes(words[2 * ct + 1], xk);
#pragma unroll
      for (int ms = 0; ms < MS; ++ms) {
        f32x4 p = mfma16(xa[ms][0], b0, f32x4{0.f, 0.f, 0.f, 0.f});
        p = mfma16(xa[ms][1], b1, p);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[ms][ct][i] = __builtin_fmaf(bp, xs[ms][i], __builtin_fmaf(sc, p[i], acc[ms][ct][i]));
      }
    }
  };
  for (int i = 0; i < ng; i += D) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      // a slot's copies are in LDS when its codes, loaded after them, are
      // in registers: wait for all but the newer slots' loads
      constexpr int kLoads = 2 * MS + NW + 1;
      wait_loads<kLoads*(D - 1)>();
      if (i + s < ng) step(s);
      // (the slot's reads are done before its next copies are issued)
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      load(s);
    }
  }

  // ---- join
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");  // every copy has landed, every ring is read
  constexpr int kPlanes = Lds::kPlanes;
  auto put = [&](int plane) {
#pragma unroll
    for (int ms = 0; ms < MS; ++ms)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) L.red[plane][16 * ms + 4 * kb + i][16 * ct + c16] = acc[ms][ct][i];
  };
  if (kPlanes == kPWaves) {
    put(wave);
  } else {
    if (wave >= kPlanes) put(wave - kPlanes);
    lds_barrier();
    if (wave < kPlanes) {
#pragma unroll
      for (int ms = 0; ms < MS; ++ms)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int ct = 0; ct < CT; ++ct) acc[ms][ct][i] += L.red[wave][16 * ms + 4 * kb + i][16 * ct + c16];
      put(wave);
    }
  }
  if (with) {
    auto finish = [&](const Entry& e, int rank, Operands& o0) {
      f32x4 d[MS][CT];
#pragma unroll
      for (int ms = 0; ms < MS; ++ms)
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) d[ms][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto add = [&](Operands& o, int s) {
        if constexpr (FUSED) fused_z(s, o);
#pragma unroll
        for (int ct = 0; ct < CT; ++ct) {
          const u32x4 b = rank_mask(o.b[ct], rank - s - 8 * kb);
#pragma unroll
          for (int ms = 0; ms < MS; ++ms) d[ms][ct] = mfma16(o.zl[ms], b, mfma16(o.zh[ms], b, d[ms][ct]));
        }
      };
      add(o0, 0);
      for (int s = 32; s < rank; s += 32) {
        Operands o;
        load_operands(e, s, o);
        add(o, s);
      }
#pragma unroll
      for (int ms = 0; ms < MS; ++ms)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * ms + 4 * kb + i;
          if (e.same >> row & 1) {
#pragma unroll
            for (int ct = 0; ct < CT; ++ct) L.red[kPlanes][row][16 * ct + c16] = d[ms][ct][i];
          }
        }
    };
#pragma unroll
    for (int k = 0; k < NE; ++k)
      if (first[k].same) finish(first[k], rank_value(a, rank_first[k]), ops[k]);
    if (distinct > kPWaves * NE) {
      const Distinct d(mine, a.n);
      for (int j = wave + kPWaves * NE; j < distinct; j += kPWaves) {
        const Entry e = entry(d, j);
        Operands o;
        load_operands(e, 0, o);
        finish(e, rank_of(a, e.ad), o);
      }
    }
  }
  __syncthreads();
  constexpr int kPairs = 8 * CT;  // column pairs per row
  for (int p = tid; p < 16 * MS * kPairs; p += kPThreads) {
    const int row = p / kPairs, c = 2 * (p % kPairs);
    if (t0 + row >= a.T) break;
    float v0 = 0.f, v1 = 0.f;
#pragma unroll
    for (int q = 0; q < kPlanes; ++q) {
      const f32x2 v = *reinterpret_cast<const f32x2*>(&L.red[q][row][c]);
      v0 += v.x;
      v1 += v.y;
    }
    if (with >> row & 1) {
      const f32x2 v = *reinterpret_cast<const f32x2*>(&L.red[kPlanes][row][c]);
      v0 += v.x;
      v1 += v.y;
    }
    *reinterpret_cast<uint32_t*>(a.y + (int64_t)(t0 + row) * a.ldy + 64 * wt + 16 * ct0 + c) = pack_bf16x2(v0, v1);
  }
}

// Many rows: a block of eight waves owns 32 RS tokens x 256 columns; wave w
// owns token half w / 4 (RS 16-token subtiles) and the 64 columns of wave
// tile w % 4. Per 64-input group each weight is expanded once, by one of the
// eight waves (half a wave tile each), to bf16 w = q s + b, and goes to LDS in
// operand order beside the activation rows; each is read by the waves that
// share it. The weights are the first operand of the matrix cores, so that a
// lane ends up with four consecutive columns of one token and stores them
// directly.
//
// The matrix cores take 16 cycles a product; the same SIMD issues about two
// vector instructions under each (two waves a SIMD), so the expansion, about
// 2.4 instructions a weight, is spread evenly over the products, one pair of
// weights per four of them. The unit of the pipeline is half a group (k half,
// 32 inputs): in half h the products of h run while h + 2 is written to LDS,
// and the first operands of h + 1 are read before the barrier that ends h
// (h + 1 was complete at the barrier before). 4096 tokens, 4096 x 2048: 60 to
// 64 us (1.1 PFLOP/s), 69 with adapters of rank 16 (76 to 82 after the first
// millisecond of such calls without a pause). The weights' one rounding leaves
// an error of 1.9e-3, 1.7e-3 of it y's own; the split kernel, which has none,
// takes three times as long.
template <int RS>
struct TileLds {
  u32x4 x[2][2][2 * RS][64];  // [group % 2][k half][16-token subtile][frag_slot]
  u32x4 w[2][2][4][4][64];    // [group % 2][k half][wave tile][column tile][lane]
};

template <int RS>
__global__ __launch_bounds__(kPThreads, 2) void project_tile_kernel(ProjectArgs a) {
  __shared__ TileLds<RS> L;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kb = lane >> 4;
  const int wr = wave >> 2, wc = wave & 3;
  const PackGeom geom = pack_geom(a.N, a.K, 0);
  const int G = geom.G;
  const int row_tiles = (a.T + 32 * RS - 1) / (32 * RS), col_tiles = (geom.n_wt + 3) / 4;
  const int units = row_tiles * col_tiles;
  // XCD x takes a contiguous range of units, column tiles fastest: the rows
  // of few row tiles stay in its L2
  const int xcd = blockIdx.x & 7;
  const int u0 = (int)((int64_t)units * xcd / 8), u1 = (int)((int64_t)units * (xcd + 1) / 8);
  const int u = u0 + (blockIdx.x >> 3);
  if (u >= u1) return;
  const int ctile = u % col_tiles, t0 = u / col_tiles * (32 * RS);
  // the groups are taken in turn from a start that depends on the column
  // tile: rows a multiple of 4 KB apart have one group of every row in the
  // same L2 channel, and blocks in step would all wait for it
  int gx = ctile * G / col_tiles, gw = gx;  // next group to load: activations, codes

  // activations: wave w stages subtiles w * RS / 4, ...
  constexpr int kXRows = RS / 4;
  const int rows = min(32 * RS, a.T - t0);
  const rsrc_t xres = make_rsrc(a.x + (int64_t)t0 * a.ldx, (uint32_t)(((int64_t)(rows - 1) * a.ldx + a.K) * 2));
  uint32_t xoff[kXRows];
#pragma unroll
  for (int f = 0; f < kXRows; ++f)
    xoff[f] = (uint32_t)min(16 * (wave * kXRows + f) + frag_row(lane), rows - 1) * (uint32_t)(a.ldx * 2) +
              16 * frag_chunk(lane);
  const int xl = frag_slot(c16, kb);  // where this lane's operand is in a fragment
  // weights: wave w expands column tiles 2 eh, 2 eh + 1 of wave tile ew
  const int ew = wave >> 1, eh = wave & 1;
  const int ewt = min(4 * ctile + ew, geom.n_wt - 1);
  const rsrc_t wres = make_rsrc(a.blob, (uint32_t)geom.expert_bytes);
  const uint32_t nbase = (uint32_t)(geom.nib_off + (int64_t)ewt * G * kNibBytes + 1024 * eh);
  const uint32_t sbase = (uint32_t)(geom.sb_off + (int64_t)ewt * G * kSbBytes);
  const WideExpand xk = wide_expand_consts();

  // (loads past the last group wrap around and are not used)
  u32x4 cw[2], sbv[2];
  auto load_x = [&](int st, int ks) {
#pragma unroll
    for (int f = 0; f < kXRows; ++f)
      bload_lds(xres, &L.x[st][ks][wave * kXRows + f][0], xoff[f] + 64 * ks, (uint32_t)gx * (2 * kGroup));
    if (ks) gx = gx + 1 < G ? gx + 1 : 0;
  };
  auto load_w = [&](int s) {
    cw[s] = bload(wres, lane * 16, nbase + (uint32_t)gw * kNibBytes);
    sbv[s] = bload(wres, c16 * 16, sbase + (uint32_t)gw * kSbBytes);
    gw = gw + 1 < G ? gw + 1 : 0;
  };
  ColAffine ca[2];
  auto affine = [&](int s) {
    const uint32_t sp = eh ? sbv[s].y : sbv[s].x, bp = eh ? sbv[s].w : sbv[s].z;
    ca[0] = col_affine(bf16lo(sp), bf16lo(bp));
    ca[1] = col_affine(bf16hi(sp), bf16hi(bp));
  };
  u32x4 ex;
  // the p-th of a k half's eight pairs of weights: column tile p / 4, pair p % 4
  auto expand_pair = [&](int s, int ks, int p) {
    ex[p & 3] = expand_bf16x2(cw[s][2 * (p >> 2) + ks], p & 3, ca[p >> 2], xk);
    if ((p & 3) == 3) L.w[s][ks][ew][2 * eh + (p >> 2)][lane] = ex;
  };

  f32x4 acc[RS][4];
#pragma unroll
  for (int ms = 0; ms < RS; ++ms)
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) acc[ms][ct] = f32x4{0.f, 0.f, 0.f, 0.f};

  // group 0 into LDS, group 1 in flight
  load_x(0, 0);
  load_x(0, 1);
  load_w(0);
  load_w(1);
  load_x(1, 0);
  affine(0);
#pragma unroll
  for (int p = 0; p < 16; ++p) expand_pair(0, p >> 3, p & 7);
  load_w(0);  // group 2
  __builtin_amdgcn_s_waitcnt(0);  // (a wait the compiler sees: the loop starts with nothing outstanding)
  lds_barrier();
  // activation operands are read kAhead subtiles ahead of their products (LDS
  // answers in about the time of eight products), the weights' half a half
  constexpr int kAhead = 3, kRing = 4;
  static_assert(RS % kRing == 0 && kAhead < kRing, "ring slots are the same in every half");
  u32x4 av[kRing], bw[2][4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) bw[0][ct] = L.w[0][0][wc][ct][lane];
#pragma unroll
  for (int f = 0; f < kAhead; ++f) av[f] = L.x[0][0][wr * RS + f][xl];
  // half ks of group i in stage S = i % 2; group i + 1's half ks is written meanwhile, from code slot 1 - S
  auto half = [&](auto S_, auto ks_) {
    constexpr int S = decltype(S_)::value, ks = decltype(ks_)::value;
    constexpr int Sn = ks ? 1 - S : S, kn = 1 - ks;  // the half after this one
    if constexpr (ks == 0) affine(1 - S);
    load_x(ks ? S : 1 - S, kn);  // three halves on, into the stage that the last half read
#pragma unroll
    for (int ms = 0; ms < RS; ++ms) {
      const int fa = ms + kAhead;
      av[fa % kRing] = fa < RS ? L.x[S][ks][wr * RS + fa][xl] : L.x[Sn][kn][wr * RS + fa - RS][xl];
      if (ms >= RS / 2) {
#pragma unroll
        for (int q = 0; q < 8 / RS; ++q) {
          const int ct = (ms - RS / 2) * (8 / RS) + q;
          bw[kn][ct] = L.w[Sn][kn][wc][ct][lane];
        }
      }
      // the eight pairs over the first three quarters of the subtiles
#pragma unroll
      for (int p = ms * 32 / (3 * RS); p < min(8, (ms + 1) * 32 / (3 * RS)); ++p) expand_pair(1 - S, ks, p);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) acc[ms][ct] = mfma16(bw[ks][ct], av[ms % kRing], acc[ms][ct]);
      // (without these fences the compiler gathers the reads and spills)
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (ks == 1) load_w(1 - S);  // group i + 3: slot 1 - S is expanded
    // Before any wave goes on: the activations of two halves on are in LDS
    // (what was issued after them may be under way: this half's copies, and
    // two loads of codes), what this half wrote too, and its reads are done
    // (LDS answers in order; the last quarter's reads, of the next half's
    // operands, may be under way).
    static_assert(RS == 8 || RS == 4, "copies per half; reads after the last write");
    if constexpr (RS == 8)
      asm volatile("s_waitcnt vmcnt(4) lgkmcnt(4)\n\ts_barrier" ::: "memory");
    else
      asm volatile("s_waitcnt vmcnt(3) lgkmcnt(3)\n\ts_barrier" ::: "memory");
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;
  for (int g = 0; g < G; g += 2) {  // G is even
    half(I0{}, I0{});
    half(I0{}, I1{});
    half(I1{}, I0{});
    half(I1{}, I1{});
  }

  // ---- B_a z, then y; lane: token c16 of each subtile, columns 4 kb .. 4 kb + 3 of each column tile
  // (the last half's copies into LDS and reads of it end here, in every wave)
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
  const int wt = 4 * ctile + wc;
  if (wt >= geom.n_wt) return;
  const int tw = t0 + 16 * RS * wr;
  if (a.adapter_of) {
    int mine[RS];
#pragma unroll
    for (int ms = 0; ms < RS; ++ms) mine[ms] = adapter_at(a, tw + 16 * ms + c16);
    for (int s = 0; s < a.R; s += 32) {
      int held = -1;
      u32x4 bv[4], zh[2], zl[2];
      auto load_z = [&](int ms) {
        const int64_t t = min(tw + 16 * ms + c16, a.T - 1);
        zh[ms & 1] = rank_chunk(z_hi(a), t, a.R, s + 8 * kb, a.R);
        zl[ms & 1] = rank_chunk(z_lo(a), t, a.R, s + 8 * kb, a.R);
      };
      load_z(0);
#pragma unroll
      for (int ms = 0; ms < RS; ++ms) {
        if (ms + 1 < RS) load_z(ms + 1);
        uint64_t rem = __ballot(mine[ms] >= 0);
        while (rem) {
          const int ad = __builtin_amdgcn_readlane(mine[ms], __builtin_ctzll(rem));
          const bool is = mine[ms] == ad;
          const uint64_t same = __ballot(is);
          rem &= ~same;
          if (ad != held) {
            held = ad;
            const int rank = rank_of(a, ad);
#pragma unroll
            for (int ct = 0; ct < 4; ++ct)
              bv[ct] = rank_chunk(a.B, (int64_t)ad * a.N + 64 * wt + 16 * ct + c16, a.R, s + 8 * kb, rank);
          }
#pragma unroll
          for (int ct = 0; ct < 4; ++ct) {
            const f32x4 d = mfma16(bv[ct], zl[ms & 1], mfma16(bv[ct], zh[ms & 1], f32x4{0.f, 0.f, 0.f, 0.f}));
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[ms][ct][i] = is ? acc[ms][ct][i] + d[i] : acc[ms][ct][i];
          }
        }
      }
    }
  }
  // through LDS, so that eight lanes store a row's 128 bytes (the stages are
  // read no more: the last half's reads wrapped around and are not used)
  constexpr int kRow = 144;  // bytes; 128 and a pad that spreads the rows over the banks
  uint8_t* tr = reinterpret_cast<uint8_t*>(&L) + wave * (2 * 16 * kRow);
#pragma unroll
  for (int ms = 0; ms < RS; ++ms) {
    uint8_t* tb = tr + (ms & 1) * (16 * kRow);
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      u32x2 o;
      o.x = pack_bf16x2(acc[ms][ct][0], acc[ms][ct][1]);
      o.y = pack_bf16x2(acc[ms][ct][2], acc[ms][ct][3]);
      *reinterpret_cast<u32x2*>(tb + c16 * kRow + 32 * ct + 8 * kb) = o;
    }
    // (a wave's LDS accesses execute in order)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = 8 * q + (lane >> 3), t = tw + 16 * ms + r;
      const u32x4 v = *reinterpret_cast<const u32x4*>(tb + r * kRow + 16 * (lane & 7));
      if (t < a.T)
        __builtin_nontemporal_store(v, reinterpret_cast<u32x4*>(a.y + (int64_t)t * a.ldy + 64 * wt + 8 * (lane & 7)));
    }
    asm volatile("" ::: "memory");
  }
}

size_t project_ws_bytes(int /*N*/, int /*K*/, int R, int T) {
  return ((size_t)T * R * 4 + 255) / 256 * 256;
}

namespace {

// Tokens of one launch: HIP takes fewer than 2^32 threads, and the tilings
// that this many tokens choose have at most 2^31 (64 x 64 with 65536 columns;
// the adapters' first product: 2^23). Longer calls are several launches, over
// the same workspace one after the other.
constexpr int kLaunchTokens = 1 << 18;

template <int MS, int CT, int D, int NE, bool FUSED = false>
hipError_t launch_split(const ProjectArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.T + 16 * MS - 1) / (16 * MS)) * (a.N / 64) * (4 / CT);
  const int64_t blocks = (units + 7) / 8 * 8;
  hipLaunchKernelGGL((project_split_kernel<MS, CT, D, NE, FUSED>), dim3((unsigned)blocks), dim3(kPThreads), 0, s, a);
  return hipGetLastError();
}

template <int RS>
hipError_t launch_tile(const ProjectArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.T + 32 * RS - 1) / (32 * RS)) * ((a.N + 255) / 256);
  const int64_t blocks = (units + 7) / 8 * 8;
  hipLaunchKernelGGL(project_tile_kernel<RS>, dim3((unsigned)blocks), dim3(kPThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_project(const ProjectArgs& a, hipStream_t s) {
  // The kernel and tile that take least, from what each measured at K = 2048
  // (all of them grow with K alike): a start and a time per round of 256
  // units, one for each compute unit, in tenths of a microsecond. Small tiles
  // start fastest and lose when there are many: 64 tokens by 4096 columns
  // take 15.2 us in 16 x 16 tiles and 5.3 in 32 x 32, 500 by 2048 31 and 10.3
  // (64 x 64), 1024 by 4096 40 in 64 x 64 and 33 in 128 x 256, 4096 by 4096
  // 77 in 128 x 256 and 62 in 256 x 256.
  struct Tiling {
    int rows, cols, start, round;
    hipError_t (*launch)(const ProjectArgs&, hipStream_t);
    hipError_t (*fused)(const ProjectArgs&, hipStream_t);
  };
  static const Tiling tilings[] = {
      {16, 16, 22, 20, launch_split<1, 1, 4, 2>, launch_split<1, 1, 4, 2, true>},
      {16, 32, 24, 20, launch_split<1, 2, 4, 2>, launch_split<1, 2, 4, 2, true>},
      {16, 64, 15, 36, launch_split<1, 4, 4, 2>, launch_split<1, 4, 4, 2, true>},
      {32, 32, 12, 39, launch_split<2, 2, 2, 4>, nullptr},
      {32, 64, 6, 57, launch_split<2, 4, 2, 1>, nullptr},
      {64, 64, 0, 100, launch_split<4, 4, 2, 1>, nullptr},
      {128, 256, 0, 330, launch_tile<4>, nullptr},
      {256, 256, 0, 600, launch_tile<8>, nullptr},
  };
  constexpr int kSplits = 6, kAll = 8;
  const int first = a.gemm == 2 ? kSplits : 0, last = a.gemm == 1 ? kSplits : kAll;
  const Tiling* best = nullptr;
  int64_t least = 0;
  for (int i = first; i < last; ++i) {
    const Tiling& t = tilings[i];
    const int64_t units = (int64_t)((a.T + t.rows - 1) / t.rows) * ((a.N + t.cols - 1) / t.cols);
    const int64_t cost = t.start + (units + 255) / 256 * t.round;
    if (!best || cost < least) {
      best = &t;
      least = cost;
    }
  }
  if (a.adapter_of && (int64_t)a.T * a.R <= kFusedRows && best->fused) return best->fused(a, s);
  for (int64_t t0 = 0; t0 < a.T; t0 += kLaunchTokens) {
    ProjectArgs c = a;
    c.T = (int)std::min<int64_t>(kLaunchTokens, a.T - t0);
    c.x += t0 * a.ldx;
    c.y += t0 * a.ldy;
    if (a.adapter_of) {
      c.adapter_of += t0;
      // blocks for each rank tile and for several adapters of a token tile while
      // there are compute units for them
      const int tiles = (c.T + 15) / 16;
      int parts = (a.R + 15) / 16, entries = std::min(std::min(16, a.n), c.T);
      while (parts > 1 && tiles * parts > 256) parts = (parts + 1) / 2;
      while (entries > 1 && tiles * parts * entries > 256) entries = (entries + 1) / 2;
      hipLaunchKernelGGL(adapter_down_kernel, dim3((unsigned)(tiles * parts * entries)), dim3(kPThreads), 0, s, c, entries,
                         parts);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
    const hipError_t e = best->launch(c, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
