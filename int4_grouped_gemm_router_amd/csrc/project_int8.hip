// A projection by 8-bit integers (gfx950 integer matrix cores):
//   y[t][n] = x_scales[t] w_scales[n] sum_k x[t][k] w[n][k] + bias[n]
// Sums are exact in 32-bit integers (K <= 65536, so at most 2^30); the scales
// and the bias are applied in fp32 and the result is rounded once.
//
// Both operands are row-major. A tile of 16 rows x 128 inputs is two matrix
// operations' operand; a wave copies it from the rows straight to LDS, eight
// lanes a row, so that each copy takes whole lines of 128 bytes (with 64 bytes a
// row, a step of one operation, L2 delivers half as much: 4096 x 12288 x 2048 took
// 115 us), and reads it back in the matrix cores' order. Three kernels:
//   int8_vector_kernel one to four tokens: whole rows of weights straight to
//                      registers, dot products of four in the vector units;
//                      memory bounds it (1 x 12288 x 2048 5.7 us, 4.4 TB/s)
//   int8_split_kernel  a block's waves split K and join through LDS: few rows,
//                      where bytes and latency count (500 x 2000 x 4096 12 us)
//   int8_tile_kernel   256 x 256 tiles, both operands shared through two stages
//                      of 128 inputs: many rows, where the matrix cores count
//                      (4096 x 12288 x 2048 112 us, 1.83 POP/s; 4096^3 62, 2.2; 8192^3
//                      464, 2.4)
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "topk.h"
#include "wide_expand.h"

namespace moe {

namespace {

constexpr int kIWaves = 8;
constexpr int kIThreads = 64 * kIWaves;
constexpr int kStep = 128;  // inputs of a tile
constexpr int kNowhere = INT32_MIN;  // a buffer offset past every end: such copies are zeros

typedef int i32x4 __attribute__((ext_vector_type(4)));

// D = A(16x64) * B(64x16) + C of signed bytes; lane l holds row (A) or column
// (B) l%16 and sixteen consecutive k of block l/16; D as of mfma16.
__device__ inline i32x4 mfma16_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Copy h of a tile (rows 8 h .. 8 h + 7): lane l takes piece piece_of(h, l) (16
// inputs) of row 8 h + l / 8 to slot 64 h + l. Lane (c16, kb) of the matrix
// cores finds piece p of row c16 in slot_of(c16, p), p = kb + 4 half. The swizzle
// puts the sixteen rows' same piece into different LDS banks.
__device__ inline int piece_of(int h, int l) { return (l & 7) ^ (4 * h + (l >> 4)); }
__device__ inline int slot_of(int c16, int p) { return 8 * c16 + (p ^ (c16 >> 1)); }

// What a wave needs to copy N tiles of one operand, from the base of rows of ld
// bytes: each lane's offsets. Rows past the last repeat it.
template <int N>
struct TileCopy {
  uint32_t off[N][2];
  __device__ void init(int lane, int first, int rows, int64_t ld) {
#pragma unroll
    for (int n = 0; n < N; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        off[n][h] = (uint32_t)min(16 * (first + n) + 8 * h + (lane >> 3), rows - 1) * (uint32_t)ld + 16 * piece_of(h, lane);
  }
  // the tiles' inputs from k on, those from K on as zeros; tile n goes to dst + 128 n
  __device__ void issue(rsrc_t r, u32x4* dst, int lane, int k, int K) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const bool past = k + 16 * piece_of(h, lane) >= K;
#pragma unroll
      for (int n = 0; n < N; ++n) bload_lds(r, dst + 128 * n + 64 * h, past ? (uint32_t)kNowhere : off[n][h], (uint32_t)k);
    }
  }
};

template <int N>
__device__ inline void wait_copies() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// Eight values to y from element `at` on, `left` of them in the row.
__device__ inline void put_eight(const Int8Args& a, int64_t at, const float (&v)[8], int left) {
  if (a.dtype == kNormF32) {
    float* p = static_cast<float*>(a.y) + at;
    if (a.wide && left >= 8) {
      reinterpret_cast<f32x4*>(p)[0] = f32x4{v[0], v[1], v[2], v[3]};
      reinterpret_cast<f32x4*>(p)[1] = f32x4{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < left) p[i] = v[i];
    }
    return;
  }
  uint32_t h[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = a.dtype == kNormBf16 ? f2bf(v[i]) : __builtin_bit_cast(uint16_t, (_Float16)v[i]);
  uint16_t* p = static_cast<uint16_t*>(a.y) + at;
  if (a.wide && left >= 8) {
    *reinterpret_cast<u32x4*>(p) = u32x4{h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < left) p[i] = (uint16_t)h[i];
  }
}

}  // namespace

// One to four tokens. Wave (r, p) of a block takes kRows outputs and the p-th
// of KS parts of K, in pieces of 16 inputs a lane: whole KBs of a row at a
// time, the next turn's pieces under way while this one's are multiplied, four
// at a time, in the vector units. The lanes' sums are joined by DPP, the parts'
// in LDS.
constexpr int kVecRows = 4;

template <int T, int KS>
__global__ __launch_bounds__(kIThreads) void int8_vector_kernel(Int8Args a) {
  constexpr int kGroups = kIWaves / KS;  // row groups of a block
  __shared__ int red[kIWaves][kVecRows][T];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int part = wave % KS, n0 = ((int)blockIdx.x * kGroups + wave / KS) * kVecRows;
  // this part's pieces: from p0 on, n of them
  const int pieces = a.K / 16, p0 = (int)((int64_t)pieces * part / KS), n = (int)((int64_t)pieces * (part + 1) / KS) - p0;
  const u32x4* w[kVecRows];
#pragma unroll
  for (int r = 0; r < kVecRows; ++r) w[r] = reinterpret_cast<const u32x4*>(a.w + (int64_t)min(n0 + r, a.N - 1) * a.K) + p0;
  const u32x4* x[T];
#pragma unroll
  for (int t = 0; t < T; ++t) x[t] = reinterpret_cast<const u32x4*>(a.x + t * a.ldx) + p0;
  int acc[kVecRows][T] = {};
  u32x4 wv[2][kVecRows], xv[2][T];
  auto load = [&](int s, int at) {
    // (pieces past the part repeat its last one, whose tokens are put to zero)
    const int i = min(at + lane, n - 1);
#pragma unroll
    for (int r = 0; r < kVecRows; ++r) wv[s][r] = __builtin_nontemporal_load(w[r] + i);
#pragma unroll
    for (int t = 0; t < T; ++t) xv[s][t] = x[t][i];
  };
  auto multiply = [&](int s, int at) {
    const bool in = at + lane < n;
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const int xd = in ? (int)xv[s][t][d] : 0;
#pragma unroll
        for (int r = 0; r < kVecRows; ++r) acc[r][t] = __builtin_amdgcn_sdot4((int)wv[s][r][d], xd, acc[r][t], false);
      }
    }
  };
  load(0, 0);
  for (int at = 0; at < n; at += 128) {
    if (at + 64 < n) load(1, at + 64);
    multiply(0, at);
    if (at + 64 >= n) break;
    if (at + 128 < n) load(0, at + 128);
    multiply(1, at + 64);
  }
  // (lane l of sixteen rows' sums; every lane gets its row's)
#pragma unroll
  for (int r = 0; r < kVecRows; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) {
      int v = acc[r][t];
      v += (int)dpp<0xB1>((uint32_t)v);
      v += (int)dpp<0x4E>((uint32_t)v);
      v += (int)dpp<0x141>((uint32_t)v);
      v += (int)dpp<0x140>((uint32_t)v);
      v = __builtin_amdgcn_readlane(v, 0) + __builtin_amdgcn_readlane(v, 16) + __builtin_amdgcn_readlane(v, 32) +
          __builtin_amdgcn_readlane(v, 48);
      if (lane == 0) red[wave][r][t] = v;
    }
  __syncthreads();
  if (tid >= kGroups * kVecRows * T) return;
  const int r = tid % kVecRows, g = tid / kVecRows % kGroups, tt = tid / (kVecRows * kGroups);
  const int row = ((int)blockIdx.x * kGroups + g) * kVecRows + r;
  if (row >= a.N) return;
  int s = 0;
#pragma unroll
  for (int p = 0; p < KS; ++p) s += red[g * KS + p][r][tt];
  float v = (float)s * a.x_scales[tt] * a.w_scales[row];
  if (a.bias) v += a.bias[row];
  const int64_t at = tt * a.ldy + row;
  if (a.dtype == kNormF32)
    static_cast<float*>(a.y)[at] = v;
  else
    static_cast<uint16_t*>(a.y)[at] = a.dtype == kNormBf16 ? f2bf(v) : __builtin_bit_cast(uint16_t, (_Float16)v);
}

// A block owns 16 MS tokens and 16 CT outputs; wave w takes the w-th of W parts
// of the steps on its own, D steps ahead in its own ring in LDS (no barrier: the
// wave waits for its copies), and the partial tiles are added in LDS.
template <int MS, int CT, int D, int W>
struct Int8SplitLds {
  static constexpr int kStride = 16 * CT + 4;  // the pad spreads the rows over the banks
  union {
    u32x4 f[W][D][MS + CT][128];
    int red[W][16 * MS][kStride];
  };
};

template <int MS, int CT, int D, int W>
__global__ __launch_bounds__(64 * W, 2) void int8_split_kernel(Int8Args a) {
  typedef Int8SplitLds<MS, CT, D, W> Lds;
  __shared__ Lds L;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kb = lane >> 4;
  const int row_tiles = (a.T + 16 * MS - 1) / (16 * MS), col_tiles = (a.N + 16 * CT - 1) / (16 * CT);
  // XCD x (blocks go to XCD b % 8 in turn) takes a contiguous range of units,
  // row tiles fastest: the row tiles of one column tile share its weights in L2
  const int64_t units = (int64_t)row_tiles * col_tiles;
  const int64_t u0 = units * (blockIdx.x & 7) / 8, u1 = units * ((blockIdx.x & 7) + 1) / 8;
  const int64_t u = u0 + (blockIdx.x >> 3);
  if (u >= u1) return;
  const int t0 = (int)(u % row_tiles) * (16 * MS), n0 = (int)(u / row_tiles) * (16 * CT);
  const int rows = min(16 * MS, a.T - t0), cols = min(16 * CT, a.N - n0);
  const int G = (a.K + kStep - 1) / kStep, g0 = (int)((int64_t)G * wave / W), ng = (int)((int64_t)G * (wave + 1) / W) - g0;
  const rsrc_t xres = make_rsrc(a.x + (int64_t)t0 * a.ldx, (uint32_t)((rows - 1) * a.ldx + a.K));
  const rsrc_t wres = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)(cols * a.K));
  TileCopy<MS> xc;
  TileCopy<CT> wc;
  xc.init(lane, 0, rows, a.ldx);
  wc.init(lane, 0, cols, a.K);
  // what the thread scales and stores in the end: eight outputs of a token,
  // whose scales are under way before the rows are
  constexpr int kEights = 16 * MS * 2 * CT, kEach = (kEights + 64 * W - 1) / (64 * W);
  float xs[kEach], ws[kEach][8], bias[kEach][8];
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int er = min((tid + 64 * W * e) / (2 * CT), rows - 1), ec = (tid + 64 * W * e) % (2 * CT) * 8;
    xs[e] = a.x_scales[t0 + er];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = min(n0 + ec + i, a.N - 1);
      ws[e][i] = a.w_scales[n];
      bias[e][i] = a.bias ? a.bias[n] : 0.f;
    }
  }
  int next = 0;
  auto load = [&](int s) {
    // (steps past the last repeat it and are not used)
    const int k = (g0 + min(next, max(ng - 1, 0))) * kStep;
    ++next;
    wc.issue(wres, L.f[wave][s][MS], lane, k, a.K);
    xc.issue(xres, L.f[wave][s][0], lane, k, a.K);
  };
#pragma unroll
  for (int s = 0; s < D; ++s) {
    load(s);
    __builtin_amdgcn_sched_barrier(0);  // the waits below count on the slots' order
  }
  i32x4 acc[MS][CT];
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[m][c] = i32x4{0, 0, 0, 0};
  for (int g = 0; g < ng; g += D) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      if (g + s < ng) {
        wait_copies<(D - 1) * 2 * (MS + CT)>();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int sl = slot_of(c16, kb + 4 * h);
          u32x4 x[MS], w[CT];
#pragma unroll
          for (int m = 0; m < MS; ++m) x[m] = L.f[wave][s][m][sl];
#pragma unroll
          for (int c = 0; c < CT; ++c) w[c] = L.f[wave][s][MS + c][sl];
#pragma unroll
          for (int m = 0; m < MS; ++m)
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[m][c] = mfma16_i8(w[c], x[m], acc[m][c]);
        }
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // read before the next copies
        load(s);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  // (every copy has landed before the ring becomes the sums)
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
#pragma unroll
  for (int m = 0; m < MS; ++m)
#pragma unroll
    for (int c = 0; c < CT; ++c)
      *reinterpret_cast<i32x4*>(&L.red[wave][16 * m + c16][16 * c + 4 * kb]) = acc[m][c];
  __syncthreads();
#pragma unroll
  for (int e = 0; e < kEach; ++e) {
    const int er = (tid + 64 * W * e) / (2 * CT), ec = (tid + 64 * W * e) % (2 * CT) * 8;
    if (er >= rows || ec >= cols) continue;
    i32x4 s[2] = {};
#pragma unroll
    for (int w = 0; w < W; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] += *reinterpret_cast<const i32x4*>(&L.red[w][er][ec + 4 * h]);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (float)s[i >> 2][i & 3] * xs[e] * ws[e][i] + bias[e][i];
    put_eight(a, (int64_t)(t0 + er) * a.ldy + n0 + ec, v, a.N - n0 - ec);
  }
}

// Many rows: tiles of 32 RS tokens x 256 outputs, eight waves of 16 RS x 64. A
// stage holds the tile's rows of one step of 128 inputs. One barrier a step,
// before the products of its last two subtiles: from there on the next step's
// operands are read, and the copies of the step after it go to where this one was.
template <int RS>
struct Int8TileLds {
  static constexpr int kTiles = 2 * RS + 16;
  u32x4 f[2][kTiles][128];  // [stage][tokens' subtiles, then outputs'][slot]
};

template <int RS>
__global__ __launch_bounds__(kIThreads, 2) void int8_tile_kernel(Int8Args a) {
  typedef Int8TileLds<RS> Lds;
  __shared__ Lds L;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kb = lane >> 4;
  const int wr = wave >> 2, wc = wave & 3;
  const int G = (a.K + kStep - 1) / kStep;
  const int row_tiles = (a.T + 32 * RS - 1) / (32 * RS), col_tiles = (a.N + 255) / 256;
  // XCD x takes a contiguous range of units, column tiles fastest: the rows of
  // few row tiles stay in its L2
  const int units = row_tiles * col_tiles;
  const int u0 = (int)((int64_t)units * (blockIdx.x & 7) / 8), u1 = (int)((int64_t)units * ((blockIdx.x & 7) + 1) / 8);
  const int u = u0 + (blockIdx.x >> 3);
  if (u >= u1) return;
  const int t0 = u / col_tiles * (32 * RS), n0 = u % col_tiles * 256;
  const int rows = min(32 * RS, a.T - t0), cols = min(256, a.N - n0);
  const rsrc_t xres = make_rsrc(a.x + (int64_t)t0 * a.ldx, (uint32_t)((rows - 1) * a.ldx + a.K));
  const rsrc_t wres = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)(cols * a.K));
  // wave w copies tokens' subtiles w RS / 4 .. and outputs' 2 w, 2 w + 1
  constexpr int kX = RS / 4;
  TileCopy<kX> xc;
  TileCopy<2> oc;
  xc.init(lane, wave * kX, rows, a.ldx);
  oc.init(lane, 2 * wave, cols, a.K);
  // the steps are taken in turn from a start that depends on the column tile:
  // rows a multiple of 4 KB apart have one step of every row in the same L2
  // channel, and blocks in step would all wait for it
  int gk = (int)((int64_t)(u % col_tiles) * G / col_tiles);
  // (steps past the last wrap around and are not used)
  auto load = [&](int st) {
    xc.issue(xres, L.f[st][wave * kX], lane, gk * kStep, a.K);
    oc.issue(wres, L.f[st][2 * RS + 2 * wave], lane, gk * kStep, a.K);
    gk = gk + 1 < G ? gk + 1 : 0;
  };
  i32x4 acc[RS][4];
#pragma unroll
  for (int m = 0; m < RS; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = i32x4{0, 0, 0, 0};
  load(0);
  load(1);
  constexpr int kCopies = 2 * (kX + 2);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kCopies) : "memory");
  const int sl[2] = {slot_of(c16, kb), slot_of(c16, kb + 4)};
  // token operands are read kAhead subtiles ahead of their products, the
  // outputs' over the end of the half before
  constexpr int kAhead = 3, kRing = 4;
  u32x4 av[kRing], bw[2][4];
#pragma unroll
  for (int c = 0; c < 4; ++c) bw[0][c] = L.f[0][2 * RS + 4 * wc + c][sl[0]];
#pragma unroll
  for (int m = 0; m < kAhead; ++m) av[m] = L.f[0][wr * RS + m][sl[0]];
  auto products = [&](int h, int m) {
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = mfma16_i8(bw[h][c], av[m % kRing], acc[m][c]);
    // (without these fences the compiler gathers the reads and spills)
    __builtin_amdgcn_sched_barrier(0);
  };
  auto step = [&](auto S_) {
    constexpr int S = decltype(S_)::value, Sn = 1 - S;
    auto token = [&](int st, int h, int m) { av[m % kRing] = L.f[st][wr * RS + m][sl[h]]; };
    auto output = [&](int st, int h, int c) { bw[h][c] = L.f[st][2 * RS + 4 * wc + c][sl[h]]; };
#pragma unroll
    for (int m = 0; m < RS; ++m) {
      const int fa = m + kAhead;
      token(S, fa < RS ? 0 : 1, fa % RS);
      if (m >= RS / 2) {
#pragma unroll
        for (int q = 0; q < 8 / RS; ++q) output(S, 1, (m - RS / 2) * (8 / RS) + q);
      }
      products(0, m);
    }
#pragma unroll
    for (int m = 0; m < RS - 2; ++m) {
      if (m + kAhead < RS) token(S, 1, m + kAhead);
      products(1, m);
    }
    // Every wave has read this step, and the next one is in LDS.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
    load(S);
    token(Sn, 0, 0);
    token(Sn, 0, 1);
    output(Sn, 0, 0);
    output(Sn, 0, 1);
    products(1, RS - 2);
    token(Sn, 0, 2);
    output(Sn, 0, 2);
    output(Sn, 0, 3);
    products(1, RS - 1);
  };
  for (int g = 0;; g += 2) {
    step(std::integral_constant<int, 0>{});
    if (g + 1 >= G) break;
    step(std::integral_constant<int, 1>{});
    if (g + 2 >= G) break;
  }
  // (the last copies and reads of the stages end here, in every wave)
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // lane: token c16 of each subtile, outputs 4 kb .. 4 kb + 3 of each sixteen;
  // through LDS, so that eight lanes store a row's 64 values
  const int tw = t0 + 16 * RS * wr, nw = n0 + 64 * wc;
  if (nw >= a.N) return;
  float ws[4][4], bias[4][4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = min(nw + 16 * c + 4 * kb + i, a.N - 1);
      ws[c][i] = a.w_scales[n];
      bias[c][i] = a.bias ? a.bias[n] : 0.f;
    }
  constexpr int kRow = 68;  // floats; the pad spreads the rows over the banks
  float* tr = reinterpret_cast<float*>(&L) + wave * (16 * kRow);
#pragma unroll
  for (int m = 0; m < RS; ++m) {
    const float xs = a.x_scales[min(tw + 16 * m + c16, a.T - 1)];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (float)acc[m][c][i] * xs * ws[c][i] + bias[c][i];
      *reinterpret_cast<f32x4*>(tr + c16 * kRow + 16 * c + 4 * kb) = v;
    }
    // (a wave's LDS accesses execute in order)
    asm volatile("" ::: "memory");
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int r = 8 * q + (lane >> 3), t = tw + 16 * m + r, n = nw + 8 * (lane & 7);
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f32x4 p = *reinterpret_cast<const f32x4*>(tr + r * kRow + 8 * (lane & 7) + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = p[i];
      }
      if (t < a.T && n < a.N) put_eight(a, (int64_t)t * a.ldy + n, v, a.N - n);
    }
    asm volatile("" ::: "memory");
  }
}

namespace {

constexpr int kVecTokens = 4;

template <int T, int KS>
hipError_t launch_vector(const Int8Args& a, hipStream_t s) {
  constexpr int kOut = kIWaves / KS * kVecRows;
  hipLaunchKernelGGL((int8_vector_kernel<T, KS>), dim3((a.N + kOut - 1) / kOut), dim3(kIThreads), 0, s, a);
  return hipGetLastError();
}

template <int T>
hipError_t launch_vector_parts(const Int8Args& a, hipStream_t s) {
  // a KB of a row for each wave, as long as the waves are not more than what
  // keeps the memory busy: one token, 12288 x 2048 with K in 1, 2, 4, 8 parts 6.3,
  // 6.2, 6.6, 8.8 us, 2048 x 4096 5.1, 4.3, 3.9, 4.0, 4096 x 8192 10.6, 8.7, 7.4,
  // 7.3, 12288 x 512 3.7, 4.0, 5.5, 8.1; four tokens, 12288 x 2048 7.9, 8.6, 11.4,
  // 19.6, 2048 x 4096 7.0, 5.7, 5.1, 5.5
  const auto fits = [&](int parts) { return a.K >= 1024 * parts && (int64_t)a.N / kVecRows * parts <= 4096; };
  if (fits(8)) return launch_vector<T, 8>(a, s);
  if (fits(4)) return launch_vector<T, 4>(a, s);
  if (fits(2)) return launch_vector<T, 2>(a, s);
  return launch_vector<T, 1>(a, s);
}

template <int MS, int CT, int D, int W>
hipError_t launch_split(const Int8Args& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.T + 16 * MS - 1) / (16 * MS)) * ((a.N + 16 * CT - 1) / (16 * CT));
  hipLaunchKernelGGL((int8_split_kernel<MS, CT, D, W>), dim3((unsigned)((units + 7) / 8 * 8)), dim3(64 * W), 0, s, a);
  return hipGetLastError();
}

template <int RS>
hipError_t launch_tile(const Int8Args& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.T + 32 * RS - 1) / (32 * RS)) * ((a.N + 255) / 256);
  hipLaunchKernelGGL(int8_tile_kernel<RS>, dim3((unsigned)((units + 7) / 8 * 8)), dim3(kIThreads), 0, s, a);
  return hipGetLastError();
}

// A start and a time per round of 256 units, one for each compute unit, in
// tenths of a microsecond, measured at K = 2048 (all of them grow with K alike).
struct Tiling {
  int rows, cols, start, round;
  hipError_t (*launch)(const Int8Args&, hipStream_t);
};

}  // namespace

hipError_t launch_project_int8(const Int8Args& in, hipStream_t s) {
  // Small tiles start fastest and lose when there are many, in us: 16 tokens by
  // 4096 outputs 4.5 in 16 x 16 tiles, 5.0 in 32 x 32, 7.2 in 64 x 64; 16 by 12288
  // 8.9, 9.3, 9.4 (16 x 64: 7.8); 64 by 4096 7.3, 5.2, 7.5; 256 by 4096 19, 11, 7.9
  // and 18 in 128 x 256; 512 by 12288 43 in 64 x 64, 26 in 128 x 256, 33 in 256 x
  // 256; 4096 by 12288 369, 154, 113.
  static const Tiling tilings[] = {
      {16, 16, 30, 10, launch_split<1, 1, 2, 4>}, {16, 32, 33, 14, launch_split<1, 2, 2, 4>},
      {16, 64, 30, 24, launch_split<1, 4, 2, 4>}, {32, 32, 33, 19, launch_split<2, 2, 2, 4>},
      {32, 64, 20, 41, launch_split<2, 4, 2, 4>}, {64, 64, 8, 71, launch_split<4, 4, 2, 4>},
      {128, 256, 0, 257, launch_tile<4>},         {256, 256, 0, 372, launch_tile<8>},
  };
  Int8Args a = in;
  const int eb = a.dtype == kNormF32 ? 4 : 2;
  a.wide = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.ldy * eb % 16 == 0;
  if (a.T <= kVecTokens) {
    switch (a.T) {
      case 1: return launch_vector_parts<1>(a, s);
      case 2: return launch_vector_parts<2>(a, s);
      case 3: return launch_vector_parts<3>(a, s);
      default: return launch_vector_parts<4>(a, s);
    }
  }
  const Tiling* best = nullptr;
  int64_t least = 0;
  for (const Tiling& t : tilings) {
    const int64_t units = (int64_t)((a.T + t.rows - 1) / t.rows) * ((a.N + t.cols - 1) / t.cols);
    const int64_t cost = t.start + (units + 255) / 256 * t.round;
    if (!best || cost < least) {
      best = &t;
      least = cost;
    }
  }
  // (as many tokens as leave fewer than 2^31 threads a launch in every tiling that so many choose)
  constexpr int kLaunchTokens = 1 << 18;
  for (int64_t t0 = 0; t0 < in.T; t0 += kLaunchTokens) {
    Int8Args c = a;
    c.T = (int)std::min<int64_t>(kLaunchTokens, in.T - t0);
    c.x += t0 * a.ldx;
    c.x_scales += t0;
    c.y = static_cast<char*>(c.y) + t0 * a.ldy * eb;
    const hipError_t e = best->launch(c, s);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace moe
