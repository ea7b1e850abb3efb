// A projection by 8-bit integers (gfx950 integer matrix cores):
//   y[t][n] = x_scales[t] w_scales[n] sum_k x[t][k] w[n][k] + bias[n]
// Sums are exact in 32-bit integers (K <= 65536, so at most 2^30); the scales
// and the bias are applied in fp32 and the result is rounded once.
//
// Both operands are row-major. A fragment, 16 rows x 64 inputs, is what one
// matrix operation takes of an operand; a wave copies it from the rows straight
// to LDS, four lanes a row (sixteen lanes that each read another row cost the
// address unit four times as long), and reads it back in the matrix cores'
// order. Two kernels:
//   int8_split_kernel  a block's eight waves split K and join through LDS:
//                      few rows, where bytes and latency count
//   int8_tile_kernel   256 x 256 tiles, both operands shared through a ring of
//                      four stages of 64 inputs: many rows, where the matrix
//                      cores count
#include <algorithm>
#include <type_traits>

#include "kernels.h"
#include "wide_expand.h"

namespace moe {

namespace {

constexpr int kIWaves = 8;
constexpr int kIThreads = 64 * kIWaves;
constexpr int kStep = 64;  // inputs of a fragment

typedef int i32x4 __attribute__((ext_vector_type(4)));

// D = A(16x64) * B(64x16) + C of signed bytes; lane l holds row (A) or column
// (B) l%16 and sixteen consecutive k of block l/16; D as of mfma16.
__device__ inline i32x4 mfma16_i8(u32x4 a, u32x4 b, i32x4 c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, a), __builtin_bit_cast(i32x4, b), c, 0, 0, 0);
}

// Lane l of a copy takes piece piece_of(l) (16 inputs) of row l / 4 to slot l;
// lane (c16, kb) of the matrix cores finds row c16, piece kb in slot_of(c16,
// kb). The swizzle spreads the sixteen rows of one piece over the LDS banks.
__device__ inline int piece_of(int l) { return (l & 3) ^ (l >> 4); }
__device__ inline int slot_of(int c16, int kb) { return 4 * c16 + (kb ^ (c16 >> 2)); }

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

// A block owns 16 MS tokens and 16 CT outputs; wave w takes the w-th eighth of
// the steps on its own, D steps ahead in its own ring in LDS (no barrier: the
// wave waits for its copies), and the eight partial tiles are added in LDS.
template <int MS, int CT, int D>
struct Int8SplitLds {
  static constexpr int kStride = 16 * CT + 4;  // the pad spreads the rows over the banks
  union {
    u32x4 f[kIWaves][D][MS + CT][64];
    int red[kIWaves][16 * MS][kStride];
  };
};

template <int MS, int CT, int D>
__global__ __launch_bounds__(kIThreads, 2) void int8_split_kernel(Int8Args a) {
  typedef Int8SplitLds<MS, CT, D> Lds;
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
  const int G = a.K / kStep, g0 = (int)((int64_t)G * wave / kIWaves), ng = (int)((int64_t)G * (wave + 1) / kIWaves) - g0;
  // (rows past the last repeat it and are not stored)
  const rsrc_t xres = make_rsrc(a.x + (int64_t)t0 * a.ldx, (uint32_t)((rows - 1) * a.ldx + a.K));
  const rsrc_t wres = make_rsrc(a.w + (int64_t)n0 * a.K, (uint32_t)(cols * a.K));
  uint32_t xoff[MS], woff[CT];
#pragma unroll
  for (int m = 0; m < MS; ++m) xoff[m] = (uint32_t)min(16 * m + (lane >> 2), rows - 1) * (uint32_t)a.ldx + 16 * piece_of(lane);
#pragma unroll
  for (int c = 0; c < CT; ++c) woff[c] = (uint32_t)min(16 * c + (lane >> 2), cols - 1) * (uint32_t)a.K + 16 * piece_of(lane);
  int next = 0;
  auto load = [&](int s) {
    // (steps past the last repeat it and are not used)
    const uint32_t k = (uint32_t)(g0 + min(next, max(ng - 1, 0))) * kStep;
    ++next;
#pragma unroll
    for (int c = 0; c < CT; ++c) bload_lds(wres, &L.f[wave][s][MS + c][0], woff[c], k);
#pragma unroll
    for (int m = 0; m < MS; ++m) bload_lds(xres, &L.f[wave][s][m][0], xoff[m], k);
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
  const int sl = slot_of(c16, kb);
  for (int g = 0; g < ng; g += D) {
#pragma unroll
    for (int s = 0; s < D; ++s) {
      if (g + s < ng) {
        wait_copies<(D - 1) * (MS + CT)>();
        u32x4 x[MS], w[CT];
#pragma unroll
        for (int m = 0; m < MS; ++m) x[m] = L.f[wave][s][m][sl];
#pragma unroll
        for (int c = 0; c < CT; ++c) w[c] = L.f[wave][s][MS + c][sl];
#pragma unroll
        for (int m = 0; m < MS; ++m)
#pragma unroll
          for (int c = 0; c < CT; ++c) acc[m][c] = mfma16_i8(w[c], x[m], acc[m][c]);
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
  constexpr int kEights = 16 * MS * 2 * CT;
  for (int e = tid; e < kEights; e += kIThreads) {
    const int r = e / (2 * CT), c = e % (2 * CT) * 8;
    if (r >= rows || c >= cols) continue;
    i32x4 s[2] = {};
#pragma unroll
    for (int w = 0; w < kIWaves; ++w)
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] += *reinterpret_cast<const i32x4*>(&L.red[w][r][c + 4 * h]);
    const float xs = a.x_scales[t0 + r];
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int n = min(n0 + c + i, a.N - 1);
      v[i] = (float)s[i >> 2][i & 3] * xs * a.w_scales[n];
      if (a.bias) v[i] += a.bias[n];
    }
    put_eight(a, (int64_t)(t0 + r) * a.ldy + n0 + c, v, a.N - n0 - c);
  }
}

// Many rows: tiles of 32 RS tokens x 256 outputs, eight waves of 16 RS x 64. A
// stage holds the tile's fragments of one step; step i is multiplied while
// step i + 1, which is in LDS already, gives its first operands and step i + 3
// is copied to where step i - 1 was. One barrier a step.
template <int RS>
struct Int8TileLds {
  static constexpr int kFrags = 2 * RS + 16;
  u32x4 f[4][kFrags][64];  // [stage][tokens' subtiles, then outputs'][slot]
};

template <int RS>
__global__ __launch_bounds__(kIThreads, 2) void int8_tile_kernel(Int8Args a) {
  typedef Int8TileLds<RS> Lds;
  __shared__ Lds L;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int c16 = lane & 15, kb = lane >> 4;
  const int wr = wave >> 2, wc = wave & 3;
  const int G = a.K / kStep;
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
  constexpr int kX = RS / 4, kCopies = kX + 2;
  uint32_t xoff[kX], woff[2];
#pragma unroll
  for (int f = 0; f < kX; ++f)
    xoff[f] = (uint32_t)min(16 * (wave * kX + f) + (lane >> 2), rows - 1) * (uint32_t)a.ldx + 16 * piece_of(lane);
#pragma unroll
  for (int f = 0; f < 2; ++f)
    woff[f] = (uint32_t)min(16 * (2 * wave + f) + (lane >> 2), cols - 1) * (uint32_t)a.K + 16 * piece_of(lane);
  // the steps are taken in turn from a start that depends on the column tile:
  // rows a multiple of 4 KB apart have one step of every row in the same L2
  // channel, and blocks in step would all wait for it
  int gk = (int)((int64_t)(u % col_tiles) * G / col_tiles);
  // (steps past the last wrap around and are not used)
  auto load = [&](int st) {
#pragma unroll
    for (int f = 0; f < kX; ++f) bload_lds(xres, &L.f[st][wave * kX + f][0], xoff[f], (uint32_t)gk * kStep);
#pragma unroll
    for (int f = 0; f < 2; ++f) bload_lds(wres, &L.f[st][2 * RS + 2 * wave + f][0], woff[f], (uint32_t)gk * kStep);
    gk = gk + 1 < G ? gk + 1 : 0;
  };
  i32x4 acc[RS][4];
#pragma unroll
  for (int m = 0; m < RS; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = i32x4{0, 0, 0, 0};
  load(0);
  load(1);
  load(2);
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(kCopies) : "memory");
  const int sl = slot_of(c16, kb);
  // token operands are read kAhead subtiles ahead of their products, the
  // outputs' over the second half of a step
  constexpr int kAhead = 3, kRing = 4;
  u32x4 av[kRing], bw[2][4];
#pragma unroll
  for (int c = 0; c < 4; ++c) bw[0][c] = L.f[0][2 * RS + 4 * wc + c][sl];
#pragma unroll
  for (int m = 0; m < kAhead; ++m) av[m] = L.f[0][wr * RS + m][sl];
  auto step = [&](auto S_) {
    constexpr int S = decltype(S_)::value, Sn = (S + 1) & 3, B = S & 1;
    load((S + 3) & 3);
#pragma unroll
    for (int m = 0; m < RS; ++m) {
      const int fa = m + kAhead;
      av[fa % kRing] = fa < RS ? L.f[S][wr * RS + fa][sl] : L.f[Sn][wr * RS + fa - RS][sl];
      if (m >= RS / 2) {
#pragma unroll
        for (int q = 0; q < 8 / RS; ++q) {
          const int c = (m - RS / 2) * (8 / RS) + q;
          bw[1 - B][c] = L.f[Sn][2 * RS + 4 * wc + c][sl];
        }
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) acc[m][c] = mfma16_i8(bw[B][c], av[m % kRing], acc[m][c]);
      // (without these fences the compiler gathers the reads and spills)
      __builtin_amdgcn_sched_barrier(0);
    }
    // Before any wave goes on: step i + 2 is in LDS (the copies of step i + 3
    // may be under way), and this wave's reads of step i are done (LDS answers
    // in order; the last quarter's reads, of step i + 1, may be under way).
    static_assert(RS == 8 || RS == 4, "reads after the last of this step");
    if constexpr (RS == 8)
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(4)\n\ts_barrier" ::"n"(kCopies) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(3)\n\ts_barrier" ::"n"(kCopies) : "memory");
  };
  for (int g = 0;; g += 4) {
    step(std::integral_constant<int, 0>{});
    if (g + 1 >= G) break;
    step(std::integral_constant<int, 1>{});
    if (g + 2 >= G) break;
    step(std::integral_constant<int, 2>{});
    if (g + 3 >= G) break;
    step(std::integral_constant<int, 3>{});
    if (g + 4 >= G) break;
  }
  // (the last copies and reads of the ring end here, in every wave)
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

size_t int8_ws_bytes(int /*N*/, int /*K*/, int /*T*/) { return 0; }

namespace {

template <int MS, int CT, int D>
hipError_t launch_split(const Int8Args& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.T + 16 * MS - 1) / (16 * MS)) * ((a.N + 16 * CT - 1) / (16 * CT));
  hipLaunchKernelGGL((int8_split_kernel<MS, CT, D>), dim3((unsigned)((units + 7) / 8 * 8)), dim3(kIThreads), 0, s, a);
  return hipGetLastError();
}

template <int RS>
hipError_t launch_tile(const Int8Args& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.T + 32 * RS - 1) / (32 * RS)) * ((a.N + 255) / 256);
  hipLaunchKernelGGL(int8_tile_kernel<RS>, dim3((unsigned)((units + 7) / 8 * 8)), dim3(kIThreads), 0, s, a);
  return hipGetLastError();
}

struct Tiling {
  int rows, cols, start, round;
  hipError_t (*launch)(const Int8Args&, hipStream_t);
};

}  // namespace

hipError_t launch_project_int8(const Int8Args& in, hipStream_t s) {
  static const Tiling tilings[] = {
      {16, 16, 22, 20, launch_split<1, 1, 4>}, {16, 32, 24, 20, launch_split<1, 2, 4>}, {16, 64, 15, 36, launch_split<1, 4, 4>},
      {32, 32, 12, 39, launch_split<2, 2, 2>}, {32, 64, 6, 57, launch_split<2, 4, 2>},  {64, 64, 0, 100, launch_split<4, 4, 2>},
      {128, 256, 0, 330, launch_tile<4>},      {256, 256, 0, 600, launch_tile<8>},
  };
  Int8Args a = in;
  const int eb = a.dtype == kNormF32 ? 4 : 2;
  a.wide = (reinterpret_cast<uintptr_t>(a.y) & 15) == 0 && a.ldy * eb % 16 == 0;
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
