// Layer norm, forward and backward, over rows of C elements (bf16 or fp32).
//
// Per row: mu = mean x, r = 1 / sqrt(mean (x - mu)^2 + eps), x^ = (x - mu) r, y = x^ w + b.
// Backward, with g = dy w:  dx = r (g - mean g - x^ mean(g x^)),  dw = sum_rows dy x^,
// db = sum_rows dy.
//
// What bounds it: HBM. The forward reads and writes each element once, the backward reads two and
// writes one, so a row stays in the registers of the threads that share it (a group of GT threads,
// NV pieces of 16 bytes each) from its load to its store: the mean, then the squares about that
// mean (two passes over registers, no cancellation), then the result. Groups are persistent: a
// group's columns do not change from row to row, so its weights, and in the backward its column
// sums of dy x^ and dy, live in registers over all its rows. The backward's column sums are added
// over the groups of a block in shared memory and over the blocks by a second kernel, both in a
// fixed order, so a call's results do not change from run to run.
// Measured (bf16, at 6.56 TB/s of copy): forward of 1,048,576 x 96 rows 73 us (5.5 TB/s) and of
// 131,072 x 768 75 us, backward 108 and 107 us (5.6 TB/s); weights in shared memory instead of
// registers, with twice the warps, took 94 and 104 us, and rows fetched two ahead 82 and 87 us.
#include <math.h>

#include "common.cuh"
#include "launch.h"
#include "vec.cuh"

namespace p3d {
namespace ln {

// E consecutive elements of T: a 16-byte piece (E > 1) or a single element (rows whose length is
// not a whole number of pieces).
template <typename T, int E> struct Piece;
template <typename T> struct Piece<T, 1> {
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = p[0]; }
  __device__ __forceinline__ void zero() { raw = from_f<T>(0.f); }
  __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = to_f(raw); }
  __device__ __forceinline__ static void store(T* p, const float (&x)[1]) { p[0] = from_f<T>(x[0]); }
};
template <> struct Piece<float, 4> {
  float4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { raw = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void get(float (&x)[4]) const {
    x[0] = raw.x; x[1] = raw.y; x[2] = raw.z; x[3] = raw.w;
  }
  __device__ __forceinline__ static void store(float* p, const float (&x)[4]) {
    Vec<float>::store(p, x);
  }
};
template <> struct Piece<__nv_bfloat16, 8> {
  uint4 raw;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    raw = *reinterpret_cast<const uint4*>(p);
  }
  __device__ __forceinline__ void zero() { raw = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void get(float (&x)[8]) const { Vec<__nv_bfloat16>::unpack(raw, x); }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&x)[8]) {
    Vec<__nv_bfloat16>::store(p, x);
  }
};

// weight or bias element of either type
__device__ __forceinline__ float param(const void* p, int wtype, int c, float none) {
  if (!p) return none;
  return wtype == PACK3D_BF16 ? to_f(static_cast<const __nv_bfloat16*>(p)[c])
                              : static_cast<const float*>(p)[c];
}

// Sums over the GT threads of a group: shuffles inside a warp, then one word per warp and value
// in shared memory (a buffer per use in a row, so one barrier per sum is enough).
template <int GT, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float* red) {
  constexpr int W = GT < 32 ? GT : 32;
#pragma unroll
  for (int o = W / 2; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if constexpr (GT > 32) {
    constexpr int NW = GT / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) red[k * NW + warp] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) s += red[k * NW + w];
      v[k] = s;
    }
  }
}

// s / n by the rounded reciprocal and one residual correction, q + (s - q n) / n, which is a Newton step
// for the quotient (a constant row has exactly its mean), and 1 / sqrt(v) by the hardware's
// approximation and one Newton step: a division and a root take as many instructions as 24 elements'
// worth of the row's arithmetic.
__device__ __forceinline__ float quotient(float s, float n, float inv) {
  const float q = s * inv;
  return fmaf(fmaf(-q, n, s), inv, q);
}
__device__ __forceinline__ float inv_sqrt(float v) {
  const float r = rsqrtf(v);
  const float e = fmaf(-v * r, r, 1.f);  // no number where r is infinite: r stands then
  return e == e ? fmaf(0.5f * r, e, r) : r;
}

constexpr int block_threads(int gt) { return gt > 32 ? gt : 256; }
// The backward keeps a row pair, the next one and the column sums in registers: one block of 384
// threads (168 registers each) has more rows on their way than one of 256 (bf16, 100 million numbers
// in rows of 96: 109 against 130 us, of 768: 108 against 129). bf16 rows of four pieces a thread do
// not fit 168 registers and spill: rows of 128 take 183 us, of 256 and 512 155, of 1,024 212, where
// 256 threads take 117.
constexpr int bwd_threads(int gt) { return gt > 32 ? gt : 384; }

// GT threads share a row; each holds NV pieces of E elements: thread t's piece i covers the
// columns (i GT + t) E ... + E - 1.
template <typename T, int GT, int NV, int E>
__global__ void __launch_bounds__(block_threads(GT))
    k_ln_fwd(const T* __restrict__ x, const void* __restrict__ w, const void* __restrict__ b,
             int wtype, int64_t rows, int cols, float eps, T* __restrict__ y,
             float* __restrict__ mean, float* __restrict__ rstd) {
  constexpr int BT = block_threads(GT), GROUPS = BT / GT;
  __shared__ float red[2][GT > 32 ? GT / 32 : 1];
  const int t = threadIdx.x % GT, grp = threadIdx.x / GT;
  const float n = (float)cols, inv = 1.f / n;
  float wr[NV][E], br[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (i * GT + t) * E + e;
      wr[i][e] = c < cols ? param(w, wtype, c, 1.f) : 0.f;
      br[i][e] = c < cols ? param(b, wtype, c, 0.f) : 0.f;
    }
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  // every group of a warp walks the same number of rows (shuffles need the whole warp)
  const int64_t first = (int64_t)blockIdx.x * GROUPS;
  Piece<T, E> nx[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * GT + t) * E;
      if (row < rows && c < cols)
        nx[i].load(x + row * cols + c);
      else
        nx[i].zero();
    }
  };
  fetch(first + grp);
  for (int64_t r0 = first; r0 < rows; r0 += step) {
    const int64_t row = r0 + grp;
    float v[NV][E];
#pragma unroll
    for (int i = 0; i < NV; ++i) nx[i].get(v[i]);
    if (r0 + step < rows) fetch(row + step);  // the next row's loads run under this one's sums
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) s[0] += v[i][e];
    group_sum<GT>(s, red[0]);
    const float mu = quotient(s[0], n, inv);
    float q[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      // a piece lies inside the row or outside (of several elements, the last alone can be outside)
      const float m = (E > 1 && i + 1 < NV) || (i * GT + t) * E < cols ? mu : 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        v[i][e] -= m;
        q[0] = fmaf(v[i][e], v[i][e], q[0]);
      }
    }
    group_sum<GT>(q, red[1]);
    const float rs = inv_sqrt(fmaf(q[0], inv, eps));
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * GT + t) * E;
        if (c < cols) {
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = fmaf(v[i][e] * rs, wr[i][e], br[i][e]);
          Piece<T, E>::store(y + row * cols + c, o);
        }
      }
      if (t == 0) {
        if (mean) mean[row] = mu;
        if (rstd) rstd[row] = rs;
      }
    }
  }
}

// Backward of the same rows. part: [gridDim.x][2][cols] column sums of dy x^ and dy (or null).
template <typename T, int GT, int NV, int E>
__global__ void __launch_bounds__(bwd_threads(GT))
    k_ln_bwd(const T* __restrict__ dy, const T* __restrict__ x, const void* __restrict__ w,
             int wtype, const float* __restrict__ mean, const float* __restrict__ rstd,
             int64_t rows, int cols, T* __restrict__ dx, float* __restrict__ part) {
  constexpr int BT = bwd_threads(GT), GROUPS = BT / GT;
  __shared__ float red[2][GT > 32 ? 2 * (GT / 32) : 2];
  const int t = threadIdx.x % GT, grp = threadIdx.x / GT;
  const float n = (float)cols, inv = 1.f / n;
  float wr[NV][E], aw[NV][E], ab[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int c = (i * GT + t) * E + e;
      wr[i][e] = c < cols ? param(w, wtype, c, 1.f) : 0.f;
      aw[i][e] = ab[i][e] = 0.f;
    }
  const int64_t step = (int64_t)gridDim.x * GROUPS;
  const int64_t first = (int64_t)blockIdx.x * GROUPS;
  Piece<T, E> nx[NV], nd[NV];
  float nmu = 0.f, nrs = 0.f;
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * GT + t) * E;
      if (row < rows && c < cols) {
        nx[i].load(x + row * cols + c);
        nd[i].load(dy + row * cols + c);
      } else {
        nx[i].zero();
        nd[i].zero();
      }
    }
    nmu = row < rows ? mean[row] : 0.f;
    nrs = row < rows ? rstd[row] : 0.f;
  };
  fetch(first + grp);
  int par = 0;
  for (int64_t r0 = first; r0 < rows; r0 += step, par ^= 1) {
    const int64_t row = r0 + grp;
    float xv[NV][E], dv[NV][E];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      nx[i].get(xv[i]);
      nd[i].get(dv[i]);
    }
    const float mu = nmu, rs = nrs;
    if (r0 + step < rows) fetch(row + step);
    float s[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        // a column past the row has dy = 0 and w = 0: it adds nothing to any sum
        const float xh = (xv[i][e] - mu) * rs;
        aw[i][e] = fmaf(dv[i][e], xh, aw[i][e]);
        ab[i][e] += dv[i][e];
        const float g = dv[i][e] * wr[i][e];
        xv[i][e] = xh;
        dv[i][e] = g;
        s[0] += g;
        s[1] = fmaf(g, xh, s[1]);
      }
    group_sum<GT>(s, red[par]);
    const float mg = s[0] * inv, mgx = s[1] * inv;
    if (row < rows) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * GT + t) * E;
        if (c < cols) {
          float o[E];
#pragma unroll
          for (int e = 0; e < E; ++e) o[e] = rs * (dv[i][e] - mg - xv[i][e] * mgx);
          Piece<T, E>::store(dx + row * cols + c, o);
        }
      }
    }
  }
  if (!part) return;
  // column sums of the block: over the groups of a warp by shuffles, then over the warps
  float* dst = part + (int64_t)blockIdx.x * 2 * cols;
  if constexpr (GT < 32) {
#pragma unroll
    for (int o = GT; o < 32; o <<= 1)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < E; ++e) {
          aw[i][e] += __shfl_xor_sync(0xffffffffu, aw[i][e], o);
          ab[i][e] += __shfl_xor_sync(0xffffffffu, ab[i][e], o);
        }
  }
  if constexpr (GT <= 32) {
    constexpr int NW = BT / 32, CW = GT * NV * E;  // columns covered, at most 32 * 4 * 8
    __shared__ float acc[NW][CW];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int pass = 0; pass < 2; ++pass) {
      __syncthreads();
      if (lane < GT)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < E; ++e) acc[warp][(i * GT + t) * E + e] = pass ? ab[i][e] : aw[i][e];
      __syncthreads();
      for (int c = threadIdx.x; c < cols; c += BT) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < NW; ++k) s += acc[k][c];
        dst[pass * cols + c] = s;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const int c = (i * GT + t) * E + e;
        if (c < cols) {
          dst[c] = aw[i][e];
          dst[cols + c] = ab[i][e];
        }
      }
  }
}

// Rows longer than a block's registers hold: one block per row, which is read once per pass (the
// later passes hit L1 / L2). A counter of columns runs a block's threads past the last of up to
// 2^31 - 1, so C, its type, has 64 bits for rows of more than kShortCounter columns. For the others
// 64 bits would cost the loops their unrolling (forward of 50 rows of 1,000,003 bf16: 1,262 against
// 670 us; backward of 5,592 rows of 9,001: 221 against 187).
constexpr int kLongThreads = 512;
constexpr int kShortCounter = 1 << 30;
template <int K> __device__ __forceinline__ void block_sum(float (&v)[K], float* red) {
  __syncthreads();  // the previous sum's words have been read
  group_sum<kLongThreads>(v, red);
}

template <typename T, typename C>
__global__ void __launch_bounds__(kLongThreads)
    k_ln_fwd_long(const T* __restrict__ x, const void* __restrict__ w, const void* __restrict__ b,
                  int wtype, int64_t rows, int cols, float eps, T* __restrict__ y,
                  float* __restrict__ mean, float* __restrict__ rstd) {
  __shared__ float red[kLongThreads / 32];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * cols;
    float s[1] = {0.f};
    for (C c = threadIdx.x; c < cols; c += kLongThreads) s[0] += to_f(xr[c]);
    block_sum(s, red);
    const float mu = s[0] / (float)cols;
    s[0] = 0.f;
    for (C c = threadIdx.x; c < cols; c += kLongThreads) {
      const float d = to_f(xr[c]) - mu;
      s[0] = fmaf(d, d, s[0]);
    }
    block_sum(s, red);
    const float rs = 1.f / sqrtf(s[0] / (float)cols + eps);
    for (C c = threadIdx.x; c < cols; c += kLongThreads)
      y[row * cols + c] = from_f<T>(fmaf((to_f(xr[c]) - mu) * rs, param(w, wtype, (int)c, 1.f),
                                         param(b, wtype, (int)c, 0.f)));
    if (threadIdx.x == 0) {
      if (mean) mean[row] = mu;
      if (rstd) rstd[row] = rs;
    }
  }
}

template <typename T, typename C>
__global__ void __launch_bounds__(kLongThreads)
    k_ln_bwd_long(const T* __restrict__ dy, const T* __restrict__ x, const void* __restrict__ w,
                  int wtype, const float* __restrict__ mean, const float* __restrict__ rstd,
                  int64_t rows, int cols, T* __restrict__ dx) {
  __shared__ float red[2 * (kLongThreads / 32)];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * cols;
    const T* dr = dy + row * cols;
    const float mu = mean[row], rs = rstd[row];
    float s[2] = {0.f, 0.f};
    for (C c = threadIdx.x; c < cols; c += kLongThreads) {
      const float g = to_f(dr[c]) * param(w, wtype, (int)c, 1.f);
      s[0] += g;
      s[1] = fmaf(g, (to_f(xr[c]) - mu) * rs, s[1]);
    }
    block_sum(s, red);
    const float mg = s[0] / (float)cols, mgx = s[1] / (float)cols;
    for (C c = threadIdx.x; c < cols; c += kLongThreads) {
      const float g = to_f(dr[c]) * param(w, wtype, (int)c, 1.f);
      dx[row * cols + c] = from_f<T>(rs * (g - mg - (to_f(xr[c]) - mu) * rs * mgx));
    }
  }
}

// Column sums of long rows: a thread per column, blockIdx.y a range of rows.
template <typename T, typename C>
__global__ void __launch_bounds__(256)
    k_ln_cols(const T* __restrict__ dy, const T* __restrict__ x, const float* __restrict__ mean,
              const float* __restrict__ rstd, int64_t rows, int cols, float* __restrict__ part) {
  const C c = (C)blockIdx.x * 256 + (C)threadIdx.x;
  if (c >= cols) return;
  float a = 0.f, b = 0.f;
  for (int64_t row = blockIdx.y; row < rows; row += gridDim.y) {
    const float d = to_f(dy[row * cols + c]);
    a = fmaf(d, (to_f(x[row * cols + c]) - mean[row]) * rstd[row], a);
    b += d;
  }
  part[(int64_t)blockIdx.y * 2 * cols + c] = a;
  part[(int64_t)blockIdx.y * 2 * cols + cols + c] = b;
}

// dw, db from the blocks' column sums: 32 threads of a block share a column, each adding every
// 32nd block's word; their sums are added in a fixed tree.
__global__ void __launch_bounds__(1024)
    k_ln_finish(const float* __restrict__ part, int nparts, int cols, int wtype,
                void* __restrict__ dw, void* __restrict__ db) {
  __shared__ float acc[32][33];
  const int lane = threadIdx.x & 31, g = threadIdx.x >> 5;
  const int64_t c = blockIdx.x * 32ll + lane;
  void* dst = blockIdx.y ? db : dw;
  if (!dst) return;
  float s = 0.f;
  if (c < cols) {
    const float* p = part + (int64_t)blockIdx.y * cols + c;
#pragma unroll 8
    for (int i = g; i < nparts; i += 32) s += p[(int64_t)i * 2 * cols];
  }
  acc[g][lane] = s;
  __syncthreads();
  float r = acc[lane][g];  // warp g adds column g
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
  const int64_t col = blockIdx.x * 32ll + g;
  if (lane == 0 && col < cols) {
    if (wtype == PACK3D_BF16)
      static_cast<__nv_bfloat16*>(dst)[col] = __float2bfloat16_rn(r);
    else
      static_cast<float*>(dst)[col] = r;
  }
}

struct Args {
  const void *dy, *x, *w, *b;
  void *y, *dx;
  float *mean, *rstd, *part;
  const float *cmean, *crstd;
  int wtype;
  int64_t rows;
  int cols;
  float eps;
  cudaStream_t s;
};

// Blocks that fill the device: the launch's blocks are persistent.
inline int grid_for(const void* fn, int threads, PerDevice& cache) {
  const int n = cache.get([&] {
    int per = 0;
    const bool ok =
        cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, fn, threads, 0) == cudaSuccess;
    return ok ? per * sm_count() : 0;
  });
  return n > 0 ? n : sm_count();
}

constexpr int kMaxParts = 2048;  // most blocks a backward launch may have (a row of sums each)

template <typename T, int GT, int NV, int E> int run(const Args& a, bool bwd) {
  constexpr int BT = block_threads(GT), GROUPS = BT / GT;
  const int64_t blocks = (a.rows + GROUPS - 1) / GROUPS;
  if (!bwd) {
    static PerDevice fit;
    const int cap = grid_for(reinterpret_cast<const void*>(k_ln_fwd<T, GT, NV, E>), BT, fit);
    const int grid = (int)(blocks < cap ? blocks : cap);
    k_ln_fwd<T, GT, NV, E><<<grid, BT, 0, a.s>>>(
        static_cast<const T*>(a.x), a.w, a.b, a.wtype, a.rows, a.cols, a.eps,
        static_cast<T*>(a.y), a.mean, a.rstd);
    return grid;
  }
  constexpr int BB = bwd_threads(GT);
  const int64_t bblocks = (a.rows + BB / GT - 1) / (BB / GT);
  static PerDevice fit;
  const int most = grid_for(reinterpret_cast<const void*>(k_ln_bwd<T, GT, NV, E>), BB, fit);
  const int cap = most < kMaxParts ? most : kMaxParts;
  const int grid = (int)(bblocks < cap ? bblocks : cap);
  k_ln_bwd<T, GT, NV, E><<<grid, BB, 0, a.s>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.w, a.wtype, a.cmean, a.crstd,
      a.rows, a.cols, static_cast<T*>(a.dx), a.part);
  return grid;
}

template <typename T, int GT, int E> int by_pieces(const Args& a, bool bwd, int nv) {
  switch (nv) {
    case 1: return run<T, GT, 1, E>(a, bwd);
    case 2: return run<T, GT, 2, E>(a, bwd);
    case 3: return run<T, GT, 3, E>(a, bwd);
    default: return run<T, GT, 4, E>(a, bwd);
  }
}

// Threads per row: the fewest whose registers hold the row in at most 4 pieces each. Few threads with
// several pieces keep the shuffles and barriers per byte low; more than 4 pieces a thread would cost
// occupancy. Rows that are no whole number of pieces go by single elements, up to 8 each, and up to 16
// where that saves the barriers of several warps per row (training, bf16: 300,001 x 333 by 128 threads
// 650 us, by 32 308; 1,000,000 x 7 by 8 threads of 8 elements 127 us, by 4 of 2 47).
constexpr int kGroups[7] = {4, 8, 16, 32, 128, 256, 512};
constexpr int kSingles = 8;
// Rows of whole pieces of e elements move by pieces as far as registers hold them; ragged and longer
// rows move by elements and may start at any.
constexpr bool moves_by_pieces(int cols, int e) {
  return cols % e == 0 && cols / e <= 4 * kGroups[6];
}

// Long rows: the launches, and the rows of column sums they leave.
template <typename T, typename C> int long_rows(const Args& a, bool bwd) {
  const int64_t cap = 4 * (int64_t)sm_count();
  const int grid = (int)(a.rows < cap ? a.rows : cap);
  if (!bwd) {
    k_ln_fwd_long<T, C><<<grid, kLongThreads, 0, a.s>>>(
        static_cast<const T*>(a.x), a.w, a.b, a.wtype, a.rows, a.cols, a.eps,
        static_cast<T*>(a.y), a.mean, a.rstd);
    return 1;
  }
  k_ln_bwd_long<T, C><<<grid, kLongThreads, 0, a.s>>>(
      static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.w, a.wtype, a.cmean, a.crstd,
      a.rows, a.cols, static_cast<T*>(a.dx));
  int parts = 0;
  if (a.part) {
    parts = (int)(a.rows < 64 ? a.rows : 64);
    k_ln_cols<T, C><<<dim3((unsigned)((a.cols + 255ll) / 256), parts), 256, 0, a.s>>>(
        static_cast<const T*>(a.dy), static_cast<const T*>(a.x), a.cmean, a.crstd, a.rows, a.cols,
        a.part);
    count_launch();
  }
  return parts;
}

template <typename T> int launch(const Args& a, bool bwd) {
  constexpr int E = 16 / (int)sizeof(T);
  if (moves_by_pieces(a.cols, E)) {
    const int pieces = a.cols / E;
    for (int gt : kGroups) {
      const int nv = (pieces + gt - 1) / gt;
      if (nv > 4) continue;
      switch (gt) {
        case 4: return by_pieces<T, 4, E>(a, bwd, nv);
        case 8: return by_pieces<T, 8, E>(a, bwd, nv);
        case 16: return by_pieces<T, 16, E>(a, bwd, nv);
        case 32: return by_pieces<T, 32, E>(a, bwd, nv);
        case 128: return by_pieces<T, 128, E>(a, bwd, nv);
        case 256: return by_pieces<T, 256, E>(a, bwd, nv);
        default: return by_pieces<T, 512, E>(a, bwd, nv);
      }
    }
  } else {
    if (a.cols <= 8) return run<T, 4, 2, 1>(a, bwd);
    if (a.cols <= 32) return run<T, 8, 4, 1>(a, bwd);
    if (a.cols <= 8 * kSingles) return run<T, 8, kSingles, 1>(a, bwd);
    if (a.cols <= 32 * kSingles) return run<T, 32, kSingles, 1>(a, bwd);
    if (a.cols <= 32 * 2 * kSingles) return run<T, 32, 2 * kSingles, 1>(a, bwd);
    if (a.cols <= 128 * kSingles) return run<T, 128, kSingles, 1>(a, bwd);
    if (a.cols <= 512 * kSingles) return run<T, 512, kSingles, 1>(a, bwd);
    if (a.cols <= 1024 * kSingles) return run<T, 512, 2 * kSingles, 1>(a, bwd);
  }
  return a.cols <= kShortCounter ? long_rows<T, int>(a, bwd) : long_rows<T, int64_t>(a, bwd);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool aligned_rows(const void* p, int dtype, int cols) {
  const int size = dtype == PACK3D_BF16 ? 2 : 4;
  const int by = moves_by_pieces(cols, 16 / size) ? 16 : size;
  return reinterpret_cast<uintptr_t>(p) % by == 0;
}

pack3d_status check(int dtype, int wtype, int64_t rows, int32_t cols) {
  if ((dtype != PACK3D_F32 && dtype != PACK3D_BF16) || (wtype != PACK3D_F32 && wtype != PACK3D_BF16))
    return PACK3D_ERR_INVALID_ARG;
  if (rows < 0 || cols <= 0) return PACK3D_ERR_INVALID_ARG;
  if (rows > INT64_MAX / 8 / cols) return PACK3D_ERR_UNSUPPORTED;
  return PACK3D_OK;
}

// Blocks a backward launch of these rows may have at most (its column sums' rows).
int64_t max_parts(int64_t rows) { return rows < kMaxParts ? rows : kMaxParts; }

}  // namespace ln
}  // namespace p3d

using namespace p3d;

extern "C" pack3d_status pack3d_layer_norm_fwd(const void* x, const void* weight, const void* bias,
                                               int dtype, int wdtype, int64_t rows, int32_t cols,
                                               float eps, void* y, float* mean, float* rstd,
                                               void* stream) {
  reset_launches();
  pack3d_status st = ln::check(dtype, wdtype, rows, cols);
  if (st != PACK3D_OK) return st;
  if (!(eps >= 0.f) || isinf(eps)) return PACK3D_ERR_INVALID_ARG;
  if (rows == 0) return PACK3D_OK;
  if (!x || !y) return PACK3D_ERR_INVALID_ARG;
  if (!ln::aligned_rows(x, dtype, cols) || !ln::aligned_rows(y, dtype, cols))
    return PACK3D_ERR_ALIGN;
  if (x == y) return PACK3D_ERR_INVALID_ARG;  // a row is fetched ahead of the stores before it
  ln::Args a{};
  a.x = x; a.w = weight; a.b = bias; a.y = y; a.mean = mean; a.rstd = rstd;
  a.wtype = wdtype; a.rows = rows; a.cols = cols; a.eps = eps;
  a.s = static_cast<cudaStream_t>(stream);
  if (dtype == PACK3D_BF16)
    ln::launch<__nv_bfloat16>(a, false);
  else
    ln::launch<float>(a, false);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? PACK3D_OK : PACK3D_ERR_CUDA;
}

extern "C" size_t pack3d_layer_norm_bwd_workspace_bytes(int dtype, int64_t rows, int32_t cols) {
  if (ln::check(dtype, PACK3D_F32, rows, cols) != PACK3D_OK) return 0;
  const size_t b = (size_t)ln::max_parts(rows) * 2 * (size_t)cols * sizeof(float);
  return b ? b : 4;
}

extern "C" pack3d_status pack3d_layer_norm_bwd(const void* dy, const void* x, const void* weight,
                                               const float* mean, const float* rstd, int dtype,
                                               int wdtype, int64_t rows, int32_t cols, void* dx,
                                               void* dweight, void* dbias, void* workspace,
                                               size_t workspace_bytes, void* stream) {
  reset_launches();
  pack3d_status st = ln::check(dtype, wdtype, rows, cols);
  if (st != PACK3D_OK) return st;
  const bool cols_out = dweight || dbias;
  if (rows > 0) {
    if (!dy || !x || !mean || !rstd || !dx) return PACK3D_ERR_INVALID_ARG;
    for (const void* p : {dy, x, static_cast<const void*>(dx)})
      if (!ln::aligned_rows(p, dtype, cols)) return PACK3D_ERR_ALIGN;
    if (dx == dy || dx == x) return PACK3D_ERR_INVALID_ARG;
    if (cols_out) {
      if (!workspace) return PACK3D_ERR_INVALID_ARG;
      if (!ln::aligned16(workspace)) return PACK3D_ERR_ALIGN;
      if (workspace_bytes < pack3d_layer_norm_bwd_workspace_bytes(dtype, rows, cols))
        return PACK3D_ERR_WORKSPACE;
    }
  }
  ln::Args a{};
  a.dy = dy; a.x = x; a.w = weight; a.cmean = mean; a.crstd = rstd; a.dx = dx;
  a.part = cols_out ? static_cast<float*>(workspace) : nullptr;
  a.wtype = wdtype; a.rows = rows; a.cols = cols;
  a.s = static_cast<cudaStream_t>(stream);
  int parts = 0;
  if (rows > 0) {
    parts = dtype == PACK3D_BF16 ? ln::launch<__nv_bfloat16>(a, true) : ln::launch<float>(a, true);
    count_launch();
  }
  if (cols_out) {  // no rows: the sums are zero
    ln::k_ln_finish<<<dim3((unsigned)((cols + 31ll) / 32), 2), 1024, 0, a.s>>>(a.part, parts, cols, wdtype,
                                                               dweight, dbias);
    count_launch();
  }
  return cudaGetLastError() == cudaSuccess ? PACK3D_OK : PACK3D_ERR_CUDA;
}
