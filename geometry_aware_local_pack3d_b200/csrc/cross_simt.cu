// Cross attention in fp32 on CUDA cores (no TF32: the 32-bit path keeps 32-bit products), forward
// and backward, head_dim 48, 64, 96 or 128.
//
// Tiles of 64 rows x 64 states; 256 threads as 16 x 16, thread (ty, tx) holding rows 4 ty .. + 3
// and states tx + 16 j of a score tile. What bounds it: shared memory and the FMA pipe in turn, with
// too few warps to fill either; a thread's 4 x 4 scores take 64 FMAs per 8 shared loads of 16 bytes
// (measured, 4 heads of 2,500 rows to 2,500 states of 128: forward 475 us, backward 1,518; FMA pipe 46
// to 50 %, shared memory 55 to 59 % busy with the 8 warps that an SM holds). The rows of a masked state
// are read as zeros, so that nothing they hold reaches a product, and their scores are -inf.
//   k_cross_fwd32   online softmax over a range of the state tiles, o and lse
//   k_cross_dq32    dq_i = sum_j dS_ij k_j,            dS = p (dO v - D) tau, over such a range
//   k_cross_dkv32   dk_j = sum_i dS_ij q_i,  dv_j = sum_i p_ij dO_i over a range of row tiles; the
//                   ranges' sums are added in order by k_cross_sum
// The state ranges (one, unless the row tiles leave SMs idle) are joined by k_cross_join (o, lse) and
// k_cross_sum32 (dq). Every sum runs in a fixed order (no atomics). A tile's 64 products are summed
// apart and then added: one sum over 16,384 states or 65,536 rows would lose three bits to its order.
// exp(s tau - lse) is formed as written, not as 2^(s tau log2 e - lse log2 e), whose rounded second
// term would move a whole row's probabilities.
#include <math.h>

#include <algorithm>

#include "cross.h"
#include "launch.h"

namespace p3d {
namespace xa {

namespace xs {
constexpr int kT = 64;          // rows, states per tile
constexpr int kThreads = 256;
constexpr int kP = kT + 4;      // pitch of a score tile
template <int D> constexpr int pitch() { return D + 4; }

template <int D>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t row0, int64_t rows,
                                          uint32_t w0, uint32_t w1) {
  constexpr int C = D / 4;
  for (int i = threadIdx.x; i < kT * C; i += kThreads) {
    const int r = i / C, c = (i % C) * 4;
    const bool on = row0 + r < rows && (((r < 32 ? w0 : w1) >> (r & 31)) & 1u);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (on) x = *reinterpret_cast<const float4*>(src + (row0 + r) * D + c);
    *reinterpret_cast<float4*>(dst + r * pitch<D>() + c) = x;
  }
}

// s[i][j] = <a row 4 ty + i, b row tx + 16 j>
template <int D>
__device__ __forceinline__ void product(const float* a, const float* b, int ty, int tx,
                                        float (&s)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
  for (int c = 0; c < D; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * pitch<D>() + c);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * pitch<D>() + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
        s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
        s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
        s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
      }
  }
}

// The D / 16 columns of thread tx: pairs of neighbours (one 8-byte load from shared memory feeds
// eight FMAs; single columns would take as many load cycles as FMAs), and one more where D is an odd
// number of sixteens.
template <int D> __device__ __forceinline__ void columns(const float* row, int tx, float (&y)[D / 16]) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    const float2 x = *reinterpret_cast<const float2*>(row + 32 * c + 2 * tx);
    y[2 * c] = x.x;
    y[2 * c + 1] = x.y;
  }
  if (D % 32) y[D / 16 - 1] = row[D / 32 * 32 + tx];
}
template <int D>
__device__ __forceinline__ void store_columns(float* row, int tx, const float (&y)[D / 16], float f) {
#pragma unroll
  for (int c = 0; c < D / 32; ++c)
    *reinterpret_cast<float2*>(row + 32 * c + 2 * tx) = make_float2(y[2 * c] * f, y[2 * c + 1] * f);
  if (D % 32) row[D / 32 * 32 + tx] = y[D / 16 - 1] * f;
}
template <int D> __device__ __forceinline__ void clear(float (&a)[4][D / 16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) a[i][c] = 0.f;
}
template <int D>
__device__ __forceinline__ void add(float (&acc)[4][D / 16], const float (&a)[4][D / 16]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[i][c] += a[i][c];
}

// out[i][c] += sum over the 64 inner rows of m[4 ty + i][inner] b[inner][column c of tx]
template <int D>
__device__ __forceinline__ void accumulate(const float* m, const float* b, int ty, int tx,
                                           float (&out)[4][D / 16]) {
  float acc[4][D / 16];
  clear<D>(acc);
#pragma unroll 2
  for (int k = 0; k < kT; k += 4) {
    float4 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(m + (4 * ty + i) * kP + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float y[D / 16];
      columns<D>(b + (k + e) * pitch<D>(), tx, y);
#pragma unroll
      for (int c = 0; c < D / 16; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc[i][c] = fmaf(e == 0 ? x[i].x : e == 1 ? x[i].y : e == 2 ? x[i].z : x[i].w, y[c],
                           acc[i][c]);
    }
  }
  add<D>(out, acc);
}

// As accumulate with m transposed: out[i][c] += sum over rows r < n of m[r][4 ty + i] b[r][column c]
template <int D>
__device__ __forceinline__ void accumulate_t(const float* m, const float* b, int n, int ty, int tx,
                                             float (&out)[4][D / 16]) {
  float acc[4][D / 16];
  clear<D>(acc);
#pragma unroll 4
  for (int r = 0; r < n; ++r) {
    const float4 x = *reinterpret_cast<const float4*>(m + r * kP + 4 * ty);
    float y[D / 16];
    columns<D>(b + r * pitch<D>(), tx, y);
#pragma unroll
    for (int c = 0; c < D / 16; ++c) {
      acc[0][c] = fmaf(x.x, y[c], acc[0][c]);
      acc[1][c] = fmaf(x.y, y[c], acc[1][c]);
      acc[2][c] = fmaf(x.z, y[c], acc[2][c]);
      acc[3][c] = fmaf(x.w, y[c], acc[3][c]);
    }
  }
  add<D>(out, acc);
}

__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct Params {
  const float *q, *k, *v, *dO, *o;
  const float *lse;       // backward
  float *out, *out_lse;   // o, lse  |  dq
  float *part, *part_lse;  // of nstate > 1 state ranges: o or dq [nstate][rows][D], lse
  float *dk, *dv;         // partial sums [nsplit][bh][l][D]
  float *delta;           // [bh][np]
  const int32_t* act;
  const uint32_t* bits;
  int64_t np, l, bh, words;
  int tiles, kv_heads;
  int nstate, nsplit;  // state ranges (o, dq); row ranges (dk, dv)
  float scale;
};

// Half-tiles (64 states) of the batch entry: number, place and bits of the i-th.
struct Halves {
  const int32_t* list;
  const uint32_t* bits;
  int n;
  int64_t l;
  __device__ __forceinline__ Halves(const Params& P, int64_t bh) {
    const int64_t b = bh / P.kv_heads;
    list = P.act ? P.act + b * (P.tiles + 1) + 1 : nullptr;
    bits = P.act ? P.bits + b * P.words : nullptr;
    n = 2 * (P.act ? list[-1] : P.tiles);
    l = P.l;
  }
  __device__ __forceinline__ int64_t at(int i, uint32_t& w0, uint32_t& w1) const {
    const int64_t at = (int64_t)(list ? list[i >> 1] : i >> 1) * kTile + (i & 1) * kT;
    uint32_t w[2];
    state_words(bits, l, at, w);
    w0 = w[0];
    w1 = w[1];
    return at;
  }
  // the half-tiles of range z of `ranges`
  __device__ __forceinline__ int begin(int z, int ranges) const {
    return (int)((int64_t)n * z / ranges);
  }
  __device__ __forceinline__ int end(int z, int ranges) const { return begin(z + 1, ranges); }
};

// Whether the warp's 8 rows of a tile hold one of the problem's: a few rows are the work of a few warps.
__device__ __forceinline__ bool warp_lives(int64_t row0, int64_t np) {
  return row0 + (threadIdx.x >> 5) * 8 < np;
}
__device__ __forceinline__ bool on(uint32_t w0, uint32_t w1, int j) {
  return ((j < 32 ? w0 : w1) >> (j & 31)) & 1u;
}
}  // namespace xs

template <int D>
__global__ void __launch_bounds__(xs::kThreads, D <= 96 ? 2 : 1) k_cross_fwd32(const xs::Params P) {
  using namespace xs;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sk = sq + kT * pitch<D>();
  float* sv = sk + kT * pitch<D>();
  float* sp = sv + kT * pitch<D>();
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int64_t bh = blockIdx.y, row0 = (int64_t)blockIdx.x * kT;
  const bool live = warp_lives(row0, P.np);
  const Halves H(P, bh);
  load_tile<D>(sq, P.q + bh * P.np * D, row0, P.np, ~0u, ~0u);
  float acc[4][D / 16], m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  clear<D>(acc);
  const float sl2 = P.scale * kLog2e;
  const int h1 = H.end(blockIdx.z, P.nstate);
  for (int h = H.begin(blockIdx.z, P.nstate); h < h1; ++h) {
    uint32_t w0, w1;
    const int64_t at = H.at(h, w0, w1);
    if (!(w0 | w1)) continue;
    __syncthreads();
    load_tile<D>(sk, P.k + bh * P.l * D, at, P.l, w0, w1);
    load_tile<D>(sv, P.v + bh * P.l * D, at, P.l, w0, w1);
    __syncthreads();
    if (!live) continue;
    float s[4][4];
    product<D>(sq, sk, ty, tx, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = on(w0, w1, tx + 16 * j) ? s[i][j] : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
      const float mn = fmaxf(m[i], row_max(top) * sl2);
      const float base = mn == -INFINITY ? 0.f : mn;
      const float f = exp2f(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(fmaf(s[i][j], sl2, -base));
        sum += p;
        sp[(4 * ty + i) * kP + tx + 16 * j] = p;
      }
      l[i] = l[i] * f + row_sum(sum);
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < D / 16; ++c) acc[i][c] *= f;
    }
    __syncwarp();  // a warp's rows of sp are its own
    accumulate<D>(sp, sv, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * ty + i;
    if (row >= P.np) continue;
    const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
    const bool parts = P.nstate > 1;
    const int64_t at = (parts ? blockIdx.z * P.bh * P.np : 0) + bh * P.np + row;
    float* const o = (parts ? P.part : P.out) + at * D;
    float* const lse = parts ? P.part_lse : P.out_lse;
    store_columns<D>(o, tx, acc[i], inv);
    if (lse && tx == 0) lse[at] = l[i] == 0.f ? -INFINITY : fmaf(m[i], kLn2, logf(l[i]));
  }
}

// delta_i = <dO_i, o_i>: 8 threads per row
template <int D>
__global__ void __launch_bounds__(256) k_cross_delta32(const xs::Params P) {
  const int64_t row = blockIdx.x * 32ll + (threadIdx.x >> 3);
  const int t = threadIdx.x & 7;
  float s = 0.f;
  if (row < P.bh * P.np)
    for (int c = t * 4; c < D; c += 32) {
      const float4 a = *reinterpret_cast<const float4*>(P.dO + row * D + c);
      const float4 b = *reinterpret_cast<const float4*>(P.o + row * D + c);
      s = fmaf(a.x, b.x, fmaf(a.y, b.y, fmaf(a.z, b.z, fmaf(a.w, b.w, s))));
    }
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (t == 0 && row < P.bh * P.np) P.delta[row] = s;
}

namespace xs {
// Scores of a tile as probabilities (into sp, if any) and dS (into sd, which may lie over sv: `over`).
template <int D, bool over>
__device__ __forceinline__ void grads(const float* sq, const float* sg, const float* sk,
                                      const float* sv, float* sp, float* sd, int ty, int tx,
                                      const float (&nl)[4], const float (&dl)[4], uint32_t w0,
                                      uint32_t w1, float scale, bool live) {
  float s[4][4], g[4][4];
  if (live) {
    product<D>(sq, sk, ty, tx, s);
    product<D>(sg, sv, ty, tx, g);
  }
  if (over) __syncthreads();  // V has been read
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool in = on(w0, w1, tx + 16 * j);
      const float p = in ? expf(fmaf(s[i][j], scale, nl[i])) : 0.f;
      const int at = (4 * ty + i) * kP + tx + 16 * j;
      if (sp) sp[at] = p;
      sd[at] = p * (g[i][j] - dl[i]) * scale;
    }
}
}  // namespace xs

template <int D>
__global__ void __launch_bounds__(xs::kThreads, D <= 96 ? 2 : 1) k_cross_dq32(const xs::Params P) {
  using namespace xs;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sg = sq + kT * pitch<D>();
  float* sk = sg + kT * pitch<D>();
  float* sv = sk + kT * pitch<D>();
  float* sd = sv;  // dS over V, so that two blocks share an SM up to d = 96
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int64_t bh = blockIdx.y, row0 = (int64_t)blockIdx.x * kT;
  const bool live = warp_lives(row0, P.np);
  const Halves H(P, bh);
  load_tile<D>(sq, P.q + bh * P.np * D, row0, P.np, ~0u, ~0u);
  load_tile<D>(sg, P.dO + bh * P.np * D, row0, P.np, ~0u, ~0u);
  float acc[4][D / 16], nl[4], dl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * ty + i;
    const bool in = row < P.np;
    const float lse = in ? P.lse[bh * P.np + row] : -INFINITY;
    nl[i] = lse == -INFINITY ? -INFINITY : -lse;  // a row without any state: p = 0
    dl[i] = in ? P.delta[bh * P.np + row] : 0.f;
  }
  clear<D>(acc);
  const int h1 = H.end(blockIdx.z, P.nstate);
  for (int h = H.begin(blockIdx.z, P.nstate); h < h1; ++h) {
    uint32_t w0, w1;
    const int64_t at = H.at(h, w0, w1);
    if (!(w0 | w1)) continue;
    __syncthreads();
    load_tile<D>(sk, P.k + bh * P.l * D, at, P.l, w0, w1);
    load_tile<D>(sv, P.v + bh * P.l * D, at, P.l, w0, w1);
    __syncthreads();
    grads<D, true>(sq, sg, sk, sv, nullptr, sd, ty, tx, nl, dl, w0, w1, P.scale, live);
    __syncwarp();
    if (live) accumulate<D>(sd, sk, ty, tx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + 4 * ty + i;
    if (row >= P.np) continue;
    float* const dq = (P.nstate > 1 ? P.part + blockIdx.z * P.bh * P.np * D : P.out) +
                      (bh * P.np + row) * D;
    store_columns<D>(dq, tx, acc[i], 1.f);
  }
}

template <int D>
__global__ void __launch_bounds__(xs::kThreads, D <= 64 ? 2 : 1) k_cross_dkv32(const xs::Params P) {
  using namespace xs;
  extern __shared__ __align__(16) float sm[];
  float* sq = sm;
  float* sg = sq + kT * pitch<D>();
  float* sk = sg + kT * pitch<D>();
  float* sv = sk + kT * pitch<D>();
  float* sp = sv + kT * pitch<D>();
  float* sd = sp + kT * kP;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int64_t bh = blockIdx.y;
  const int half = blockIdx.x / P.nsplit, split = blockIdx.x % P.nsplit;
  const int64_t at = (int64_t)half * kT;
  uint32_t w[2];
  state_words(P.act ? P.bits + bh / P.kv_heads * P.words : nullptr, P.l, at, w);
  const uint32_t w0 = w[0], w1 = w[1];
  load_tile<D>(sk, P.k + bh * P.l * D, at, P.l, w0, w1);
  load_tile<D>(sv, P.v + bh * P.l * D, at, P.l, w0, w1);
  float ak[4][D / 16], av[4][D / 16];
  clear<D>(ak);
  clear<D>(av);
  const int64_t qt = (P.np + kT - 1) / kT;
  const int64_t t0 = qt * split / P.nsplit, t1 = (w0 | w1) ? qt * (split + 1) / P.nsplit : t0;
  for (int64_t t = t0; t < t1; ++t) {
    const int64_t row0 = t * kT;
    __syncthreads();
    load_tile<D>(sq, P.q + bh * P.np * D, row0, P.np, ~0u, ~0u);
    load_tile<D>(sg, P.dO + bh * P.np * D, row0, P.np, ~0u, ~0u);
    float nl[4], dl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + 4 * ty + i;
      const bool in = row < P.np;
      const float lse = in ? P.lse[bh * P.np + row] : -INFINITY;
      nl[i] = lse == -INFINITY ? -INFINITY : -lse;  // a row without any state: p = 0
      dl[i] = in ? P.delta[bh * P.np + row] : 0.f;
    }
    __syncthreads();
    grads<D, false>(sq, sg, sk, sv, sp, sd, ty, tx, nl, dl, w0, w1, P.scale,
                    warp_lives(row0, P.np));
    __syncthreads();
    const int n = P.np - row0 < kT ? (int)(P.np - row0 + 7) & ~7 : kT;  // rows of warps that live
    accumulate_t<D>(sp, sg, n, ty, tx, av);
    accumulate_t<D>(sd, sq, n, ty, tx, ak);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t row = at + 4 * ty + i;
    if (row >= P.l) continue;
    const int64_t dst = ((split * P.bh + bh) * P.l + row) * D;
    if (P.act && !((P.bits[bh / P.kv_heads * P.words + (row >> 5)] >> (row & 31)) & 1u)) {
      // A masked state: zeros, not 0 x dO and 0 x q of rows that may not be finite. (The words above,
      // kept until here, would take registers from the loop: d = 64 769 against 749 us on 4 x 2,500.)
#pragma unroll
      for (int c = 0; c < D / 16; ++c) ak[i][c] = av[i][c] = 0.f;
    }
    store_columns<D>(P.dk + dst, tx, ak[i], 1.f);
    store_columns<D>(P.dv + dst, tx, av[i], 1.f);
  }
}

// out = sum over the ranges of part, in order
__global__ void __launch_bounds__(256)
    k_cross_sum32(const float* __restrict__ part, int nsplit, int64_t n, float* __restrict__ dk,
                  const float* __restrict__ part2, float* __restrict__ dv) {
  const int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 4;
  if (i >= n) return;
  const float* p = blockIdx.y ? part2 : part;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int k = 0; k < nsplit; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(p + k * n + i);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  *reinterpret_cast<float4*>((blockIdx.y ? dv : dk) + i) = s;
}

// Ranges that `items` blocks of `steps` tiles each are cut into: the count whose blocks fill the last
// wave of `slots` best, at least 5 % better than fewer (partial rows are written and read again); a
// block's fixed cost is about that of one tile. (A single row over a long context would otherwise be
// the work of one block per problem: 8 heads over 16,384 states of 64, forward 660 -> 83 us; 160
// blocks on 148 SMs would take two waves.)
static int ranges(int64_t items, int64_t steps, int64_t slots) {
  const int64_t most = std::min<int64_t>((4 * slots + items - 1) / items, kMaxSplits);
  int best = 1;
  double eff = 0.0;
  for (int64_t n = 1; n <= most && n <= steps; ++n) {
    const int64_t waves = (items * n + slots - 1) / slots;
    const double e = (double)steps * items / (waves * slots * ((double)((steps + n - 1) / n) + 1.0));
    if (e > eff * 1.05) {
      eff = e;
      best = (int)n;
    }
  }
  return best;
}
static int64_t tiles64(int64_t n) { return (n + xs::kT - 1) / xs::kT; }
// Ranges of states for o and dq (two blocks per SM up to d = 96), of rows for dk and dv (two up to 64).
static int state_ranges(const Problem& p) {
  return ranges(p.bh * tiles64(p.np), tiles64(p.l), (p.d <= 96 ? 2 : 1) * (int64_t)sm_count());
}
static int row_ranges(const Problem& p) {
  return ranges(p.bh * tiles64(p.l), tiles64(p.np), (p.d <= 64 ? 2 : 1) * (int64_t)sm_count());
}
static size_t part_bytes(const Problem& p, int n) {
  return n > 1 ? align256((size_t)n * p.bh * p.np * p.d * sizeof(float)) : 0;
}

static xs::Params simt_params(const Problem& p, const MaskTables& m) {
  xs::Params P{};
  P.q = static_cast<const float*>(p.q);
  P.k = static_cast<const float*>(p.k);
  P.v = static_cast<const float*>(p.v);
  P.act = m.act;
  P.bits = m.bits;
  P.np = p.np;
  P.l = p.l;
  P.bh = p.bh;
  P.words = m.words;
  P.tiles = m.tiles;
  P.kv_heads = p.kv_heads;
  P.nstate = state_ranges(p);
  P.nsplit = 1;
  P.scale = p.scale;
  return P;
}

template <int D> static cudaError_t launch_fwd32(const Problem& p, xs::Params P) {
  constexpr int bytes = 4 * (3 * xs::kT * xs::pitch<D>() + xs::kT * xs::kP);
  static std::atomic<uint64_t> attr{0};
  const cudaError_t e =
      smem_attr_once(reinterpret_cast<const void*>(k_cross_fwd32<D>), bytes, attr);
  if (e != cudaSuccess) return e;
  k_cross_fwd32<D><<<dim3((unsigned)((p.np + xs::kT - 1) / xs::kT), (unsigned)p.bh, P.nstate),
                     xs::kThreads, bytes, p.s>>>(P);
  count_launch();
  if (P.nstate > 1) return join_splits(p, P.part, P.part_lse, P.nstate, P.out, P.out_lse);
  return cudaGetLastError();
}

size_t fwd_simt_bytes(const Problem& p) {
  const int n = state_ranges(p);
  return n > 1 ? part_bytes(p, n) + align256((size_t)n * p.bh * p.np * sizeof(float)) : 0;
}

cudaError_t fwd_simt(const Problem& p, const MaskTables& m, void* o, float* lse, void* ws) {
  xs::Params P = simt_params(p, m);
  if (P.nstate > 1) {
    P.part = static_cast<float*>(ws);
    P.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + part_bytes(p, P.nstate));
  }
  P.out = static_cast<float*>(o);
  P.out_lse = lse;
  switch (p.d) {
    case 48: return launch_fwd32<48>(p, P);
    case 64: return launch_fwd32<64>(p, P);
    case 96: return launch_fwd32<96>(p, P);
    default: return launch_fwd32<128>(p, P);
  }
}

size_t bwd_simt_bytes(const Problem& p) {
  const size_t n = row_ranges(p), e = (size_t)p.bh * p.l * p.d * sizeof(float);
  return align256((size_t)p.bh * p.np * sizeof(float)) + part_bytes(p, state_ranges(p)) +
         (n > 1 ? 2 * align256(n * e) : 0);
}

template <int D> static cudaError_t launch_bwd32(const Problem& p, xs::Params P, float* dk, float* dv) {
  constexpr int tile = xs::kT * xs::pitch<D>();
  constexpr int score = xs::kT * xs::kP;
  constexpr int bq = 4 * (3 * tile + (tile > score ? tile : score)), bk = 4 * (4 * tile + 2 * score);
  static std::atomic<uint64_t> aq{0}, ak{0};
  cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(k_cross_dq32<D>), bq, aq);
  if (e == cudaSuccess)
    e = smem_attr_once(reinterpret_cast<const void*>(k_cross_dkv32<D>), bk, ak);
  if (e != cudaSuccess) return e;
  k_cross_delta32<D><<<(unsigned)((p.bh * p.np + 31) / 32), 256, 0, p.s>>>(P);
  k_cross_dq32<D><<<dim3((unsigned)((p.np + xs::kT - 1) / xs::kT), (unsigned)p.bh, P.nstate),
                    xs::kThreads, bq, p.s>>>(P);
  if (P.nstate > 1) {
    const int64_t n = p.bh * p.np * D;
    k_cross_sum32<<<dim3((unsigned)((n / 4 + 255) / 256), 1), 256, 0, p.s>>>(
        P.part, P.nstate, n, P.out, nullptr, nullptr);
    count_launch();
  }
  const int64_t halves = (p.l + xs::kT - 1) / xs::kT;
  k_cross_dkv32<D><<<dim3((unsigned)(halves * P.nsplit), (unsigned)p.bh), xs::kThreads, bk, p.s>>>(P);
  count_launch(3);
  if (P.nsplit > 1) {
    const int64_t n = p.bh * p.l * D;
    k_cross_sum32<<<dim3((unsigned)((n / 4 + 255) / 256), 2), 256, 0, p.s>>>(P.dk, P.nsplit, n, dk,
                                                                           P.dv, dv);
    count_launch();
  }
  return cudaGetLastError();
}

cudaError_t bwd_simt(const Problem& p, const MaskTables& m, const void* o, const float* lse,
                     const void* dO, void* dq, void* dk, void* dv, void* ws) {
  xs::Params P = simt_params(p, m);
  P.o = static_cast<const float*>(o);
  P.dO = static_cast<const float*>(dO);
  P.lse = lse;
  P.out = static_cast<float*>(dq);
  uint8_t* at = static_cast<uint8_t*>(ws);
  P.delta = reinterpret_cast<float*>(at);
  at += align256((size_t)p.bh * p.np * sizeof(float));
  P.part = reinterpret_cast<float*>(at);
  at += part_bytes(p, P.nstate);
  P.nsplit = row_ranges(p);
  P.dk = static_cast<float*>(dk);
  P.dv = static_cast<float*>(dv);
  if (P.nsplit > 1) {
    const size_t e = (size_t)P.nsplit * p.bh * p.l * p.d * sizeof(float);
    P.dk = reinterpret_cast<float*>(at);
    P.dv = reinterpret_cast<float*>(at + align256(e));
  }
  float *k = static_cast<float*>(dk), *v = static_cast<float*>(dv);
  switch (p.d) {
    case 48: return launch_bwd32<48>(p, P, k, v);
    case 64: return launch_bwd32<64>(p, P, k, v);
    case 96: return launch_bwd32<96>(p, P, k, v);
    default: return launch_bwd32<128>(p, P, k, v);
  }
}

}  // namespace xa
}  // namespace p3d
