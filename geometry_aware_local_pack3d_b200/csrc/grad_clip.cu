// Global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum over tensors and elements of g^2),   out = g min(1, max_norm / (norm + 1e-6)).
//
// What bounds it: HBM. The norm reads every gradient once; the scaling reads it again and writes
// it. Each launch covers up to kPerLaunch tensors, whose addresses and lengths travel in the
// kernel's parameters (nothing to upload, and a captured graph keeps them). The tensors are cut
// into chunks of kChunkBytes at 16-byte boundaries; a block takes a contiguous range of chunks.
// The scaling walks every range backwards, so that it starts with the lines the norm left in L2,
// and does nothing at all when the result would be the input in place.
// Measured, 300 tensors of 150 million numbers, half of them bf16: norm 72 us (6.0 TB/s), scaling 150
// us (5.5 TB/s), 237 us in all; 12 tensors of 1.2 million 14 us, the launches.
// Sums: the squares of one thread's 16-byte pieces in fp32, a chunk's in double (where a chunk's
// fp32 sum is out of the range that fp32 squares keep exact, the squares are taken again in
// double), the blocks' words in double in block order: no atomics, the same result every run.
#include <math.h>

#include <algorithm>
#include <vector>

#include "common.cuh"
#include "launch.h"
#include "vec.cuh"

namespace p3d {
namespace gc {

constexpr int kPerLaunch = 512;
constexpr int kThreads = 256;
constexpr int kPieces = 4;                                // 16-byte pieces per thread and chunk
constexpr int kChunkBytes = kThreads * kPieces * 16;
constexpr int kBlocksPerSm = 4;
constexpr int kMaxBlocks = 1024;                          // words of the workspace per launch

struct Tensor {
  const uint8_t* g;
  uint8_t* o;        // out; null: norm only
  int64_t n;         // elements
  int32_t chunk0;    // first chunk of this tensor within the launch
  int32_t dtype;
};
// (a short list travels in a short block of parameters: copying one takes longer than a small norm)
constexpr int kShort = 48;
template <int N> struct Launch {
  int32_t count, chunks, per_block;  // tensors, chunks, chunks per block
  int32_t words;                     // scaling: words of the norm's sum (every launch's blocks)
  Tensor t[N];
};

// The tensor that holds chunk c (the last one whose first chunk is not after c).
template <int N> __device__ __forceinline__ int find(const Launch<N>& L, int c) {
  int lo = 0, hi = L.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (L.t[mid].chunk0 <= c) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ void unpack(const uint4 v, int dtype, float (&x)[8]) {
  if (dtype == PACK3D_BF16) {
    Vec<__nv_bfloat16>::unpack(v, x);
  } else {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
    x[4] = x[5] = x[6] = x[7] = 0.f;
  }
}

// Piece `p` of a tensor: its 16 bytes counted from the tensor's address rounded down to 16. Pieces
// that stick out of the tensor are read element by element (the rest reads as zero).
struct View {
  const uint8_t* base;   // address rounded down
  int64_t lo, hi;        // the tensor's bytes within it
  __device__ __forceinline__ View(const uint8_t* g, int64_t bytes) {
    const int head = (int)(reinterpret_cast<uintptr_t>(g) & 15);
    base = g - head;
    lo = head;
    hi = head + bytes;
  }
  __device__ __forceinline__ bool whole(int64_t at) const { return at >= lo && at + 16 <= hi; }
  __device__ __forceinline__ bool none(int64_t at) const { return at + 16 <= lo || at >= hi; }
  __device__ uint4 edge(int64_t at, int es) const {
    alignas(16) uint8_t b[16] = {};
    for (int i = 0; i < 16; i += es)
      if (at + i >= lo && at + i < hi)
        for (int j = 0; j < es; ++j) b[i + j] = base[at + i + j];
    return *reinterpret_cast<const uint4*>(b);
  }
  __device__ __forceinline__ uint4 load(int64_t at, int es) const {
    if (whole(at)) return *reinterpret_cast<const uint4*>(base + at);
    if (none(at)) return make_uint4(0u, 0u, 0u, 0u);
    return edge(at, es);
  }
};

__device__ __forceinline__ double block_sum(double s, double* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  double r = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) r += red[w];
  return r;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    k_grad_sq(const __grid_constant__ Launch<N> L, double* __restrict__ words) {
  __shared__ double red[kThreads / 32];
  const int c0 = blockIdx.x * L.per_block, c1 = min(L.chunks, c0 + L.per_block);
  double total = 0.0;
  int ti = c0 < c1 ? find(L, c0) : 0;
  for (int c = c0; c < c1; ++c) {
    while (ti + 1 < L.count && L.t[ti + 1].chunk0 <= c) ++ti;
    const int dt = L.t[ti].dtype, es = dt == PACK3D_BF16 ? 2 : 4;
    const View v(L.t[ti].g, L.t[ti].n * es);
    const int64_t at = (int64_t)(c - L.t[ti].chunk0) * kChunkBytes + threadIdx.x * 16;
    uint4 p[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) p[i] = v.load(at + i * (kThreads * 16), es);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float x[8];
      unpack(p[i], dt, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
    }
    // below 1e-25 a square may have lost bits or vanished, above 1e37 it may have overflowed
    if (s > 1e-25f && s < 1e37f) {
      total += (double)s;
    } else {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        float x[8];
        unpack(p[i], dt, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) total = fma((double)x[e], (double)x[e], total);
      }
    }
  }
  const double r = block_sum(total, red);
  if (threadIdx.x == 0) words[blockIdx.x] = r;
}

// The words' sum, the same in every block: thread t adds words t, t + 256, ..., then the block.
__device__ __forceinline__ float norm_of(const double* words, int n, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) s += words[i];
  return (float)sqrt(block_sum(s, red));
}

__global__ void __launch_bounds__(kThreads)
    k_grad_norm(const double* __restrict__ words, int n, float* __restrict__ norm) {
  __shared__ double red[kThreads / 32];
  const float r = norm_of(words, n, red);
  if (threadIdx.x == 0) *norm = r;
}

__device__ __forceinline__ void scale_piece(uint4 v, int dt, float coef, uint4* out) {
  float x[8];
  unpack(v, dt, x);
  if (dt == PACK3D_BF16) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] *= coef;
    Vec<__nv_bfloat16>::store(reinterpret_cast<__nv_bfloat16*>(out), x);
  } else {
    *out = make_uint4(__float_as_uint(x[0] * coef), __float_as_uint(x[1] * coef),
                      __float_as_uint(x[2] * coef), __float_as_uint(x[3] * coef));
  }
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    k_grad_scale(const __grid_constant__ Launch<N> L, const double* __restrict__ words,
                 float max_norm, float* __restrict__ norm) {
  __shared__ double red[kThreads / 32];
  const float nrm = norm_of(words, L.words, red);
  if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = nrm;
  float coef = max_norm / (nrm + 1e-6f);
  coef = coef > 1.f ? 1.f : coef;  // a norm that is no number gives a coefficient that is none
  const int c0 = blockIdx.x * L.per_block, c1 = min(L.chunks, c0 + L.per_block);
  int ti = c0 < c1 ? find(L, c1 - 1) : 0;
  for (int c = c1 - 1; c >= c0; --c) {
    while (L.t[ti].chunk0 > c) --ti;
    if (coef == 1.f && L.t[ti].o == L.t[ti].g) continue;
    const int dt = L.t[ti].dtype, es = dt == PACK3D_BF16 ? 2 : 4;
    const View v(L.t[ti].g, L.t[ti].n * es);
    uint8_t* const out = L.t[ti].o - v.lo;  // where byte 0 of the view would go
    const bool vec = (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    const int64_t at = (int64_t)(c - L.t[ti].chunk0) * kChunkBytes + threadIdx.x * 16;
    uint4 p[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) p[i] = v.load(at + i * (kThreads * 16), es);
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int64_t a = at + i * (kThreads * 16);
      if (v.none(a)) continue;
      if (vec && v.whole(a)) {
        scale_piece(p[i], dt, coef, reinterpret_cast<uint4*>(out + a));
      } else {
        alignas(16) uint8_t b[16];
        scale_piece(p[i], dt, coef, reinterpret_cast<uint4*>(b));
        for (int k = 0; k < 16; k += es)
          if (a + k >= v.lo && a + k < v.hi) {
            if (es == 2)
              *reinterpret_cast<uint16_t*>(out + a + k) = *reinterpret_cast<uint16_t*>(b + k);
            else
              *reinterpret_cast<uint32_t*>(out + a + k) = *reinterpret_cast<uint32_t*>(b + k);
          }
      }
    }
  }
}

struct Span {
  uintptr_t a, b;  // bytes [a, b)
};

int elem(int dtype) { return dtype == PACK3D_BF16 ? 2 : 4; }

pack3d_status check(const void* const* grads, const int64_t* counts, const int* dtypes, int n) {
  if (n < 0) return PACK3D_ERR_INVALID_ARG;
  if (n > 0 && (!grads || !counts || !dtypes)) return PACK3D_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i) {
    if (dtypes[i] != PACK3D_F32 && dtypes[i] != PACK3D_BF16) return PACK3D_ERR_INVALID_ARG;
    if (counts[i] < 0) return PACK3D_ERR_INVALID_ARG;
    // chunk numbers of a launch are 32-bit
    if (counts[i] > (int64_t)1 << 38) return PACK3D_ERR_UNSUPPORTED;
    if (counts[i] == 0) continue;
    if (!grads[i]) return PACK3D_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(grads[i]) % elem(dtypes[i])) return PACK3D_ERR_ALIGN;
  }
  return PACK3D_OK;
}

// Results may be written where their own gradient is read, and nowhere else where anything is
// read or written: blocks run in any order.
bool overlapping(const void* const* grads, void* const* outs, const int64_t* counts,
                 const int* dtypes, int n) {
  std::vector<Span> o, g;
  o.reserve(n);
  for (int i = 0; i < n; ++i) {
    if (!counts[i]) continue;
    const uintptr_t bytes = (uintptr_t)counts[i] * elem(dtypes[i]);
    const uintptr_t a = reinterpret_cast<uintptr_t>(outs[i]), b = reinterpret_cast<uintptr_t>(grads[i]);
    o.push_back({a, a + bytes});
    if (a != b) g.push_back({b, b + bytes});
  }
  auto less = [](const Span& x, const Span& y) { return x.a < y.a; };
  if (!std::is_sorted(o.begin(), o.end(), less)) std::sort(o.begin(), o.end(), less);
  for (size_t i = 1; i < o.size(); ++i)
    if (o[i].a < o[i - 1].b) return true;
  for (const Span& s : g) {  // the outputs are disjoint and sorted: look at the neighbours of s
    auto it = std::upper_bound(o.begin(), o.end(), s, less);
    if (it != o.end() && it->a < s.b) return true;
    if (it != o.begin() && (it - 1)->b > s.a) return true;
  }
  return false;
}

// One launch's tensors [i0, i1): as many as fit.
template <int N>
int fill(Launch<N>* L, const void* const* grads, void* const* outs, const int64_t* counts,
         const int* dtypes, int n, int i0) {
  int i = i0;
  int64_t chunks = 0;
  L->count = 0;
  for (; i < n && L->count < N; ++i) {
    if (!counts[i]) continue;
    const int64_t head = reinterpret_cast<uintptr_t>(grads[i]) & 15;
    const int64_t c = (head + counts[i] * elem(dtypes[i]) + kChunkBytes - 1) / kChunkBytes;
    if (L->count && chunks + c > INT32_MAX) break;
    Tensor& t = L->t[L->count++];
    t.g = static_cast<const uint8_t*>(grads[i]);
    t.o = outs ? static_cast<uint8_t*>(outs[i]) : nullptr;
    t.n = counts[i];
    t.chunk0 = (int32_t)chunks;
    t.dtype = dtypes[i];
    chunks += c;
  }
  L->chunks = (int32_t)chunks;
  return i;
}

template <int N> int grid_of(Launch<N>* L) {
  int cap = kBlocksPerSm * sm_count();
  if (cap > kMaxBlocks) cap = kMaxBlocks;
  const int blocks = L->chunks < cap ? L->chunks : cap;
  if (!blocks) return 0;
  L->per_block = (L->chunks + blocks - 1) / blocks;
  return (L->chunks + L->per_block - 1) / L->per_block;
}

size_t workspace_bytes(int n) {
  const size_t launches = ((size_t)n + kPerLaunch - 1) / kPerLaunch;
  return (launches ? launches : 1) * kMaxBlocks * sizeof(double);
}

// The sum of squares: returns the words written.
template <int N>
int sum_squares(const void* const* grads, const int64_t* counts, const int* dtypes, int n,
                double* words, cudaStream_t s) {
  Launch<N> L;
  int used = 0;
  for (int i = 0; i < n;) {
    i = fill(&L, grads, nullptr, counts, dtypes, n, i);
    const int grid = grid_of(&L);
    if (!grid) continue;
    L.words = 0;
    k_grad_sq<N><<<grid, kThreads, 0, s>>>(L, words + used);
    count_launch();
    used += grid;
  }
  return used;
}

// The scaling; the norm is written by the first launch, or by none if every tensor is empty.
template <int N>
bool scale(const void* const* grads, void* const* outs, const int64_t* counts, const int* dtypes,
           int n, float max_norm, float* norm, const double* words, int used, cudaStream_t s) {
  Launch<N> L;
  bool told = false;
  for (int i = 0; i < n;) {
    i = fill(&L, grads, outs, counts, dtypes, n, i);
    const int grid = grid_of(&L);
    if (!grid) continue;
    L.words = used;
    k_grad_scale<N><<<grid, kThreads, 0, s>>>(L, words, max_norm, told ? nullptr : norm);
    told = true;
    count_launch();
  }
  return told;
}

int sum_squares_of(const void* const* grads, const int64_t* counts, const int* dtypes, int n,
                   double* words, cudaStream_t s) {
  return n <= kShort ? sum_squares<kShort>(grads, counts, dtypes, n, words, s)
                     : sum_squares<kPerLaunch>(grads, counts, dtypes, n, words, s);
}

pack3d_status check_workspace(void* workspace, size_t bytes, int n) {
  if (!workspace) return PACK3D_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(workspace) & 15) return PACK3D_ERR_ALIGN;
  return bytes < workspace_bytes(n) ? PACK3D_ERR_WORKSPACE : PACK3D_OK;
}

}  // namespace gc
}  // namespace p3d

using namespace p3d;

extern "C" size_t pack3d_grad_norm_workspace_bytes(int n_tensors) {
  return n_tensors < 0 ? 0 : gc::workspace_bytes(n_tensors);
}

extern "C" pack3d_status pack3d_grad_norm(const void* const* grads, const int64_t* counts,
                                          const int* dtypes, int n_tensors, float* norm,
                                          void* workspace, size_t workspace_bytes, void* stream) {
  reset_launches();
  pack3d_status st = gc::check(grads, counts, dtypes, n_tensors);
  if (st != PACK3D_OK) return st;
  if (!norm) return PACK3D_ERR_INVALID_ARG;
  if ((st = gc::check_workspace(workspace, workspace_bytes, n_tensors)) != PACK3D_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* words = static_cast<double*>(workspace);
  const int used = gc::sum_squares_of(grads, counts, dtypes, n_tensors, words, s);
  gc::k_grad_norm<<<1, gc::kThreads, 0, s>>>(words, used, norm);
  count_launch();
  return cudaGetLastError() == cudaSuccess ? PACK3D_OK : PACK3D_ERR_CUDA;
}

extern "C" pack3d_status pack3d_clip_grad_norm(const void* const* grads, void* const* outs,
                                               const int64_t* counts, const int* dtypes,
                                               int n_tensors, float max_norm, float* norm,
                                               void* workspace, size_t workspace_bytes,
                                               void* stream) try {
  reset_launches();
  pack3d_status st = gc::check(grads, counts, dtypes, n_tensors);
  if (st != PACK3D_OK) return st;
  if (!norm || (n_tensors > 0 && !outs) || !(max_norm >= 0.f)) return PACK3D_ERR_INVALID_ARG;
  for (int i = 0; i < n_tensors; ++i) {
    if (!counts[i]) continue;
    if (!outs[i]) return PACK3D_ERR_INVALID_ARG;
    if (reinterpret_cast<uintptr_t>(outs[i]) % gc::elem(dtypes[i])) return PACK3D_ERR_ALIGN;
  }
  if ((st = gc::check_workspace(workspace, workspace_bytes, n_tensors)) != PACK3D_OK) return st;
  if (gc::overlapping(grads, outs, counts, dtypes, n_tensors)) return PACK3D_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* words = static_cast<double*>(workspace);
  const int used = gc::sum_squares_of(grads, counts, dtypes, n_tensors, words, s);
  const bool told =
      n_tensors <= gc::kShort
          ? gc::scale<gc::kShort>(grads, outs, counts, dtypes, n_tensors, max_norm, norm, words, used, s)
          : gc::scale<gc::kPerLaunch>(grads, outs, counts, dtypes, n_tensors, max_norm, norm, words,
                                      used, s);
  if (!told) {  // nothing but empty tensors: the norm is zero
    gc::k_grad_norm<<<1, gc::kThreads, 0, s>>>(words, used, norm);
    count_launch();
  }
  return cudaGetLastError() == cudaSuccess ? PACK3D_OK : PACK3D_ERR_CUDA;
} catch (...) {  // the host's memory ran out
  return PACK3D_ERR_INVALID_ARG;
}
