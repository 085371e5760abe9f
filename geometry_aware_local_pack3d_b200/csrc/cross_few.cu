// Cross attention of few rows (N' = G N <= 16: single tokens) to long contexts, bf16.
//
// Every state is read once and meets at most 16 rows: 16 FLOP a byte, far below the tensor cores'
// ratio, so K and V at the memory's rate are all that counts. The tile of tcgen05 has 128 rows and a
// round trip through tensor memory per step of states, a chain of ~1,500 cycles for 64 states that
// one CTA per SM cannot hide (8 sequences of one token, 2 KV heads of 4 heads, d = 96, 16,384 padded
// states: 45 us with that kernel, its mask tables and its join). Here a warp owns its states: 32 at a
// time by asynchronous copies into its own two buffers (the next 12 KB in flight while it works, no
// barrier with another warp), m16n8k16 products on registers, the softmax's maximum and sum in
// registers (fp32). Masked states are not read at all: their copies fill zeros, chunks without a
// state are left out, and the mask's bytes become words in the warp itself: 25.5 us for the case above
// with the join (75 MB in all, 2.9 TB/s).
//
// Chunks go to the warps of a problem in turn, so that a padded batch entry keeps all of them busy.
// The block's warps join through shared memory, the blocks of a problem through k_cross_join.
#include "cross.h"
#include "launch.h"
#include "tc.cuh"

namespace p3d {
namespace xa {

namespace fw {
constexpr int kRows = 16, kChunk = 32;
template <int D> struct Cfg {
  // two blocks per SM: 8 warps, or 6 at d = 128
  static constexpr int kWarps = D == 128 ? 3 : 4;
  static constexpr int kPitch = 2 * D + 16;  // bytes: eight rows' pieces lie in distinct banks
  static constexpr int kTileB = kChunk * kPitch, kStage = 2 * kTileB;
  static constexpr int kBytes = kWarps * 2 * kStage;
  static_assert(kWarps * kRows * (D + 2) * 4 <= kBytes, "the join's partial rows");
};
struct Params {
  const __nv_bfloat16 *q, *k, *v;
  const uint8_t* mask;
  __nv_bfloat16* o;
  float *lse, *part_o, *part_lse;
  int64_t l, rows;  // states; rows of all problems
  int np, kv_heads, nsplit;
  float scale_log2;
};
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
template <int N> __device__ __forceinline__ void copies_but() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
template <bool T> __device__ __forceinline__ void ldm4(uint32_t (&r)[4], uint32_t addr) {
  if (T)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                    uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
}  // namespace fw

// Block (split, problem). Thread `lane` of a warp holds, of a 16 x 8 tile of S or O, rows lane / 4
// and lane / 4 + 8, columns 2 (lane mod 4) and the next.
template <int D>
__global__ void __launch_bounds__(32 * fw::Cfg<D>::kWarps, 2) k_cross_few(const fw::Params P) {
  using namespace fw;
  using C = Cfg<D>;
  constexpr int KS = D / 16, NT = D / 8;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r0 = lane >> 2, c0 = 2 * (lane & 3);
  const int split = blockIdx.x;
  const int64_t bh = blockIdx.y;
  const __nv_bfloat16 *k = P.k + bh * P.l * D, *v = P.v + bh * P.l * D;
  const uint8_t* mask = P.mask ? P.mask + bh / P.kv_heads * P.l : nullptr;
  const uint32_t buf = tc::smem_u32(smem) + warp * 2 * C::kStage;
  // the join may be launched; it waits for this kernel's end
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  uint32_t qa[KS][4];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = r0 + 8 * (i & 1), c = 16 * ks + c0 + 8 * (i >> 1);
      qa[ks][i] = r < P.np ? *reinterpret_cast<const uint32_t*>(P.q + (bh * P.np + r) * D + c) : 0u;
    }
  float o[NT][4], top[2] = {-INFINITY, -INFINITY}, sum[2] = {0.f, 0.f};
#pragma unroll
  for (int t = 0; t < NT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.f;

  const int64_t chunks = (P.l + kChunk - 1) / kChunk, step = (int64_t)P.nsplit * C::kWarps;
  // 32 of the warp's chunks a round: lane i keeps the word of the i-th
  for (int64_t first = split * C::kWarps + warp; first < chunks; first += 32 * step) {
    uint32_t word = 0u;
#pragma unroll 8
    for (int i = 0; i < 32; ++i) {
      const int64_t at = (first + i * step) * kChunk + lane;
      const bool on = at < P.l && (!mask || mask[at] != 0);
      const uint32_t w = __ballot_sync(0xffffffffu, on);
      if (lane == i) word = w;
    }
    uint32_t todo = __ballot_sync(0xffffffffu, word != 0u);
    // the lowest listed chunk: its copies into stage `st`, one group (empty once none is left)
    auto load = [&](int st) {
      if (todo) {
        const int i = __ffs(todo) - 1;
        todo &= todo - 1;
        const uint32_t w = __shfl_sync(0xffffffffu, word, i);
        const int64_t at = (first + i * step) * kChunk;
        const uint32_t dst = buf + st * C::kStage;
#pragma unroll
        for (int x = 0; x < D / 8; ++x) {
          const int f = 32 * x + lane, s = f / (D / 8), pc = f % (D / 8);
          const bool on = (w >> s) & 1u;
          const int64_t src = on ? (at + s) * D + pc * 8 : 0;
          copy16(dst + s * C::kPitch + pc * 16, k + src, on);
          copy16(dst + C::kTileB + s * C::kPitch + pc * 16, v + src, on);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint32_t left = todo;
    load(0);
    for (int st = 0; left; left &= left - 1, st ^= 1) {
      load(st ^ 1);
      copies_but<1>();
      __syncwarp();
      const uint32_t w = __shfl_sync(0xffffffffu, word, __ffs(left) - 1);
      const uint32_t kt = buf + st * C::kStage, vt = kt + C::kTileB;
      float s[4][4];
#pragma unroll
      for (int t = 0; t < 4; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h) {  // 16 states
          uint32_t b[4];
          ldm4<false>(b, kt + (16 * h + 8 * (lane >> 4) + (lane & 7)) * C::kPitch +
                             (16 * ks + 8 * ((lane >> 3) & 1)) * 2);
          mma(s[2 * h], qa[ks], b[0], b[1]);
          mma(s[2 * h + 1], qa[ks], b[2], b[3]);
        }
      // scores in base 2, masked states at -inf; the running maximum of the two rows
      float m[2] = {top[0], top[1]};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][i] = (w >> (8 * t + c0 + (i & 1))) & 1u ? s[t][i] * P.scale_log2 : -INFINITY;
          m[i >> 1] = fmaxf(m[i >> 1], s[t][i]);
        }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 1));
        m[r] = fmaxf(m[r], __shfl_xor_sync(0xffffffffu, m[r], 2));
      }
      if (__any_sync(0xffffffffu, m[0] > top[0] || m[1] > top[1])) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float f = m[r] > top[r] ? ex2(top[r] - m[r]) : 1.f;
          top[r] = m[r];
          sum[r] *= f;
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            o[t][2 * r] *= f;
            o[t][2 * r + 1] *= f;
          }
        }
      }
      const float base[2] = {top[0] == -INFINITY ? 0.f : top[0],
                             top[1] == -INFINITY ? 0.f : top[1]};
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s[t][i] = ex2(s[t][i] - base[i >> 1]);
          sum[i >> 1] += s[t][i];
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        // P in bf16, rounded as the products take it (relative 2^-8 a state, the sum unrounded)
        const uint32_t pa[4] = {tc::pack_bf16(s[2 * h][0], s[2 * h][1]),
                                tc::pack_bf16(s[2 * h][2], s[2 * h][3]),
                                tc::pack_bf16(s[2 * h + 1][0], s[2 * h + 1][1]),
                                tc::pack_bf16(s[2 * h + 1][2], s[2 * h + 1][3])};
#pragma unroll
        for (int t = 0; t < NT; t += 2) {
          uint32_t b[4];
          ldm4<true>(b, vt + (16 * h + 8 * ((lane >> 3) & 1) + (lane & 7)) * C::kPitch +
                            (8 * t + 8 * (lane >> 4)) * 2);
          mma(o[t], pa, b[0], b[1]);
          mma(o[t + 1], pa, b[2], b[3]);
        }
      }
      __syncwarp();  // the buffer may be filled again
    }
    copies_but<0>();
    __syncwarp();
  }

  // ---- the block's warps: (maximum, sum) and O of each in shared memory
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 1);
    sum[r] += __shfl_xor_sync(0xffffffffu, sum[r], 2);
  }
  __syncthreads();  // (over the warps' buffers)
  float* po = reinterpret_cast<float*>(smem);             // [warps][16][D]
  float* pm = po + C::kWarps * kRows * D;                 // [warps][16][2]
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int row = warp * kRows + r0 + 8 * r;
#pragma unroll
    for (int t = 0; t < NT; ++t)
      *reinterpret_cast<float2*>(po + row * D + 8 * t + c0) =
          make_float2(o[t][2 * r], o[t][2 * r + 1]);
    if ((lane & 3) == 0) *reinterpret_cast<float2*>(pm + 2 * row) = make_float2(top[r], sum[r]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < P.np * (D / 4); i += 32 * C::kWarps) {
    const int r = i / (D / 4), c = 4 * (i % (D / 4));
    float m = -INFINITY;
#pragma unroll
    for (int x = 0; x < C::kWarps; ++x) m = fmaxf(m, pm[2 * (x * kRows + r)]);
    const float base = m == -INFINITY ? 0.f : m;
    float l = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int x = 0; x < C::kWarps; ++x) {
      const float2 ms = *reinterpret_cast<const float2*>(pm + 2 * (x * kRows + r));
      const float4 y = *reinterpret_cast<const float4*>(po + (x * kRows + r) * D + c);
      const float f = ex2(ms.x - base);
      l = fmaf(f, ms.y, l);
      a.x = fmaf(f, y.x, a.x);
      a.y = fmaf(f, y.y, a.y);
      a.z = fmaf(f, y.z, a.z);
      a.w = fmaf(f, y.w, a.w);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    const float lse = l == 0.f ? -INFINITY : (base + log2f(l)) * kLn2;
    const int64_t row = bh * P.np + r;
    if (P.nsplit > 1) {
      *reinterpret_cast<float4*>(P.part_o + (split * P.rows + row) * D + c) = a;
      if (c == 0) P.part_lse[split * P.rows + row] = lse;
    } else {
      *reinterpret_cast<uint2*>(P.o + row * D + c) =
          make_uint2(tc::pack_bf16(a.x, a.y), tc::pack_bf16(a.z, a.w));
      if (c == 0 && P.lse) P.lse[row] = lse;
    }
  }
}

bool few_fwd(const Problem& p) {
  return p.dtype == PACK3D_BF16 && p.np <= fw::kRows && !short_fwd(p);
}

// Blocks per problem: two per SM in all, at least two chunks of 32 states for a warp.
static int few_splits(const Problem& p) {
  const int64_t chunks = (p.l + fw::kChunk - 1) / fw::kChunk, warps = p.d == 128 ? 3 : 4;
  const int64_t most = chunks / (2 * warps);
  int64_t n = 2 * (int64_t)sm_count() / p.bh;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)(n < kMaxSplits ? n : kMaxSplits);
}

size_t few_bytes(const Problem& p) {
  const int n = few_splits(p);
  if (n == 1) return 0;
  const size_t rows = (size_t)n * p.bh * p.np;
  return align256(rows * p.d * sizeof(float)) + align256(rows * sizeof(float));
}

template <int D>
static cudaError_t launch_few(const Problem& p, void* o, float* lse, void* ws) {
  using C = fw::Cfg<D>;
  static std::atomic<uint64_t> attr{0};
  const cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(k_cross_few<D>), C::kBytes, attr);
  if (e != cudaSuccess) return e;
  fw::Params P{};
  P.q = static_cast<const __nv_bfloat16*>(p.q);
  P.k = static_cast<const __nv_bfloat16*>(p.k);
  P.v = static_cast<const __nv_bfloat16*>(p.v);
  P.mask = p.mask;
  P.o = static_cast<__nv_bfloat16*>(o);
  P.lse = lse;
  P.l = p.l;
  P.rows = p.bh * p.np;
  P.np = (int)p.np;
  P.kv_heads = p.kv_heads;
  P.nsplit = few_splits(p);
  P.scale_log2 = p.scale * kLog2e;
  if (P.nsplit > 1) {
    P.part_o = static_cast<float*>(ws);
    P.part_lse = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) +
                                          align256((size_t)P.nsplit * P.rows * D * sizeof(float)));
  }
  k_cross_few<D><<<dim3(P.nsplit, (unsigned)p.bh), 32 * C::kWarps, C::kBytes, p.s>>>(P);
  count_launch();
  if (P.nsplit > 1) return join_splits(p, P.part_o, P.part_lse, P.nsplit, o, lse);
  return cudaGetLastError();
}

cudaError_t fwd_few(const Problem& p, void* o, float* lse, void* ws) {
  switch (p.d) {
    case 48: return launch_few<48>(p, o, lse, ws);
    case 64: return launch_few<64>(p, o, lse, ws);
    case 96: return launch_few<96>(p, o, lse, ws);
    default: return launch_few<128>(p, o, lse, ws);
  }
}

}  // namespace xa
}  // namespace p3d
