// Cross attention, backward, bf16 on tcgen05 tensor cores (head_dim 48, 64, 96 or 128).
//
//   p_ij = exp(tau <q_i, k_j> - lse_i),  D_i = <dO_i, o_i>,  dS_ij = p_ij (<dO_i, v_j> - D_i) tau,
//   dq_i = sum_j dS_ij k_j,   dk_j = sum_i dS_ij q_i,   dv_j = sum_i p_ij dO_i.
//
//   k_cross_dq    row-major: a CTA walks 128-row tiles; first D of the tile's rows (left for
//                 k_cross_dkv too); per 64 states S = q K^T and dP = dO V^T, dS in bf16, dq += dS K.
//                 Two CTAs per SM, so that one tile's products run under the other's elementwise
//                 pass and epilogue. Few row tiles: the states in ranges, a unit each, whose fp32
//                 sums k_cross_sum adds in order.
//   k_cross_dkv   state-major: a CTA owns 128 states of one problem and a range of rows; per 64 rows
//                 S^T = K q^T and dP^T = V dO^T (double-buffered in TMEM), P^T and dS^T in bf16 over
//                 them, dv += P^T dO and dk += dS^T q. Two groups of elementwise warps take turns.
//   k_cross_sum   the row ranges' partial dk, dv, added in range order (no atomics anywhere).
// What bounds them: the chain of a step (scores, elementwise pass, second products) through tensor
// memory, which two CTAs or two warp groups overlap only in part. Measured, 2 x 8 heads of 32,768 rows
// to 500 padded states of 96: dq 224 us with the tensor pipe 28 % busy and the exponential unit 26 %,
// dk and dv 189 us with 45 % and 30 %; backward 400 to 490 us from box to box, 390 to 480 TFLOP/s over
// its five products (seven are formed: S and dP in both kernels).
// A KV head's gradients sum over its query heads, which are rows of the same problem.
// P and dS are rounded to bf16 for the second products (relative 2^-8, as the outputs).
// Masked states: in k_cross_dq their dS is zero whatever S and dP hold, and their K rows (which may
// hold NaN) are zeroed in shared memory; in k_cross_dkv each state is an output row of its own, so
// the masked rows' sums are simply not written and zeros are.
#include <math.h>

#include "cross_tc.cuh"
#include "launch.h"

namespace p3d {
namespace xa {

namespace xb {
constexpr int kHalf = 64;  // states per step (dq), rows per step (dkv)

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 d;
  asm("{\n\t.reg .b64 ra, rb, rd;\n\t"
      "mov.b64 ra, {%2, %3};\n\tmov.b64 rb, {%4, %5};\n\t"
      "mul.rn.f32x2 rd, ra, rb;\n\tmov.b64 {%0, %1}, rd;\n\t}"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 f2(uint32_t a, uint32_t b) {
  return make_float2(__uint_as_float(a), __uint_as_float(b));
}

struct Params {
  float2* rows;  // [bh][npad] (-lse log2(e), D tau): written by k_cross_dq, read by k_cross_dkv
  const __nv_bfloat16* o;
  const float* lse;
  const int32_t* act;
  const uint32_t* bits;
  int32_t* status;
  long long budget;
  int64_t np, npad, l, bh, units, words;
  int rtiles, tiles, kv_heads, nsplit;
  int nstate;               // k_cross_dq: ranges of states
  float* part_q;            // [nstate][bh][np][D] where there are several
  float scale, scale_log2;
  __nv_bfloat16 *dk, *dv;   // written when nsplit is 1
  float *part_k, *part_v;   // [nsplit][bh][l][D] otherwise
};
}  // namespace xb

// -------------------------------------------------------------------------------------- dq
namespace xq {
constexpr int kThreads = 256;  // elementwise 0-3, TMA 4, S and dP 5, masked rows of K 6, dq 7
// Registers: two CTAs per SM leave 128 per thread at the launch; the elementwise warps, which hold
// 64 columns of S and of dP, take 176, the others keep 80: 128 (176 + 80) = 256 * 128.
constexpr int kRegs = 128, kMore = 176, kLess = 80;
static_assert(128 * (kMore + kLess) <= kThreads * kRegs, "registers of the launch");
template <int D> struct Smem {
  static constexpr int TB = Lay<D>::bytes(kTile), HB = Lay<D>::bytes(xb::kHalf);
  static constexpr int kQ = 0, kG = TB, kRing = 2 * TB;
  // V and K take turns (V first: its slot is free before K's, which the step's last product reads)
  static constexpr int kSlots = dq_slots(D);
  static_assert(kRing == dq_ring_at(D), "shared memory");
  static constexpr int kBar = kRing + kSlots * HB;
  static constexpr int kBytes = kBar + 512;
};
constexpr int kMaxSlots = 6, kReady = kDqReady;
enum {
  B_QFULL = 0, B_QEMPTY = 1, B_FULL = 2, B_EMPTY = B_FULL + kMaxSlots,
  B_READY = B_EMPTY + kMaxSlots, B_SFULL = B_READY + kReady, B_SFREE, B_PFULL, B_DONE, B_STAGED,
  B_DRAIN, B_COUNT
};
static_assert(8 * B_COUNT + 16 <= 512, "barrier area");
// TMEM columns of 256: S, dP, dS (bf16), dq. Where dS has columns of its own (d <= 96), the next
// step's S and dP are formed as soon as this step's have been read; at d = 128 dS lies over S and
// they wait for this step's last product.
template <int D> struct Cols {
  static constexpr bool kOwn = dq_own(D);
  static constexpr uint32_t kS = 0, kP = 64, kD = kOwn ? 128 : 0, kO = kOwn ? 160 : 128;
  static_assert(kO + D <= 256, "tensor memory");
};

// A unit's problem, first row and steps of 64 states (the batch entry's listed tiles, halved): its
// range z of them, from step j0 on. Range 0 is empty only if all are.
struct Unit {
  int64_t bh, row0;
  int n, z, j0;
  const int32_t* list;
  const uint32_t* bits;
  __device__ __forceinline__ Unit(const xb::Params& P, int64_t u) {
    z = j0 = 0;
    if (P.nstate > 1) {
      z = (int)(u % P.nstate);
      u /= P.nstate;
    }
    bh = u / P.rtiles;
    row0 = (u % P.rtiles) * kTile;
    const int64_t b = bh / P.kv_heads;
    list = nullptr;
    bits = nullptr;
    n = (int)((P.l + xb::kHalf - 1) / xb::kHalf);
    if (P.act) {
      list = P.act + b * (P.tiles + 1) + 1;
      bits = P.bits + b * P.words;
      n = 2 * list[-1];
    }
    if (P.nstate > 1) {
      j0 = (int)(((int64_t)n * z + P.nstate - 1) / P.nstate);
      n = (int)(((int64_t)n * (z + 1) + P.nstate - 1) / P.nstate) - j0;
    }
  }
  __device__ __forceinline__ int64_t at(int j) const {
    j += j0;
    return list ? (int64_t)list[j >> 1] * kTile + (j & 1) * xb::kHalf : (int64_t)j * xb::kHalf;
  }
  __device__ __forceinline__ void words(int64_t l, int j, uint32_t (&w)[2]) const {
    state_words(bits, l, at(j), w);
  }
};
}  // namespace xq

template <int D>
__global__ void __launch_bounds__(xq::kThreads, 2)
    k_cross_dq(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
               const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
               const __grid_constant__ CUtensorMap mo, const xb::Params P) {
  using namespace xq;
  using S = Smem<D>;
  using Ly = Lay<D>;
  using C = Cols<D>;
  constexpr int NS = S::kSlots;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kBar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kBar + 8 * B_COUNT + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Waiter ab(abort_flag, P.budget);
  const uint32_t sb = tc::smem_u32(bars);  // barrier i at sb + 8 i
  if (tid == 0) {
    tc::mbar_init(&bars[B_QFULL], 1);
    tc::mbar_init(&bars[B_QEMPTY], 1);
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&bars[B_FULL + i], 1);
      tc::mbar_init(&bars[B_EMPTY + i], 1);
    }
    for (int i = 0; i < kReady; ++i) tc::mbar_init(&bars[B_READY + i], 1);
    tc::mbar_init(&bars[B_SFULL], 1);
    tc::mbar_init(&bars[B_SFREE], 128);
    tc::mbar_init(&bars[B_PFULL], 128);
    tc::mbar_init(&bars[B_DONE], 1);
    tc::mbar_init(&bars[B_STAGED], 128);
    tc::mbar_init(&bars[B_DRAIN], 2);
    abort_flag[0] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 5) tc::tmem_alloc(tmem_slot, 256);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp < 4) {
    // ------------------------------------------------------------ elementwise and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMore));
    const int rin = warp * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
    uint32_t gc = 0, uc = 0, staged = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
      // the row's D = <dO, o> and lse, for this kernel and for k_cross_dkv; a row without any state,
      // and the padding, get P = 0
      float2 rd = make_float2(-INFINITY, 0.f);
      {
        const int64_t row = U.row0 + rin, at = U.bh * P.np + row;
        uint4 o[D / 8];
        const bool in = row < P.np && U.n;
        float le = -INFINITY, d = 0.f;
        if (in) {
          le = P.lse[at];
#pragma unroll
          for (int pc = 0; pc < D / 8; ++pc)
            o[pc] = *reinterpret_cast<const uint4*>(P.o + at * D + pc * 8);
        }
        if (U.n) ok = ab.all(sb + 8 * (B_QFULL), uc++);
        if (!ok) break;
        if (in) {
#pragma unroll
          for (int pc = 0; pc < D / 8; ++pc) {
            float a[8], b[8];
            Vec<__nv_bfloat16>::unpack(o[pc], a);
            Vec<__nv_bfloat16>::load_shared(
                reinterpret_cast<const __nv_bfloat16*>(smem + S::kG + Ly::piece(kTile, rin, pc)), b);
#pragma unroll
            for (int e = 0; e < 8; ++e) d = fmaf(a[e], b[e], d);
          }
          if (le != -INFINITY) rd = make_float2(-le * kLog2e, d * P.scale);
        }
        if (U.z == 0) P.rows[U.bh * P.npad + row] = rd;
      }
      const float2 nl2 = make_float2(rd.x, rd.x), nd2 = make_float2(-rd.y, -rd.y);
      const float2 sl2 = make_float2(P.scale_log2, P.scale_log2);
      const float2 sc2 = make_float2(P.scale, P.scale);
      uint32_t seen = 0;
#pragma unroll 1
      for (int j = 0; j < U.n; ++j, ++gc) {
        uint32_t w[2];
        U.words(P.l, j, w);
        ok = ab.all(seen, sb + 8 * (B_SFULL), gc);
        if (!ok) break;
        tc::tc_fence_after();
        const uint32_t done = ab.probe(sb + 8 * (B_DONE), gc - 1);
        uint32_t sv[2][32], dv[2][32];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          tc::tmem_ld32(tl + C::kS + 32 * h, sv[h]);
          tc::tmem_ld32(tl + C::kP + 32 * h, dv[h]);
        }
        tc::tmem_wait_ld();
        if (C::kOwn) {
          tc::tc_fence_before();
          arrive32(sb + 8 * (B_SFREE));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int k = 0; k < 32; k += 2) {
            const float2 x = tc::fma2(xb::f2(sv[h][k], sv[h][k + 1]), sl2, nl2);
            const float2 t = tc::fma2(xb::f2(dv[h][k], dv[h][k + 1]), sc2, nd2);
            float2 ds = xb::mul2(make_float2(ex2(x.x), ex2(x.y)), t);
            if (w[h] != 0xffffffffu) {
              ds.x = ((w[h] >> k) & 1u) ? ds.x : 0.f;
              ds.y = ((w[h] >> (k + 1)) & 1u) ? ds.y : 0.f;
            }
            pk[k >> 1] = tc::pack_bf16(ds.x, ds.y);
          }
          if (C::kOwn && h == 0 && gc) {
            // dS is the previous step's until its product has completed
            ok = ab.all(done, sb + 8 * (B_DONE), gc - 1);
            if (!ok) break;
            tc::tc_fence_after();
          }
          tc::tmem_st16(tl + C::kD + 16 * h, pk);
        }
        if (!ok) break;
        if (C::kOwn) seen = ab.probe(sb + 8 * (B_SFULL), gc + 1);
        tc::tmem_wait_st();
        tc::tc_fence_before();
        arrive32(sb + 8 * (B_PFULL));
      }
      if (!ok) break;
      if (U.n && !ab.all(sb + 8 * (B_DONE), (gc - 1) & 1)) break;
      if (!U.n) {
        // no state: zero rows
        if (U.row0 + rin < P.np && P.nstate > 1) {
          float* dst = P.part_q + ((U.z * P.bh + U.bh) * P.np + U.row0 + rin) * D;
#pragma unroll
          for (int e = 0; e < D; e += 4)
            *reinterpret_cast<float4*>(dst + e) = make_float4(0.f, 0.f, 0.f, 0.f);
        } else if (U.row0 + rin < P.np) {
          __nv_bfloat16* dst = P.dk + (U.bh * P.np + U.row0 + rin) * D;
#pragma unroll
          for (int e = 0; e < D; e += 8)
            *reinterpret_cast<uint4*>(dst + e) = make_uint4(0u, 0u, 0u, 0u);
        }
        continue;
      }
      tc::tc_fence_after();
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tc::tmem_ld16(tl + C::kO + c, o);
        tc::tmem_wait_ld();
        if (P.nstate > 1) {
          if (U.row0 + rin < P.np) {
            float* dst = P.part_q + ((U.z * P.bh + U.bh) * P.np + U.row0 + rin) * D + c;
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<uint4*>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
          }
          continue;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pk[i] = tc::pack_bf16(__uint_as_float(o[8 * h + 2 * i]),
                                  __uint_as_float(o[8 * h + 2 * i + 1]));
          // the q tile has been consumed: its buffer takes the gradient's rows
          *reinterpret_cast<uint4*>(smem + S::kQ + Ly::piece(kTile, rin, c / 8 + h)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      tc::tc_fence_before();
      tc::fence_proxy_async_smem();
      arrive32(sb + 8 * (B_STAGED));
      if (rin == 0) {
        if (!ab.wait(sb + 8 * (B_STAGED), staged++ & 1)) ok = false;
#pragma unroll
        for (int c = 0; c < Ly::NB && ok && P.nstate == 1; ++c)
          tma_store_3d(&mo, smem + S::kQ + c * kTile * Ly::RB, c * Ly::CW, (int)U.row0, (int)U.bh);
        bulk_commit();
        bulk_wait_read();
        arrive32(sb + 8 * (B_QEMPTY));
      }
      ok = __all_sync(0xffffffffu, ok);  // a warp leaves the loop as one
    }
    if (rin == 0) bulk_wait();
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLess));
  if (warp == 4) {
    // ------------------------------------------------------------ TMA loads
    if (lane == 0) {
      uint32_t kv = 0, uc = 0;
      bool ok = true;
      for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
        const Unit U(P, u);
        if (!U.n) continue;
        if (uc && !ab.wait(sb + 8 * (B_QEMPTY), (uc - 1) & 1)) break;
        tc::mbar_expect_tx(&bars[B_QFULL], 2 * S::TB);
        load_rows<D>(smem + S::kQ, &mq, kTile, U.row0, (int)U.bh, &bars[B_QFULL]);
        load_rows<D>(smem + S::kG, &mg, kTile, U.row0, (int)U.bh, &bars[B_QFULL]);
        ++uc;
        for (int j = 0; j < U.n && ok; ++j) {
          const int64_t at = U.at(j);
          for (int x = 0; x < 2; ++x, ++kv) {
            const int st = kv % NS;
            if (kv >= (uint32_t)NS && !ab.wait(sb + 8 * (B_EMPTY + st), ((kv / NS) - 1) & 1)) {
              ok = false;
              break;
            }
            tc::mbar_expect_tx(&bars[B_FULL + st], S::HB);
            load_rows<D>(smem + S::kRing + st * S::HB, x ? &mk : &mv, xb::kHalf, at, (int)U.bh,
                         &bars[B_FULL + st]);
          }
        }
      }
      for (uint32_t k = kv > (uint32_t)NS ? kv - NS : 0; k < kv; ++k)
        tc::mbar_wait(&bars[B_FULL + (k % NS)], (k / NS) & 1);
      if (uc) tc::mbar_wait(&bars[B_QFULL], (uc - 1) & 1);
    }
  } else if (warp == 5) {
    // ------------------------------------------------------------ S and dP
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t id_s = tc::idesc_bf16_f32(128, xb::kHalf, false, false);
    const uint64_t qd = Ly::kdesc(tc::smem_u32(smem + S::kQ));
    const uint64_t gd = Ly::kdesc(tc::smem_u32(smem + S::kG));
    const uint64_t kd0 = Ly::kdesc(tc::smem_u32(smem + S::kRing));
    const bool masked = P.act != nullptr;
    uint32_t g = 0, uc = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
      if (!U.n) continue;
      if (!ab.all(sb + 8 * (B_QFULL), uc & 1)) break;
      ++uc;
#pragma unroll 1
      for (int j = 0; j < U.n; ++j, ++g) {
        const int sv = 2 * g % NS, sk = (2 * g + 1) % NS;
        ok = masked ? ab.all(sb + 8 * (B_READY + g % kReady), g / kReady)
                    : ab.all(sb + 8 * (B_FULL + sk), (2 * g + 1) / NS);
        ok = ok && ab.all(sb + 8 * (B_FULL + sv), 2 * g / NS);
        // the last step's S and dP have been read (with dS over S: its product has completed)
        if (g >= 1) ok = ok && ab.all(sb + 8 * (C::kOwn ? B_SFREE : B_DONE), g - 1);
        if (!ok) break;
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint64_t ko = (uint64_t)((sk * S::HB) >> 4), vo = (uint64_t)((sv * S::HB) >> 4);
#pragma unroll
          for (int ks = 0; ks < Ly::kSteps; ++ks) {
            tc::mma_ss(tb + C::kS, qd + Ly::koff(kTile, ks), kd0 + ko + Ly::koff(xb::kHalf, ks),
                       id_s, ks > 0);
            tc::mma_ss(tb + C::kP, gd + Ly::koff(kTile, ks), kd0 + vo + Ly::koff(xb::kHalf, ks),
                       id_s, ks > 0);
          }
          commit32(sb + 8 * (B_SFULL));
          commit32(sb + 8 * (B_EMPTY + sv));
        }
        __syncwarp();
      }
    }
    if (tc::elect_one()) commit32(sb + 8 * (B_DRAIN));
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) *abort_flag = 1;
  } else if (warp == 7) {
    // ------------------------------------------------------------ dq += dS K
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t id_o = tc::idesc_bf16_f32(128, D, false, true);
    const uint64_t km0 = Ly::mdesc(tc::smem_u32(smem + S::kRing), xb::kHalf);
    uint32_t g = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
#pragma unroll 1
      for (int j = 0; j < U.n; ++j, ++g) {
        const int sk = (2 * g + 1) % NS;
        ok = ab.all(sb + 8 * (B_PFULL), g);
        if (!ok) break;
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint64_t ko = (uint64_t)((sk * S::HB) >> 4);
#pragma unroll
          for (int ks = 0; ks < xb::kHalf / 16; ++ks)
            tc::mma_ts(tb + C::kO, tb + C::kD + ks * 8, km0 + ko + Ly::moff(ks), id_o,
                       (j > 0 || ks > 0) ? 1u : 0u);
          commit32(sb + 8 * (B_DONE));
          commit32(sb + 8 * (B_EMPTY + sk));
        }
        __syncwarp();
      }
    }
    if (tc::elect_one()) commit32(sb + 8 * (B_DRAIN));
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) *abort_flag = 1;
  } else if (warp == 6 && P.act) {
    // ------------------------------------------------------------ masked rows of K
    uint32_t g = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
      for (int j = 0; j < U.n; ++j, ++g) {
        uint32_t w[2];
        U.words(P.l, j, w);
        const uint32_t kv = 2 * g + 1;
        const int st = kv % NS;
        // V first: a slot holds V and K in turn, and every phase of its barrier has to be followed
        ok = ab.all(sb + 8 * (B_FULL + (kv - 1) % NS), (kv - 1) / NS) &&
             ab.all(sb + 8 * (B_FULL + st), kv / NS);
        if (!ok) break;
        if ((w[0] & w[1]) != 0xffffffffu) {
          uint8_t* kt = smem + S::kRing + st * S::HB;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            if (!((w[i] >> lane) & 1u))
#pragma unroll
              for (int pc = 0; pc < D / 8; ++pc)
                *reinterpret_cast<uint4*>(kt + Ly::piece(xb::kHalf, 32 * i + lane, pc)) =
                    make_uint4(0u, 0u, 0u, 0u);
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) arrive32(sb + 8 * (B_READY + g % kReady));
      }
    }
  }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(P.status, PACK3D_ERR_TIMEOUT);
  if (warp == 5) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tbase, 256);
  }
}

// ---------------------------------------------------------------------------------- dk, dv
namespace xk {
constexpr int kThreads = 384;  // elementwise 0-3 (even steps), 4-7 (odd), TMA 8, S and dP 9, dk and dv 10
// Registers: 168 per thread at the launch; the elementwise warps, which hold 64 columns of S^T and
// of dP^T, take 208, the others keep 88: 256 * 208 + 128 * 88 = 384 * 168.
constexpr int kRegs = 168, kMore = 208, kLess = 88;
static_assert(256 * kMore + 128 * kLess <= kThreads * kRegs, "registers of the launch");
template <int D> struct Smem {
  static constexpr int TB = Lay<D>::bytes(kTile), HB = Lay<D>::bytes(xb::kHalf);
  static constexpr int kK = 0, kV = TB, kRing = 2 * TB;
  static constexpr int kRowB = xb::kHalf * 8;               // (-lse log2(e), D tau) of a step's rows
  static constexpr int kStages = dkv_stages(D);
  static_assert(kStages % 2 == 0, "a group of warps sees the same slots");
  static constexpr int kRows = kRing + kStages * 2 * HB;    // [stages]
  static constexpr int kBar = kRows + kStages * kRowB;
  static constexpr int kBytes = kBar + 512;
};
constexpr int kMaxStages = 6;
enum {
  B_AFULL = 0, B_QFULL = 1, B_QEMPTY = B_QFULL + kMaxStages, B_SFULL = B_QEMPTY + kMaxStages,
  B_SFREE = B_SFULL + 2, B_PFULL = B_SFREE + 2, B_DONE = B_PFULL + kDkvTurns,
  B_ALL = B_DONE + kDkvTurns, B_DRAIN, B_COUNT
};
static_assert(8 * B_COUNT + 16 <= 512, "barrier area");
// TMEM columns: dk, dv and slots of 64. Step i has S^T in slot s(i), over which its P and dS (bf16)
// go, and dP^T in slot g(i). With five slots (d <= 96) s(i) = i mod 5 and g(i) = s(i + 2): S^T of
// step i + 2 goes where dP^T of step i has been read, dP^T where P and dS of step i - 1 were, so
// that the products of steps i and i + 2 need not wait for one another. At d = 128 there are four:
// steps i and i + 2 share theirs.
template <int D> struct Cols {
  static constexpr bool kFive = dkv_five(D);
  static constexpr uint32_t kK = 0, kV = D, kS = 2 * D;
  static_assert(kS + 64 * (kFive ? 5 : 4) <= 512, "tensor memory");
  __device__ __forceinline__ static uint32_t s(int i) {
    return kS + 64u * (kFive ? (uint32_t)i % 5u : 2u * ((uint32_t)i & 1u));
  }
  __device__ __forceinline__ static uint32_t g(int i) { return kFive ? s(i + 2) : s(i) + 64u; }
  // P of 16 rows; dS 16 columns further
  __device__ __forceinline__ static uint32_t p(int i, int ks) {
    return s(i) + 32u * (ks >> 1) + 8u * (ks & 1);
  }
};
}  // namespace xk

template <int D>
__global__ void __launch_bounds__(xk::kThreads, 1)
    k_cross_dkv(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                const xb::Params P) {
  using namespace xk;
  using S = Smem<D>;
  using Ly = Lay<D>;
  using C = Cols<D>;
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kBar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kBar + 8 * B_COUNT + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Waiter ab(abort_flag, P.budget);
  const uint32_t sb = tc::smem_u32(bars);  // barrier i at sb + 8 i
  const int64_t item = blockIdx.x;
  const int split = (int)(item % P.nsplit);
  const int kt = (int)((item / P.nsplit) % P.tiles);
  const int64_t bh = item / ((int64_t)P.nsplit * P.tiles);
  uint32_t w[4];
  state_words(P.act ? P.bits + bh / P.kv_heads * P.words : nullptr, P.l, (int64_t)kt * kTile, w);
  const bool any = (w[0] | w[1] | w[2] | w[3]) != 0u;
  const int64_t steps = (P.np + xb::kHalf - 1) / xb::kHalf;
  const int64_t i0 = steps * split / P.nsplit;
  const int NT = any ? (int)(steps * (split + 1) / P.nsplit - i0) : 0;
  if (tid == 0) {
    tc::mbar_init(&bars[B_AFULL], 1);
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&bars[B_QFULL + i], 1);
      tc::mbar_init(&bars[B_QEMPTY + i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&bars[B_SFULL + i], 1);
      tc::mbar_init(&bars[B_SFREE + i], 128);
    }
    for (int i = 0; i < kDkvTurns; ++i) {
      tc::mbar_init(&bars[B_PFULL + i], 128);
      tc::mbar_init(&bars[B_DONE + i], 1);
    }
    tc::mbar_init(&bars[B_ALL], 1);
    tc::mbar_init(&bars[B_DRAIN], 2);
    abort_flag[0] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------------------ elementwise and epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMore));
    const int b = warp >> 2, rin = (warp & 3) * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    const float2 sl2 = make_float2(P.scale_log2, P.scale_log2);
    const float2 sc2 = make_float2(P.scale, P.scale);
    bool ok = true;
    uint32_t seen = 0;
#pragma unroll 1
    for (int i = b; i < NT; i += 2) {
      // (the row data came with the step's tiles)
      ok = ab.all(seen, sb + 8 * (B_SFULL + b), i >> 1) &&
           ab.all(sb + 8 * (B_QFULL + i % kStages), i / kStages);
      if (!ok) break;
      tc::tc_fence_after();
      // one 16-byte read brings two rows' data (every thread reads the same)
      const float4* rd =
          reinterpret_cast<const float4*>(smem + S::kRows + (i % kStages) * S::kRowB);
      uint32_t sv[2][32], dv[2][32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        tc::tmem_ld32(tl + C::s(i) + 32 * h, sv[h]);
        tc::tmem_ld32(tl + C::g(i) + 32 * h, dv[h]);
      }
      tc::tmem_wait_ld();
      if (C::kFive) {
        tc::tc_fence_before();
        arrive32(sb + 8 * (B_SFREE + b));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t pp[16], pd[16];
#pragma unroll
        for (int k = 0; k < 32; k += 2) {
          const float4 r = rd[16 * h + (k >> 1)];
          const float2 x =
              tc::fma2(xb::f2(sv[h][k], sv[h][k + 1]), sl2, make_float2(r.x, r.z));
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          const float2 t =
              tc::fma2(xb::f2(dv[h][k], dv[h][k + 1]), sc2, make_float2(-r.y, -r.w));
          const float2 ds = xb::mul2(p, t);
          pp[k >> 1] = tc::pack_bf16(p.x, p.y);
          pd[k >> 1] = tc::pack_bf16(ds.x, ds.y);
        }
        tc::tmem_st16(tl + C::s(i) + 32 * h, pp);
        tc::tmem_st16(tl + C::s(i) + 32 * h + 16, pd);
      }
      seen = C::kFive ? ab.probe(sb + 8 * (B_SFULL + b), (i >> 1) + 1) : 0u;
      tc::tmem_wait_st();
      tc::tc_fence_before();
      arrive32(sb + 8 * (B_PFULL + i % kDkvTurns));
    }
    // warps 0-3 write dk, warps 4-7 dv, once every step's products have completed (a barrier of
    // its own: a group has not followed the other group's phases of B_DONE)
    const int64_t row = (int64_t)kt * kTile + rin;
    const bool in = (w[rin >> 5] >> (rin & 31)) & 1u;
    if (ok && NT > 0) ok = ab.all(sb + 8 * (B_ALL), 0);
    tc::tc_fence_after();
    if (ok) {
#pragma unroll
      for (int c = 0; c < D; c += 16) {
        uint32_t a[16];
        if (NT > 0) {
          tc::tmem_ld16(tl + (b ? C::kV : C::kK) + c, a);
          tc::tmem_wait_ld();
        }
        if (NT == 0 || !in)
#pragma unroll
          for (int e = 0; e < 16; ++e) a[e] = 0u;
        if (row < P.l) {
          if (P.nsplit > 1) {
            float* dst = (b ? P.part_v : P.part_k) + ((split * P.bh + bh) * P.l + row) * D + c;
#pragma unroll
            for (int e = 0; e < 16; e += 4)
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(a[e], a[e + 1], a[e + 2], a[e + 3]);
          } else {
            __nv_bfloat16* dst = (b ? P.dv : P.dk) + (bh * P.l + row) * D + c;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                pk[e] = tc::pack_bf16(__uint_as_float(a[8 * h + 2 * e]),
                                      __uint_as_float(a[8 * h + 2 * e + 1]));
              *reinterpret_cast<uint4*>(dst + 8 * h) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
            }
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLess));
  if (warp == 8) {
    // ------------------------------------------------------------ loads
    if (lane == 0 && NT > 0) {
      tc::mbar_expect_tx(&bars[B_AFULL], 2 * S::TB);
      load_rows<D>(smem + S::kK, &mk, kTile, (int64_t)kt * kTile, (int)bh, &bars[B_AFULL]);
      load_rows<D>(smem + S::kV, &mv, kTile, (int64_t)kt * kTile, (int)bh, &bars[B_AFULL]);
      int i = 0;
      for (; i < NT; ++i) {
        const int st = i % kStages;
        if (i >= kStages && !ab.wait(sb + 8 * (B_QEMPTY + st), ((i / kStages) - 1) & 1)) break;
        const int64_t row = (i0 + i) * xb::kHalf;
        tc::mbar_expect_tx(&bars[B_QFULL + st], 2 * S::HB + S::kRowB);
        load_rows<D>(smem + S::kRing + 2 * st * S::HB, &mq, xb::kHalf, row, (int)bh,
                     &bars[B_QFULL + st]);
        load_rows<D>(smem + S::kRing + (2 * st + 1) * S::HB, &mg, xb::kHalf, row, (int)bh,
                     &bars[B_QFULL + st]);
        tc::bulk_g2s(smem + S::kRows + st * S::kRowB, P.rows + bh * P.npad + row, S::kRowB,
                     &bars[B_QFULL + st]);
      }
      tc::mbar_wait(&bars[B_AFULL], 0);
      for (int k = i > kStages ? i - kStages : 0; k < i; ++k)
        tc::mbar_wait(&bars[B_QFULL + (k % kStages)], (k / kStages) & 1);
    }
  } else if (warp == 9) {
    // ------------------------------------------------------------ S^T and dP^T
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t id_s = tc::idesc_bf16_f32(128, xb::kHalf, false, false);
    const uint64_t kd = Ly::kdesc(tc::smem_u32(smem + S::kK));
    const uint64_t vd = Ly::kdesc(tc::smem_u32(smem + S::kV));
    const uint64_t r0 = Ly::kdesc(tc::smem_u32(smem + S::kRing));
    constexpr uint64_t HO = (uint64_t)(S::HB >> 4);
    bool ok = NT > 0 && ab.all(sb + 8 * (B_AFULL), 0);
#pragma unroll 1
    for (int i = 0; i < NT && ok; ++i) {
      const int st = i % kStages, b = i & 1;
      ok = ab.all(sb + 8 * (B_QFULL + st), i / kStages);
      // once those of step i - 2 have been read and the products of step i - 3 have completed; with
      // four slots, the products of step i - 2
      const int done = i - (C::kFive ? 3 : 2);
      if (C::kFive && i >= 2) ok = ok && ab.all(sb + 8 * (B_SFREE + b), (i - 2) >> 1);
      if (done >= 0) ok = ok && ab.all(sb + 8 * (B_DONE + done % kDkvTurns), done / kDkvTurns);
      if (!ok) break;
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint64_t qo = r0 + 2 * st * HO, go = qo + HO;
#pragma unroll
        for (int ks = 0; ks < Ly::kSteps; ++ks) {
          tc::mma_ss(tb + C::s(i), kd + Ly::koff(kTile, ks), qo + Ly::koff(xb::kHalf, ks), id_s,
                     ks > 0);
          tc::mma_ss(tb + C::g(i), vd + Ly::koff(kTile, ks), go + Ly::koff(xb::kHalf, ks), id_s,
                     ks > 0);
        }
        commit32(sb + 8 * (B_SFULL + b));
      }
      __syncwarp();
    }
    if (tc::elect_one()) commit32(sb + 8 * (B_DRAIN));
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) *abort_flag = 1;
  } else if (warp == 10) {
    // ------------------------------------------------------------ dv += P^T dO, dk += dS^T q
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t id_o = tc::idesc_bf16_f32(128, D, false, true);
    const uint64_t r0 = Ly::mdesc(tc::smem_u32(smem + S::kRing), xb::kHalf);
    constexpr uint64_t HO = (uint64_t)(S::HB >> 4);
#pragma unroll 1
    for (int i = 0; i < NT; ++i) {
      const int st = i % kStages, turn = i % kDkvTurns;
      if (!ab.all(sb + 8 * (B_PFULL + turn), i / kDkvTurns)) break;
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint64_t qm = r0 + 2 * st * HO, gm = qm + HO;
#pragma unroll
        for (int ks = 0; ks < xb::kHalf / 16; ++ks) {
          tc::mma_ts(tb + C::kV, tb + C::p(i, ks), gm + Ly::moff(ks), id_o,
                     (i > 0 || ks > 0) ? 1u : 0u);
          tc::mma_ts(tb + C::kK, tb + C::p(i, ks) + 16u, qm + Ly::moff(ks), id_o,
                     (i > 0 || ks > 0) ? 1u : 0u);
        }
        commit32(sb + 8 * (B_QEMPTY + st));
        commit32(sb + 8 * (B_DONE + turn));
        if (i == NT - 1) commit32(sb + 8 * (B_ALL));
      }
      __syncwarp();
    }
    if (tc::elect_one()) commit32(sb + 8 * (B_DRAIN));
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) *abort_flag = 1;
  }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(P.status, PACK3D_ERR_TIMEOUT);
  if (warp == 9) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

// dk, dv = sum over the row ranges, in order: four elements per thread
__global__ void __launch_bounds__(256)
    k_cross_sum(const float* __restrict__ pk, const float* __restrict__ pv, int nsplit, int64_t n,
                __nv_bfloat16* __restrict__ dk, __nv_bfloat16* __restrict__ dv) {
  const int64_t i = (blockIdx.x * 256ll + threadIdx.x) * 4;
  if (i >= n) return;
  const float* p = (blockIdx.y ? pv : pk) + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int k = 0; k < nsplit; ++k) {
    const float4 x = *reinterpret_cast<const float4*>(p + k * n);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  *reinterpret_cast<uint2*>((blockIdx.y ? dv : dk) + i) =
      make_uint2(tc::pack_bf16(s.x, s.y), tc::pack_bf16(s.z, s.w));
}

// Row ranges of the state-major kernel (one CTA per SM): the count whose CTAs fill the last wave
// best, the fewest on a tie, with at least four steps of 64 rows in a range.
static int dkv_ranges(const Problem& p) {
  const int64_t items = p.bh * p.tiles(), sms = sm_count();
  const int64_t steps = (p.np + xb::kHalf - 1) / xb::kHalf;
  const int64_t most = (8 * sms + items - 1) / items;
  int best = 1;
  double eff = 0.0;
  for (int64_t n = 1; n <= most && (n == 1 || n * 4 <= steps); ++n) {
    const int64_t waves = (items * n + sms - 1) / sms;
    // a range's fixed cost (loads, epilogue) is about two steps
    const double per = (double)((steps + n - 1) / n) + 2.0;
    const double e = (double)steps * items / (waves * sms * per);
    if (e > eff * 1.001) {
      eff = e;
      best = (int)n;
    }
  }
  return best;
}

// State ranges of the row-major kernel (two CTAs per SM): only when the row tiles leave half of the SMs
// without a CTA, at least four steps of 64 states each. (8 heads of one token over 16,384 states of 64:
// training step 252 -> 92 us; two ranges of 16,000 rows over 1,000 states, whose partial rows are 8 MB,
// took 86 us against 82.)
static int dq_ranges(const Problem& p) {
  const int64_t units = p.bh * ((p.np + kTile - 1) / kTile);
  const int64_t steps = (p.l + xb::kHalf - 1) / xb::kHalf;
  int64_t n = 2 * (int64_t)sm_count() / units;
  if (n > steps / 4) n = steps / 4;
  return n < 4 ? 1 : (int)n;
}
static size_t dq_part_bytes(const Problem& p) {
  const int n = dq_ranges(p);
  return n > 1 ? align256((size_t)n * p.bh * p.np * p.d * sizeof(float)) : 0;
}

size_t bwd_tc_bytes(const Problem& p) {
  const int64_t npad = (p.np + kTile - 1) / kTile * kTile;
  const int n = dkv_ranges(p);
  const size_t e = (size_t)n * p.bh * p.l * p.d * sizeof(float);
  return align256((size_t)p.bh * npad * sizeof(float2)) + dq_part_bytes(p) +
         (n > 1 ? 2 * align256(e) : 0);
}

template <int D>
static cudaError_t launch_bwd(const Problem& p, const MaskTables& m, const void* o,
                              const float* lse, const void* dO, void* dq, void* dk, void* dv,
                              void* ws) {
  using Sq = xq::Smem<D>;
  using Sk = xk::Smem<D>;
  static std::atomic<uint64_t> aq{0}, ak{0};
  cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(k_cross_dq<D>), Sq::kBytes, aq);
  if (e == cudaSuccess)
    e = smem_attr_once(reinterpret_cast<const void*>(k_cross_dkv<D>), Sk::kBytes, ak);
  if (e != cudaSuccess) return e;
  // the split of registers needs every one of the launch's
  static PerDevice split_fits;
  if (!split_fits.get([] {
        cudaFuncAttributes a, b;
        return cudaFuncGetAttributes(&a, k_cross_dq<D>) == cudaSuccess &&
               cudaFuncGetAttributes(&b, k_cross_dkv<D>) == cudaSuccess && a.numRegs >= xq::kRegs &&
               b.numRegs >= xk::kRegs;
      }))
    return cudaErrorLaunchOutOfResources;
  CUtensorMap q128, g128, k64, v64, o128, q64, g64, k128, v128;
  if (!encode_rows<D>(&q128, p.q, p.np, p.bh, kTile) ||
      !encode_rows<D>(&g128, dO, p.np, p.bh, kTile) ||
      !encode_rows<D>(&o128, dq, p.np, p.bh, kTile) ||
      !encode_rows<D>(&k64, p.k, p.l, p.bh, xb::kHalf) ||
      !encode_rows<D>(&v64, p.v, p.l, p.bh, xb::kHalf) ||
      !encode_rows<D>(&q64, p.q, p.np, p.bh, xb::kHalf) ||
      !encode_rows<D>(&g64, dO, p.np, p.bh, xb::kHalf) ||
      !encode_rows<D>(&k128, p.k, p.l, p.bh, kTile) ||
      !encode_rows<D>(&v128, p.v, p.l, p.bh, kTile))
    return cudaErrorInvalidValue;
  const int64_t npad = (p.np + kTile - 1) / kTile * kTile;
  float2* rows = static_cast<float2*>(ws);
  xb::Params P{};
  P.rows = rows;
  P.o = static_cast<const __nv_bfloat16*>(o);
  P.lse = lse;
  P.act = m.act;
  P.bits = m.bits;
  P.status = p.status;
  P.budget = wait_budget_cycles();
  P.np = p.np;
  P.npad = npad;
  P.l = p.l;
  P.bh = p.bh;
  P.rtiles = (int)(npad / kTile);
  P.tiles = (int)p.tiles();
  P.words = m.words;
  P.kv_heads = p.kv_heads;
  P.scale = p.scale;
  P.scale_log2 = p.scale * kLog2e;
  // dq: persistent, two CTAs per SM
  P.nsplit = 1;
  P.nstate = dq_ranges(p);
  P.units = p.bh * P.rtiles * P.nstate;
  uint8_t* at = static_cast<uint8_t*>(ws) + align256((size_t)p.bh * npad * sizeof(float2));
  P.part_q = reinterpret_cast<float*>(at);
  at += dq_part_bytes(p);
  P.dk = static_cast<__nv_bfloat16*>(dq);
  const int64_t cap = 2 * (int64_t)sm_count();
  k_cross_dq<D><<<(unsigned)(P.units < cap ? P.units : cap), xq::kThreads, Sq::kBytes, p.s>>>(
      q128, g128, k64, v64, o128, P);
  if (P.nstate > 1) {
    const int64_t n = p.bh * p.np * D;
    k_cross_sum<<<dim3((unsigned)((n / 4 + 255) / 256), 1), 256, 0, p.s>>>(
        P.part_q, nullptr, P.nstate, n, P.dk, nullptr);
    count_launch();
  }
  // dk, dv
  P.nsplit = dkv_ranges(p);
  P.dk = static_cast<__nv_bfloat16*>(dk);
  P.dv = static_cast<__nv_bfloat16*>(dv);
  if (P.nsplit > 1) {
    P.part_k = reinterpret_cast<float*>(at);
    P.part_v = reinterpret_cast<float*>(
        at + align256((size_t)P.nsplit * p.bh * p.l * D * sizeof(float)));
  }
  const int64_t items = p.bh * P.tiles * P.nsplit;
  if (items > 0x7fffffffLL) return cudaErrorInvalidValue;
  k_cross_dkv<D><<<(unsigned)items, xk::kThreads, Sk::kBytes, p.s>>>(q64, g64, k128, v128, P);
  count_launch(2);
  if (P.nsplit > 1) {
    const int64_t n = p.bh * p.l * D;
    k_cross_sum<<<dim3((unsigned)((n / 4 + 255) / 256), 2), 256, 0, p.s>>>(
        P.part_k, P.part_v, P.nsplit, n, P.dk, P.dv);
    count_launch();
  }
  return cudaGetLastError();
}

cudaError_t bwd_tc(const Problem& p, const MaskTables& m, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, void* ws) {
  switch (p.d) {
    case 48: return launch_bwd<48>(p, m, o, lse, dO, dq, dk, dv, ws);
    case 64: return launch_bwd<64>(p, m, o, lse, dO, dq, dk, dv, ws);
    case 96: return launch_bwd<96>(p, m, o, lse, dO, dq, dk, dv, ws);
    default: return launch_bwd<128>(p, m, o, lse, dO, dq, dk, dv, ws);
  }
}

}  // namespace xa
}  // namespace p3d
