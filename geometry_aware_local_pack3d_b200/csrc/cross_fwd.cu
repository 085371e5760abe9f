// Cross attention, forward, bf16 on tcgen05 tensor cores (head_dim 48, 64, 96 or 128).
//
//   s_ij = tau <q_i, k_j>,  p = softmax over the unmasked states j,  o_i = sum_j p_ij v_j,
//   lse_i = log sum_j exp s_ij;   a row with no unmasked state has o = 0, lse = -inf.
//
// Work unit: 256 rows of one problem = two 128-row tiles that share every K and V tile of 128
// states. Persistent CTAs; warps 0-3 and 4-7 are the softmax and epilogue of tile 0 and 1 (thread
// = row = TMEM lane), warp 8 loads by TMA, warps 9 and 10 issue the MMAs of tile 0 and 1, warp 11
// clears the masked rows of V. Per state tile: S = q K^T (fp32 in TMEM), the softmax threads write
// P = 2^(s - m) in bf16 over S, O += P V (P read from TMEM). The two tiles' chains S -> P -> O are
// independent, so that one tile's products run under the other's softmax.
// The running reference m of a row moves only when its maximum has grown by more than 2^8 (p is at
// most 2^8 and its sum and O are fp32, so nothing overflows and no digits are lost); O is then
// rescaled in TMEM, which few tiles need after the first.
// P is rounded to bf16 for the second product (relative 2^-9, as the output itself); the row sum is
// taken from the unrounded values.
// Masked states: their S is replaced by -inf whatever it holds, and their V rows (which may hold
// NaN) are zeroed in shared memory, in the tiles that mix masked and unmasked states; tiles without
// an unmasked state are not in the list and are never loaded.
// When there are fewer units than SMs and several state tiles, the states are split over nsplit
// CTAs; each writes its normalised fp32 rows and lse, and k_cross_join adds them with the weights
// exp(lse_s - lse).
#include <math.h>

#include "cross_tc.cuh"
#include "launch.h"

namespace p3d {
namespace xa {

namespace xf {
constexpr int kThreads = 384;
constexpr int kSmemLimit = 232448;
template <int D> struct Smem {
  static constexpr int TB = Lay<D>::bytes(kTile);
  static constexpr int kQ = 0;                       // [2 buffers][2 tiles]
  static constexpr int kRing = 4 * TB;
  static constexpr int kFit = (kSmemLimit - 2048 - kRing) / TB;
  static constexpr int kSlots = kFit < 8 ? kFit : 8; // K and V tiles take turns
  static constexpr int kBar = kRing + kSlots * TB;
  static constexpr int kBytes = kBar + 512 + 1024;   // + room to align the base to 1,024
};
// barriers
constexpr int kMaxSlots = 8;
// V tiles the row-clearing warp may be ahead of the MMA warps: fewer than the ring holds
constexpr int kReady = 8;
enum {
  B_QFULL = 0, B_QEMPTY = 4, B_FULL = 8, B_EMPTY = B_FULL + kMaxSlots,
  B_READY = B_EMPTY + kMaxSlots, B_SFULL = B_READY + kReady, B_PFULL = B_SFULL + 2,
  B_DONE = B_PFULL + 2, B_STAGED = B_DONE + 2, B_DRAIN = B_STAGED + 2, B_COUNT = B_DRAIN + 2
};
static_assert(8 * B_COUNT + 16 <= 512, "barrier area");

struct Params {
  float* lse;        // [bh][np] or null
  __nv_bfloat16* o;  // [bh][np][D]
  float* part_o;     // [nsplit][bh][np][D], split launches
  float* part_lse;   // [nsplit][bh][np]
  const int32_t* act;
  const uint4* bits;
  int32_t* status;
  long long budget;
  int64_t np, l, bh, units;
  int pairs, tiles, kv_heads, nsplit;
  float scale_log2;
};

// A unit's place: problem, first row, and its range [j0, j1) of the batch entry's list of tiles.
struct Unit {
  int64_t bh, row0;
  int split, j0, j1;
  const int32_t* list;  // null: tile j is j
  const uint4* bits;
  bool two;             // has rows for the second tile
  __device__ __forceinline__ Unit(const Params& P, int64_t u) {
    split = (int)(u % P.nsplit);
    const int64_t r = u / P.nsplit;
    bh = r / P.pairs;
    row0 = (r % P.pairs) * (2 * kTile);
    two = row0 + kTile < P.np;
    const int64_t b = bh / P.kv_heads;
    int n = P.tiles;
    list = nullptr;
    bits = nullptr;
    if (P.act) {
      list = P.act + b * (P.tiles + 1) + 1;
      n = list[-1];
      bits = P.bits + b * P.tiles;
    }
    j0 = (int)((int64_t)n * split / P.nsplit);
    j1 = (int)((int64_t)n * (split + 1) / P.nsplit);
  }
  __device__ __forceinline__ int tile(int j) const { return list ? list[j] : j; }
};
}  // namespace xf

template <int D>
__global__ void __launch_bounds__(xf::kThreads, 1)
    k_cross_fwd(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo,
                const xf::Params P) {
  using namespace xf;
  using S = Smem<D>;
  using Ly = Lay<D>;
  constexpr int NS = S::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kBar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kBar + 8 * B_COUNT + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  tc::Abort ab{abort_flag, P.status, P.budget};
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      tc::mbar_init(&bars[B_QFULL + i], 1);
      tc::mbar_init(&bars[B_QEMPTY + i], 1);
    }
    for (int i = 0; i < NS; ++i) {
      tc::mbar_init(&bars[B_FULL + i], 1);
      tc::mbar_init(&bars[B_EMPTY + i], 2);
    }
    for (int i = 0; i < kReady; ++i) tc::mbar_init(&bars[B_READY + i], 1);
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(&bars[B_SFULL + t], 1);
      tc::mbar_init(&bars[B_PFULL + t], 128);
      tc::mbar_init(&bars[B_DONE + t], 1);
      tc::mbar_init(&bars[B_STAGED + t], 128);
      tc::mbar_init(&bars[B_DRAIN + t], 1);
    }
    abort_flag[0] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp < 8) {
    // ------------------------------------------------------------ softmax and epilogue
    // a row's 128 logits stay in registers: 2 x 128 x 208 + 128 x 88 = 384 x 168
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int t = warp >> 2, wt = warp & 3;
    const int rin = wt * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(wt * 32) << 16);
    const uint32_t ts = tl + 128u * t, to = tl + 256u + 128u * t;
    uint32_t gc = 0, uc = 0, staged = 0;  // state tiles, units and stores this tile has had
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
      if (t == 1 && !U.two) continue;
      const int64_t row = U.row0 + t * kTile + rin;
      const int64_t grow = U.bh * P.np + row;
      const bool valid = row < P.np;
      const bool busy = row - lane < P.np;  // the warp has a row at all
      if (U.j0 == U.j1) {
        // no state takes part: zeros
        if (valid) {
          if (P.nsplit > 1) {
            P.part_lse[U.split * P.bh * P.np + grow] = -INFINITY;
          } else {
            const uint4 z = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
            for (int e = 0; e < D; e += 8) *reinterpret_cast<uint4*>(P.o + grow * D + e) = z;
            if (P.lse) P.lse[grow] = -INFINITY;
          }
        }
        continue;
      }
      float m = -INFINITY, lsum = 0.f;  // reference (in powers of two) and sum
      uint4 nb = U.bits ? U.bits[U.tile(U.j0)] : make_uint4(0u, 0u, 0u, 0u);
      for (int j = U.j0; j < U.j1; ++j, ++gc) {
        uint32_t w[4] = {nb.x, nb.y, nb.z, nb.w};
        if (!U.bits) tail_words(P.l, j, w);
        if (U.bits && j + 1 < U.j1) nb = U.bits[U.tile(j + 1)];
        if (!__all_sync(0xffffffffu, ab.wait(&bars[B_SFULL + t], gc & 1))) { ok = false; break; }
        if (busy) {
          tc::tc_fence_after();
          uint32_t s[2][64];
          tc::tmem_ld64(ts, s[0]);
          tc::tmem_ld64(ts + 64, s[1]);
          tc::tmem_wait_ld();
          if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
#pragma unroll
            for (int c = 0; c < 128; ++c)
              s[c >> 6][c & 63] = ((w[c >> 5] >> (c & 31)) & 1u) ? s[c >> 6][c & 63] : 0xff800000u;
          }
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int c = 0; c < 128; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              mx[i] = tc::max3f(mx[i], __uint_as_float(s[c >> 6][(c & 63) + 2 * i]),
                                __uint_as_float(s[c >> 6][(c & 63) + 2 * i + 1]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * P.scale_log2;
          const bool grow_m = top > m + 8.f;
          if (__any_sync(0xffffffffu, grow_m)) {
            // no earlier tile: O holds nothing yet and the first product overwrites it
            const float f = grow_m ? ex2(m - top) : 1.f;
            lsum *= f;
            if (grow_m) m = top;
            if (j > U.j0) {
#pragma unroll
              for (int c = 0; c < D; c += 16) {
                uint32_t o[16];
                tc::tmem_ld16(to + c, o);
                tc::tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                tc::tmem_st16(to + c, o);
              }
            }
          }
          const float nm = m == -INFINITY ? 0.f : -m;
          const float2 sl2 = make_float2(P.scale_log2, P.scale_log2), nm2 = make_float2(nm, nm);
          float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = 32 * h + 2 * i;
              const float2 x = tc::fma2(make_float2(__uint_as_float(s[c >> 6][c & 63]),
                                                    __uint_as_float(s[c >> 6][(c & 63) + 1])),
                                        sl2, nm2);
              const float2 p = make_float2(ex2(x.x), ex2(x.y));
              sum[i & 1] = tc::add2(sum[i & 1], p);
              pk[i] = tc::pack_bf16(p.x, p.y);
            }
            tc::tmem_st16(ts + 16 * h, pk);
          }
          lsum += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
          tc::tmem_wait_st();
          tc::tc_fence_before();
        }
        tc::mbar_arrive(&bars[B_PFULL + t]);
      }
      if (!ok) break;
      if (!__all_sync(0xffffffffu, ab.wait(&bars[B_DONE + t], (gc - 1) & 1))) break;
      tc::tc_fence_after();
      const float inv = lsum > 0.f ? 1.f / lsum : (lsum == 0.f ? 0.f : lsum);
      const float le = lsum == 0.f ? -INFINITY : (m + log2f(lsum)) * kLn2;
      const int buf = uc & 1;
      if (P.nsplit > 1) {
        const int64_t at = U.split * P.bh * P.np + grow;
        if (valid) P.part_lse[at] = le;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tc::tmem_ld16(to + c, o);
          tc::tmem_wait_ld();
          if (valid) {
#pragma unroll
            for (int i = 0; i < 16; i += 4)
              *reinterpret_cast<float4*>(P.part_o + at * D + c + i) = make_float4(
                  __uint_as_float(o[i]) * inv, __uint_as_float(o[i + 1]) * inv,
                  __uint_as_float(o[i + 2]) * inv, __uint_as_float(o[i + 3]) * inv);
          }
        }
        tc::tc_fence_before();
        if (rin == 0) tc::mbar_arrive(&bars[B_QEMPTY + 2 * buf + t]);
      } else {
        // the tile's q rows have been consumed: their buffer takes the output rows
        uint8_t* stage = smem + S::kQ + (2 * buf + t) * S::TB;
        if (valid && P.lse) P.lse[grow] = le;
#pragma unroll
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tc::tmem_ld16(to + c, o);
          tc::tmem_wait_ld();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              pk[i] = tc::pack_bf16(__uint_as_float(o[8 * h + 2 * i]) * inv,
                                    __uint_as_float(o[8 * h + 2 * i + 1]) * inv);
            *reinterpret_cast<uint4*>(stage + Ly::piece(kTile, rin, c / 8 + h)) =
                make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        tc::tc_fence_before();
        tc::fence_proxy_async_smem();
        tc::mbar_arrive(&bars[B_STAGED + t]);
        if (rin == 0) {
          // an aborting warp may never arrive: the wait is bounded as the others
          if (!ab.wait(&bars[B_STAGED + t], staged++ & 1)) ok = false;
#pragma unroll
          for (int c = 0; c < Ly::NB && ok; ++c)
            tma_store_3d(&mo, stage + c * kTile * Ly::RB, c * Ly::CW, (int)(U.row0 + t * kTile),
                         (int)U.bh);
          bulk_commit();
          bulk_wait_read();
          tc::mbar_arrive(&bars[B_QEMPTY + 2 * buf + t]);
        }
        ok = __all_sync(0xffffffffu, ok);  // a warp leaves the loop as one
      }
      ++uc;
    }
    if (rin == 0) bulk_wait();
  } else {
   asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
   if (warp == 8) {
    // ------------------------------------------------------------ TMA loads
    if (lane == 0) {
      tc::tma_prefetch_desc(&mq);
      tc::tma_prefetch_desc(&mk);
      tc::tma_prefetch_desc(&mv);
      uint32_t kv = 0, uc[2] = {0, 0};
      bool ok = true;
      for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
        const Unit U(P, u);
        if (U.j0 == U.j1) continue;
        for (int t = 0; t < (U.two ? 2 : 1) && ok; ++t, ++uc[t - 1]) {
          const int i = 2 * (uc[t] & 1) + t;
          if (uc[t] >= 2 && !ab.wait(&bars[B_QEMPTY + i], ((uc[t] >> 1) - 1) & 1)) {
            ok = false;
            break;
          }
          tc::mbar_expect_tx(&bars[B_QFULL + i], S::TB);
          load_rows<D>(smem + S::kQ + i * S::TB, &mq, kTile, U.row0 + t * kTile, (int)U.bh,
                       &bars[B_QFULL + i]);
        }
        for (int j = U.j0; j < U.j1 && ok; ++j) {
          const int64_t at = (int64_t)U.tile(j) * kTile;
          for (int x = 0; x < 2; ++x, ++kv) {
            const int st = kv % NS;
            if (kv >= (uint32_t)NS && !ab.wait(&bars[B_EMPTY + st], ((kv / NS) - 1) & 1)) {
              ok = false;
              break;
            }
            tc::mbar_expect_tx(&bars[B_FULL + st], S::TB);
            load_rows<D>(smem + S::kRing + st * S::TB, x ? &mv : &mk, kTile, at, (int)U.bh,
                         &bars[B_FULL + st]);
          }
        }
      }
      // an aborted run leaves no copy in flight
      for (uint32_t k = kv > (uint32_t)NS ? kv - NS : 0; k < kv; ++k)
        tc::mbar_wait(&bars[B_FULL + (k % NS)], (k / NS) & 1);
      for (int t = 0; t < 2; ++t)
        for (uint32_t k = uc[t] > 2 ? uc[t] - 2 : 0; k < uc[t]; ++k)
          tc::mbar_wait(&bars[B_QFULL + 2 * (k & 1) + t], (k >> 1) & 1);
    }
  } else if (warp < 11) {
    // ------------------------------------------------------------ MMA issuer of tile t
    const int t = warp - 9;
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t ts = tb + 128u * t, to = tb + 256u + 128u * t;
    const uint32_t id_s = tc::idesc_bf16_f32(128, 128, false, false);
    const uint32_t id_o = tc::idesc_bf16_f32(128, D, false, true);
    const uint64_t qd0 = Ly::kdesc(tc::smem_u32(smem + S::kQ + t * S::TB));
    const uint64_t kd0 = Ly::kdesc(tc::smem_u32(smem + S::kRing));
    const uint64_t vd0 = Ly::mdesc(tc::smem_u32(smem + S::kRing), kTile);
    auto wwait = [&](uint64_t* bar, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, ab.wait(bar, parity, false));
    };
    const bool masked = P.act != nullptr;
    uint32_t kv = 0, gc = 0, uc = 0;
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
      if (U.j0 == U.j1) continue;
      if (t == 1 && !U.two) {
        // no rows: give the state tiles back as they come
        for (int j = 0; j < 2 * (U.j1 - U.j0) && ok; ++j, ++kv) {
          ok = wwait(&bars[B_FULL + kv % NS], (kv / NS) & 1);
          if (ok && lane == 0) tc::mbar_arrive(&bars[B_EMPTY + kv % NS]);
        }
        continue;
      }
      const int buf = uc & 1;
      if (!wwait(&bars[B_QFULL + 2 * buf + t], (uc >> 1) & 1)) break;
      ++uc;
      for (int j = U.j0; j < U.j1; ++j, ++gc) {
        int st = kv % NS;
        if (!wwait(&bars[B_FULL + st], (kv / NS) & 1)) { ok = false; break; }
        // S holds the previous tile's P until its product has completed
        if (gc >= 1 && !wwait(&bars[B_DONE + t], (gc - 1) & 1)) { ok = false; break; }
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint64_t qd = qd0 + (uint64_t)((2 * buf * S::TB) >> 4);
          const uint64_t kd = kd0 + (uint64_t)((st * S::TB) >> 4);
#pragma unroll
          for (int ks = 0; ks < Ly::kSteps; ++ks)
            tc::mma_ss(ts, qd + Ly::koff(kTile, ks), kd + Ly::koff(kTile, ks), id_s, ks > 0);
          tc::tc_commit(&bars[B_SFULL + t]);
          tc::tc_commit(&bars[B_EMPTY + st]);
        }
        __syncwarp();
        ++kv;
        st = kv % NS;
        if (!(masked ? wwait(&bars[B_READY + (kv >> 1) % kReady], ((kv >> 1) / kReady) & 1)
                     : wwait(&bars[B_FULL + st], (kv / NS) & 1))) {
          ok = false;
          break;
        }
        if (!wwait(&bars[B_PFULL + t], gc & 1)) { ok = false; break; }
        tc::tc_fence_after();
        if (tc::elect_one()) {
          const uint64_t vd = vd0 + (uint64_t)((st * S::TB) >> 4);
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            tc::mma_ts(to, ts + ks * 8, vd + Ly::moff(ks), id_o, (j > U.j0 || ks > 0) ? 1u : 0u);
          tc::tc_commit(&bars[B_DONE + t]);
          tc::tc_commit(&bars[B_EMPTY + st]);
        }
        __syncwarp();
        ++kv;
      }
    }
    if (tc::elect_one()) tc::tc_commit(&bars[B_DRAIN + t]);
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN + t], 0, 100000000LL))
      set_status(P.status, PACK3D_ERR_TIMEOUT);
  } else if (P.act) {
    // ------------------------------------------------------------ masked rows of V
    uint32_t g = 0;  // V tiles (ring items 2 g + 1)
    bool ok = true;
    for (int64_t u = blockIdx.x; u < P.units && ok; u += gridDim.x) {
      const Unit U(P, u);
      for (int j = U.j0; j < U.j1; ++j, ++g) {
        const uint4 b4 = U.bits[U.tile(j)];
        const uint32_t w[4] = {b4.x, b4.y, b4.z, b4.w};
        const uint32_t kv = 2 * g + 1;
        const int st = kv % NS;
        ok = __all_sync(0xffffffffu, ab.wait(&bars[B_FULL + st], (kv / NS) & 1));
        if (!ok) break;
        if ((w[0] & w[1] & w[2] & w[3]) != 0xffffffffu) {
          uint8_t* vt = smem + S::kRing + st * S::TB;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (!((w[i] >> lane) & 1u))
#pragma unroll
              for (int pc = 0; pc < D / 8; ++pc)
                *reinterpret_cast<uint4*>(vt + Ly::piece(kTile, 32 * i + lane, pc)) =
                    make_uint4(0u, 0u, 0u, 0u);
          tc::fence_proxy_async_smem();
        }
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[B_READY + g % kReady]);
      }
    }
   }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

// Joins the splits of each row: lse = log sum_s exp(lse_s), o = sum_s exp(lse_s - lse) o_s, in
// split order. A group of 16 threads per row.
template <int D>
__global__ void __launch_bounds__(128)
    k_cross_join(const float* __restrict__ part_o, const float* __restrict__ part_lse, int nsplit,
                 int64_t rows, __nv_bfloat16* __restrict__ o, float* __restrict__ lse) {
  const int64_t row = blockIdx.x * 8ll + (threadIdx.x >> 4);
  const int t = threadIdx.x & 15;
  if (row >= rows) return;
  float top = -INFINITY;
  for (int s = 0; s < nsplit; ++s) top = fmaxf(top, part_lse[s * rows + row]);
  const float base = top == -INFINITY ? 0.f : top;
  constexpr int NP = (D / 4 + 15) / 16;
  float4 a[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) a[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.f;
  for (int s = 0; s < nsplit; ++s) {
    const float ls = part_lse[s * rows + row];
    if (ls == -INFINITY) continue;  // nothing in this range: its rows were not written
    const float f = exp2f((ls - base) * kLog2e);
    sum += f;
#pragma unroll
    for (int i = 0; i < NP; ++i) {
      const int c = (i * 16 + t) * 4;
      if (c < D) {
        const float4 x = *reinterpret_cast<const float4*>(part_o + (s * rows + row) * D + c);
        a[i].x = fmaf(f, x.x, a[i].x);
        a[i].y = fmaf(f, x.y, a[i].y);
        a[i].z = fmaf(f, x.z, a[i].z);
        a[i].w = fmaf(f, x.w, a[i].w);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int c = (i * 16 + t) * 4;
    if (c < D)
      *reinterpret_cast<uint2*>(o + row * D + c) =
          make_uint2(tc::pack_bf16(a[i].x * inv, a[i].y * inv),
                     tc::pack_bf16(a[i].z * inv, a[i].w * inv));
  }
  if (lse && t == 0) lse[row] = sum == 0.f ? -INFINITY : base + logf(sum);
}

// One block per batch entry: the bits and the list of tiles with an unmasked state.
__global__ void __launch_bounds__(512)
    k_cross_mask(const uint8_t* __restrict__ mask, int64_t l, int tiles, int32_t* __restrict__ act,
                 uint4* __restrict__ bits) {
  __shared__ uint8_t some[512];
  __shared__ int32_t warp_n[16];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* m = mask + b * l;
  int32_t* list = act + (int64_t)b * (tiles + 1);
  int total = 0;
  // 512 tiles a round; a warp forms the words of four tiles at a time (16 loads in flight)
  for (int base = 0; base < tiles; base += 512) {
    const int end = min(512, tiles - base);
    for (int i = warp * 4; i < end; i += 64) {
      bool on[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int64_t at = (int64_t)(base + i) * kTile + 32 * k + lane;
        on[k] = at < l && m[at] != 0;
      }
      uint32_t w[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) w[k] = __ballot_sync(0xffffffffu, on[k]);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (lane == k && i + k < end) {
          bits[(int64_t)b * tiles + base + i + k] =
              make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          some[i + k] = (w[4 * k] | w[4 * k + 1] | w[4 * k + 2] | w[4 * k + 3]) != 0u;
        }
    }
    __syncthreads();
    const bool mine = threadIdx.x < end && some[threadIdx.x];
    const uint32_t have = __ballot_sync(0xffffffffu, mine);
    if (lane == 0) warp_n[warp] = __popc(have);
    __syncthreads();
    int at = total;
    for (int k = 0; k < 16; ++k) {
      if (k < warp) at += warp_n[k];
      total += warp_n[k];
    }
    if (mine) list[1 + at + __popc(have & ((1u << lane) - 1u))] = base + threadIdx.x;
    __syncthreads();
  }
  if (threadIdx.x == 0) list[0] = total;
}

cudaError_t build_mask(const Problem& p, const MaskTables& m) {
  if (!m.act) return cudaSuccess;
  k_cross_mask<<<p.batch, 512, 0, p.s>>>(p.mask, p.l, (int)p.tiles(), m.act, m.bits);
  count_launch();
  return cudaGetLastError();
}

// State ranges per unit: only when the units leave SMs idle, at least two tiles each.
static int fwd_splits(const Problem& p) {
  const int64_t units = p.bh * ((p.np + 2 * kTile - 1) / (2 * kTile));
  const int64_t tiles = p.tiles();
  const int64_t room = sm_count() / (units > 0 ? units : 1);
  int64_t n = tiles / 2 < room ? tiles / 2 : room;
  return n < 1 ? 1 : (int)n;
}

size_t fwd_tc_bytes(const Problem& p) {
  const int n = fwd_splits(p);
  if (n == 1) return 0;
  const size_t rows = (size_t)n * p.bh * p.np;
  return align256(rows * p.d * sizeof(float)) + align256(rows * sizeof(float));
}

template <int D>
static cudaError_t launch_fwd(const Problem& p, const MaskTables& m, void* o, float* lse, void* ws) {
  using S = xf::Smem<D>;
  static std::atomic<uint64_t> attr{0};
  cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(k_cross_fwd<D>), S::kBytes, attr);
  if (e != cudaSuccess) return e;
  CUtensorMap mq, mk, mv, mo;
  if (!encode_rows<D>(&mq, p.q, p.np, p.bh, kTile) || !encode_rows<D>(&mk, p.k, p.l, p.bh, kTile) ||
      !encode_rows<D>(&mv, p.v, p.l, p.bh, kTile) || !encode_rows<D>(&mo, o, p.np, p.bh, kTile))
    return cudaErrorInvalidValue;
  xf::Params P{};
  P.lse = lse;
  P.o = static_cast<__nv_bfloat16*>(o);
  P.act = m.act;
  P.bits = m.bits;
  P.status = p.status;
  P.budget = wait_budget_cycles();
  P.np = p.np;
  P.l = p.l;
  P.bh = p.bh;
  P.pairs = (int)((p.np + 2 * kTile - 1) / (2 * kTile));
  P.tiles = (int)p.tiles();
  P.kv_heads = p.kv_heads;
  P.nsplit = fwd_splits(p);
  P.scale_log2 = p.scale * kLog2e;
  P.units = p.bh * P.pairs * P.nsplit;
  if (P.nsplit > 1) {
    P.part_o = static_cast<float*>(ws);
    P.part_lse = reinterpret_cast<float*>(
        static_cast<uint8_t*>(ws) +
        align256((size_t)P.nsplit * p.bh * p.np * D * sizeof(float)));
  }
  const int64_t cap = sm_count();
  k_cross_fwd<D><<<(unsigned)(P.units < cap ? P.units : cap), xf::kThreads, S::kBytes, p.s>>>(
      mq, mk, mv, mo, P);
  count_launch();
  if (P.nsplit > 1) {
    const int64_t rows = p.bh * p.np;
    k_cross_join<D><<<(unsigned)((rows + 7) / 8), 128, 0, p.s>>>(P.part_o, P.part_lse, P.nsplit,
                                                               rows, P.o, lse);
    count_launch();
  }
  return cudaGetLastError();
}

cudaError_t fwd_tc(const Problem& p, const MaskTables& m, void* o, float* lse, void* ws) {
  switch (p.d) {
    case 48: return launch_fwd<48>(p, m, o, lse, ws);
    case 64: return launch_fwd<64>(p, m, o, lse, ws);
    case 96: return launch_fwd<96>(p, m, o, lse, ws);
    default: return launch_fwd<128>(p, m, o, lse, ws);
  }
}

}  // namespace xa
}  // namespace p3d
