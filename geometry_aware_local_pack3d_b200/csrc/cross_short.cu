// Cross attention to a short context, bf16 on tcgen05 tensor cores: at most 128 states, which stay
// in shared memory while the rows of their problem pass by.
//
// What bounds both directions is HBM: a row is read once (q; q, dO and o) and written once (o; dq),
// the products of so few states take less than that. So the pieces are small and simple: a CTA takes
// a run of consecutive 128-row tiles, and only rows move.
//
// Forward (k_cross_fwd_short), two CTAs per SM, whose steps fill each other's gaps:
//   S = q K^T, P = 2^(S - m) over S in TMEM, O = P V, o = O / sum through the tile's q buffer. One
//   pass: a row sees all its states at once, its maximum is exact.
// Backward (k_cross_bwd_short), one CTA per SM, every product formed once (five of them):
//   S = q K^T and dP = dO V^T (rows of the tile x states, TMEM); P and dS = P (dP - D) tau as bf16
//   tiles [row][state] in shared memory; dq = dS K (dS as the K-major operand), and dv += P^T dO,
//   dk += dS^T q, which read the same tiles as MN-major operands (states along M). D = <dO, o> is
//   taken from the rows as they pass. dk and dv stay in TMEM for the CTA's share of a problem's
//   rows; the shares are added in order by k_cross_sum_shares (no atomics).
// Measured: 2 x 8 heads of 32,768 rows to 77 padded states of 96, forward 48 us (4.2 TB/s of the 6.56
// of a copy); 65,536 x 8 rows to 77 of 48, forward 38 us and backward 82 us (2.4 TB/s): there the chain
// of a tile through its barriers is longer than its bytes take.
// The mask is read as bytes by each CTA, once per problem: one bit per state in four words. Masked
// logits become -inf, masked dS zero, and the masked rows of the tile that a product sums over (V
// forward, K backward) are zeroed in shared memory, whatever they hold.
#include <math.h>

#include "cross_tc.cuh"
#include "launch.h"

namespace p3d {
namespace xa {

namespace sh {
constexpr int kSmem = 232448;         // of a CTA
constexpr int kSmemOfTwo = 115712;    // of each of two CTAs on an SM

struct Params {
  const uint8_t* mask;   // [B, L] or null
  const __nv_bfloat16* o;
  const float* lse;      // backward
  float* out_lse;        // forward, or null
  float *part_k, *part_v;  // [CTAs + problems][lp][D]
  int32_t* status;
  long long budget;
  int64_t np;
  int l, lp;             // states; rounded up to a multiple of 32
  int bh, tiles, kv_heads;
  int bufs;              // backward: buffers of P and dS
  int per, more;         // units of a CTA: per, or one more for the first `more`
  float scale, scale_log2;
};

// The CTA's run of units (problem, row tile).
struct Run {
  int left, bh, tile;
  bool fresh;  // the problem's first unit here
  __device__ __forceinline__ explicit Run(const Params& P) {
    const int b = blockIdx.x, first = b * P.per + min(b, P.more);
    left = P.per + (b < P.more ? 1 : 0);
    bh = first / P.tiles;
    tile = first - bh * P.tiles;
    fresh = true;
  }
  __device__ __forceinline__ bool last(const Params& P) const {  // the problem's last unit here
    return left == 1 || tile + 1 == P.tiles;
  }
  __device__ __forceinline__ void next(const Params& P) {
    --left;
    fresh = ++tile == P.tiles;
    if (fresh) {
      tile = 0;
      ++bh;
    }
  }
};

// One bit per state of the problem's batch entry, by a whole warp.
__device__ __forceinline__ void problem_words(const Params& P, int bh, uint32_t (&w)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int at = 32 * i + lane;
    const bool on =
        at < P.l && (!P.mask || P.mask[(int64_t)(bh / P.kv_heads) * P.l + at] != 0);
    w[i] = __ballot_sync(0xffffffffu, on);
  }
}
__device__ __forceinline__ uint32_t word_of(const uint32_t (&w)[4], int i) {
  return i == 0 ? w[0] : i == 1 ? w[1] : i == 2 ? w[2] : w[3];
}
// Zeroes row r of a tile of `rows` rows.
template <int D> __device__ __forceinline__ void zero_row(uint8_t* tile, int rows, int r) {
#pragma unroll 1
  for (int pc = 0; pc < D / 8; ++pc)
    *reinterpret_cast<uint4*>(tile + Lay<D>::piece(rows, r, pc)) = make_uint4(0u, 0u, 0u, 0u);
}
// K-major operand of `rows` rows: byte offset >> 4 of K step ks (rows known at run time)
template <int D> __device__ __forceinline__ uint64_t koff(int rows, int ks) {
  constexpr int RB = Lay<D>::RB;
  return (uint64_t)((uint32_t)(ks * 32 / RB * rows * RB + ks * 32 % RB) >> 4);
}
}  // namespace sh

// --------------------------------------------------------------------------------- forward
namespace shf {
constexpr int kThreads = 192;  // softmax and epilogue 0-3, TMA loads and MMA 4, TMA stores 5
template <int D> constexpr int bytes(int lp) {
  return 2 * Lay<D>::bytes(kTile) + 2 * Lay<D>::bytes(lp) + 256 + 1024;
}
enum {
  B_Q = 0, B_QFREE = 2, B_KV = 4, B_VREADY, B_S, B_P, B_O, B_STAGED, B_DRAIN = B_STAGED + kShortTurns,
  B_COUNT
};
constexpr uint32_t kS = 0, kO = 128;  // TMEM columns (of 256): S, then P over it; O
}  // namespace shf

template <int D>
__global__ void __launch_bounds__(shf::kThreads, 2)
    k_cross_fwd_short(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                      const __grid_constant__ CUtensorMap mv,
                      const __grid_constant__ CUtensorMap mo, const sh::Params P) {
  using namespace shf;
  using Ly = Lay<D>;
  constexpr int QB = Ly::bytes(kTile);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  const int KB = Ly::bytes(P.lp);
  uint8_t* const sk = smem + 2 * QB;
  uint8_t* const sv = sk + KB;
  uint64_t* bars = reinterpret_cast<uint64_t*>(sv + KB);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + B_COUNT + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Waiter ab(abort_flag, P.budget);
  const uint32_t sb = tc::smem_u32(bars);  // barrier i at sb + 8 i
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      tc::mbar_init(&bars[i],
                    i == B_P || i == B_VREADY || (i >= B_STAGED && i < B_DRAIN) ? 128 : 1);
    abort_flag[0] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 4) tc::tmem_alloc(tmem_slot, 256);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  const int chunks = P.lp >> 5;

  if (warp < 4) {
    // ------------------------------------------------------------ softmax and epilogue
    const int rin = warp * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
    uint32_t n = 0, gen = 0;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    bool ok = true, full = true;
#pragma unroll 1
    for (sh::Run R(P); R.left > 0 && ok; R.next(P), ++n) {
      if (R.fresh) {
        sh::problem_words(P, R.bh, w);
        full = all_states(w);
        ok = ab.all(sb + 8 * B_KV, gen++);
        if (!ok) break;
        if (P.mask && rin < P.lp && !((sh::word_of(w, warp) >> lane) & 1u))
          sh::zero_row<D>(sv, P.lp, rin);
        tc::fence_proxy_async_smem();
        arrive32(sb + 8 * B_VREADY);
      }
      const int64_t row = (int64_t)R.tile * kTile + rin;
      ok = ab.all(sb + 8 * B_S, n);
      if (!ok) break;
      tc::tc_fence_after();
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
      for (int h = 0; h < chunks; ++h) {
        uint32_t s[32];
        tc::tmem_ld32(tl + kS + 32 * h, s);
        tc::tmem_wait_ld();
        const uint32_t wh = sh::word_of(w, h);
        if (wh != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 32; ++c) s[c] = ((wh >> c) & 1u) ? s[c] : 0xff800000u;
          tc::tmem_st16(tl + kS + 32 * h, reinterpret_cast<uint32_t(&)[16]>(s[0]));
          tc::tmem_st16(tl + kS + 32 * h + 16, reinterpret_cast<uint32_t(&)[16]>(s[16]));
        }
#pragma unroll
        for (int c = 0; c < 32; c += 4)
#pragma unroll
          for (int i = 0; i < 2; ++i)
            mx[i] = tc::max3f(mx[i], __uint_as_float(s[c + 2 * i]),
                              __uint_as_float(s[c + 2 * i + 1]));
      }
      if (!full) tc::tmem_wait_st();
      const float m = fmaxf(mx[0], mx[1]) * P.scale_log2;
      const float nm = m == -INFINITY ? 0.f : -m;
      const float2 sl2 = make_float2(P.scale_log2, P.scale_log2), nm2 = make_float2(nm, nm);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int h = 0; h < chunks; ++h) {
        uint32_t s[32], pk[16];
        tc::tmem_ld32(tl + kS + 32 * h, s);
        tc::tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 32; c += 2) {
          const float2 x =
              tc::fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2, nm2);
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          sum = tc::add2(sum, p);
          pk[c >> 1] = tc::pack_bf16(p.x, p.y);
        }
        // over columns that this thread has read
        tc::tmem_st16(tl + kS + 16 * h, pk);
      }
      tc::tmem_wait_st();
      tc::tc_fence_before();
      arrive32(sb + 8 * B_P);
      const float lsum = sum.x + sum.y;
      const float inv = lsum > 0.f ? 1.f / lsum : lsum;  // no state: 0
      if (P.out_lse && row < P.np)
        P.out_lse[R.bh * P.np + row] = lsum == 0.f ? -INFINITY : (m + log2f(lsum)) * kLn2;
      ok = ab.all(sb + 8 * B_O, n);
      if (!ok) break;
      tc::tc_fence_after();
      // the tile's q rows have been consumed: their buffer takes the output rows
      uint8_t* stage = smem + (n & 1) * QB;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tc::tmem_ld16(tl + kO + c, o);
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
      arrive32(sb + 8 * (B_STAGED + n % kShortTurns));
    }
  } else if (warp == 4) {
    // ------------------------------------------------------------ loads and products
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t id_s = tc::idesc_bf16_f32(128, 16, false, false) - (2u << 17) +
                          ((uint32_t)(P.lp >> 3) << 17);  // N = lp
    const uint32_t id_o = tc::idesc_bf16_f32(128, D, false, true);
    const uint64_t qd0 = Ly::kdesc(tc::smem_u32(smem));
    const uint64_t kd = Ly::kdesc(tc::smem_u32(sk)), vd = Ly::mdesc(tc::smem_u32(sv), P.lp);
    uint32_t n = 0, gen = 0, loaded = 0;
    bool ok = true;
    sh::Run ahead(P);  // whose rows are loaded next
    auto load_q = [&]() {
      const uint32_t i = loaded++;
      if (lane == 0) {
        tc::mbar_expect_tx(&bars[B_Q + (i & 1)], QB);
        load_rows<D>(smem + (i & 1) * QB, &mq, kTile, (int64_t)ahead.tile * kTile, ahead.bh,
                     &bars[B_Q + (i & 1)]);
      }
      ahead.next(P);
    };
    load_q();
#pragma unroll 1
    for (sh::Run R(P); R.left > 0; R.next(P), ++n) {
      // the products before have read S, and K and V if these change (n == 0: nothing yet)
      ok = n == 0 || ab.all(sb + 8 * B_O, n - 1);
      if (!ok) break;
      if (R.fresh) {
        if (lane == 0) {
          tc::mbar_expect_tx(&bars[B_KV], 2 * KB);
          load_rows<D>(sk, &mk, P.lp, 0, R.bh, &bars[B_KV]);
          load_rows<D>(sv, &mv, P.lp, 0, R.bh, &bars[B_KV]);
        }
        ok = ab.all(sb + 8 * B_KV, gen++);
        if (!ok) break;
      }
      ok = ab.all(sb + 8 * (B_Q + (n & 1)), n >> 1);
      if (!ok) break;
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint64_t qd = qd0 + (((n & 1) * QB) >> 4);
#pragma unroll
        for (int ks = 0; ks < Ly::kSteps; ++ks)
          tc::mma_ss(tb + kS, qd + Ly::koff(kTile, ks), kd + sh::koff<D>(P.lp, ks), id_s, ks > 0);
        commit32(sb + 8 * B_S);
      }
      __syncwarp();
      if (ahead.left > 0) {
        // the next rows, into the other buffer once its output rows have left
        if (n >= 1) ok = ab.all(sb + 8 * (B_QFREE + ((n + 1) & 1)), ((n + 1) >> 1) - 1);
        if (!ok) break;
        load_q();
      }
      if (R.fresh) ok = ab.all(sb + 8 * B_VREADY, gen - 1);
      ok = ok && ab.all(sb + 8 * B_P, n);
      if (!ok) break;
      tc::tc_fence_after();
      if (tc::elect_one()) {
#pragma unroll 1
        for (int ks = 0; ks < P.lp / 16; ++ks)
          tc::mma_ts(tb + kO, tb + kS + ks * 8, vd + Ly::moff(ks), id_o, ks > 0 ? 1u : 0u);
        commit32(sb + 8 * B_O);
      }
      __syncwarp();
    }
    if (tc::elect_one()) commit32(sb + 8 * B_DRAIN);
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) *abort_flag = 1;
    if (!ok) {
      // an aborted run leaves no copy in flight
      for (uint32_t i = loaded > 2 ? loaded - 2 : 0; i < loaded; ++i)
        tc::mbar_wait(&bars[B_Q + (i & 1)], (i >> 1) & 1);
      if (gen) tc::mbar_wait(&bars[B_KV], (gen - 1) & 1);
    }
  } else {
    // ------------------------------------------------------------ stores
    if (lane == 0) {
      uint32_t n = 0;
#pragma unroll 1
      for (sh::Run R(P); R.left > 0; R.next(P), ++n) {
        if (!ab.wait(sb + 8 * (B_STAGED + n % kShortTurns), n / kShortTurns)) break;
#pragma unroll 1
        for (int c = 0; c < Ly::NB; ++c)
          tma_store_3d(&mo, smem + (n & 1) * QB + c * kTile * Ly::RB, c * Ly::CW, R.tile * kTile,
                       R.bh);
        bulk_commit();
        bulk_wait_read();
        arrive32(sb + 8 * (B_QFREE + (n & 1)));
      }
      bulk_wait();
    }
  }
  tc::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) set_status(P.status, PACK3D_ERR_TIMEOUT);
  if (warp == 4) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tbase, 256);
  }
}

// -------------------------------------------------------------------------------- backward
namespace shb {
constexpr int kThreads = 320;  // elementwise 0-3, row data and dq 4-7, TMA 8, MMA 9
// P and dS come first: as M = 128 operands of fewer than 128 states they reach past their tiles,
// into the operands behind them (rows of dk, dv that no state owns and nobody reads)
template <int D> constexpr int bytes(int lp, int bufs) {
  return bufs * 2 * Lay<64>::RB * kTile * (lp / 32) + 2 * Lay<D>::bytes(lp) +
         5 * Lay<D>::bytes(kTile) + 2 * kTile * 8 + 512;
}
// Buffers of P and dS: two where they fit, so that a tile's elementwise pass runs under the products
// of the one before (65,536 rows x 8 heads to 77 states of 48: backward 88 -> 82 us).
template <int D> constexpr int buffers(int lp) { return bytes<D>(lp, 2) <= sh::kSmem ? 2 : 1; }
enum {
  B_Q = 0, B_KV = 2, B_KREADY, B_S, B_SFREE, B_ROWS, B_PD = B_ROWS + 2, B_MM = B_PD + 2,
  B_DQFREE = B_MM + 2,
  B_FLUSH, B_STAGED, B_STFREE, B_DRAIN, B_COUNT
};
}  // namespace shb

template <int D>
__global__ void __launch_bounds__(shb::kThreads, 1)
    k_cross_bwd_short(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mg,
                      const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv,
                      const __grid_constant__ CUtensorMap mo, const sh::Params P) {
  using namespace shb;
  using Ly = Lay<D>;
  using Lp = Lay<64>;  // P and dS: blocks of 32 states
  constexpr int QB = Ly::bytes(kTile);
  extern __shared__ __align__(1024) uint8_t smem[];
  const int KB = Ly::bytes(P.lp), PB = kTile * P.lp * 2;
  const int bufs = P.bufs;
  uint8_t* const sp = smem;             // [buffers] P and dS
  uint8_t* const sd = sp + PB;
  uint8_t* const sq = sp + bufs * 2 * PB;  // [2 buffers] q, [2] dO
  uint8_t* const sg = sq + 2 * QB;
  uint8_t* const sk = sg + 2 * QB;
  uint8_t* const sv = sk + KB;
  uint8_t* const so = sv + KB;          // dq rows on their way out
  float2* const srow = reinterpret_cast<float2*>(so + QB);  // [2][128] (-lse log2(e), D tau)
  uint64_t* bars = reinterpret_cast<uint64_t*>(srow + 2 * kTile);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + B_COUNT + 1);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Waiter ab(abort_flag, P.budget);
  const uint32_t sb = tc::smem_u32(bars);
  if (tid == 0) {
    for (int i = 0; i < B_COUNT; ++i)
      tc::mbar_init(&bars[i], i == B_KREADY || i == B_SFREE || i == B_ROWS || i == B_ROWS + 1 ||
                                      i == B_PD || i == B_PD + 1 || i == B_DQFREE || i == B_FLUSH || i == B_STAGED
                                  ? 128
                                  : 1);
    abort_flag[0] = 0;
    tc::fence_mbar_init();
  }
  if (warp == 9) tc::tmem_alloc(tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_slot;
  // TMEM columns: S, dP, dq, dk, dv (2 lp + 3 D <= 512)
  const uint32_t cP = (uint32_t)P.lp, cQ = 2 * cP, cK = cQ + D, cV = cK + D;
  const int chunks = P.lp >> 5;

  if (warp < 4) {
    // ------------------------------------------------------------ P and dS
    const int rin = warp * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)(warp * 32) << 16);
    uint32_t n = 0, gen = 0;
    uint32_t w[4] = {0u, 0u, 0u, 0u};
    bool ok = true;
#pragma unroll 1
    for (sh::Run R(P); R.left > 0 && ok; R.next(P), ++n) {
      if (R.fresh) {
        sh::problem_words(P, R.bh, w);
        ok = ab.all(sb + 8 * B_KV, gen++);
        if (!ok) break;
        if (P.mask && rin < P.lp && !((sh::word_of(w, warp) >> lane) & 1u))
          sh::zero_row<D>(sk, P.lp, rin);
        tc::fence_proxy_async_smem();
        arrive32(sb + 8 * B_KREADY);
      }
      ok = ab.all(sb + 8 * (B_ROWS + (n & 1)), n >> 1) && ab.all(sb + 8 * B_S, n);
      // P and dS are the tile's before (or the one before that) until its products have completed
      if (n >= (uint32_t)bufs)
        ok = ok && ab.all(sb + 8 * (B_MM + ((n - bufs) & 1)), (n - bufs) >> 1);
      const int buf = bufs == 2 ? (n & 1) * 2 * PB : 0;
      if (!ok) break;
      tc::tc_fence_after();
      const float2 rd = srow[(n & 1) * kTile + rin];
      const float2 nl2 = make_float2(rd.x, rd.x), nd2 = make_float2(-rd.y, -rd.y);
      const float2 sl2 = make_float2(P.scale_log2, P.scale_log2);
      const float2 sc2 = make_float2(P.scale, P.scale);
#pragma unroll 1
      for (int h = 0; h < chunks; ++h) {
        const uint32_t wh = sh::word_of(w, h);
        uint32_t s[32], g[32];
        tc::tmem_ld32(tl + 32 * h, s);
        tc::tmem_ld32(tl + cP + 32 * h, g);
        tc::tmem_wait_ld();
        if (h + 1 == chunks) {  // S and dP have been read: the next tile's may be formed
          tc::tc_fence_before();
          arrive32(sb + 8 * B_SFREE);
        }
        if (wh != 0xffffffffu) {
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            s[c] = ((wh >> c) & 1u) ? s[c] : 0xff800000u;
            g[c] = ((wh >> c) & 1u) ? g[c] : 0u;
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t pp[4], pd[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int c = 8 * q + 2 * i;
            const float2 x = tc::fma2(
                make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2, nl2);
            const float2 p = make_float2(ex2(x.x), ex2(x.y));
            const float2 t = tc::fma2(
                make_float2(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), sc2, nd2);
            pp[i] = tc::pack_bf16(p.x, p.y);
            pd[i] = tc::pack_bf16(p.x * t.x, p.y * t.y);
          }
          const int at = buf + Lp::piece(kTile, rin, 4 * h + q);
          *reinterpret_cast<uint4*>(sp + at) = make_uint4(pp[0], pp[1], pp[2], pp[3]);
          *reinterpret_cast<uint4*>(sd + at) = make_uint4(pd[0], pd[1], pd[2], pd[3]);
        }
      }
      tc::fence_proxy_async_smem();
      arrive32(sb + 8 * (B_PD + (n & 1)));
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ row data, dq, dk and dv
    const int rin = (warp - 4) * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)((warp - 4) * 32) << 16);
    sh::Run ahead(P);
    bool ok = true;
    // the o row and lse of unit `ahead`: asked for a unit before they are used, since a trip to HBM
    // per tile in this chain took as long as the tile (training step of 65,536 x 8 heads to 77 states of 48:
    // 143 -> 126 us)
    uint4 orow[D / 8];
    float le = -INFINITY;
    auto fetch = [&]() {
      const int64_t row = (int64_t)ahead.tile * kTile + rin, at = ahead.bh * P.np + row;
      const bool in = ahead.left > 0 && row < P.np;
      le = in ? P.lse[at] : -INFINITY;
#pragma unroll
      for (int pc = 0; pc < D / 8; ++pc)
        orow[pc] = in ? *reinterpret_cast<const uint4*>(P.o + at * D + pc * 8)
                      : make_uint4(0u, 0u, 0u, 0u);
    };
    fetch();
    // D = <dO, o> and lse of the rows of unit i
    auto rows = [&](uint32_t i) -> bool {
      if (!ab.all(sb + 8 * (B_Q + (i & 1)), i >> 1)) return false;
      const int64_t row = (int64_t)ahead.tile * kTile + rin;
      float s = 0.f;
      if (row < P.np) {
#pragma unroll
        for (int pc = 0; pc < D / 8; ++pc) {
          float a[8], b[8];
          Vec<__nv_bfloat16>::unpack(orow[pc], a);
          Vec<__nv_bfloat16>::load_shared(
              reinterpret_cast<const __nv_bfloat16*>(sg + (i & 1) * QB + Ly::piece(kTile, rin, pc)),
              b);
#pragma unroll
          for (int e = 0; e < 8; ++e) s = fmaf(a[e], b[e], s);
        }
      }
      // a row without any state, and the rows past the last: P = 0, and no D of whatever dO holds
      srow[(i & 1) * kTile + rin] = le == -INFINITY ? make_float2(-INFINITY, 0.f)
                                                    : make_float2(-le * kLog2e, s * P.scale);
      arrive32(sb + 8 * (B_ROWS + (i & 1)));
      ahead.next(P);
      fetch();
      return true;
    };
    ok = rows(0);
    uint32_t n = 0;
#pragma unroll 1
    for (sh::Run R(P); R.left > 0 && ok; R.next(P), ++n) {
      // the next unit's rows while this one's products are under way
      if (ahead.left > 0) ok = rows(n + 1);
      ok = ok && ab.all(sb + 8 * (B_MM + (n & 1)), n >> 1);
      if (!ok) break;
      tc::tc_fence_after();
      if (n) ok = ab.all(sb + 8 * B_STFREE, n - 1);
      if (!ok) break;
#pragma unroll 1
      for (int c = 0; c < D; c += 16) {
        uint32_t o[16];
        tc::tmem_ld16(tl + cQ + c, o);
        tc::tmem_wait_ld();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t pk[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            pk[i] = tc::pack_bf16(__uint_as_float(o[8 * h + 2 * i]),
                                  __uint_as_float(o[8 * h + 2 * i + 1]));
          *reinterpret_cast<uint4*>(so + Ly::piece(kTile, rin, c / 8 + h)) =
              make_uint4(pk[0], pk[1], pk[2], pk[3]);
        }
      }
      tc::tc_fence_before();
      tc::fence_proxy_async_smem();
      arrive32(sb + 8 * B_STAGED);
      arrive32(sb + 8 * B_DQFREE);
      if (R.last(P)) {
        // this CTA's share of the problem's dk, dv: a slot of its own for each (CTA, problem)
        const int64_t at = ((int64_t)(blockIdx.x + R.bh) * P.lp + rin) * D;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t a[16], b[16];
          tc::tmem_ld16(tl + cK + c, a);
          tc::tmem_ld16(tl + cV + c, b);
          tc::tmem_wait_ld();
          if (rin < P.lp)
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              *reinterpret_cast<uint4*>(P.part_k + at + c + i) =
                  make_uint4(a[i], a[i + 1], a[i + 2], a[i + 3]);
              *reinterpret_cast<uint4*>(P.part_v + at + c + i) =
                  make_uint4(b[i], b[i + 1], b[i + 2], b[i + 3]);
            }
        }
        tc::tc_fence_before();
        arrive32(sb + 8 * B_FLUSH);
      }
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ loads and stores of rows
    if (lane == 0) {
      sh::Run ahead(P);
      uint32_t loaded = 0;
      auto load = [&]() {
        const uint32_t i = loaded++;
        tc::mbar_expect_tx(&bars[B_Q + (i & 1)], 2 * QB);
        load_rows<D>(sq + (i & 1) * QB, &mq, kTile, (int64_t)ahead.tile * kTile, ahead.bh,
                     &bars[B_Q + (i & 1)]);
        load_rows<D>(sg + (i & 1) * QB, &mg, kTile, (int64_t)ahead.tile * kTile, ahead.bh,
                     &bars[B_Q + (i & 1)]);
        ahead.next(P);
      };
      load();
      if (ahead.left > 0) load();
      uint32_t n = 0;
#pragma unroll 1
      for (sh::Run R(P); R.left > 0; R.next(P), ++n) {
        // the next rows as soon as the products that read their buffers have completed
        if (ahead.left > 0) {
          if (!ab.wait(sb + 8 * (B_MM + (n & 1)), n >> 1)) break;
          load();
        }
        if (!ab.wait(sb + 8 * B_STAGED, n)) break;
#pragma unroll 1
        for (int c = 0; c < Ly::NB; ++c)
          tma_store_3d(&mo, so + c * kTile * Ly::RB, c * Ly::CW, R.tile * kTile, R.bh);
        bulk_commit();
        bulk_wait_read();
        arrive32(sb + 8 * B_STFREE);
      }
      bulk_wait();
      // an aborted run leaves no copy in flight
      for (uint32_t i = loaded > 2 ? loaded - 2 : 0; i < loaded; ++i)
        tc::mbar_wait(&bars[B_Q + (i & 1)], (i >> 1) & 1);
    }
  } else {
    // ------------------------------------------------------------ products
    const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0);
    const uint32_t nl = (uint32_t)(P.lp >> 3) << 17;
    const uint32_t id_s = tc::idesc_bf16_f32(128, 0, false, false) + nl;
    const uint32_t id_q = tc::idesc_bf16_f32(128, D, false, true);
    const uint32_t id_k = tc::idesc_bf16_f32(128, D, true, true);
    const uint64_t qk0 = Ly::kdesc(tc::smem_u32(sq)), gk0 = Ly::kdesc(tc::smem_u32(sg));
    const uint64_t qm0 = Ly::mdesc(tc::smem_u32(sq), kTile), gm0 = Ly::mdesc(tc::smem_u32(sg), kTile);
    const uint64_t kk = Ly::kdesc(tc::smem_u32(sk)), vk = Ly::kdesc(tc::smem_u32(sv));
    const uint64_t km = Ly::mdesc(tc::smem_u32(sk), P.lp);
    const uint64_t dk = Lp::kdesc(tc::smem_u32(sd));
    const uint64_t pm = Lp::mdesc(tc::smem_u32(sp), kTile), dm = Lp::mdesc(tc::smem_u32(sd), kTile);
    uint32_t n = 0, gen = 0;
    bool ok = true;
    // S and dP of unit i (its problem's K and V are there; S and dP have been read)
    auto scores = [&](uint32_t i) {
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint64_t bo = (uint64_t)(((i & 1) * QB) >> 4);
#pragma unroll 1
        for (int ks = 0; ks < Ly::kSteps; ++ks) {
          const uint64_t a = sh::koff<D>(kTile, ks), b = sh::koff<D>(P.lp, ks);
          tc::mma_ss(tb, qk0 + bo + a, kk + b, id_s, ks > 0);
          tc::mma_ss(tb + cP, gk0 + bo + a, vk + b, id_s, ks > 0);
        }
        commit32(sb + 8 * B_S);
      }
      __syncwarp();
    };
    sh::Run ahead(P);
    uint32_t issued = 0;
#pragma unroll 1
    for (sh::Run R(P); R.left > 0; R.next(P), ++n) {
      if (issued == n) {
        // the unit's scores have not been formed ahead
        if (R.fresh) {
          // the products before have read K and V, and their dk, dv have been taken out
          if (n)
            ok = ab.all(sb + 8 * (B_MM + ((n - 1) & 1)), (n - 1) >> 1) &&
                 ab.all(sb + 8 * B_FLUSH, gen - 1);
          if (!ok) break;
          if (lane == 0) {
            tc::mbar_expect_tx(&bars[B_KV], 2 * KB);
            load_rows<D>(sk, &mk, P.lp, 0, R.bh, &bars[B_KV]);
            load_rows<D>(sv, &mv, P.lp, 0, R.bh, &bars[B_KV]);
          }
          __syncwarp();
          ++gen;
          ok = ab.all(sb + 8 * B_KV, gen - 1) && ab.all(sb + 8 * B_KREADY, gen - 1);
          if (!ok) break;
        }
        ok = ab.all(sb + 8 * (B_Q + (n & 1)), n >> 1) && (n == 0 || ab.all(sb + 8 * B_SFREE, n - 1));
        if (!ok) break;
        scores(n);
        ++issued;
        ahead.next(P);
      }
      ok = ab.all(sb + 8 * B_SFREE, n);
      if (!ok) break;
      // the next unit's scores go first if its rows are there and its states the same
      if (ahead.left > 0 && !ahead.fresh &&
          __all_sync(0xffffffffu, ab.probe(sb + 8 * (B_Q + ((n + 1) & 1)), (n + 1) >> 1))) {
        scores(n + 1);
        ++issued;
        ahead.next(P);
      }
      ok = ab.all(sb + 8 * (B_PD + (n & 1)), n >> 1) && (n == 0 || ab.all(sb + 8 * B_DQFREE, n - 1));
      if (!ok) break;
      tc::tc_fence_after();
      if (tc::elect_one()) {
        const uint64_t bo = (uint64_t)(((n & 1) * QB) >> 4);
        const uint64_t po = bufs == 2 ? (uint64_t)(((n & 1) * 2 * PB) >> 4) : 0;
        const uint32_t more = R.fresh ? 0u : 1u;
#pragma unroll 1
        for (int ks = 0; ks < P.lp / 16; ++ks)
          tc::mma_ss(tb + cQ, dk + po + sh::koff<64>(kTile, ks), km + Ly::moff(ks),
                     id_q, ks > 0);
#pragma unroll 1
        for (int ks = 0; ks < kTile / 16; ++ks) {
          const uint32_t acc = ks > 0 ? 1u : more;
          tc::mma_ss(tb + cV, pm + po + Lp::moff(ks), gm0 + bo + Ly::moff(ks), id_k, acc);
          tc::mma_ss(tb + cK, dm + po + Lp::moff(ks), qm0 + bo + Ly::moff(ks), id_k, acc);
        }
        commit32(sb + 8 * (B_MM + (n & 1)));
      }
      __syncwarp();
    }
    if (tc::elect_one()) commit32(sb + 8 * B_DRAIN);
    __syncwarp();
    if (!tc::mbar_wait(&bars[B_DRAIN], 0, 100000000LL)) *abort_flag = 1;
    if (!ok && gen) tc::mbar_wait(&bars[B_KV], (gen - 1) & 1);  // no copy is left in flight
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

// dk, dv of problem blockIdx.y: the shares of the CTAs c0 .. c1 that walked its rows, in order. Four
// elements per thread. A masked state's are zero by selection: its shares hold 0 x dO and 0 x q, which
// are no zeros where a row is not finite.
__global__ void __launch_bounds__(128)
    k_cross_sum_shares(const float* __restrict__ pk, const float* __restrict__ pv,
                       const uint8_t* __restrict__ mask, int kv_heads, int l, int lp, int d,
                       int tiles, int per, int more, __nv_bfloat16* __restrict__ dk,
                       __nv_bfloat16* __restrict__ dv) {
  const int e = (blockIdx.x * 128 + threadIdx.x) * 4, bh = blockIdx.y;
  if (e >= l * d) return;
  // the CTA that holds unit u: the first `more` hold one unit more
  auto cta = [&](int u) {
    const int big = more * (per + 1);
    return u < big ? u / (per + 1) : more + (u - big) / per;
  };
  const int c0 = cta(bh * tiles), c1 = cta(bh * tiles + tiles - 1);
  const float* p = (blockIdx.z ? pv : pk) + (int64_t)bh * lp * d + e;
  const bool in = !mask || mask[(int64_t)(bh / kv_heads) * l + e / d] != 0;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int c = c0; c <= c1; ++c) {
    const float4 x = *reinterpret_cast<const float4*>(p + (int64_t)c * lp * d);
    s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
  }
  if (!in) s = make_float4(0.f, 0.f, 0.f, 0.f);
  *reinterpret_cast<uint2*>((blockIdx.z ? dv : dk) + (int64_t)bh * l * d + e) =
      make_uint2(tc::pack_bf16(s.x, s.y), tc::pack_bf16(s.z, s.w));
}

// -------------------------------------------------------------------------------------- host
static int lp_of(const Problem& p) { return (int)((p.l + 31) / 32 * 32); }

// The forward's rule: each of two CTAs of an SM holds the states and two tiles of rows.
bool short_fwd(const Problem& p) {
  if (p.dtype != PACK3D_BF16 || p.l > kTile) return false;
  const int lp = lp_of(p);
  const int b = p.d == 48   ? shf::bytes<48>(lp)
                : p.d == 64 ? shf::bytes<64>(lp)
                : p.d == 96 ? shf::bytes<96>(lp)
                            : shf::bytes<128>(lp);
  return b <= sh::kSmemOfTwo;
}
// The backward's: S, dP, dq, dk and dv of all states share the 512 columns of TMEM.
bool short_bwd(const Problem& p) {
  return p.dtype == PACK3D_BF16 && p.l <= kTile && 2 * lp_of(p) + 3 * p.d <= 512;
}

static bool fill(const Problem& p, int ctas, sh::Params* P, int* grid) {
  const int64_t tiles = (p.np + kTile - 1) / kTile, units = tiles * p.bh;
  if (units > INT32_MAX / 2) return false;  // more than the memory holds
  *grid = (int)(units < ctas ? units : ctas);
  P->mask = p.mask;
  P->status = p.status;
  P->budget = wait_budget_cycles();
  P->np = p.np;
  P->l = (int)p.l;
  P->lp = lp_of(p);
  P->bh = (int)p.bh;
  P->tiles = (int)tiles;
  P->kv_heads = p.kv_heads;
  P->per = (int)(units / *grid);
  P->more = (int)(units % *grid);
  P->scale = p.scale;
  P->scale_log2 = p.scale * kLog2e;
  return true;
}

template <int D> static cudaError_t launch_fwd_short(const Problem& p, void* o, float* lse) {
  static std::atomic<uint64_t> attr{0};
  cudaError_t e = smem_attr_once(reinterpret_cast<const void*>(k_cross_fwd_short<D>),
                                 sh::kSmemOfTwo, attr);
  if (e != cudaSuccess) return e;
  sh::Params P{};
  int grid = 0;
  CUtensorMap mq, mk, mv, mo;
  if (!fill(p, 2 * sm_count(), &P, &grid) || !encode_rows<D>(&mq, p.q, p.np, p.bh, kTile) ||
      !encode_rows<D>(&mk, p.k, p.l, p.bh, P.lp) || !encode_rows<D>(&mv, p.v, p.l, p.bh, P.lp) ||
      !encode_rows<D>(&mo, o, p.np, p.bh, kTile))
    return cudaErrorInvalidValue;
  P.out_lse = lse;
  k_cross_fwd_short<D><<<grid, shf::kThreads, shf::bytes<D>(P.lp), p.s>>>(mq, mk, mv, mo, P);
  count_launch();
  return cudaGetLastError();
}

cudaError_t fwd_short(const Problem& p, void* o, float* lse) {
  switch (p.d) {
    case 48: return launch_fwd_short<48>(p, o, lse);
    case 64: return launch_fwd_short<64>(p, o, lse);
    case 96: return launch_fwd_short<96>(p, o, lse);
    default: return launch_fwd_short<128>(p, o, lse);
  }
}

size_t bwd_short_bytes(const Problem& p) {
  const size_t slots = (size_t)sm_count() + p.bh;
  return 2 * align256(slots * lp_of(p) * p.d * sizeof(float));
}

template <int D>
static cudaError_t launch_bwd_short(const Problem& p, const void* o, const float* lse,
                                    const void* dO, void* dq, void* dk, void* dv, void* ws) {
  static std::atomic<uint64_t> attr{0};
  cudaError_t e =
      smem_attr_once(reinterpret_cast<const void*>(k_cross_bwd_short<D>), sh::kSmem, attr);
  if (e != cudaSuccess) return e;
  sh::Params P{};
  int grid = 0;
  CUtensorMap mq, mg, mk, mv, mo;
  if (!fill(p, sm_count(), &P, &grid) || !encode_rows<D>(&mq, p.q, p.np, p.bh, kTile) ||
      !encode_rows<D>(&mg, dO, p.np, p.bh, kTile) || !encode_rows<D>(&mk, p.k, p.l, p.bh, P.lp) ||
      !encode_rows<D>(&mv, p.v, p.l, p.bh, P.lp) || !encode_rows<D>(&mo, dq, p.np, p.bh, kTile))
    return cudaErrorInvalidValue;
  P.o = static_cast<const __nv_bfloat16*>(o);
  P.lse = lse;
  P.bufs = shb::buffers<D>(P.lp);
  P.part_k = static_cast<float*>(ws);
  P.part_v = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + bwd_short_bytes(p) / 2);
  k_cross_bwd_short<D><<<grid, shb::kThreads, shb::bytes<D>(P.lp, P.bufs), p.s>>>(mq, mg, mk, mv, mo, P);
  k_cross_sum_shares<<<dim3((unsigned)((p.l * D / 4 + 127) / 128), (unsigned)p.bh, 2), 128, 0, p.s>>>(
      P.part_k, P.part_v, P.mask, P.kv_heads, P.l, P.lp, D, P.tiles, P.per, P.more, static_cast<__nv_bfloat16*>(dk),
      static_cast<__nv_bfloat16*>(dv));
  count_launch(2);
  return cudaGetLastError();
}

cudaError_t bwd_short(const Problem& p, const void* o, const float* lse, const void* dO, void* dq,
                      void* dk, void* dv, void* ws) {
  switch (p.d) {
    case 48: return launch_bwd_short<48>(p, o, lse, dO, dq, dk, dv, ws);
    case 64: return launch_bwd_short<64>(p, o, lse, dO, dq, dk, dv, ws);
    case 96: return launch_bwd_short<96>(p, o, lse, dO, dq, dk, dv, ws);
    default: return launch_bwd_short<128>(p, o, lse, dO, dq, dk, dv, ws);
  }
}

}  // namespace xa
}  // namespace p3d
