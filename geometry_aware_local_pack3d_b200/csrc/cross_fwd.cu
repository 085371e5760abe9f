// Cross attention, forward, bf16 on tcgen05 tensor cores (head_dim 48, 64, 96 or 128).
//
//   s_ij = tau <q_i, k_j>,  p = softmax over the unmasked states j,  o_i = sum_j p_ij v_j,
//   lse_i = log sum_j exp s_ij;   a row with no unmasked state has o = 0, lse = -inf.
//
// Work unit: 256 rows of one problem = two 128-row tiles that share every K and V tile of KT = 64
// states. Persistent CTAs of 18 warps:
//   0-3, 4-7  softmax of tile 0 and 1 (thread = row = TMEM lane)
//   8-11      epilogue of both tiles: O / sum in bf16, through the tile's consumed q rows, by TMA
//   12        TMA loads;  13, 14  S products of tile 0 and 1;  15, 16  O products of them
//   17        clears the masked rows of V
// Per state tile: S = q K^T (fp32 in TMEM); the softmax threads read S into registers and hand its
// columns back at once, so that the next tile's S is formed under this tile's exponentials;
// P = 2^(s - m) in bf16 goes to columns of its own and O += P V (P read from TMEM).
// What bounds it: a row tile's chain through tensor memory and barriers (S, maximum, exponentials, P,
// product), with the exponentials as its longest part (16 a cycle and SM: 1,024 cycles per 256 x 64
// scores against 768 of tensor work at d = 96, 2^13 FLOP a cycle): their unit is 52 % busy, the tensor
// pipe 39 %. Eight softmax warps, two per sub-partition: a warp alone keeps its sub-partition's unit
// busy half the time (it waits for S, takes maxima, packs, stores). Measured, 2 x 8 heads of 65,536
// rows to 1,024 states of 96: 550 us, 750 TFLOP/s.
// The running reference m of a row moves only when its maximum has grown by more than 2^8 (p is at
// most 2^8 and its sum and O are fp32, so nothing overflows and no digits are lost); O is then
// rescaled in TMEM, which few tiles need after the first.
// P is rounded to bf16 for the second product (relative 2^-8, as the output itself); the row sum is
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
constexpr int kThreads = 640;  // whole groups of four warps (two warps idle): they split registers
// Registers of a thread at launch, and of the softmax warps and the others once they have split the
// block's.
constexpr int kRegs = 96, kMore = 144, kLess = 64;
static_assert(256 * kMore + (kThreads - 256) * kLess <= kThreads * kRegs, "registers of the block");
template <int D> struct Smem {
  static constexpr int KT = kFwdTile;                  // states per tile
  static constexpr int QB = Lay<D>::bytes(kTile), KB = Lay<D>::bytes(KT);
  static constexpr int kSum = 0;                       // [2 turns][2 tiles][128] row sums
  static constexpr int kRef = kSum + 2048;             // the same of the references
  static constexpr int kQ = kRef + 2048;               // [2 buffers][2 tiles]
  static constexpr int kRing = kQ + 4 * QB;
  static constexpr int kSlots = fwd_slots(D);          // K and V tiles take turns
  static constexpr int kBar = kRing + kSlots * KB;
  static constexpr int kBytes = kBar + 512 + 1024;     // + room to align the base to 1,024
  // TMEM columns of tile t: S, P, O at t * 256 + ...
  static constexpr int kBufs = fwd_bufs(D);            // of S
  static constexpr uint32_t kS = 0, kP = kBufs * KT, kO = kP + KT / 2;
  static_assert(kO + D <= 256, "tensor memory of a tile");
  static_assert(kRing == fwd_ring_at(D) && kBytes <= kSmemLimit, "shared memory");
  static_assert(kSlots >= 4 && kSlots % 2 == 0, "two K and two V tiles, each in slots of their own");
};
constexpr int kMaxSlots = 8;
// V tiles the row-clearing warp may be ahead of the MMA warps: fewer than the ring holds
constexpr int kReady = kFwdReady;
enum {
  B_QFULL = 0, B_QEMPTY = 4, B_FULL = 8, B_EMPTY = B_FULL + kMaxSlots,
  B_READY = B_EMPTY + kMaxSlots, B_SFULL = B_READY + kReady, B_SFREE = B_SFULL + 4,
  B_PFULL = B_SFREE + 4, B_DONE = B_PFULL + 2, B_SUM = B_DONE + 2,
  B_OFULL = B_SUM + 4, B_OFREE = B_OFULL + 2, B_STAGED = B_OFREE + 2, B_DRAIN = B_STAGED + 2,
  B_COUNT = B_DRAIN + 4
};
static_assert(8 * B_COUNT + 16 <= 512, "barrier area");

struct Params {
  float* lse;        // [bh][np] or null
  __nv_bfloat16* o;  // [bh][np][D]
  float* part_o;     // [nsplit][bh][np][D], split launches
  float* part_lse;   // [nsplit][bh][np]
  const int32_t* act;
  const uint32_t* bits;
  int32_t* status;
  long long budget;
  int64_t np, l, bh, words;
  int units, pairs, tiles, kv_heads, nsplit;
  int step_pr, step_bh;  // pairs and problems from one unit of a CTA to its next
  float scale_log2;
};

// The units of a CTA in order: every gridDim-th. A unit is a pair of row tiles of one problem, with its
// range [j0, j1) of the batch entry's list of state tiles. A problem has two state tiles or more:
// shorter contexts have a kernel of their own.
struct Units {
  int left;              // units still to come, this one included
  int bh, pr, split, j0, j1;
  const int32_t* list;   // null: tile j is j
  const uint32_t* bits;
  __device__ __forceinline__ explicit Units(const Params& P) {
    uint32_t first = blockIdx.x;
    left = (int)(((uint32_t)P.units - first + gridDim.x - 1) / gridDim.x);
    split = 0;
    if (P.nsplit > 1) {  // (the units are then at most the CTAs: one each)
      split = (int)(first % (uint32_t)P.nsplit);
      first /= (uint32_t)P.nsplit;
    }
    bh = (int)(first / (uint32_t)P.pairs);
    pr = (int)(first - (uint32_t)bh * P.pairs);
    place(P);
  }
  __device__ __forceinline__ void place(const Params& P) {
    list = nullptr;
    bits = nullptr;
    j0 = 0;
    j1 = P.tiles;
    if (P.act) {
      const int b = (int)((uint32_t)bh / (uint32_t)P.kv_heads);
      list = P.act + (int64_t)b * (P.tiles + 1) + 1;
      j1 = left > 0 ? list[-1] : 0;
      bits = P.bits + b * P.words;
    }
    if (P.nsplit > 1) {
      // (below 2^32: at most 2^24 tiles and kMaxSplits ranges)
      const uint32_t n = (uint32_t)j1;
      j0 = (int)(n * (uint32_t)split / (uint32_t)P.nsplit);
      j1 = (int)(n * (uint32_t)(split + 1) / (uint32_t)P.nsplit);
    }
  }
  __device__ __forceinline__ void next(const Params& P) {
    --left;
    const int was = bh;
    pr += P.step_pr;
    bh += P.step_bh;
    if (pr >= P.pairs) {
      pr -= P.pairs;
      ++bh;
    }
    if (P.act && bh != was) place(P);
  }
  __device__ __forceinline__ bool any() const { return j0 != j1; }
  __device__ __forceinline__ int64_t row0() const { return (int64_t)pr * (2 * kTile); }
  __device__ __forceinline__ bool two(const Params& P) const { return row0() + kTile < P.np; }
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
  constexpr int NS = S::kSlots, KT = S::KT, KW = KT / 32;
  constexpr int kEpi = 8, kLoad = 12, kMma = 13, kClear = 17;  // first warp of each role
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~(uintptr_t)1023);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + S::kBar + 8 * B_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + S::kBar + 8 * B_COUNT + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Waiter ab{abort_flag, P.budget};
  const uint32_t sb = tc::smem_u32(bars);  // barrier i at sb + 8 i
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
      for (int b = 0; b < 4; b += 2) {  // a barrier per buffer of S: they run one ahead
        tc::mbar_init(&bars[B_SFULL + b + t], 1);
        tc::mbar_init(&bars[B_SFREE + b + t], 128);
      }
      tc::mbar_init(&bars[B_PFULL + t], 128);
      tc::mbar_init(&bars[B_DONE + t], 1);
      tc::mbar_init(&bars[B_SUM + t], 128);      // a barrier per turn: the softmax may be two
      tc::mbar_init(&bars[B_SUM + 2 + t], 128);  // units ahead of the epilogue
      tc::mbar_init(&bars[B_OFULL + t], 1);
      tc::mbar_init(&bars[B_OFREE + t], 128);
      tc::mbar_init(&bars[B_STAGED + t], 128);
      tc::mbar_init(&bars[B_DRAIN + t], 1);
      tc::mbar_init(&bars[B_DRAIN + 2 + t], 1);
    }
    abort_flag[0] = 0;
    tc::fence_mbar_init();
  }
  if (warp == kMma) tc::tmem_alloc(tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  const uint32_t tbase = *tmem_slot;

  if (warp < kEpi) {
    // ------------------------------------------------------------ softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMore));
    const int t = warp >> 2;
    const int rin = (warp & 3) * 32 + lane;
    const uint32_t tl = tbase + ((uint32_t)((warp & 3) * 32) << 16) + 256u * t;
    const uint32_t tp = tl + S::kP, to = tl + S::kO;
    uint32_t gc = 0, uc = 0;  // state tiles and units this row tile has had
    bool ok = true;
    for (Units U(P); U.left > 0 && ok; U.next(P)) {
      if ((t == 1 && !U.two(P)) || !U.any()) continue;
      if (U.row0() + t * kTile + (warp & 3) * 32 >= P.np) {
        // the warp has no row: nothing to compute, but it follows every phase of the barriers
        for (int j = U.j0; j < U.j1; ++j, ++gc) {
          const int b = gc % S::kBufs;
          ok = ab.all(sb + 8 * (B_SFULL + 2 * b + t), gc / S::kBufs);
          if (!ok) break;
          arrive32(sb + 8 * (B_SFREE + 2 * b + t));
          if (gc) ok = ab.all(sb + 8 * (B_DONE + t), gc - 1);
          if (!ok) break;
          if (j + 1 == U.j1) arrive32(sb + 8 * (B_SUM + 2 * (uc & 1) + t));
          arrive32(sb + 8 * (B_PFULL + t));
        }
        ++uc;
        continue;
      }
      float m = -INFINITY, lsum = 0.f;  // reference (in powers of two) and sum
      uint32_t seen = 0;  // the next S was there when the tile before looked
#pragma unroll 1
      for (int j = U.j0; j < U.j1; ++j, ++gc) {
        const int b = gc % S::kBufs;
        const uint32_t ts = tl + S::kS + b * KT;
        ok = ab.all(seen, sb + 8 * (B_SFULL + 2 * b + t), gc / S::kBufs);
        if (!ok) break;
        tc::tc_fence_after();
        if (U.bits || j + 1 == P.tiles) {
          // the masked logits become -inf whatever they hold
          uint32_t w[KW];
          state_words(U.bits, P.l, (int64_t)U.tile(j) * KT, w);
          if (!all_states(w)) {
#pragma unroll 1
            for (int h = 0; h < KW; ++h) {
              const uint32_t wh = h == 0 ? w[0] : w[KW - 1];
              uint32_t s[32];
              tc::tmem_ld32(ts + 32 * h, s);
              tc::tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) s[c] = ((wh >> c) & 1u) ? s[c] : 0xff800000u;
              tc::tmem_st16(ts + 32 * h, reinterpret_cast<uint32_t(&)[16]>(s[0]));
              tc::tmem_st16(ts + 32 * h + 16, reinterpret_cast<uint32_t(&)[16]>(s[16]));
            }
            tc::tmem_wait_st();
          }
        }
        uint32_t s[KT];
#pragma unroll
        for (int c = 0; c < KT; c += 32)
          tc::tmem_ld32(ts + c, reinterpret_cast<uint32_t(&)[32]>(s[c]));
        tc::tmem_wait_ld();
        tc::tc_fence_before();
        arrive32(sb + 8 * (B_SFREE + 2 * b + t));
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < KT; c += 8)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = tc::max3f(mx[i], __uint_as_float(s[c + 2 * i]), __uint_as_float(s[c + 2 * i + 1]));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * P.scale_log2;
        const bool up = top > m + 8.f;
        if (__any_sync(0xffffffffu, up)) {
          const float f = up ? ex2(m - top) : 1.f;
          lsum *= f;
          if (up) m = top;
          // (first tile: O holds nothing of this unit, and the first product overwrites it)
          if (j > U.j0) {
            ok = ab.all(sb + 8 * (B_DONE + t), gc - 1);
            if (!ok) break;
            tc::tc_fence_after();
#pragma unroll 1
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
        float2 sum = make_float2(0.f, 0.f);
        uint32_t pk[KT / 2], done = 0;
#pragma unroll
        for (int c = 0; c < KT; c += 2) {
          if (c == KT - 16) {
            // looked at here, used below
            done = ab.probe(sb + 8 * (B_DONE + t), gc - 1);
            const int nb = (gc + 1) % S::kBufs;
            seen = ab.probe(sb + 8 * (B_SFULL + 2 * nb + t), (gc + 1) / S::kBufs);
          }
          const float2 x =
              tc::fma2(make_float2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl2, nm2);
          const float2 p = make_float2(ex2(x.x), ex2(x.y));
          sum = tc::add2(sum, p);
          pk[c >> 1] = tc::pack_bf16(p.x, p.y);
        }
        lsum += sum.x + sum.y;
        // O and the columns of P are the previous tile's until its product has completed
        if (gc) {
          ok = ab.all(done, sb + 8 * (B_DONE + t), gc - 1);
          if (!ok) break;
          tc::tc_fence_after();
        }
#pragma unroll
        for (int c = 0; c < KT / 2; c += 16)
          tc::tmem_st16(tp + c, reinterpret_cast<uint32_t(&)[16]>(pk[c]));
        tc::tmem_wait_st();
        tc::tc_fence_before();
        if (j + 1 == U.j1) {
          // The row's sum and reference go to the epilogue. Its reads of this turn's slots two
          // units ago came before the product that the wait above saw complete; and this arrival
          // comes before the last P's, so that none can belong to the next unit's phase.
          reinterpret_cast<float*>(smem + S::kSum)[(uc & 1) * 256 + t * 128 + rin] = lsum;
          reinterpret_cast<float*>(smem + S::kRef)[(uc & 1) * 256 + t * 128 + rin] = m;
          arrive32(sb + 8 * (B_SUM + 2 * (uc & 1) + t));
        }
        arrive32(sb + 8 * (B_PFULL + t));
      }
      tc::tmem_wait_ld();  // (an aborted run leaves no load of S in flight)
      ++uc;
    }
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLess));
    if (warp < kLoad) {
      // ---------------------------------------------------------- epilogue
      const int rin = (warp & 3) * 32 + lane;
      uint32_t uc[2] = {0, 0};
      bool ok = true;
      for (Units U(P); U.left > 0 && ok; U.next(P)) {
        const int nt = U.two(P) ? 2 : 1;
#pragma unroll 1
        for (int t = 0; t < nt && ok; ++t) {
          const int64_t row = U.row0() + t * kTile + rin;
          const int64_t grow = U.bh * P.np + row;
          const bool valid = row < P.np, part = P.nsplit > 1;
          const int64_t at = U.split * P.bh * P.np + grow;
          const bool any = U.any();
          const uint32_t turn = (t ? uc[1] : uc[0]) & 1;
          float inv = 0.f, le = -INFINITY;  // a row without any state: zeros
          if (any) {
            if (!ab.all(sb + 8 * (B_SUM + 2 * turn + t), (t ? uc[1] : uc[0]) >> 1) ||
                !ab.all(sb + 8 * (B_OFULL + t), turn)) {
              ok = false;
              break;
            }
            tc::tc_fence_after();
            const int slot = turn * 256 + t * 128 + rin;
            const float lsum = reinterpret_cast<const float*>(smem + S::kSum)[slot];
            const float m = reinterpret_cast<const float*>(smem + S::kRef)[slot];
            if (lsum != 0.f) {
              inv = lsum > 0.f ? 1.f / lsum : lsum;
              le = (m + log2f(lsum)) * kLn2;
            }
          }
          if (valid) {
            if (part)
              P.part_lse[at] = le;
            else if (P.lse)
              P.lse[grow] = le;
          }
          if (part && !any) continue;  // the join skips it
          // the tile's q rows have been consumed: their buffer takes the output rows
          uint8_t* stage = smem + S::kQ + (2 * turn + t) * S::QB;
          const uint32_t to = tbase + ((uint32_t)((warp & 3) * 32) << 16) + 256u * t + S::kO;
#pragma unroll 1
          for (int c = 0; c < D; c += 16) {
            uint32_t o[16];
            if (any) {
              tc::tmem_ld16(to + c, o);
              tc::tmem_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 16; ++i)
              o[i] = any ? __float_as_uint(__uint_as_float(o[i]) * inv) : 0u;
            if (part) {
              if (valid)
#pragma unroll
                for (int i = 0; i < 16; i += 4)
                  *reinterpret_cast<uint4*>(P.part_o + at * D + c + i) =
                      make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
              continue;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t pk[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                pk[i] = tc::pack_bf16(__uint_as_float(o[8 * h + 2 * i]),
                                      __uint_as_float(o[8 * h + 2 * i + 1]));
              const uint4 v = make_uint4(pk[0], pk[1], pk[2], pk[3]);
              if (any)
                *reinterpret_cast<uint4*>(stage + Ly::piece(kTile, rin, c / 8 + h)) = v;
              else if (valid)
                *reinterpret_cast<uint4*>(P.o + grow * D + c + 8 * h) = v;
            }
          }
          if (!any) continue;
          tc::tc_fence_before();
          // (staged before free: a thread a unit ahead of another cannot meet its phase)
          tc::fence_proxy_async_smem();
          if (!part) arrive32(sb + 8 * (B_STAGED + t));
          arrive32(sb + 8 * (B_OFREE + t));
          if (rin == 0) {
            if (!part) {
              // an aborting warp may never arrive: the wait is bounded as the others
              if (!ab.wait(sb + 8 * (B_STAGED + t), turn)) ok = false;
#pragma unroll 1
              for (int c = 0; c < Ly::NB && ok; ++c)
                tma_store_3d(&mo, stage + c * kTile * Ly::RB, c * Ly::CW,
                             (int)(U.row0() + t * kTile), U.bh);
              bulk_commit();
              bulk_wait_read();
            }
            arrive32(sb + 8 * (B_QEMPTY + 2 * turn + t));
          }
          ok = __all_sync(0xffffffffu, ok);  // a warp leaves the loop as one
          if (t) ++uc[1]; else ++uc[0];
        }
      }
      if (rin == 0) bulk_wait();
    } else if (warp == kLoad) {
      // ---------------------------------------------------------- TMA loads
      if (lane == 0) {
        tc::tma_prefetch_desc(&mq);
        tc::tma_prefetch_desc(&mk);
        tc::tma_prefetch_desc(&mv);
        uint32_t kv = 0, uc[2] = {0, 0};
        bool ok = true;
        for (Units U(P); U.left > 0 && ok; U.next(P)) {
          if (!U.any()) continue;
          const int nt = U.two(P) ? 2 : 1;
#pragma unroll 1
          for (int t = 0; t < nt && ok; ++t) {
            const uint32_t n = t ? uc[1] : uc[0];
            const int i = 2 * (n & 1) + t;
            if (n >= 2) ok = ab.wait(sb + 8 * (B_QEMPTY + i), (n >> 1) - 1);
            if (!ok) break;
            tc::mbar_expect_tx(&bars[B_QFULL + i], S::QB);
            load_rows<D>(smem + S::kQ + i * S::QB, &mq, kTile, U.row0() + t * kTile, U.bh,
                         &bars[B_QFULL + i]);
            if (t) ++uc[1]; else ++uc[0];
          }
#pragma unroll 1
          for (int j = 2 * U.j0; j < 2 * U.j1 && ok; ++j, ++kv) {
            // K and V of a tile take turns
            const int st = kv % NS;
            if (kv >= (uint32_t)NS) ok = ab.wait(sb + 8 * (B_EMPTY + st), kv / NS - 1);
            if (!ok) break;
            tc::mbar_expect_tx(&bars[B_FULL + st], S::KB);
            load_rows<D>(smem + S::kRing + st * S::KB, j & 1 ? &mv : &mk, KT,
                         (int64_t)U.tile(j >> 1) * KT, U.bh, &bars[B_FULL + st]);
          }
        }
        // an aborted run leaves no copy in flight
        for (uint32_t k = kv > (uint32_t)NS ? kv - NS : 0; k < kv; ++k)
          tc::mbar_wait(&bars[B_FULL + (k % NS)], (k / NS) & 1);
        for (int t = 0; t < 2; ++t)
          for (uint32_t k = uc[t] > 2 ? uc[t] - 2 : 0; k < uc[t]; ++k)
            tc::mbar_wait(&bars[B_QFULL + 2 * (k & 1) + t], (k >> 1) & 1);
      }
    } else if (warp < kMma + 2) {
      // ---------------------------------------------------------- S products of tile t
      // S needs only what the softmax threads have read, and is there when they come back for it
      const int t = warp - kMma;
      const uint32_t ts = __shfl_sync(0xffffffffu, tbase, 0) + 256u * t + S::kS;
      const uint32_t id_s = tc::idesc_bf16_f32(128, KT, false, false);
      const uint64_t qd0 = Ly::kdesc(tc::smem_u32(smem + S::kQ + t * S::QB));
      const uint64_t kd0 = Ly::kdesc(tc::smem_u32(smem + S::kRing));
      uint32_t kv = 0, n = 0, uc = 0;  // state tiles; those and the units of this row tile
      bool ok = true;
#pragma unroll 1
      for (Units U(P); U.left > 0 && ok; U.next(P)) {
        if (!U.any()) continue;
        const bool mine = t == 0 || U.two(P);
        if (mine) ok = ab.all(sb + 8 * (B_QFULL + 2 * (uc & 1) + t), uc >> 1);
        const uint64_t qd = qd0 + ((2 * (uc & 1) * S::QB) >> 4);
#pragma unroll 1
        for (int j = U.j0; j < U.j1 && ok; ++j) {
          const uint32_t st = (2 * kv) % NS, b = n % S::kBufs;
          const uint32_t fb = sb + 8 * (B_FULL + st), eb = sb + 8 * (B_SFREE + 2 * b + t);
          const bool wait = mine && n >= S::kBufs;
          const uint32_t pf = ab.probe(fb, 2 * kv / NS);
          const uint32_t pe = wait ? ab.probe(eb, n / S::kBufs - 1) : 1u;
          ok = ab.all(pf, fb, 2 * kv / NS) && (!wait || ab.all(pe, eb, n / S::kBufs - 1));
          if (!ok) break;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            if (mine) {
              const uint64_t kd = kd0 + ((st * S::KB) >> 4);
#pragma unroll
              for (int ks = 0; ks < Ly::kSteps; ++ks)
                tc::mma_ss(ts + b * KT, qd + Ly::koff(kTile, ks), kd + Ly::koff(KT, ks), id_s,
                           ks > 0);
              commit32(sb + 8 * (B_SFULL + 2 * b + t));
            }
            commit32(sb + 8 * (B_EMPTY + st));
          }
          __syncwarp();
          n += mine;
          ++kv;
        }
        uc += mine;
      }
      if (tc::elect_one()) commit32(sb + 8 * (B_DRAIN + t));
      __syncwarp();
      if (!tc::mbar_wait(&bars[B_DRAIN + t], 0, 100000000LL)) *abort_flag = 1;
    } else if (warp < kClear) {
      // ---------------------------------------------------------- O products of tile t
      const int t = warp - kMma - 2;
      const uint32_t tb = __shfl_sync(0xffffffffu, tbase, 0) + 256u * t;
      const uint32_t tp = tb + S::kP, to = tb + S::kO;
      const uint32_t id_o = tc::idesc_bf16_f32(128, D, false, true);
      const uint64_t vd0 = Ly::mdesc(tc::smem_u32(smem + S::kRing), KT);
      const bool masked = P.act != nullptr;
      uint32_t kv = 0, n = 0, uc = 0;
      bool ok = true;
#pragma unroll 1
      for (Units U(P); U.left > 0 && ok; U.next(P)) {
        if (!U.any()) continue;
        const bool mine = t == 0 || U.two(P);
        // O still holds the previous unit's rows until the epilogue has read them
        if (mine && uc) ok = ab.all(sb + 8 * (B_OFREE + t), uc - 1);
#pragma unroll 1
        for (int j = U.j0; j < U.j1 && ok; ++j) {
          const uint32_t st = (2 * kv + 1) % NS;
          const uint32_t vb = sb + 8 * (masked ? B_READY + kv % kReady : B_FULL + st);
          const uint32_t vp = masked ? kv / kReady : (2 * kv + 1) / NS;
          const uint32_t pv = ab.probe(vb, vp);
          if (mine) ok = ab.all(sb + 8 * (B_PFULL + t), n);
          ok = ok && ab.all(pv, vb, vp);
          if (!ok) break;
          tc::tc_fence_after();
          if (tc::elect_one()) {
            if (mine) {
              const uint64_t vd = vd0 + ((st * S::KB) >> 4);
#pragma unroll
              for (int ks = 0; ks < KT / 16; ++ks)
                tc::mma_ts(to, tp + ks * 8, vd + Ly::moff(ks), id_o, (j > U.j0 || ks > 0) ? 1u : 0u);
              commit32(sb + 8 * (B_DONE + t));
              if (j + 1 == U.j1) commit32(sb + 8 * (B_OFULL + t));
            }
            commit32(sb + 8 * (B_EMPTY + st));
          }
          __syncwarp();
          n += mine;
          ++kv;
        }
        uc += mine;
      }
      if (tc::elect_one()) commit32(sb + 8 * (B_DRAIN + 2 + t));
      __syncwarp();
      if (!tc::mbar_wait(&bars[B_DRAIN + 2 + t], 0, 100000000LL)) *abort_flag = 1;
    } else if (warp == kClear && P.act) {
      // ---------------------------------------------------------- masked rows of V
      uint32_t g = 0;  // V tiles loaded (ring items 2 g + 1)
      bool ok = true;
      for (Units U(P); U.left > 0 && ok; U.next(P)) {
#pragma unroll 1
        for (int j = U.j0; j < U.j1; ++j, ++g) {
          uint32_t w[KW];
          state_words(U.bits, P.l, (int64_t)U.tile(j) * KT, w);
          const uint32_t kv = 2 * g + 1;
          const int st = kv % NS;
          ok = ab.all(sb + 8 * (B_FULL + st), (kv / NS));
          if (!ok) break;
          if (!all_states(w)) {
            uint8_t* vt = smem + S::kRing + st * S::KB;
#pragma unroll
            for (int i = 0; i < KW; ++i)
              if (!((w[i] >> lane) & 1u))
#pragma unroll 1
                for (int pc = 0; pc < D / 8; ++pc)
                  *reinterpret_cast<uint4*>(vt + Ly::piece(KT, 32 * i + lane, pc)) =
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
  if (warp == kMma) {
    __syncwarp();
    tc::tc_fence_after();
    tc::tmem_dealloc(tbase, 512);
  }
}

// Joins the splits of each row: lse = log sum_s exp(lse_s), o = sum_s exp(lse_s - lse) o_s. A block
// per row: every warp forms the weights (a few loads), sums every fourth split, four columns per
// lane, and the four sums are added in order. Latency is all of it: it is launched while the kernel
// before it still runs and waits for that kernel's end here.
template <int D, typename T>
__global__ void __launch_bounds__(128)
    k_cross_join(const float* __restrict__ part_o, const float* __restrict__ part_lse, int nsplit,
                 int64_t rows, T* __restrict__ o, float* __restrict__ lse) {
  __shared__ float wgt[4][kMaxSplits];
  __shared__ float4 sums[4][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float top = -INFINITY;
  for (int s = lane; s < nsplit; s += 32) {
    const float x = part_lse[s * rows + row];
    wgt[warp][s] = x;
    top = fmaxf(top, x);
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
  const float base = top == -INFINITY ? 0.f : top;
  float sum = 0.f;
  for (int s = lane; s < nsplit; s += 32) {
    const float f = exp2f((wgt[warp][s] - base) * kLog2e);
    wgt[warp][s] = f;
    sum += f;
  }
#pragma unroll
  for (int x = 16; x > 0; x >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, x);
  __syncwarp();
  if (lane < D / 4) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 5
    for (int s = warp; s < nsplit; s += 4) {
      const float f = wgt[warp][s];
      // a split without any state has written no row
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (f != 0.f) x = *reinterpret_cast<const float4*>(part_o + (s * rows + row) * D + 4 * lane);
      a.x = fmaf(f, x.x, a.x);
      a.y = fmaf(f, x.y, a.y);
      a.z = fmaf(f, x.z, a.z);
      a.w = fmaf(f, x.w, a.w);
    }
    sums[warp][lane] = a;
  }
  __syncthreads();
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (threadIdx.x < D / 4) {
    float4 a = sums[0][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) {
      const float4 x = sums[w][lane];
      a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
    }
    a = make_float4(a.x * inv, a.y * inv, a.z * inv, a.w * inv);
    if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint2*>(o + row * D + 4 * lane) =
          make_uint2(tc::pack_bf16(a.x, a.y), tc::pack_bf16(a.z, a.w));
    else
      *reinterpret_cast<float4*>(o + row * D + 4 * lane) = a;
  }
  if (lse && threadIdx.x == 0) lse[row] = sum == 0.f ? -INFINITY : base + logf(sum);
}

template <int D>
static cudaError_t launch_join(const Problem& p, const float* part_o, const float* part_lse,
                               int nsplit, void* o, float* lse) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t c{};
  c.gridDim = dim3((unsigned)(p.bh * p.np));
  c.blockDim = dim3(128);
  c.stream = p.s;
  c.attrs = &early;
  c.numAttrs = 1;
  count_launch();
  const int64_t rows = p.bh * p.np;
  return p.dtype == PACK3D_BF16
             ? cudaLaunchKernelEx(&c, k_cross_join<D, __nv_bfloat16>, part_o, part_lse, nsplit, rows,
                                  static_cast<__nv_bfloat16*>(o), lse)
             : cudaLaunchKernelEx(&c, k_cross_join<D, float>, part_o, part_lse, nsplit, rows,
                                  static_cast<float*>(o), lse);
}

cudaError_t join_splits(const Problem& p, const float* part_o, const float* part_lse, int nsplit,
                        void* o, float* lse) {
  switch (p.d) {
    case 48: return launch_join<48>(p, part_o, part_lse, nsplit, o, lse);
    case 64: return launch_join<64>(p, part_o, part_lse, nsplit, o, lse);
    case 96: return launch_join<96>(p, part_o, part_lse, nsplit, o, lse);
    default: return launch_join<128>(p, part_o, part_lse, nsplit, o, lse);
  }
}

// One block per batch entry: the bits and the list of tiles with an unmasked state.
__global__ void __launch_bounds__(512)
    k_cross_mask(const uint8_t* __restrict__ mask, int64_t l, int tiles, int tw, int64_t words,
                 int32_t* __restrict__ act, uint32_t* __restrict__ bits) {
  __shared__ uint32_t sw[512 * 4 + 16];
  __shared__ int32_t warp_n[16];
  const int b = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint8_t* m = mask + b * l;
  int32_t* list = act + (int64_t)b * (tiles + 1);
  uint32_t* out = bits + b * words;
  int total = 0;
  // 512 tiles a round (every word of the run, the last round's zero padding included); a warp
  // forms 16 words at a time, their loads in flight together
  for (int base = 0; base < tiles; base += 512) {
    const int64_t w0 = (int64_t)base * tw;
    const int nw = (int)(base + 512 < tiles ? 512 * tw : words - w0);
    for (int i = warp * 16; i < nw; i += 256) {
      bool on[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const int64_t at = (w0 + i + k) * 32 + lane;
        on[k] = at < l && m[at] != 0;
      }
      uint32_t mine = 0u;
#pragma unroll
      for (int k = 0; k < 16; ++k) {
        const uint32_t w = __ballot_sync(0xffffffffu, on[k]);
        if (lane == k) mine = w;
      }
      if (lane < 16 && i + lane < nw) {
        out[w0 + i + lane] = mine;
        sw[i + lane] = mine;
      }
    }
    __syncthreads();
    bool mine = false;
    if (base + (int)threadIdx.x < tiles)
      for (int k = 0; k < tw; ++k) mine = mine || sw[threadIdx.x * tw + k] != 0u;
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

// A wait for a barrier on which nothing arrives (pack3d_testing_wait): out = gave up, cycles.
__global__ void __launch_bounds__(32) k_cross_wait(long long budget, long long* __restrict__ out) {
  __shared__ uint64_t bar;
  __shared__ int flag;
  if (threadIdx.x == 0) {
    tc::mbar_init(&bar, 1);
    flag = 0;
    tc::fence_mbar_init();
  }
  __syncwarp();
  const Waiter ab(&flag, budget);
  const long long t0 = clock64();
  const bool ok = ab.all(tc::smem_u32(&bar), 0);
  const long long t = clock64() - t0;
  if (threadIdx.x == 0) {
    out[0] = !ok && *const_cast<volatile int*>(&flag) == 1;
    out[1] = t;
  }
}

cudaError_t wait_in_vain(long long* out, cudaStream_t s) {
  k_cross_wait<<<1, 32, 0, s>>>(wait_budget_cycles(), out);
  count_launch();
  return cudaGetLastError();
}

cudaError_t build_mask(const Problem& p, const MaskTables& m) {
  if (!m.act) return cudaSuccess;
  k_cross_mask<<<p.batch, 512, 0, p.s>>>(p.mask, p.l, m.tiles, m.tw, m.words, m.act, m.bits);
  count_launch();
  return cudaGetLastError();
}

// State ranges per unit: only when the units leave SMs idle, at least two tiles each.
static int fwd_splits(const Problem& p) {
  const int64_t units = p.bh * ((p.np + 2 * kTile - 1) / (2 * kTile));
  const int64_t tiles = (p.l + kFwdTile - 1) / kFwdTile;
  const int64_t room = sm_count() / (units > 0 ? units : 1);
  int64_t n = tiles / 2 < room ? tiles / 2 : room;
  if (n > kMaxSplits) n = kMaxSplits;
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
  // a split of more registers than the block was launched with would wait for ever
  static PerDevice split_fits;
  if (!split_fits.get([] {
        cudaFuncAttributes a;
        return cudaFuncGetAttributes(&a, k_cross_fwd<D>) == cudaSuccess && a.numRegs >= xf::kRegs;
      }))
    return cudaErrorLaunchOutOfResources;
  CUtensorMap mq, mk, mv, mo;
  if (!encode_rows<D>(&mq, p.q, p.np, p.bh, kTile) || !encode_rows<D>(&mk, p.k, p.l, p.bh, S::KT) ||
      !encode_rows<D>(&mv, p.v, p.l, p.bh, S::KT) || !encode_rows<D>(&mo, o, p.np, p.bh, kTile))
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
  P.words = m.words;
  P.tiles = m.tiles;
  P.kv_heads = p.kv_heads;
  P.nsplit = fwd_splits(p);
  P.scale_log2 = p.scale * kLog2e;
  const int64_t units = p.bh * P.pairs * P.nsplit;
  if (units > INT32_MAX / 2) return cudaErrorInvalidValue;  // more than the memory holds
  P.units = (int)units;
  if (P.nsplit > 1) {
    P.part_o = static_cast<float*>(ws);
    P.part_lse = reinterpret_cast<float*>(
        static_cast<uint8_t*>(ws) +
        align256((size_t)P.nsplit * p.bh * p.np * D * sizeof(float)));
  }
  const int grid = P.units < sm_count() ? P.units : sm_count();
  P.step_pr = grid % P.pairs;
  P.step_bh = grid / P.pairs;
  k_cross_fwd<D><<<grid, xf::kThreads, S::kBytes, p.s>>>(
      mq, mk, mv, mo, P);
  count_launch();
  if (P.nsplit > 1) return join_splits(p, P.part_o, P.part_lse, P.nsplit, o, lse);
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
