// Tensor-core building blocks of the cross-attention kernels: swizzled operand tiles that TMA
// writes and tcgen05 reads.
//
// A tile of R rows x D bf16 lies in shared memory as D / CW blocks of R rows x CW elements, each
// row of a block RB = 2 CW bytes (64 with the 64-byte swizzle; 32 with the 32-byte one where D is
// no multiple of 32): one TMA box per block. The 16-byte pieces of 8 consecutive rows are permuted
// so that both the K-major reads (rows = M or N) and the MN-major reads (rows = K) of an 8 x 16
// byte core matrix touch 8 different bank groups. The same tile serves both kinds of read.
#pragma once

#include "cross.h"
#include "tc.cuh"
#include "tmap.h"
#include "vec.cuh"

namespace p3d {
namespace xa {

template <int D> struct Lay {
  static constexpr int CW = D % 32 == 0 ? 32 : 16;
  static constexpr int RB = 2 * CW;
  static constexpr int NB = D / CW;
  static constexpr int kSteps = D / 16;                    // K steps of a product over D
  static constexpr int kPieces = RB / 16;                  // 16-byte pieces of a block's row
  static constexpr uint64_t kType = RB == 64 ? 4ull : 6ull;  // 64-byte / 32-byte swizzle
  static constexpr int bytes(int rows) { return rows * D * 2; }
  // byte offset of 16-byte piece `pc` (of D / 8) of row r
  __device__ __forceinline__ static int piece(int rows, int r, int pc) {
    const int c = pc / kPieces, i = pc % kPieces;
    const int x = RB == 64 ? (r >> 1) & 3 : (r >> 2) & 1;
    return c * rows * RB + r * RB + ((i ^ x) << 4);
  }
  // K-major operand (rows M or N, D contiguous): descriptor and the offset of K step ks
  __device__ __forceinline__ static uint64_t kdesc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fff) | (1ull << 16) | ((uint64_t)(8 * RB >> 4) << 32) |
           (1ull << 46) | (kType << 61);
  }
  __device__ __forceinline__ static constexpr uint64_t koff(int rows, int ks) {
    return (uint64_t)(((ks * 32 / RB) * rows * RB + ks * 32 % RB) >> 4);
  }
  // MN-major operand (rows K, D = N contiguous): K step ks covers rows 16 ks .. 16 ks + 15
  __device__ __forceinline__ static uint64_t mdesc(uint32_t addr, int rows) {
    return (uint64_t)((addr >> 4) & 0x3fff) | ((uint64_t)(rows * RB >> 4) << 16) |
           ((uint64_t)(8 * RB >> 4) << 32) | (1ull << 46) | (kType << 61);
  }
  __device__ __forceinline__ static constexpr uint64_t moff(int ks) {
    return (uint64_t)((ks * 16 * RB) >> 4);
  }
};

// [count][rows][d] bf16 as a 3D box source / target: boxes of CW elements x box_rows rows.
template <int D>
inline bool encode_rows(CUtensorMap* map, const void* base, int64_t rows, int64_t count,
                        int box_rows) {
  EncodeTiledFn fn = encode_tiled_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)count};
  cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)rows * D * 2};
  cuuint32_t box[3] = {(cuuint32_t)Lay<D>::CW, (cuuint32_t)box_rows, 1};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            es, CU_TENSOR_MAP_INTERLEAVE_NONE,
            Lay<D>::RB == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// All blocks of the tile that starts at row `row` of problem `p`.
template <int D>
__device__ __forceinline__ void load_rows(void* smem_dst, const CUtensorMap* map, int rows,
                                          int64_t row, int p, uint64_t* bar) {
#pragma unroll
  for (int c = 0; c < Lay<D>::NB; ++c)
    tc::tma_load_3d(static_cast<uint8_t*>(smem_dst) + c * rows * Lay<D>::RB, map, c * Lay<D>::CW,
                    (int)row, p, bar);
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x,
                                             int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(tc::smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// the committed stores have read their shared memory / have completed
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// Barrier operations on 32-bit shared addresses (a generic pointer costs several instructions at
// each use).
__device__ __forceinline__ void arrive32(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void commit32(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   bar)
               : "memory");
}

// Bounded, abortable wait (as tc::Abort: `budget` SM clock cycles from the first look that fails)
// that suspends on the barrier instead of polling it: a polling warp takes issue slots from the warps
// of its sub-partition that compute. A suspension lasts kNap ns at most, so a wait outlasts its budget
// by about that. A wait that runs out raises the CTA's abort word, every other wait then gives up, and
// the kernel records PACK3D_ERR_TIMEOUT once at its end. The wait is inlined at many places and stays
// short: these kernels have many roles, and code beyond the instruction cache costs them more than
// waiting.
struct Waiter {
  static constexpr uint32_t kNap = 20000;
  uint32_t flag;     // shared address of the abort word
  long long budget;  // cycles
  __device__ __forceinline__ Waiter(volatile int* f, long long b)
      : flag(tc::smem_u32(const_cast<int*>(f))), budget(b) {}
  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t phase) const {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .u32 f;\n\t.reg .u64 t0, t;\n\t"
        "mov.u32 %0, 1;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "@p bra DONE;\n\t"
        "mov.u64 t0, %%clock64;\n"
        "WAIT:\n\t"
        "ld.volatile.shared.u32 f, [%4];\n\t"
        "setp.ne.u32 q, f, 0;\n\t"
        "@q bra FAIL;\n\t"
        "mov.u64 t, %%clock64;\n\t"
        "sub.u64 t, t, t0;\n\t"
        "setp.gt.s64 q, t, %5;\n\t"
        "@q st.volatile.shared.u32 [%4], 1;\n\t"
        "@q bra FAIL;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "@!p bra WAIT;\n\t"
        "bra DONE;\n"
        "FAIL:\n\t"
        "mov.u32 %0, 0;\n"
        "DONE:\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(phase & 1), "r"(kNap), "r"(flag), "l"(budget)
        : "memory");
    return ok != 0;
  }
  // by a whole warp
  __device__ __forceinline__ bool all(uint32_t bar, uint32_t phase) const {
    return __all_sync(0xffffffffu, wait(bar, phase));
  }
  // A look at a barrier whose answer is used later: barrier operations queue behind the other
  // warps' exponentials, and a wait that is satisfied still takes a few hundred cycles.
  __device__ __forceinline__ static uint32_t probe(uint32_t bar, uint32_t phase) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(phase & 1)
        : "memory");
    return ok;
  }
  // by a whole warp, after a probe of the same phase
  __device__ __forceinline__ bool all(uint32_t probed, uint32_t bar, uint32_t phase) const {
    if (__all_sync(0xffffffffu, probed)) return true;
    return all(bar, phase);
  }
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

}  // namespace xa
}  // namespace p3d
