// Cross attention: what its kernels share on the host and the device.
//
// The G = H / H_kv query heads of a KV head are contiguous in [B, H, N, d], so their rows are one
// run of N' = G N rows: every kernel sees B H_kv independent problems of N' rows against L states.
#pragma once

#include "common.cuh"
#include "cross_phases.h"

namespace p3d {
namespace xa {

struct Problem {
  const void *q, *k, *v;
  const uint8_t* mask;  // [B, L] or null
  int dtype, batch, kv_heads, d;
  int64_t bh;           // B H_kv problems
  int64_t np;           // rows of each, G N
  int64_t l;            // states
  float scale;
  int32_t* status;
  cudaStream_t s;
  int64_t tiles() const { return (l + kTile - 1) / kTile; }
};

// Tables of the mask, built by k_cross_mask in the workspace: one bit per state (bits: a run of
// words per batch entry, states past L count as masked) and, for tiles of 32 tw states, the tiles
// that hold an unmasked one (act: their number, then their indices in order).
struct MaskTables {
  int32_t* act;    // [B][tiles + 1]; null: no mask
  uint32_t* bits;  // [B][words]
  int tw, tiles;   // words per tile; tiles
  int64_t words;   // words per batch entry, a multiple of 12: whole tiles of 2, 3 and 4 words
};
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline MaskTables mask_at(const Problem& p, int tw, void* ws) {
  MaskTables m{};
  m.tw = tw;
  m.tiles = (int)((p.l + 32 * tw - 1) / (32 * tw));
  m.words = ((p.l + 31) / 32 + 11) / 12 * 12;
  if (p.mask) {
    m.act = static_cast<int32_t*>(ws);
    m.bits = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(ws) +
                                         align256(sizeof(int32_t) * p.batch * (m.tiles + 1)));
  }
  return m;
}
inline size_t mask_bytes(const Problem& p, int tw) {
  const MaskTables m = mask_at(p, tw, nullptr);
  return align256(sizeof(int32_t) * p.batch * (m.tiles + 1)) +
         align256(sizeof(uint32_t) * p.batch * m.words);
}

// Words per tile of the mask's list, forward and backward.
inline int mask_tile_words(const Problem& p, bool backward) {
  return !backward && p.dtype == PACK3D_BF16 ? kFwdTile / 32 : kTile / 32;
}

cudaError_t build_mask(const Problem& p, const MaskTables& m);
cudaError_t wait_in_vain(long long* out, cudaStream_t s);  // testing

// forward (o, lse), bf16 and fp32; `ws` follows the mask's tables
size_t fwd_tc_bytes(const Problem& p);
cudaError_t fwd_tc(const Problem& p, const MaskTables& m, void* o, float* lse, void* ws);
size_t fwd_simt_bytes(const Problem& p);
cudaError_t fwd_simt(const Problem& p, const MaskTables& m, void* o, float* lse, void* ws);
// bf16 forward of few rows (no mask tables)
bool few_fwd(const Problem& p);
size_t few_bytes(const Problem& p);
cudaError_t fwd_few(const Problem& p, void* o, float* lse, void* ws);
// o and lse of rows whose states went to `nsplit` ranges: part_o [nsplit][rows][d], part_lse
// [nsplit][rows]
constexpr int kMaxSplits = 160;
cudaError_t join_splits(const Problem& p, const float* part_o, const float* part_lse, int nsplit,
                        void* o, float* lse);
// bf16 forward and backward of a short context (no mask tables)
bool short_fwd(const Problem& p);
cudaError_t fwd_short(const Problem& p, void* o, float* lse);
bool short_bwd(const Problem& p);
size_t bwd_short_bytes(const Problem& p);
cudaError_t bwd_short(const Problem& p, const void* o, const float* lse, const void* dO, void* dq,
                      void* dk, void* dv, void* ws);
// backward
size_t bwd_tc_bytes(const Problem& p);
cudaError_t bwd_tc(const Problem& p, const MaskTables& m, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, void* ws);
size_t bwd_simt_bytes(const Problem& p);
cudaError_t bwd_simt(const Problem& p, const MaskTables& m, const void* o, const float* lse,
                     const void* dO, void* dq, void* dk, void* dv, void* ws);

// The W words of states from `at` on: of the batch entry's bits, or the states before L.
template <int W>
__device__ __forceinline__ void state_words(const uint32_t* bits, int64_t l, int64_t at,
                                            uint32_t (&w)[W]) {
  if (!bits && at + 32 * W <= l) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = 0xffffffffu;
    return;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (bits) {
      w[i] = bits[(at >> 5) + i];
    } else {
      const int64_t left = l - at - 32 * i;
      w[i] = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
    }
  }
}
template <int W> __device__ __forceinline__ bool all_states(const uint32_t (&w)[W]) {
  uint32_t a = 0xffffffffu;
#pragma unroll
  for (int i = 0; i < W; ++i) a &= w[i];
  return a == 0xffffffffu;
}

}  // namespace xa
}  // namespace p3d
