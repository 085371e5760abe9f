// Cross attention: what its kernels share on the host and the device.
//
// The G = H / H_kv query heads of a KV head are contiguous in [B, H, N, d], so their rows are one
// run of N' = G N rows: every kernel sees B H_kv independent problems of N' rows against L states.
#pragma once

#include "common.cuh"

namespace p3d {
namespace xa {

constexpr int kTile = 128;  // rows or states of a tile

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

// Tables of the mask, built by k_cross_mask in the workspace: for each batch entry, the tiles of
// 128 states that hold an unmasked one (act: their number, then their indices in order) and one
// bit per state (bits: four words per tile; states past L count as masked).
struct MaskTables {
  int32_t* act;  // [B][tiles + 1]; null: no mask
  uint4* bits;   // [B][tiles]
};
inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
inline size_t mask_bytes(const Problem& p) {
  return align256(sizeof(int32_t) * p.batch * (p.tiles() + 1)) +
         align256(sizeof(uint4) * p.batch * p.tiles());
}
inline MaskTables mask_at(const Problem& p, void* ws) {
  if (!p.mask) return MaskTables{nullptr, nullptr};
  uint8_t* at = static_cast<uint8_t*>(ws);
  return MaskTables{reinterpret_cast<int32_t*>(at),
                    reinterpret_cast<uint4*>(
                        at + align256(sizeof(int32_t) * p.batch * (p.tiles() + 1)))};
}

cudaError_t build_mask(const Problem& p, const MaskTables& m);

// forward (o, lse), bf16 and fp32; `ws` follows the mask's tables
size_t fwd_tc_bytes(const Problem& p);
cudaError_t fwd_tc(const Problem& p, const MaskTables& m, void* o, float* lse, void* ws);
cudaError_t fwd_simt(const Problem& p, const MaskTables& m, void* o, float* lse);
// backward
size_t bwd_tc_bytes(const Problem& p);
cudaError_t bwd_tc(const Problem& p, const MaskTables& m, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, void* ws);
size_t bwd_simt_bytes(const Problem& p);
cudaError_t bwd_simt(const Problem& p, const MaskTables& m, const void* o, const float* lse,
                     const void* dO, void* dq, void* dk, void* dv, void* ws);

// Does state j of the tile whose words are `w` take part?
__device__ __forceinline__ bool state_bit(const uint32_t (&w)[4], int j) {
  return (w[j >> 5] >> (j & 31)) & 1u;
}
// The words of tile `tile` without a mask: the states before L.
__device__ __forceinline__ void tail_words(int64_t l, int tile, uint32_t (&w)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t left = l - (int64_t)tile * kTile - 32 * i;
    w[i] = left >= 32 ? 0xffffffffu : (left <= 0 ? 0u : (1u << left) - 1u);
  }
}

}  // namespace xa
}  // namespace p3d
