// C ABI of cross attention: argument checks, workspace layout and dispatch.
#include <math.h>

#include "cross.h"
#include "launch.h"

namespace p3d {
pack3d_status kv_group_of(int heads, int kv_heads, int* group);
}
using namespace p3d;

namespace {

// Rows without states: o = 0, lse = -inf.
__global__ void __launch_bounds__(256)
    k_cross_empty(uint4* __restrict__ o, int64_t n16, float* __restrict__ lse, int64_t rows) {
  const int64_t i = blockIdx.x * 256ll + threadIdx.x;
  if (i < n16) o[i] = make_uint4(0u, 0u, 0u, 0u);
  if (lse && i < rows) lse[i] = -INFINITY;
}

cudaError_t empty_rows(void* o, int64_t bytes, float* lse, int64_t rows, cudaStream_t s) {
  const int64_t n16 = bytes / 16, n = n16 > rows ? n16 : rows;  // a row is a multiple of 16 bytes
  if (n == 0) return cudaSuccess;
  k_cross_empty<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(static_cast<uint4*>(o), n16, lse, rows);
  count_launch();
  return cudaGetLastError();
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
pack3d_status cuda_status(cudaError_t e) { return e == cudaSuccess ? PACK3D_OK : PACK3D_ERR_CUDA; }

// The sizes alone. Coordinates of a copy are 32-bit: G n and l up to 2^30.
pack3d_status make(xa::Problem* p, int dtype, int batch, int heads, int kv_heads, int64_t n,
                   int64_t l, int head_dim) {
  if (dtype != PACK3D_F32 && dtype != PACK3D_BF16) return PACK3D_ERR_INVALID_ARG;
  if (batch <= 0 || heads <= 0 || n < 0 || l < 0) return PACK3D_ERR_INVALID_ARG;
  int group = 1;
  const pack3d_status st = kv_group_of(heads, kv_heads, &group);
  if (st != PACK3D_OK) return st;
  if ((int64_t)batch * heads > 65535) return PACK3D_ERR_UNSUPPORTED;
  if (head_dim != 48 && head_dim != 64 && head_dim != 96 && head_dim != 128)
    return PACK3D_ERR_UNSUPPORTED;
  if (l > (int64_t)1 << 30 || n > ((int64_t)1 << 30) / group) return PACK3D_ERR_UNSUPPORTED;
  p->dtype = dtype;
  p->batch = batch;
  p->kv_heads = heads / group;
  p->d = head_dim;
  p->bh = (int64_t)batch * p->kv_heads;
  p->np = n * group;
  p->l = l;
  return PACK3D_OK;
}

size_t bytes_of(const xa::Problem& p, bool mask, bool backward) {
  if (p.l == 0 || p.np == 0) return 0;
  if (backward ? xa::short_bwd(p) : xa::short_fwd(p)) return backward ? xa::bwd_short_bytes(p) : 0;
  if (!backward && xa::few_fwd(p)) return xa::few_bytes(p);
  const bool tc = p.dtype == PACK3D_BF16;
  const size_t own = backward ? (tc ? xa::bwd_tc_bytes(p) : xa::bwd_simt_bytes(p))
                              : (tc ? xa::fwd_tc_bytes(p) : xa::fwd_simt_bytes(p));
  return own + (mask ? xa::mask_bytes(p, xa::mask_tile_words(p, backward)) : 0);
}

pack3d_status check_workspace(const xa::Problem& p, const void* ws, size_t bytes, bool backward) {
  const size_t need = bytes_of(p, p.mask != nullptr, backward);
  if (need == 0) return PACK3D_OK;
  if (!ws) return PACK3D_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 255) return PACK3D_ERR_ALIGN;
  return bytes < need ? PACK3D_ERR_WORKSPACE : PACK3D_OK;
}

void* after_mask(const xa::Problem& p, int tw, void* ws) {
  return p.mask ? static_cast<uint8_t*>(ws) + xa::mask_bytes(p, tw) : ws;
}
}  // namespace

extern "C" size_t pack3d_cross_attn_workspace_bytes(int dtype, int batch, int heads, int kv_heads,
                                                    int64_t n, int64_t l, int head_dim,
                                                    int has_mask, int backward) {
  xa::Problem p{};
  if (make(&p, dtype, batch, heads, kv_heads, n, l, head_dim) != PACK3D_OK) return 0;
  return bytes_of(p, has_mask != 0, backward != 0);
}

extern "C" pack3d_status pack3d_cross_attn_fwd(const void* q, const void* k, const void* v,
                                               const uint8_t* mask, int dtype, int batch,
                                               int heads, int kv_heads, int64_t n, int64_t l,
                                               int head_dim, float scale, void* o, float* lse,
                                               void* workspace, size_t workspace_bytes,
                                               int32_t* status, void* stream) {
  reset_launches();
  xa::Problem p{};
  pack3d_status st = make(&p, dtype, batch, heads, kv_heads, n, l, head_dim);
  if (st != PACK3D_OK) return st;
  if (!(scale > 0.f) || isinf(scale)) return PACK3D_ERR_INVALID_ARG;
  if (p.np > 0) {
    if (!q || !o) return PACK3D_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o)) return PACK3D_ERR_ALIGN;
    if (l > 0) {
      if (!k || !v) return PACK3D_ERR_INVALID_ARG;
      if (!aligned16(k) || !aligned16(v)) return PACK3D_ERR_ALIGN;
    }
  }
  p.q = q; p.k = k; p.v = v; p.mask = mask;
  p.scale = scale;
  p.status = status;
  p.s = static_cast<cudaStream_t>(stream);
  if (p.np == 0) return PACK3D_OK;
  const int64_t rows = p.bh * p.np;
  if (l == 0)
    return cuda_status(empty_rows(o, rows * p.d * (dtype == PACK3D_BF16 ? 2 : 4), lse, rows, p.s));
  if ((st = check_workspace(p, workspace, workspace_bytes, false)) != PACK3D_OK) return st;
  if (xa::short_fwd(p)) return cuda_status(xa::fwd_short(p, o, lse));
  if (xa::few_fwd(p)) return cuda_status(xa::fwd_few(p, o, lse, workspace));
  const int tw = xa::mask_tile_words(p, false);
  const xa::MaskTables m = xa::mask_at(p, tw, workspace);
  cudaError_t e = xa::build_mask(p, m);
  if (e == cudaSuccess)
    e = dtype == PACK3D_BF16 ? xa::fwd_tc(p, m, o, lse, after_mask(p, tw, workspace))
                             : xa::fwd_simt(p, m, o, lse, after_mask(p, tw, workspace));
  return cuda_status(e);
}

extern "C" pack3d_status pack3d_cross_attn_bwd(const void* q, const void* k, const void* v,
                                               const uint8_t* mask, const void* o,
                                               const float* lse, const void* dO, int dtype,
                                               int batch, int heads, int kv_heads, int64_t n,
                                               int64_t l, int head_dim, float scale, void* dq,
                                               void* dk, void* dv, void* workspace,
                                               size_t workspace_bytes, int32_t* status,
                                               void* stream) {
  reset_launches();
  xa::Problem p{};
  pack3d_status st = make(&p, dtype, batch, heads, kv_heads, n, l, head_dim);
  if (st != PACK3D_OK) return st;
  if (!(scale > 0.f) || isinf(scale)) return PACK3D_ERR_INVALID_ARG;
  if (p.np > 0) {
    if (!q || !o || !lse || !dO || !dq) return PACK3D_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(o) || !aligned16(dO) || !aligned16(dq))
      return PACK3D_ERR_ALIGN;
  }
  if (l > 0) {
    if (!k || !v || !dk || !dv) return PACK3D_ERR_INVALID_ARG;
    if (!aligned16(k) || !aligned16(v) || !aligned16(dk) || !aligned16(dv))
      return PACK3D_ERR_ALIGN;
  }
  p.q = q; p.k = k; p.v = v; p.mask = mask;
  p.scale = scale;
  p.status = status;
  p.s = static_cast<cudaStream_t>(stream);
  const int64_t el = dtype == PACK3D_BF16 ? 2 : 4;
  if (p.np == 0 || l == 0) {
    // nothing attends to anything: every gradient is zero
    cudaError_t e = empty_rows(dq, p.bh * p.np * p.d * el, nullptr, 0, p.s);
    if (e == cudaSuccess) e = empty_rows(dk, p.bh * l * p.d * el, nullptr, 0, p.s);
    if (e == cudaSuccess) e = empty_rows(dv, p.bh * l * p.d * el, nullptr, 0, p.s);
    return cuda_status(e);
  }
  if ((st = check_workspace(p, workspace, workspace_bytes, true)) != PACK3D_OK) return st;
  if (xa::short_bwd(p)) return cuda_status(xa::bwd_short(p, o, lse, dO, dq, dk, dv, workspace));
  const int tw = xa::mask_tile_words(p, true);
  const xa::MaskTables m = xa::mask_at(p, tw, workspace);
  cudaError_t e = xa::build_mask(p, m);
  void* ws = after_mask(p, tw, workspace);
  if (e == cudaSuccess)
    e = dtype == PACK3D_BF16 ? xa::bwd_tc(p, m, o, lse, dO, dq, dk, dv, ws)
                             : xa::bwd_simt(p, m, o, lse, dO, dq, dk, dv, ws);
  return cuda_status(e);
}

extern "C" pack3d_status pack3d_read_status(int32_t* status, void* stream) {
  if (!status) return PACK3D_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t h = 0;
  if (cudaMemcpyAsync(&h, status, sizeof(h), cudaMemcpyDeviceToHost, s) != cudaSuccess ||
      cudaStreamSynchronize(s) != cudaSuccess)
    return PACK3D_ERR_CUDA;
  if (h != 0 && cudaMemsetAsync(status, 0, sizeof(h), s) != cudaSuccess) return PACK3D_ERR_CUDA;
  return static_cast<pack3d_status>(h);
}

extern "C" pack3d_status pack3d_testing_wait(int64_t* out, void* stream) {
  reset_launches();
  if (!out) return PACK3D_ERR_INVALID_ARG;
  return cuda_status(xa::wait_in_vain(reinterpret_cast<long long*>(out),
                                      static_cast<cudaStream_t>(stream)));
}
