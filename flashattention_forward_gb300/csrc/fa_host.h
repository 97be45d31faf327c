// fa_host.h -- host-side helpers of the C-ABI units: error text, tensor
// descriptor checks, tensor-map encoding.
#pragma once
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "../../include/fa_gb300.h"
#include "fa_internal.h"

namespace fa {
namespace host {

// The calling thread's fa_last_error() text (defined in fa_api.cu).
extern thread_local char g_msg[512];

inline fa_status_t fail(fa_status_t st, const char *fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof g_msg, fmt, ap);
  va_end(ap);
  return st;
}

inline fa_status_t cuda_fail(cudaError_t e, const char *where) {
  return fail(FA_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (!fn) {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// Tiled map with 128-byte swizzle; strides in bytes for dims 1..rank-1.
inline fa_status_t make_map(CUtensorMap *m, CUtensorMapDataType dt, int rank, const void *base, const uint64_t *dims,
                     const uint64_t *strides, const uint32_t *box, const char *what,
                     CUtensorMapSwizzle swz = CU_TENSOR_MAP_SWIZZLE_128B) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled is not available from the driver");
  cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  CUresult r = fn(m, dt, rank, const_cast<void *>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(FA_ERR_CUDA, "cuTensorMapEncodeTiled(%s) failed with %d", what, (int)r);
  return FA_OK;
}

inline int dtype_size(int dt) {
  switch (dt) {
    case FA_BF16: return 2;
    case FA_E4M3: return 1;
    case FA_I8: return 1;
    case FA_F32: return 4;
    case FA_I32: return 4;
    case FA_U8: return 1;
    default: return 0;
  }
}

inline bool is_pow2(int64_t x) { return x > 0 && (x & (x - 1)) == 0; }
inline int ilog2(int64_t x) {
  int s = 0;
  while ((int64_t(1) << s) < x) ++s;
  return s;
}

// Basic shape/dtype check of a tensor descriptor.
inline fa_status_t check_tensor(const fa_tensor_t *t, const char *name, int dtype, int ndim) {
  if (!t) return fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if (t->dtype != dtype) return fail(FA_ERR_INVALID_ARG, "%s has dtype %d, expected %d", name, t->dtype, dtype);
  if (t->ndim != ndim) return fail(FA_ERR_INVALID_ARG, "%s has %d dims, expected %d", name, t->ndim, ndim);
  for (int i = 0; i < ndim; ++i)
    if (t->shape[i] < 0) return fail(FA_ERR_INVALID_ARG, "%s has a negative extent", name);
  return FA_OK;
}

inline bool contiguous(const fa_tensor_t *t) {
  int64_t s = 1;
  for (int i = t->ndim - 1; i >= 0; --i) {
    if (t->shape[i] != 1 && t->stride[i] != s) return false;
    s *= t->shape[i];
  }
  return true;
}

inline int64_t numel(const fa_tensor_t *t) {
  int64_t n = 1;
  for (int i = 0; i < t->ndim; ++i) n *= t->shape[i];
  return n;
}

inline int64_t span_bytes(const fa_tensor_t *t) {
  int64_t hi = 0;
  for (int i = 0; i < t->ndim; ++i) hi += (t->shape[i] - 1) * t->stride[i];
  return (hi + 1) * dtype_size(t->dtype);
}

inline bool overlaps(const fa_tensor_t *a, const fa_tensor_t *b) {
  if (!a || !b || numel(a) == 0 || numel(b) == 0) return false;
  const char *a0 = (const char *)a->data, *b0 = (const char *)b->data;
  return a0 < b0 + span_bytes(b) && b0 < a0 + span_bytes(a);
}

inline size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Device address of the error word on the current device (fa_api.cu).
int *error_word();

// Score mod (kind 0 none, 1 ALiBi, 2 soft-cap; NULL = none) and 128 x 128
// block mask checks shared by the forward and backward entry points.
inline fa_status_t check_mods(const fa_score_mod_t *score_mod, const fa_block_mask_t *block_mask, const fa_launch_t *launch,
                       int *mod, float *slope, float *cap) {
  *mod = 0;
  *slope = *cap = 0.f;
  if (score_mod) {
    *mod = score_mod->kind;
    if (*mod < 0 || *mod > 2) return fail(FA_ERR_INVALID_ARG, "score_mod.kind %d", *mod);
    *slope = score_mod->alibi_slope;
    *cap = score_mod->softcap;
    if (*mod == 1 && !std::isfinite(*slope)) return fail(FA_ERR_INVALID_ARG, "alibi_slope must be finite");
    if (*mod == 2 && !(*cap > 0.f && std::isfinite(*cap)))
      return fail(FA_ERR_INVALID_ARG, "softcap must be positive and finite");
  }
  if (block_mask) {
    if (!block_mask->data) return fail(FA_ERR_INVALID_ARG, "block_mask.data is NULL");
    if (block_mask->blk_q != 128 || block_mask->blk_k != 128)
      return fail(FA_ERR_UNSUPPORTED, "block masks use 128x128 blocks");
    if ((int64_t)block_mask->n_qblk * 128 < launch->max_seqlen_q || (int64_t)block_mask->n_kblk * 128 < launch->max_seqlen_k)
      return fail(FA_ERR_INVALID_ARG, "block_mask does not cover max_seqlen_q/k");
  }
  return FA_OK;
}

// Byte geometry of a paged cache [N_pg, P_s, Hkv, D] for the row gather.
inline fa::KvGather kv_gather(const fa_tensor_t *t, int esz) {
  fa::KvGather g;
  g.base = (const uint8_t *)t->data;
  g.page_stride = t->stride[0] * esz;
  g.slot_stride = t->stride[1] * esz;
  g.head_stride = t->stride[2] * esz;
  return g;
}

}  // namespace host
}  // namespace fa
