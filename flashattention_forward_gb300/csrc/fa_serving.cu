// fa_serving.cu -- the C ABI of the operators around the paged decode:
// shared-prefix attention, key weights and cache eviction (fa_gb300.h).  As in
// fa_api.cu, every check runs on the host before anything is enqueued, and no
// device memory is read back or allocated.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "fa_host.h"
#include "fa_internal.h"

using namespace fa::host;

namespace {

int sm_count() {
  int sms = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    sms = 148;
  return sms;
}

// Positions are int32 and windows are added to them: both stay below 2^30.
constexpr int64_t kMaxLen = int64_t(1) << 30;

// One token-major cache tensor: packed [T_k, Hkv, D] or pages [N_pg, P_s, Hkv, D].
fa_status_t check_cache(const fa_tensor_t *t, const char *name, bool paged, int32_t page_size) {
  if (!t) return fail(FA_ERR_INVALID_ARG, "%s is NULL", name);
  if (t->dtype != FA_BF16 && t->dtype != FA_E4M3 && t->dtype != FA_I8)
    return fail(FA_ERR_INVALID_ARG, "%s dtype must be bf16, e4m3 or int8", name);
  if (paged && t->ndim == 5) return fail(FA_ERR_UNSUPPORTED, "%s: token-major pages only, not the vectorized 5-D layout", name);
  const int nd = paged ? 4 : 3;
  fa_status_t st = check_tensor(t, name, t->dtype, nd);
  if (st) return st;
  const int esz = dtype_size(t->dtype);
  const int64_t d = t->shape[nd - 1];
  if (d != 64 && d != 128 && d != 192) return fail(FA_ERR_UNSUPPORTED, "%s head dim %lld is not compiled", name, (long long)d);
  if (t->stride[nd - 1] != 1) return fail(FA_ERR_INVALID_ARG, "%s needs a contiguous last dim", name);
  for (int i = 0; i < nd - 1; ++i)
    if ((t->stride[i] * esz) % 16) return fail(FA_ERR_INVALID_ARG, "%s strides must be multiples of 16 bytes", name);
  if ((uintptr_t)t->data & 15) return fail(FA_ERR_INVALID_ARG, "%s base must be 16-byte aligned", name);
  if (t->shape[nd - 2] <= 0) return fail(FA_ERR_INVALID_ARG, "%s has no kv heads", name);
  if (paged) {
    if (!is_pow2(page_size) || page_size > 1024)
      return fail(FA_ERR_UNSUPPORTED, "page_size %d: supported sizes are powers of two from 1 to 1024", page_size);
    if (t->shape[1] != page_size)
      return fail(FA_ERR_INVALID_ARG, "the %s page holds %lld keys, page_size=%d", name, (long long)t->shape[1], page_size);
  }
  if (t->shape[0] >= (int64_t(1) << 31)) return fail(FA_ERR_OVERFLOW, "%s: pages or rows must fit int32", name);
  return FA_OK;
}

// Per-token scales of a byte cache, as k_scale in fa_fwd_varlen; none for bf16.
fa_status_t check_scale(const fa_tensor_t *s, const char *name, const fa_tensor_t *cache, bool paged) {
  if (cache->dtype == FA_BF16) {
    if (s) return fail(FA_ERR_INVALID_ARG, "%s is only valid with an e4m3 or int8 cache", name);
    return FA_OK;
  }
  if (!s) return fail(FA_ERR_INVALID_ARG, "e4m3 and int8 caches need %s", name);
  fa_status_t st = check_tensor(s, name, FA_F32, paged ? 3 : 2);
  if (st) return st;
  for (int i = 0; i < s->ndim; ++i)
    if (s->shape[i] != cache->shape[i])
      return fail(FA_ERR_INVALID_ARG, "%s must be [N_pg, P_s, Hkv] (paged) or [T_k, Hkv]", name);
  if (!contiguous(s)) return fail(FA_ERR_INVALID_ARG, "%s must be contiguous", name);
  return FA_OK;
}

fa_status_t check_table(const fa_tensor_t *t, const char *name, int64_t num_seqs, int64_t keys, int32_t page_size) {
  fa_status_t st = check_tensor(t, name, FA_I32, 2);
  if (st) return st;
  if (t->shape[0] != num_seqs)
    return fail(FA_ERR_INVALID_ARG, "%s has %lld rows, expected num_seqs=%lld", name, (long long)t->shape[0], (long long)num_seqs);
  if (t->stride[1] != 1 && t->shape[1] > 1) return fail(FA_ERR_INVALID_ARG, "%s rows must be contiguous", name);
  if (keys > t->shape[1] * page_size)
    return fail(FA_ERR_INVALID_ARG, "%s holds %lld keys a sequence, %lld are needed", name,
                (long long)(t->shape[1] * page_size), (long long)keys);
  return FA_OK;
}

fa_status_t check_cu(const fa_tensor_t *t, const char *name, int64_t num_seqs) {
  fa_status_t st = check_tensor(t, name, FA_I32, 1);
  if (st) return st;
  if (t->shape[0] != num_seqs + 1 || !contiguous(t))
    return fail(FA_ERR_INVALID_ARG, "%s must be contiguous with num_seqs+1 = %lld entries", name, (long long)(num_seqs + 1));
  if (!t->data) return fail(FA_ERR_INVALID_ARG, "%s data is NULL", name);
  return FA_OK;
}

fa_status_t check_launch(const fa_launch_t *L) {
  if (!L) return fail(FA_ERR_INVALID_ARG, "launch is NULL");
  if (L->num_seqs < 0 || L->max_seqlen_q < 0 || L->max_seqlen_k < 0 || L->total_q < 0 || L->total_k < 0)
    return fail(FA_ERR_INVALID_ARG, "negative size in launch");
  if (L->flags) return fail(FA_ERR_INVALID_ARG, "unknown launch flags 0x%x", L->flags);
  if (L->max_seqlen_k >= kMaxLen || L->max_seqlen_q >= kMaxLen || L->total_q >= (int64_t(1) << 31) ||
      L->total_k >= (int64_t(1) << 31))
    return fail(FA_ERR_OVERFLOW, "lengths must stay below 2^30 a sequence and 2^31 in all");
  if (L->num_seqs > 65535) return fail(FA_ERR_UNSUPPORTED, "at most 65535 sequences");
  return FA_OK;
}

// bf16 query rows [T_q, Hq, D].
fa_status_t check_q(const fa_tensor_t *q, const fa_launch_t *L) {
  fa_status_t st = check_tensor(q, "q", FA_BF16, 3);
  if (st) return st;
  if (q->shape[0] != L->total_q)
    return fail(FA_ERR_INVALID_ARG, "q.shape[0]=%lld != launch.total_q=%lld", (long long)q->shape[0], (long long)L->total_q);
  if (q->stride[2] != 1 || q->stride[1] % 8 || q->stride[0] % 8 || ((uintptr_t)q->data & 15))
    return fail(FA_ERR_INVALID_ARG, "q needs a contiguous last dim, strides that are multiples of 16 bytes and a 16-byte aligned base");
  return FA_OK;
}

fa_status_t check_heads(int64_t hq, int64_t hkv) {
  if (hkv <= 0 || hq <= 0 || hq % hkv)
    return fail(FA_ERR_INVALID_ARG, "Hq=%lld must be a positive multiple of Hkv=%lld", (long long)hq, (long long)hkv);
  if (hkv > 65535) return fail(FA_ERR_UNSUPPORTED, "too many kv heads");
  return FA_OK;
}

// fp32 [num_seqs, Hkv, L] rows with a contiguous last dim, apart from each other.
fa_status_t check_rows3(const fa_tensor_t *t, const char *name, int64_t b, int64_t hkv, bool written) {
  fa_status_t st = check_tensor(t, name, FA_F32, 3);
  if (st) return st;
  if (t->shape[0] != b || t->shape[1] != hkv)
    return fail(FA_ERR_INVALID_ARG, "%s must be [num_seqs=%lld, Hkv=%lld, keys]", name, (long long)b, (long long)hkv);
  if (t->stride[2] != 1 && t->shape[2] > 1) return fail(FA_ERR_INVALID_ARG, "%s needs a contiguous last dim", name);
  if (!t->data && numel(t) > 0) return fail(FA_ERR_INVALID_ARG, "%s data is NULL", name);
  if (written && numel(t) > 0) {
    struct { int64_t n, s; } d[2] = {{b, t->stride[0]}, {hkv, t->stride[1]}};
    if (d[0].s < d[1].s) std::swap(d[0], d[1]);
    int64_t span = t->shape[2];
    for (int i = 1; i >= 0; --i) {
      if (d[i].n <= 1) continue;
      if (d[i].s < span) return fail(FA_ERR_INVALID_ARG, "%s rows overlap each other", name);
      span += (d[i].n - 1) * d[i].s;
    }
  }
  return FA_OK;
}

bool same_view(const fa_tensor_t *a, const fa_tensor_t *b) {
  if (a->data != b->data || a->ndim != b->ndim) return false;
  for (int i = 0; i < a->ndim; ++i)
    if (a->shape[i] != b->shape[i] || (a->shape[i] > 1 && a->stride[i] != b->stride[i])) return false;
  return true;
}

// TMA map over q [T_q, Hq, D] whose boxes hold the `group` heads of a kv head
// for 128 / group tokens, 64 columns at a time: the rows of a tile.
fa_status_t packed_q_map(CUtensorMap *m, const fa_tensor_t *q, int group) {
  const uint64_t dims[3] = {(uint64_t)q->shape[2], (uint64_t)q->shape[1], (uint64_t)q->shape[0]};
  const uint64_t strides[2] = {(uint64_t)(q->stride[1] * 2), (uint64_t)(q->stride[0] * 2)};
  const uint32_t box[3] = {64, (uint32_t)group, (uint32_t)(128 / group)};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q->data, dims, strides, box, "q");
}

// TMA map over a token-major cache for the ring of fa_rows.cuh: boxes of 16 keys
// of one kv head, one block of 128 or 64 bytes wide.
fa_status_t rows_map(CUtensorMap *m, const fa_tensor_t *t, bool paged, const char *what) {
  const int esz = dtype_size(t->dtype), nd = paged ? 4 : 3;
  const int64_t d = t->shape[nd - 1], row = d * esz;
  const bool sw = row % 128 == 0;
  uint64_t dims[4], str[3];
  uint32_t box[4] = {(uint32_t)((sw ? 128 : 64) / esz), 1, 16, 1};
  dims[0] = (uint64_t)d;
  dims[1] = (uint64_t)t->shape[nd - 2];
  dims[2] = (uint64_t)t->shape[nd - 3];
  str[0] = (uint64_t)(t->stride[nd - 2] * esz);
  str[1] = (uint64_t)(t->stride[nd - 3] * esz);
  if (paged) {
    dims[3] = (uint64_t)t->shape[0];
    str[2] = (uint64_t)(t->stride[0] * esz);
  }
  return make_map(m, esz == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, nd, t->data, dims, str, box,
                  what, sw ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE);
}

int32_t clamp_window(int32_t window) { return window <= 0 ? 0 : (int32_t)std::min<int64_t>(window, kMaxLen); }

int kv_code(int dtype) { return dtype == FA_E4M3 ? 1 : (dtype == FA_I8 ? 2 : 0); }

// ------------------------------------------------------- shared prefix --

size_t part_bytes(int64_t splits, int64_t tq, int64_t hq, int64_t dv, size_t *lse_at) {
  const size_t o = align256((size_t)splits * tq * hq * dv * sizeof(float));
  if (lse_at) *lse_at = o;
  return o + align256((size_t)splits * hq * tq * sizeof(float));
}

fa_status_t prefix_build(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *v_cache,
                         const fa_tensor_t *block_table, const fa_tensor_t *cu_seqlens_q,
                         const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale, const fa_tensor_t *v_scale,
                         fa_tensor_t *out, fa_tensor_t *lse, float softmax_scale, int32_t causal, int32_t window,
                         const fa_score_mod_t *score_mod, const fa_shared_prefix_t *prefix, int32_t page_size,
                         const fa_launch_t *launch, fa_fwd_plan_s &P) {
  g_msg[0] = 0;
  fa_status_t st;
  if ((st = check_launch(launch))) return st;
  if (!prefix) return fail(FA_ERR_INVALID_ARG, "prefix is NULL");
  if ((st = check_q(q, launch))) return st;
  if (!block_table) return fail(FA_ERR_UNSUPPORTED, "shared prefixes need a paged cache (block_table)");
  if ((st = check_cache(k_cache, "k_cache", true, page_size)) || (st = check_cache(v_cache, "v_cache", true, page_size)))
    return st;
  const int64_t B = launch->num_seqs, Tq = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t Hkv = k_cache->shape[2], n_pages = k_cache->shape[0];
  for (int i = 0; i < 3; ++i)
    if (v_cache->shape[i] != k_cache->shape[i]) return fail(FA_ERR_INVALID_ARG, "k_cache and v_cache shapes disagree");
  if (v_cache->dtype != k_cache->dtype) return fail(FA_ERR_INVALID_ARG, "k_cache and v_cache types differ");
  if (k_cache->shape[3] != D) return fail(FA_ERR_INVALID_ARG, "k_cache head dim %lld != q head dim %lld", (long long)k_cache->shape[3], (long long)D);
  if (v_cache->shape[3] != D || (D != 64 && D != 128))
    return fail(FA_ERR_UNSUPPORTED, "shared-prefix decode supports Dk = Dv in {64, 128}");
  if ((st = check_heads(Hq, Hkv))) return st;
  if ((st = check_scale(k_scale, "k_scale", k_cache, true)) || (st = check_scale(v_scale, "v_scale", v_cache, true))) return st;
  if ((st = check_table(block_table, "block_table", B, launch->max_seqlen_k, page_size))) return st;
  if ((st = check_cu(cu_seqlens_q, "cu_seqlens_q", B)) || (st = check_cu(cu_seqlens_k, "cu_seqlens_k", B))) return st;
  if ((st = check_tensor(out, "out", FA_BF16, 3))) return st;
  if (out->shape[0] != Tq || out->shape[1] != Hq || out->shape[2] != D || (numel(out) > 0 && !contiguous(out)))
    return fail(FA_ERR_INVALID_ARG, "out must be contiguous [%lld, %lld, %lld]", (long long)Tq, (long long)Hq, (long long)D);
  if ((uintptr_t)out->data & 15) return fail(FA_ERR_INVALID_ARG, "out must be 16-byte aligned");
  if (lse) {
    if ((st = check_tensor(lse, "lse", FA_F32, 2))) return st;
    if (lse->shape[0] != Hq || lse->shape[1] != Tq || (numel(lse) > 0 && !contiguous(lse)))
      return fail(FA_ERR_INVALID_ARG, "lse must be contiguous [Hq=%lld, T_q=%lld]", (long long)Hq, (long long)Tq);
    if (overlaps(lse, out)) return fail(FA_ERR_INVALID_ARG, "lse must not alias out");
  }
  for (const fa_tensor_t *i : {q, k_cache, v_cache})
    if (overlaps(out, i) || (lse && overlaps(lse, i))) return fail(FA_ERR_INVALID_ARG, "out and lse must not alias q/k/v");
  if (!std::isfinite(softmax_scale)) return fail(FA_ERR_INVALID_ARG, "softmax_scale must be finite");
  int mod = 0;
  float slope = 0.f, cap = 0.f;
  if ((st = check_mods(score_mod, nullptr, launch, &mod, &slope, &cap))) return st;
  if (prefix->num_groups < 1 || prefix->max_len < 0 || prefix->num_splits < 1)
    return fail(FA_ERR_INVALID_ARG, "prefix needs num_groups >= 1, max_len >= 0 and num_splits >= 1");
  if (launch->num_splits < 1) return fail(FA_ERR_INVALID_ARG, "launch.num_splits must be at least 1");
  if (prefix->num_splits > 1024 || launch->num_splits > 1024) return fail(FA_ERR_UNSUPPORTED, "at most 1024 splits");
  if (!prefix->cu_groups || !prefix->lens) return fail(FA_ERR_INVALID_ARG, "prefix.cu_groups and prefix.lens are required");
  const int group = (int)(Hq / Hkv);
  if ((int64_t)launch->max_seqlen_q * group > fa::kDecRows)
    return fail(FA_ERR_UNSUPPORTED, "shared-prefix decode needs max_seqlen_q * Hq/Hkv <= %d", fa::kDecRows);
  if (group > fa::kDecRows) return fail(FA_ERR_UNSUPPORTED, "shared-prefix decode needs Hq/Hkv <= %d", fa::kDecRows);
  P.kind = 0;
  if (B == 0 || Tq == 0) return FA_OK;
  if (launch->max_seqlen_q <= 0) return fail(FA_ERR_INVALID_ARG, "max_seqlen_q must be > 0 when total_q > 0");
  if (!q->data || !out->data || !block_table->data) return fail(FA_ERR_INVALID_ARG, "a required data pointer is NULL");
  if (n_pages > 0 && (!k_cache->data || !v_cache->data)) return fail(FA_ERR_INVALID_ARG, "a cache data pointer is NULL");
  const int Sp = prefix->num_splits, Ss = launch->num_splits, S = Sp + Ss;
  size_t lse_at = 0;
  const size_t need = part_bytes(S, Tq, Hq, D, &lse_at);
  if (!launch->workspace || launch->workspace_bytes < need)
    return fail(FA_ERR_INVALID_ARG, "this call needs a workspace of %zu bytes (fa_shared_prefix_workspace_bytes)", need);
  if ((uintptr_t)launch->workspace & 255) return fail(FA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  // CTAs along the rows: one (bf16) or two (byte caches) tiles each, every group
  // with at most one that is not full
  const int64_t cta_tokens = (128 / group) * (k_cache->dtype == FA_BF16 ? 1 : 2);
  const int64_t tiles = (Tq + cta_tokens - 1) / cta_tokens + prefix->num_groups - 1;
  if (tiles > 65535) return fail(FA_ERR_UNSUPPORTED, "too many query tiles (rows / 128 + groups)");
  if (Tq * Hq >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "too many query rows");

  window = clamp_window(window);
  const int esz = dtype_size(k_cache->dtype), kv = kv_code(k_cache->dtype);
  const int D_ = (int)D;
  float *o_part = (float *)launch->workspace, *lse_part = (float *)((char *)launch->workspace + lse_at);
  auto cache_map = [&](CUtensorMap *m, const fa_tensor_t *t, uint32_t cols, int rows, CUtensorMapSwizzle swz, const char *what) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)Hkv, (uint64_t)page_size, (uint64_t)n_pages};
    const uint64_t str[3] = {(uint64_t)(t->stride[2] * esz), (uint64_t)(t->stride[1] * esz), (uint64_t)(t->stride[0] * esz)};
    const uint32_t box[4] = {cols, 1, (uint32_t)rows, 1};
    return make_map(m, kv ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, t->data, dims, str, box, what, swz);
  };
  // (an empty pool has no map: its pages are all out of range, and rows become zeros)
  const bool gather = page_size < 16 || n_pages == 0;
  // ---- the prefix pass
  fa::PrefixLaunch &X = P.px;
  memset(&X, 0, sizeof X);
  if ((st = packed_q_map(&X.tm_q, q, group))) return st;
  const int rows_p = std::min(page_size, kv ? 32 : fa::kBlockN);
  if (n_pages > 0) {
    const CUtensorMapSwizzle swz = kv ? CU_TENSOR_MAP_SWIZZLE_NONE : CU_TENSOR_MAP_SWIZZLE_128B;
    if ((st = cache_map(&X.tm_k, k_cache, 64, rows_p, swz, "prefix k")) || (st = cache_map(&X.tm_v, v_cache, 64, rows_p, swz, "prefix v")))
      return st;
  }
  fa::PrefixParams &p = X.p;
  p.cu_q = (const int32_t *)cu_seqlens_q->data;
  p.cu_k = (const int32_t *)cu_seqlens_k->data;
  p.cu_groups = prefix->cu_groups;
  p.prefix_lens = prefix->lens;
  p.num_groups = prefix->num_groups;
  p.num_seqs = (int)B;
  p.block_table = (const int32_t *)block_table->data;
  p.bt_stride = block_table->stride[0];
  p.max_pages = block_table->shape[1];
  p.n_pages = n_pages;
  p.page_size = page_size;
  p.page_shift = ilog2(page_size);
  p.rows_per_box = rows_p;
  p.gather = gather;
  if (gather) {
    p.gk = kv_gather(k_cache, esz);
    p.gv = kv_gather(v_cache, esz);
  }
  p.k_scale = kv ? (const float *)k_scale->data : nullptr;
  p.v_scale = kv ? (const float *)v_scale->data : nullptr;
  p.total_q = Tq;
  p.hq = (int)Hq;
  p.hkv = (int)Hkv;
  p.group = group;
  p.tokens_per_tile = 128 / group;
  p.num_splits = Sp;
  p.split_tiles = (int)std::max<int64_t>(1, (((int64_t)prefix->max_len + 127) / 128 + Sp - 1) / Sp);
  p.o_part = o_part;
  p.lse_part = lse_part;
  p.causal = causal != 0;
  p.window = window;
  p.scale_log2 = softmax_scale * fa::kLog2e;
  p.alibi_log2 = mod == 1 ? slope * fa::kLog2e : 0.f;
  p.softcap_arg = mod == 2 ? softmax_scale / cap : 0.f;
  p.softcap_log2 = mod == 2 ? cap * fa::kLog2e : 0.f;
  p.err = error_word();
  X.kv = kv;
  // the plain kernel takes the maximum of raw scores: positive scales only
  X.mod = (mod == 0 && !(softmax_scale > 0.f)) ? 1 : mod;
  X.grid = dim3((unsigned)Sp, (unsigned)Hkv, (unsigned)tiles);
  // ---- the sequences' own keys
  fa::SuffixLaunch &L = P.sx;
  memset(&L, 0, sizeof L);
  fa::SuffixParams &d = L.p;
  d.q = (const __nv_bfloat16 *)q->data;
  d.q_stride_t = q->stride[0];
  d.q_stride_h = q->stride[1];
  d.cu_q = p.cu_q;
  d.cu_k = p.cu_k;
  d.cu_groups = p.cu_groups;
  d.prefix_lens = p.prefix_lens;
  d.num_groups = p.num_groups;
  d.block_table = p.block_table;
  d.bt_stride = p.bt_stride;
  d.max_pages = p.max_pages;
  d.n_pages = n_pages;
  d.page_size = page_size;
  d.page_shift = p.page_shift;
  d.small_pages = gather;
  if (!gather && ((st = rows_map(&L.tm_k, k_cache, true, "k rows")) || (st = rows_map(&L.tm_v, v_cache, true, "v rows"))))
    return st;
  d.k = (const uint8_t *)k_cache->data;
  d.v = (const uint8_t *)v_cache->data;
  d.k_page = k_cache->stride[0] * esz;
  d.k_slot = k_cache->stride[1] * esz;
  d.k_head = k_cache->stride[2] * esz;
  d.v_page = v_cache->stride[0] * esz;
  d.v_slot = v_cache->stride[1] * esz;
  d.v_head = v_cache->stride[2] * esz;
  d.k_scale = p.k_scale;
  d.v_scale = p.v_scale;
  d.num_seqs = (int)B;
  d.hq = p.hq;
  d.hkv = p.hkv;
  d.group = group;
  const int64_t own_keys = std::max<int64_t>(launch->max_seqlen_k - (int64_t)prefix->max_len, 1);
  d.split_keys = (int)(((own_keys + Ss - 1) / Ss + 15) / 16 * 16);
  d.num_splits = Ss;
  d.o_part = o_part + (int64_t)Sp * Tq * Hq * D;
  d.lse_part = lse_part + (int64_t)Sp * Hq * Tq;
  d.total_q = Tq;
  d.mod = mod;
  d.causal = p.causal;
  d.window = window;
  d.scale_log2 = p.scale_log2;
  d.alibi_log2 = p.alibi_log2;
  d.softcap_arg = p.softcap_arg;
  d.softcap_log2 = p.softcap_log2;
  d.err = p.err;
  L.kv = kv;
  L.row_tiles = (int64_t)launch->max_seqlen_q * group <= 8 ? 1 : 2;
  const int64_t units = (int64_t)Ss * Hkv * B;
  if (units >= (int64_t(1) << 31)) return fail(FA_ERR_UNSUPPORTED, "too many key ranges (splits * kv heads * sequences)");
  L.grid = dim3((unsigned)((units + fa::kSufWarps - 1) / fa::kSufWarps));
  P.kind = 3;
  P.dk = D_;
  P.splits = S;
  P.rows = Tq;
  P.hq = (int)Hq;
  P.dv = D_;
  P.out = out->data;
  P.lse = lse ? (float *)lse->data : nullptr;
  return FA_OK;
}

// --------------------------------------------------------- key weights --

fa_status_t weights_build(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *block_table,
                          const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                          const fa_tensor_t *lse, const fa_tensor_t *weights, float beta, fa_tensor_t *out,
                          float softmax_scale, int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                          int32_t page_size, const fa_launch_t *launch, fa_fwd_plan_s &P) {
  g_msg[0] = 0;
  fa_status_t st;
  if ((st = check_launch(launch))) return st;
  if ((st = check_q(q, launch))) return st;
  const bool paged = block_table != nullptr;
  if ((st = check_cache(k_cache, "k_cache", paged, page_size))) return st;
  const int nd = paged ? 4 : 3;
  const int64_t B = launch->num_seqs, Tq = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t Hkv = k_cache->shape[nd - 2];
  if (k_cache->shape[nd - 1] != D)
    return fail(FA_ERR_INVALID_ARG, "k_cache head dim %lld != q head dim %lld", (long long)k_cache->shape[nd - 1], (long long)D);
  if ((st = check_heads(Hq, Hkv))) return st;
  const int64_t group = Hq / Hkv;
  if (group > 128) return fail(FA_ERR_UNSUPPORTED, "key weights need Hq/Hkv <= 128");
  if ((st = check_scale(k_scale, "k_scale", k_cache, paged))) return st;
  if (paged && (st = check_table(block_table, "block_table", B, launch->max_seqlen_k, page_size))) return st;
  if (!paged && k_cache->shape[0] < launch->total_k) return fail(FA_ERR_INVALID_ARG, "packed k_cache has fewer rows than total_k");
  if ((st = check_cu(cu_seqlens_q, "cu_seqlens_q", B)) || (st = check_cu(cu_seqlens_k, "cu_seqlens_k", B))) return st;
  if ((st = check_tensor(lse, "lse", FA_F32, 2))) return st;
  if (lse->shape[0] != Hq || lse->shape[1] != Tq || (numel(lse) > 0 && !contiguous(lse)))
    return fail(FA_ERR_INVALID_ARG, "lse must be contiguous [Hq=%lld, T_q=%lld]", (long long)Hq, (long long)Tq);
  if ((st = check_rows3(out, "out", B, Hkv, true))) return st;
  const int64_t extent = out->shape[2];
  if (extent < launch->max_seqlen_k) return fail(FA_ERR_INVALID_ARG, "out holds %lld keys, max_seqlen_k is %d", (long long)extent, launch->max_seqlen_k);
  if (extent >= kMaxLen) return fail(FA_ERR_OVERFLOW, "out rows must stay below 2^30 entries");
  if (!std::isfinite(beta)) return fail(FA_ERR_INVALID_ARG, "beta must be finite");
  bool inplace = false;
  if (weights) {
    if ((st = check_rows3(weights, "weights", B, Hkv, false))) return st;
    if (weights->shape[2] != extent) return fail(FA_ERR_INVALID_ARG, "weights and out must have the same shape");
    inplace = same_view(weights, out);
    if (!inplace && overlaps(weights, out)) return fail(FA_ERR_INVALID_ARG, "out must be weights itself or not overlap it");
  }
  for (const fa_tensor_t *i : {q, k_cache, lse, cu_seqlens_q, cu_seqlens_k})
    if (overlaps(out, i)) return fail(FA_ERR_INVALID_ARG, "out must not alias the inputs");
  if ((k_scale && overlaps(out, k_scale)) || (paged && overlaps(out, block_table)))
    return fail(FA_ERR_INVALID_ARG, "out must not alias the inputs");
  if (!std::isfinite(softmax_scale)) return fail(FA_ERR_INVALID_ARG, "softmax_scale must be finite");
  int mod = 0;
  float slope = 0.f, cap = 0.f;
  if ((st = check_mods(score_mod, nullptr, launch, &mod, &slope, &cap))) return st;
  P.kind = 0;
  if (B == 0 || extent == 0) return FA_OK;
  if (Tq > 0 && (launch->max_seqlen_q <= 0 || !q->data || !lse->data))
    return fail(FA_ERR_INVALID_ARG, "max_seqlen_q must be > 0 and q and lse given when total_q > 0");

  fa::KeyWeightsLaunch &L = P.kw;
  memset(&L, 0, sizeof L);
  fa::KeyWeightsParams &p = L.p;
  const int esz = dtype_size(k_cache->dtype);
  p.q = (const __nv_bfloat16 *)q->data;
  p.q_stride_t = q->stride[0];
  p.q_stride_h = q->stride[1];
  p.cu_q = (const int32_t *)cu_seqlens_q->data;
  p.cu_k = (const int32_t *)cu_seqlens_k->data;
  p.block_table = paged ? (const int32_t *)block_table->data : nullptr;
  p.bt_stride = paged ? block_table->stride[0] : 0;
  p.max_pages = paged ? block_table->shape[1] : 0;
  p.page_size = paged ? page_size : 1;
  p.page_shift = paged ? ilog2(page_size) : 0;
  p.n_pages = k_cache->shape[0];
  p.k = (const uint8_t *)k_cache->data;
  p.s_page = k_cache->stride[0] * esz;
  p.s_slot = paged ? k_cache->stride[1] * esz : 0;
  p.s_head = k_cache->stride[nd - 2] * esz;
  p.k_scale = k_scale ? (const float *)k_scale->data : nullptr;
  p.lse = (const float *)lse->data;
  p.total_q = Tq;
  const bool reads = weights && beta != 0.f;
  p.w_in = reads ? (const float *)weights->data : nullptr;
  p.wi_stride_b = reads ? weights->stride[0] : 0;
  p.wi_stride_h = reads ? weights->stride[1] : 0;
  p.beta = beta;
  p.inplace = inplace && reads && beta == 1.f;
  p.w_out = (float *)out->data;
  p.wo_stride_b = out->stride[0];
  p.wo_stride_h = out->stride[1];
  p.extent = extent;
  p.max_keys = launch->max_seqlen_k;
  p.hq = (int)Hq;
  p.hkv = (int)Hkv;
  p.group = (int)group;
  p.kv = kv_code(k_cache->dtype);
  p.mod = mod;
  p.causal = causal != 0;
  p.window = clamp_window(window);
  p.scale_log2 = softmax_scale * fa::kLog2e;
  p.alibi_log2 = mod == 1 ? slope * fa::kLog2e : 0.f;
  p.softcap_arg = mod == 2 ? softmax_scale / cap : 0.f;
  p.softcap_log2 = mod == 2 ? cap * fa::kLog2e : 0.f;
  p.err = error_word();
  p.tokens_per_tile = (int)(128 / group);
  const int64_t rows = (int64_t)launch->max_seqlen_q * group;
  // keys a launch has to cover: entries past the sequences change unless they are kept as they are
  const int64_t cover = p.inplace ? std::max<int64_t>(launch->max_seqlen_k, 1) : extent;
  if (rows <= fa::kDecRows) {
    L.row_tiles = rows <= 8 ? 1 : 2;
    p.small_pages = (paged && page_size < 16) || p.n_pages == 0;
    if (!p.small_pages && (st = rows_map(&L.tm_k, k_cache, paged, "k rows"))) return st;
    // Key ranges of about twelve waves of CTAs (two per SM) if all sequences
    // had max_seqlen_k keys; ragged batches then make six or so.
    const int64_t per = B * Hkv * (int64_t)launch->max_seqlen_k / (24 * (int64_t)sm_count());
    p.keys_per_cta = (int)std::min<int64_t>(4096, std::max<int64_t>(256, (per + 255) / 256 * 256));
    L.grid = dim3((unsigned)((cover + p.keys_per_cta - 1) / p.keys_per_cta), (unsigned)Hkv, (unsigned)B);
  } else {
    if ((st = packed_q_map(&L.tm_q, q, (int)group))) return st;
    const int64_t tiles = (cover + 127) / 128;
    if (tiles > 65535) return fail(FA_ERR_UNSUPPORTED, "more than 65535 key tiles of 128");
    L.grid = dim3((unsigned)Hkv, (unsigned)B, (unsigned)tiles);
    // the plain tile kernel divides the LSE by the scale
    if (mod == 0 && !(std::fabs(softmax_scale) >= 0x1p-60f)) p.mod = 1;
  }
  P.kind = 4;
  P.dk = (int)D;
  return FA_OK;
}

// ------------------------------------------------------------ eviction --

fa_status_t evict_build(const fa_tensor_t *weights, fa_tensor_t *weights_out, const fa_tensor_t *k_cache,
                        const fa_tensor_t *v_cache, const fa_tensor_t *k_scale, const fa_tensor_t *v_scale,
                        const fa_tensor_t *block_table, const fa_tensor_t *block_table_out,
                        const fa_tensor_t *cu_seqlens_k, fa_tensor_t *cu_seqlens_k_out, fa_tensor_t *kept,
                        int32_t budget, int32_t sink, int32_t recent, int32_t page_size, const fa_launch_t *launch,
                        fa_fwd_plan_s &P) {
  g_msg[0] = 0;
  fa_status_t st;
  if ((st = check_launch(launch))) return st;
  if (!block_table) return fail(FA_ERR_UNSUPPORTED, "eviction needs a paged cache (block_table)");
  if ((st = check_cache(k_cache, "k_cache", true, page_size)) || (st = check_cache(v_cache, "v_cache", true, page_size)))
    return st;
  for (int i = 0; i < 3; ++i)
    if (v_cache->shape[i] != k_cache->shape[i]) return fail(FA_ERR_INVALID_ARG, "k_cache and v_cache shapes disagree");
  if (v_cache->dtype != k_cache->dtype) return fail(FA_ERR_INVALID_ARG, "k_cache and v_cache types differ");
  const int64_t dk = k_cache->shape[3], dv = v_cache->shape[3];
  if (!((dk == 64 && dv == 64) || (dk == 128 && dv == 128) || (dk == 192 && dv == 128)))
    return fail(FA_ERR_UNSUPPORTED, "(Dk, Dv) = (%lld, %lld) is not compiled", (long long)dk, (long long)dv);
  if ((st = check_scale(k_scale, "k_scale", k_cache, true)) || (st = check_scale(v_scale, "v_scale", v_cache, true))) return st;
  const int64_t B = launch->num_seqs, Hkv = k_cache->shape[2];
  if (Hkv > 4096) return fail(FA_ERR_UNSUPPORTED, "too many kv heads");
  if (budget < 1 || sink < 0 || recent < 0 || (int64_t)sink + recent > budget)
    return fail(FA_ERR_INVALID_ARG, "budget %d, sink %d, recent %d: budget >= 1 and sink + recent <= budget", budget, sink, recent);
  if ((st = check_table(block_table, "block_table", B, launch->max_seqlen_k, page_size))) return st;
  const int64_t most = std::min<int64_t>(budget, launch->max_seqlen_k);
  if (block_table_out && (st = check_table(block_table_out, "block_table_out", B, most, page_size))) return st;
  if ((st = check_cu(cu_seqlens_k, "cu_seqlens_k", B)) || (st = check_cu(cu_seqlens_k_out, "cu_seqlens_k_out", B))) return st;
  const bool apart = weights_out && !(weights && same_view(weights, weights_out));
  if ((st = check_rows3(weights, "weights", B, Hkv, !apart))) return st;
  if (weights->shape[2] < launch->max_seqlen_k)
    return fail(FA_ERR_INVALID_ARG, "weights hold %lld keys, max_seqlen_k is %d", (long long)weights->shape[2], launch->max_seqlen_k);
  if (weights->shape[2] >= kMaxLen) return fail(FA_ERR_OVERFLOW, "weights rows must stay below 2^30 entries");
  const fa_tensor_t *wo = apart ? weights_out : weights;
  if (apart) {
    if ((st = check_rows3(weights_out, "weights_out", B, Hkv, true))) return st;
    if (weights_out->shape[2] < most)
      return fail(FA_ERR_INVALID_ARG, "weights_out holds %lld keys, %lld may stay", (long long)weights_out->shape[2], (long long)most);
    if (overlaps(weights, weights_out)) return fail(FA_ERR_INVALID_ARG, "weights_out must be weights itself or not overlap it");
  }
  if ((st = check_tensor(kept, "kept", FA_I32, 3))) return st;
  if (kept->shape[0] != B || kept->shape[1] != Hkv || kept->shape[2] != budget || !contiguous(kept))
    return fail(FA_ERR_INVALID_ARG, "kept must be contiguous [%lld, %lld, %d]", (long long)B, (long long)Hkv, budget);
  const fa_tensor_t *ins[] = {k_cache, v_cache, k_scale, v_scale, block_table, block_table_out, cu_seqlens_k};
  const fa_tensor_t *outs[] = {wo, weights, cu_seqlens_k_out, kept};
  for (const fa_tensor_t *o : outs)
    for (const fa_tensor_t *i : ins)
      if (overlaps(o, i)) return fail(FA_ERR_INVALID_ARG, "the outputs must not overlap the inputs or the cache");
  if (overlaps(kept, cu_seqlens_k_out) || overlaps(kept, wo) || overlaps(cu_seqlens_k_out, wo) || overlaps(kept, weights) ||
      overlaps(cu_seqlens_k_out, weights))
    return fail(FA_ERR_INVALID_ARG, "the outputs must not overlap each other");
  const fa_tensor_t *moved[] = {k_cache, v_cache, k_scale, v_scale};
  const fa_tensor_t *read[] = {block_table, block_table_out, cu_seqlens_k};
  for (int i = 0; i < 4; ++i) {
    for (int j = 0; j < i; ++j) {
      // K and V may be interleaved views of one pool: only the same start is surely wrong
      const bool both_caches = i == 1;
      if (both_caches ? (numel(k_cache) > 0 && k_cache->data == v_cache->data) : overlaps(moved[i], moved[j]))
        return fail(FA_ERR_INVALID_ARG, "caches and scales must not overlap each other");
    }
    for (const fa_tensor_t *r : read)
      if (overlaps(moved[i], r)) return fail(FA_ERR_INVALID_ARG, "the cache must not overlap the tables or lengths");
  }
  fa::EvictParams &p = P.ev.p;
  memset(&P.ev, 0, sizeof P.ev);
  P.kind = 5;
  p.cu_out = (int32_t *)cu_seqlens_k_out->data;
  if (B == 0) return FA_OK;   // its one entry is 0 all the same
  if (!kept->data) return fail(FA_ERR_INVALID_ARG, "kept data is NULL");
  if (launch->max_seqlen_k > 0 && (!k_cache->data || !v_cache->data || !block_table->data))
    return fail(FA_ERR_INVALID_ARG, "a required data pointer is NULL");

  const int esz = dtype_size(k_cache->dtype);
  p.w = (const float *)weights->data;
  p.w_stride_b = weights->stride[0];
  p.w_stride_h = weights->stride[1];
  p.extent_in = weights->shape[2];
  p.w_out = (float *)wo->data;
  p.wo_stride_b = wo->stride[0];
  p.wo_stride_h = wo->stride[1];
  p.extent_out = wo->shape[2];
  p.cu_k = (const int32_t *)cu_seqlens_k->data;
  p.bt = (const int32_t *)block_table->data;
  p.bt_stride = block_table->stride[0];
  p.max_pages = block_table->shape[1];
  if (block_table_out) {
    p.bt_out = (const int32_t *)block_table_out->data;
    p.bto_stride = block_table_out->stride[0];
    p.max_pages_out = block_table_out->shape[1];
  }
  p.n_pages = k_cache->shape[0];
  p.page_size = page_size;
  p.page_shift = ilog2(page_size);
  p.k = (uint8_t *)k_cache->data;
  p.v = (uint8_t *)v_cache->data;
  p.k_page = k_cache->stride[0] * esz;
  p.k_slot = k_cache->stride[1] * esz;
  p.k_head = k_cache->stride[2] * esz;
  p.v_page = v_cache->stride[0] * esz;
  p.v_slot = v_cache->stride[1] * esz;
  p.v_head = v_cache->stride[2] * esz;
  p.k_row = (int32_t)(dk * esz);
  p.v_row = (int32_t)(dv * esz);
  p.k_scale = k_scale ? (float *)k_scale->data : nullptr;
  p.v_scale = v_scale ? (float *)v_scale->data : nullptr;
  p.hkv = (int32_t)Hkv;
  p.num_seqs = (int32_t)B;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.max_keys = launch->max_seqlen_k;
  p.kept = (int32_t *)kept->data;
  p.err = error_word();
  // A row of long weights is shared by the CTAs of a cluster where the rows do
  // not fill the GPU by themselves (two CTAs per SM), as far as a segment fits
  // its shared memory.  Measured (us; 1, 4, 8 CTAs): 12 rows of 30000 weights 30,
  // 19, 21, of 100000 95, -, 28; 384 rows of 30000 67, 99, 264; 32 rows of 8192
  // 12, 14, - .
  const int64_t keys = std::min(p.max_keys, p.extent_in), rows = B * Hkv;
  const auto fits = [&](int64_t ctas) { return rows * ctas <= 2 * sm_count() && keys <= ctas * fa::kEvictSegKeys; };
  P.ev.ctas = keys > 32768 && fits(8) ? 8 : keys > 8192 && fits(4) ? 4 : 1;
  return FA_OK;
}

// Runs `build` into a plan of its own for the caller to keep.
template <typename Build>
fa_status_t make_plan(fa_fwd_plan_t *plan, Build build) {
  if (!plan) return fail(FA_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  fa_fwd_plan_s *P = new (std::nothrow) fa_fwd_plan_s();
  if (!P) return fail(FA_ERR_INVALID_ARG, "out of host memory");
  fa_status_t st = build(*P);
  if (st == FA_OK && cudaGetDevice(&P->device) != cudaSuccess) st = fail(FA_ERR_CUDA, "cudaGetDevice failed");
  if (st != FA_OK) {
    delete P;
    return st;
  }
  *plan = P;
  return FA_OK;
}

fa_status_t enqueue(const fa_fwd_plan_s &P, cudaStream_t s) {
  cudaError_t e = cudaSuccess;
  const char *what = "";
  if (P.kind == 3) {
    fa::PrefixLaunch X = P.px;
    X.stream = s;
    e = fa::launch_prefix(P.dk, X);
    what = "prefix launch";
    if (e == cudaSuccess) {
      fa::SuffixLaunch L = P.sx;
      L.stream = s;
      e = fa::launch_suffix(P.dk, L);
      what = "suffix launch";
    }
    if (e == cudaSuccess) {
      e = fa::launch_prefix_merge(P.dk, P.px.p.o_part, P.px.p.lse_part, P.px.p.cu_q, P.px.p.num_seqs, P.splits, P.rows,
                                  P.hq, P.out, P.lse, s);
      what = "merge launch";
    }
  } else if (P.kind == 4) {
    fa::KeyWeightsLaunch L = P.kw;
    L.stream = s;
    e = fa::launch_key_weights(P.dk, L);
    what = "key-weights launch";
  } else if (P.kind == 5) {
    fa::EvictLaunch L = P.ev;
    L.stream = s;
    e = fa::launch_evict(L);
    what = "eviction launch";
  }
  if (e != cudaSuccess) return cuda_fail(e, what);
  return FA_OK;
}

}  // namespace

namespace fa {
fa_status_t run_serving(const fa_fwd_plan_s &P, cudaStream_t stream) {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(FA_ERR_CUDA, "cudaGetDevice failed");
  if (dev != P.device)
    return fail(FA_ERR_INVALID_ARG, "the plan was made on device %d, device %d is current", P.device, dev);
  return enqueue(P, stream);
}
}  // namespace fa

extern "C" {

size_t fa_shared_prefix_workspace_bytes(const fa_launch_t *launch, const fa_shared_prefix_t *prefix, int32_t hq, int32_t dv) {
  if (!launch || !prefix || launch->total_q <= 0 || hq <= 0 || dv <= 0) return 0;
  if (prefix->num_splits < 1 || launch->num_splits < 1) return 0;
  return part_bytes((int64_t)prefix->num_splits + launch->num_splits, launch->total_q, hq, dv, nullptr);
}

int32_t fa_shared_prefix_default_splits(int64_t total_q, int32_t num_groups, int32_t max_len, int32_t hq, int32_t hkv,
                                        int32_t kv_dtype) {
  if (total_q <= 0 || num_groups <= 0 || hkv <= 0 || hq <= 0 || hq % hkv || max_len <= 0) return 1;
  // One CTA per SM, of 128 rows (bf16) or 256: at most one wave, since a second
  // doubles the time.  Two bf16 CTAs fit an SM, which pays once each has five
  // key tiles.  Measured (us, ranges per prefix): 64 rows of 32 heads behind
  // 8192 keys 54 (6), 50 (9), 48 (12), 49 (19); 34 rows of 12 heads behind 11
  // key tiles 22 (2), 15.6 (6), 18.8 (12).
  const bool bf16 = kv_dtype == FA_BF16;
  const int64_t tokens = std::max(1, 128 / (hq / hkv)) * (bf16 ? 1 : 2);
  const int64_t tiles = std::max<int64_t>((total_q + tokens - 1) / tokens, num_groups) * hkv;
  const int64_t by_keys = ((int64_t)max_len + 127) / 128;
  int64_t n = sm_count() / tiles;
  if (bf16) n = std::max(n, std::min<int64_t>(2 * (int64_t)sm_count() / tiles, by_keys / 5));
  return (int32_t)std::max<int64_t>(1, std::min<int64_t>(std::min(n, by_keys), 64));
}

int32_t fa_shared_prefix_default_own_splits(int32_t num_seqs, int32_t max_own_len, int64_t total_own, int32_t hkv) {
  if (num_seqs <= 0 || hkv <= 0 || max_own_len <= 0) return 1;
  // Ranges for about eight warps per SM (12 or 16 fit), 64 to 512 keys each:
  // short ones balance ragged batches, long ones write fewer partials.
  // Measured (us, ranges per sequence 1, 2, 4, 8, 16): 64 sequences of up to 1024
  // such keys 87, 61, 52, 54, 56; 192 of up to 2048 432, 370, 358, 350, 360.
  const double total = total_own > 0 ? (double)total_own : 0.5 * max_own_len * num_seqs;
  double per = total * hkv / (8.0 * sm_count());
  per = std::min(512.0, std::max(64.0, per));
  return (int32_t)std::min<int64_t>(1024, std::max<int64_t>(1, (int64_t)std::ceil(max_own_len / per)));
}

fa_status_t fa_fwd_shared_prefix(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *v_cache,
                                 const fa_tensor_t *block_table, const fa_tensor_t *cu_seqlens_q,
                                 const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                                 const fa_tensor_t *v_scale, fa_tensor_t *out, fa_tensor_t *lse, float softmax_scale,
                                 int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                                 const fa_shared_prefix_t *prefix, int32_t page_size, const fa_launch_t *launch,
                                 void *stream) {
  fa_fwd_plan_s P;
  const fa_status_t st = prefix_build(q, k_cache, v_cache, block_table, cu_seqlens_q, cu_seqlens_k, k_scale, v_scale, out,
                                      lse, softmax_scale, causal, window, score_mod, prefix, page_size, launch, P);
  return st == FA_OK ? enqueue(P, (cudaStream_t)stream) : st;
}

fa_status_t fa_shared_prefix_plan_create(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *v_cache,
                                         const fa_tensor_t *block_table, const fa_tensor_t *cu_seqlens_q,
                                         const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                                         const fa_tensor_t *v_scale, fa_tensor_t *out, fa_tensor_t *lse,
                                         float softmax_scale, int32_t causal, int32_t window,
                                         const fa_score_mod_t *score_mod, const fa_shared_prefix_t *prefix,
                                         int32_t page_size, const fa_launch_t *launch, fa_fwd_plan_t *plan) {
  return make_plan(plan, [&](fa_fwd_plan_s &P) {
    return prefix_build(q, k_cache, v_cache, block_table, cu_seqlens_q, cu_seqlens_k, k_scale, v_scale, out, lse,
                        softmax_scale, causal, window, score_mod, prefix, page_size, launch, P);
  });
}

fa_status_t fa_key_weights(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *block_table,
                           const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k, const fa_tensor_t *k_scale,
                           const fa_tensor_t *lse, const fa_tensor_t *weights, float beta, fa_tensor_t *out,
                           float softmax_scale, int32_t causal, int32_t window, const fa_score_mod_t *score_mod,
                           int32_t page_size, const fa_launch_t *launch, void *stream) {
  fa_fwd_plan_s P;
  const fa_status_t st = weights_build(q, k_cache, block_table, cu_seqlens_q, cu_seqlens_k, k_scale, lse, weights, beta, out,
                                       softmax_scale, causal, window, score_mod, page_size, launch, P);
  return st == FA_OK ? enqueue(P, (cudaStream_t)stream) : st;
}

fa_status_t fa_key_weights_plan_create(const fa_tensor_t *q, const fa_tensor_t *k_cache, const fa_tensor_t *block_table,
                                       const fa_tensor_t *cu_seqlens_q, const fa_tensor_t *cu_seqlens_k,
                                       const fa_tensor_t *k_scale, const fa_tensor_t *lse, const fa_tensor_t *weights,
                                       float beta, fa_tensor_t *out, float softmax_scale, int32_t causal, int32_t window,
                                       const fa_score_mod_t *score_mod, int32_t page_size, const fa_launch_t *launch,
                                       fa_fwd_plan_t *plan) {
  return make_plan(plan, [&](fa_fwd_plan_s &P) {
    return weights_build(q, k_cache, block_table, cu_seqlens_q, cu_seqlens_k, k_scale, lse, weights, beta, out,
                         softmax_scale, causal, window, score_mod, page_size, launch, P);
  });
}

fa_status_t fa_cache_evict(const fa_tensor_t *weights, fa_tensor_t *weights_out, const fa_tensor_t *k_cache,
                           const fa_tensor_t *v_cache, const fa_tensor_t *k_scale, const fa_tensor_t *v_scale,
                           const fa_tensor_t *block_table, const fa_tensor_t *block_table_out,
                           const fa_tensor_t *cu_seqlens_k, fa_tensor_t *cu_seqlens_k_out, fa_tensor_t *kept,
                           int32_t budget, int32_t sink, int32_t recent, int32_t page_size, const fa_launch_t *launch,
                           void *stream) {
  fa_fwd_plan_s P;
  const fa_status_t st = evict_build(weights, weights_out, k_cache, v_cache, k_scale, v_scale, block_table, block_table_out,
                                     cu_seqlens_k, cu_seqlens_k_out, kept, budget, sink, recent, page_size, launch, P);
  return st == FA_OK ? enqueue(P, (cudaStream_t)stream) : st;
}

}  // extern "C"
