// fa_evict.cuh -- parameters of the cache eviction kernels (fa_evict.cu).
#pragma once
#include <cstdint>

namespace fa {

// Weights that a CTA of a cluster holds in shared memory (two CTAs per SM).
constexpr int kEvictSegKeys = 24 * 1024;

struct EvictParams {
  const float *w;                     // [B, Hkv, extent_in]
  int64_t w_stride_b, w_stride_h, extent_in;
  float *w_out;                       // [B, Hkv, extent_out]; may be w itself
  int64_t wo_stride_b, wo_stride_h, extent_out;
  const int32_t *cu_k;
  int32_t *cu_out;
  const int32_t *bt, *bt_out;         // bt_out null: in place
  int64_t bt_stride, bto_stride, max_pages, max_pages_out, n_pages;
  int32_t page_size, page_shift;
  uint8_t *k, *v;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;   // bytes
  int32_t k_row, v_row;               // bytes of one key's row
  float *k_scale, *v_scale;           // [N_pg, P_s, Hkv] or null
  int32_t hkv, num_seqs;
  int32_t budget, sink, recent;
  int64_t max_keys;                   // the host's bound on a sequence's keys
  int32_t *kept;                      // [B, Hkv, budget]
  int *err;
};

}  // namespace fa
