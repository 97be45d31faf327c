// fa_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// For every (sequence, kv head) of more than `budget` keys: the first `sink`
// and the last `recent` keys stay, and of the others the budget - sink -
// recent with the largest weights (ties: the lowest index; NaN ranks below
// every number).  The keys that stay keep their order and move to slots
// 0 .. budget - 1, so the causal mask's bottom-right alignment and the
// meaning of "recent" hold for the shortened cache.
//
// Selection (fa_evict_select_kernel, one CTA per (sequence, kv head)): the
// weight that divides the kept from the others is found by radix selection on
// the weights' bits -- three histograms of 11, 11 and 10 bits -- and one ordered
// pass then writes the kept indices and moves the weights.  No sort: the
// weights are read four times, after the first time from L2 or L1.
//
// Moving (fa_evict_move_kernel): 16-byte copies.  In place, the row of rank r
// comes from a slot >= r, so a CTA that takes a (sequence, kv head, column
// slice)'s ranks in ascending blocks, reading a whole block before it writes
// it, never overwrites a row that is still to be read; rows of other heads,
// of K and V and of other column slices are disjoint.  Into other pages the
// blocks are independent.
#include <algorithm>

#include "fa_internal.h"

namespace fa {
namespace {

constexpr int kSelThreads = 512;
constexpr int kSelItems = 4;                        // consecutive keys per thread and step
constexpr int kSelChunk = kSelThreads * kSelItems;
constexpr int kBins = 2048;

// The keys of sequence b, held to what the weights and the table cover.
__device__ __forceinline__ int evict_keys(const EvictParams &p, int b) {
  const int sk = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
  const int64_t cap = min(min(p.extent_in, p.max_pages * p.page_size), p.max_keys);
  return (int)min((int64_t)max(sk, 0), cap);
}

// Weight -> unsigned order (NaN lowest, -0 equal to +0).
__device__ __forceinline__ uint32_t evict_order(float w) {
  uint32_t u = __float_as_uint(w);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0u;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive prefix sum over the block's threads; `total` gets the sum.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int NW = kSelThreads / 32;
  uint32_t incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += x;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  uint32_t before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    const uint32_t x = warp_sums[w];
    if (w < warp) before += x;
    total += x;
  }
  __syncthreads();
  return before + incl - v;
}

__global__ void __launch_bounds__(kSelThreads) fa_evict_select_kernel(const EvictParams p) {
  __shared__ uint32_t hist[kBins];
  __shared__ uint32_t warp_sums[kSelThreads / 32];
  __shared__ uint32_t pick[2];                      // digit and what is still to be taken inside it
  const int hk = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  if (hk == p.hkv) {
    // the new lengths' prefix sums
    if (b != 0) return;
    uint32_t run = 0, total;
    for (int base = 0; base < p.num_seqs; base += kSelThreads) {
      const int x = base + tid;
      const uint32_t n = x < p.num_seqs ? (uint32_t)min(evict_keys(p, x), p.budget) : 0u;
      const uint32_t before = block_scan(n, warp_sums, total);
      if (x < p.num_seqs) p.cu_out[x + 1] = (int32_t)(run + before + n);
      run += total;
    }
    if (tid == 0) p.cu_out[0] = 0;
    return;
  }
  const int n = evict_keys(p, b);
  if (tid == 0 && hk == 0 && __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b) != n) record_error(p.err, kErrBounds);
  const float *w = p.w + (int64_t)b * p.w_stride_b + (int64_t)hk * p.w_stride_h;
  float *wo = p.w_out + (int64_t)b * p.wo_stride_b + (int64_t)hk * p.wo_stride_h;
  int32_t *kept = p.kept + ((int64_t)b * p.hkv + hk) * p.budget;
  const int n_keep = min(n, p.budget);
  // Keys of [lo, hi) compete; those outside stay.
  const int lo = n > p.budget ? p.sink : n, hi = n > p.budget ? n - p.recent : n;
  uint32_t need = n > p.budget ? (uint32_t)(p.budget - p.sink - p.recent) : 0u;
  // Threshold: keys above it stay, and of those equal to it the first `need`.
  uint32_t thr = 0xFFFFFFFFu;
  if (need > 0) {
    uint32_t prefix = 0, mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t dmask = pass == 2 ? 1023u : 2047u;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t u = evict_order(w[j]);
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & dmask], 1u);
      }
      __syncthreads();
      // bins from the highest: thread t owns four, counted from the top
      uint32_t c[4], mine = 0, total;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        c[k] = hist[kBins - 1 - (4 * tid + k)];
        mine += c[k];
      }
      uint32_t above = block_scan(mine, warp_sums, total);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < need && need <= above + c[k]) {
          pick[0] = (uint32_t)(kBins - 1 - (4 * tid + k));
          pick[1] = need - above;
        }
        above += c[k];
      }
      __syncthreads();
      prefix |= pick[0] << shift;
      mask |= dmask << shift;
      need = pick[1];
      __syncthreads();
    }
    thr = prefix;
  }
  // One ordered pass: (sure to stay, equal to the threshold) counted together
  // in the halves of one word (a step has at most kSelChunk of each).
  uint32_t sure_run = 0, eq_run = 0;
  for (int base = 0; base < n; base += kSelChunk) {
    const int j0 = base + tid * kSelItems;
    float wv[kSelItems];
    uint32_t flag[kSelItems], mine = 0;
#pragma unroll
    for (int k = 0; k < kSelItems; ++k) {
      const int j = j0 + k;
      flag[k] = 0;
      wv[k] = 0.f;
      if (j < n) {
        wv[k] = w[j];
        const uint32_t u = evict_order(wv[k]);
        if (j < lo || j >= hi || u > thr) flag[k] = 1u;
        else if (u == thr) flag[k] = 0x10000u;
      }
      mine += flag[k];
    }
    uint32_t total;
    const uint32_t before = block_scan(mine, warp_sums, total);   // its barriers also end this step's reads of w
    uint32_t sure = sure_run + (before & 0xFFFFu), eq = eq_run + (before >> 16);
#pragma unroll
    for (int k = 0; k < kSelItems; ++k) {
      const bool take = flag[k] == 1u || (flag[k] == 0x10000u && eq < need);
      if (take) {
        const uint32_t rank = sure + min(eq, need);
        if (rank < (uint32_t)n_keep) {
          kept[rank] = j0 + k;
          wo[rank] = wv[k];
        }
      }
      sure += flag[k] & 0xFFFFu;
      eq += flag[k] >> 16;
    }
    sure_run += total & 0xFFFFu;
    eq_run += total >> 16;
  }
  __syncthreads();
  for (int r = n_keep + tid; r < p.budget; r += kSelThreads) kept[r] = -1;
  for (int64_t r = n_keep + tid; r < p.extent_out; r += kSelThreads) wo[r] = 0.f;
}

constexpr int kMoveThreads = 256;
constexpr int kMoveItems = 8;                       // 16-byte pieces per thread and block of ranks

// P: 16-byte pieces of a row slice.  A block is ROWS ranks.
template <int P, bool INPLACE>
__global__ void __launch_bounds__(kMoveThreads) fa_evict_move_kernel(const EvictParams p, int slices, int is_v) {
  constexpr int ROWS = kMoveThreads * kMoveItems / P;
  const int slice = blockIdx.y % slices, hk = blockIdx.y / slices, b = blockIdx.z;
  const int n = evict_keys(p, b);
  const int n_keep = min(n, p.budget);
  if (INPLACE && n <= p.budget) return;             // nothing moves
  const int32_t *kept = p.kept + ((int64_t)b * p.hkv + hk) * p.budget;
  const int32_t *bs = p.bt + (int64_t)b * p.bt_stride;
  const int32_t *bd = INPLACE ? bs : p.bt_out + (int64_t)b * p.bto_stride;
  uint8_t *cache = is_v ? p.v : p.k;
  float *scale = is_v ? p.v_scale : p.k_scale;
  const int64_t s_page = is_v ? p.v_page : p.k_page, s_slot = is_v ? p.v_slot : p.k_slot;
  uint8_t *head = cache + (int64_t)hk * (is_v ? p.v_head : p.k_head) + slice * (P * 16);
  auto page_of = [&](const int32_t *t, int64_t cap, int j) -> int {
    const int64_t i = j >> p.page_shift;
    const int pg = i < cap ? __ldg(t + i) : -1;
    if (pg < 0 || pg >= p.n_pages) {
      record_error(p.err, kErrBounds);
      return -1;
    }
    return pg;
  };
  const int64_t cap_d = INPLACE ? p.max_pages : p.max_pages_out;
  for (int r0 = (INPLACE ? p.sink : (int)blockIdx.x * ROWS); r0 < n_keep; r0 += ROWS * (INPLACE ? 1 : gridDim.x)) {
    uint4 v[kMoveItems];
    uint8_t *dst[kMoveItems];
#pragma unroll
    for (int i = 0; i < kMoveItems; ++i) {
      const int e = threadIdx.x + i * kMoveThreads, rr = e / P, r = r0 + rr;
      dst[i] = nullptr;
      if (rr < ROWS && r < n_keep) {
        const int j = kept[r];
        if (!INPLACE || j != r) {
          const int ps = page_of(bs, p.max_pages, j), pd = page_of(bd, cap_d, r);
          if (ps >= 0 && pd >= 0) {
            const int piece = (e % P) * 16;
            v[i] = *reinterpret_cast<const uint4 *>(head + (int64_t)ps * s_page + (int64_t)(j & (p.page_size - 1)) * s_slot +
                                                    piece);
            dst[i] = head + (int64_t)pd * s_page + (int64_t)(r & (p.page_size - 1)) * s_slot + piece;
          }
        }
      }
    }
    // scales of the block's ranks, by the first slice
    constexpr int NSC = (ROWS + kMoveThreads - 1) / kMoveThreads;
    float sv[NSC];
    float *sd[NSC];
#pragma unroll
    for (int i = 0; i < NSC; ++i) {
      const int rr = threadIdx.x + i * kMoveThreads, r = r0 + rr;
      sd[i] = nullptr;
      if (scale && slice == 0 && rr < ROWS && r < n_keep) {
        const int j = kept[r];
        if (!INPLACE || j != r) {
          const int ps = page_of(bs, p.max_pages, j), pd = page_of(bd, cap_d, r);
          if (ps >= 0 && pd >= 0) {
            sv[i] = scale[((int64_t)ps * p.page_size + (j & (p.page_size - 1))) * p.hkv + hk];
            sd[i] = scale + ((int64_t)pd * p.page_size + (r & (p.page_size - 1))) * p.hkv + hk;
          }
        }
      }
    }
    if (INPLACE) __syncthreads();                   // the block is read: its slots may be written
#pragma unroll
    for (int i = 0; i < kMoveItems; ++i)
      if (dst[i]) *reinterpret_cast<uint4 *>(dst[i]) = v[i];
#pragma unroll
    for (int i = 0; i < NSC; ++i)
      if (sd[i]) *sd[i] = sv[i];
  }
}

template <int P>
cudaError_t move_p(const EvictLaunch &L, int slices, int is_v) {
  const EvictParams &p = L.p;
  constexpr int ROWS = kMoveThreads * kMoveItems / P;
  const unsigned y = (unsigned)(slices * p.hkv), z = (unsigned)p.num_seqs;
  if (p.bt_out) {
    const unsigned x = (unsigned)std::max<int64_t>(1, (std::min<int64_t>(p.budget, p.max_keys) + ROWS - 1) / ROWS);
    fa_evict_move_kernel<P, false><<<dim3(x, y, z), kMoveThreads, 0, L.stream>>>(p, slices, is_v);
  } else {
    fa_evict_move_kernel<P, true><<<dim3(1, y, z), kMoveThreads, 0, L.stream>>>(p, slices, is_v);
  }
  return cudaGetLastError();
}

cudaError_t move_rows(const EvictLaunch &L, int is_v) {
  const int pieces = (is_v ? L.p.v_row : L.p.k_row) / 16;   // 4, 8, 12, 16 or 24
  switch (pieces) {
    case 4: return move_p<4>(L, 1, is_v);
    case 8: return move_p<8>(L, 1, is_v);
    case 12: return move_p<12>(L, 1, is_v);
    case 16: return move_p<16>(L, 1, is_v);
    case 24: return move_p<24>(L, 1, is_v);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch &L) {
  fa_evict_select_kernel<<<dim3((unsigned)L.p.hkv + 1, (unsigned)L.p.num_seqs), kSelThreads, 0, L.stream>>>(L.p);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = move_rows(L, 0);
  if (e == cudaSuccess) e = move_rows(L, 1);
  return e;
}

}  // namespace fa
