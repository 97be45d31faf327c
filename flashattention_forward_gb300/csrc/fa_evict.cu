// fa_evict.cu -- eviction from a paged cache by accumulated attention weight.
//
// For every (sequence, kv head) of more than `budget` keys: the first `sink`
// and the last `recent` keys stay, and of the others the budget - sink -
// recent with the largest weights (ties: the lowest index; NaN ranks below
// every number).  The keys that stay keep their order and move to slots
// 0 .. budget - 1, so the causal mask's bottom-right alignment and the
// meaning of "recent" hold for the shortened cache.
//
// Selection (fa_evict_select_kernel, one CTA or cluster per (sequence, kv
// head)): the weight that divides the kept from the others is found by radix
// selection on the weights' bits -- three histograms of 11, 11 and 10 bits --
// and one ordered pass then writes the kept indices and moves the weights.  No
// sort, and the weights are read once.
//
// Moving (fa_evict_move_kernel, K and V in one launch): 16-byte copies.  In place, the row of rank r
// comes from a slot >= r, so a CTA that takes a (sequence, kv head, column
// slice)'s ranks in ascending blocks, reading a whole block before it writes
// it, never overwrites a row that is still to be read; rows of other heads,
// of K and V and of other column slices are disjoint.  Into other pages the
// blocks are independent.
#include <cooperative_groups.h>

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

// Shared memory of the selection besides the cached weights.
struct SelShared {
  uint32_t hist[2][kBins];                          // passes alternate
  uint32_t warp_sums[kSelThreads / 32];
  uint32_t pick[2];                                 // digit, and what is still to be taken inside it
  uint32_t count;                                   // this CTA's (sure, equal) keys
};

// The new lengths' prefix sums, by one CTA.
__device__ __forceinline__ void evict_lengths(const EvictParams &p, uint32_t *warp_sums) {
  uint32_t run = 0, total;
  for (int base = 0; base < p.num_seqs; base += kSelThreads) {
    const int x = base + threadIdx.x;
    const uint32_t n = x < p.num_seqs ? (uint32_t)min(evict_keys(p, x), p.budget) : 0u;
    const uint32_t before = block_scan(n, warp_sums, total);
    if (x < p.num_seqs) p.cu_out[x + 1] = (int32_t)(run + before + n);
    run += total;
  }
  if (threadIdx.x == 0) p.cu_out[0] = 0;
}

// CTAS CTAs (a cluster) share one (sequence, kv head): each takes a segment of
// the weights, and the histograms and counts are read across the cluster.
// CACHED: the segment is read once into shared memory, before any CTA writes a
// weight, so that the update in place is safe.  Rows too long for that take
// one CTA that reads the weights again in every pass; it writes a weight only
// behind those it has read.
template <int CTAS, bool CACHED>
__global__ void __launch_bounds__(kSelThreads) fa_evict_select_kernel(const EvictParams p) {
  static_assert(CACHED || CTAS == 1, "only cached segments are shared out");
  extern __shared__ float cache[];
  __shared__ SelShared sh;
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x, part = CTAS > 1 ? (int)(blockIdx.x % CTAS) : 0;
  const int hk = blockIdx.x / CTAS, b = blockIdx.y;
  if (hk == p.hkv) {
    if (b == 0 && part == 0) evict_lengths(p, sh.warp_sums);
    return;
  }
  const int n = evict_keys(p, b);
  if (tid == 0 && hk == 0 && part == 0 && __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b) != n) record_error(p.err, kErrBounds);
  const float *w = p.w + (int64_t)b * p.w_stride_b + (int64_t)hk * p.w_stride_h;
  float *wo = p.w_out + (int64_t)b * p.wo_stride_b + (int64_t)hk * p.wo_stride_h;
  int32_t *kept = p.kept + ((int64_t)b * p.hkv + hk) * p.budget;
  const int n_keep = min(n, p.budget);
  // this CTA's keys [s0, s1), and of them those that compete, [lo, hi)
  const int seg = (n + CTAS - 1) / CTAS, s0 = min(n, part * seg), s1 = min(n, s0 + seg);
  const bool cut = n > p.budget;
  const int lo = cut ? max(s0, p.sink) : s1, hi = cut ? min(s1, n - p.recent) : s1;
  if (CACHED) {
#pragma unroll 8
    for (int j = s0 + tid; j < s1; j += kSelThreads) cache[j - s0] = w[j];
  }
  auto weight = [&](int j) { return CACHED ? cache[j - s0] : w[j]; };
  // Threshold: competitors above it stay, and of those equal to it the first `need`.
  uint32_t need = cut ? (uint32_t)(p.budget - p.sink - p.recent) : 0u;
  uint32_t thr = 0xFFFFFFFFu;
  for (int i = tid; i < kBins; i += kSelThreads) sh.hist[0][i] = 0;
  __syncthreads();
  if (need > 0) {
    uint32_t prefix = 0, mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t dmask = pass == 2 ? 1023u : 2047u;
      uint32_t *hist = sh.hist[pass & 1];
#pragma unroll 4
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t u = evict_order(weight(j));
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & dmask], 1u);
      }
      if (CTAS > 1) cg::this_cluster().sync();
      else __syncthreads();
      // bins from the highest: thread t owns four, counted from the top
      uint32_t c[4] = {0, 0, 0, 0}, mine, total;
      const int top = kBins - 4 - 4 * tid;
#pragma unroll
      for (int x = 0; x < CTAS; ++x) {
        const uint32_t *h = CTAS > 1 ? cg::this_cluster().map_shared_rank(hist, x) : hist;
        const uint4 v = *reinterpret_cast<const uint4 *>(h + top);
        c[0] += v.w;
        c[1] += v.z;
        c[2] += v.y;
        c[3] += v.x;
      }
      mine = c[0] + c[1] + c[2] + c[3];
      // the other buffer's readers passed the barrier above
      for (int i = tid; i < kBins; i += kSelThreads) sh.hist[(pass + 1) & 1][i] = 0;
      uint32_t above = block_scan(mine, sh.warp_sums, total);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < need && need <= above + c[k]) {
          sh.pick[0] = (uint32_t)(top + 3 - k);
          sh.pick[1] = need - above;
        }
        above += c[k];
      }
      __syncthreads();
      prefix |= sh.pick[0] << shift;
      mask |= dmask << shift;
      need = sh.pick[1];
      __syncthreads();
    }
    thr = prefix;
  }
  // (sure to stay, equal to the threshold) of a key
  auto classify = [&](int j, float x) -> uint32_t {
    if (j < lo || j >= hi) return 1u;
    const uint32_t u = evict_order(x);
    return u > thr ? 1u : (u == thr ? 0x10000u : 0u);
  };
  uint32_t sure_run = 0, eq_run = 0;
  if (CTAS > 1) {
    // what the segments before this one hold (a segment has at most 32767 keys)
    uint32_t mine = 0, total;
    for (int j = s0 + tid; j < s1; j += kSelThreads) mine += classify(j, cache[j - s0]);
    block_scan(mine, sh.warp_sums, total);
    if (tid == 0) sh.count = total;
    cg::this_cluster().sync();
    for (int x = 0; x < part; ++x) {
      const uint32_t v = *cg::this_cluster().map_shared_rank(&sh.count, x);
      sure_run += v & 0xFFFFu;
      eq_run += v >> 16;
    }
  }
  // One ordered pass, both counts in the halves of one word (a step has at
  // most kSelChunk of each).
  for (int base = s0; base < s1; base += kSelChunk) {
    const int j0 = base + tid * kSelItems;
    float wv[kSelItems];
    uint32_t flag[kSelItems], mine = 0;
#pragma unroll
    for (int k = 0; k < kSelItems; ++k) {
      const int j = j0 + k;
      wv[k] = j < s1 ? weight(j) : 0.f;
      flag[k] = j < s1 ? classify(j, wv[k]) : 0u;
      mine += flag[k];
    }
    uint32_t total;
    const uint32_t before = block_scan(mine, sh.warp_sums, total);   // its barriers also end this step's reads of w
    uint32_t sure = sure_run + (before & 0xFFFFu), eq = eq_run + (before >> 16);
#pragma unroll
    for (int k = 0; k < kSelItems; ++k) {
      if (flag[k] == 1u || (flag[k] == 0x10000u && eq < need)) {
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
  // the rest of the rows, once every weight is read
  if (!CACHED) __syncthreads();
  for (int r = n_keep + part * kSelThreads + tid; r < p.budget; r += CTAS * kSelThreads) kept[r] = -1;
  for (int64_t r = n_keep + part * kSelThreads + tid; r < p.extent_out; r += CTAS * kSelThreads) wo[r] = 0.f;
  if (CTAS > 1) cg::this_cluster().sync();   // no CTA leaves while another may read its counts
}

// Cached segments: up to this many keys per CTA (two CTAs per SM), and up to
// eight CTAs; beyond, the row streams through one CTA.
constexpr int kSegKeys = 24 * 1024;
// A CTA takes a row alone up to this many keys (measured: see launch_select).
constexpr int kAloneKeys = 4096;

template <int CTAS, bool CACHED>
cudaError_t select_one(const EvictLaunch &L, int64_t keys) {
  auto kern = fa_evict_select_kernel<CTAS, CACHED>;
  const size_t smem = CACHED ? (size_t)((keys + CTAS - 1) / CTAS + 1) * sizeof(float) : 0;
  if (smem > 30 * 1024) {   // with the static part, past the 48 KB that need no opt-in
    static unsigned long long done = 0;
    cudaError_t e = ensure_smem_attr(kern, (kSegKeys + 1) * (int)sizeof(float), &done);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((L.p.hkv + 1) * CTAS), (unsigned)L.p.num_seqs);
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = L.stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = CTAS;
  at[0].val.clusterDim.y = 1;
  at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = CTAS > 1 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, L.p);
}

cudaError_t launch_select(const EvictLaunch &L) {
  const int64_t keys = std::min(L.p.max_keys, L.p.extent_in);
  if (keys > 8 * (int64_t)kSegKeys) return select_one<1, false>(L, keys);
  if (keys > 4 * kAloneKeys) return select_one<8, true>(L, keys);
  if (keys > 2 * kAloneKeys) return select_one<4, true>(L, keys);
  if (keys > kAloneKeys) return select_one<2, true>(L, keys);
  return select_one<1, true>(L, keys);
}

constexpr int kMoveThreads = 256;
constexpr int kMoveItems = 8;                       // 16-byte pieces per thread and block of ranks

__device__ __forceinline__ uint4 ld_row(const uint8_t *a) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a)
               : "memory");
  return v;
}

// One tensor's rows of one (sequence, kv head): P 16-byte pieces of each, from
// byte col0 on; a block is ROWS ranks.  Indices, then pages, then data: the
// reads of a block are in flight together.
template <int P, bool INPLACE>
__device__ __forceinline__ void move_rows(const EvictParams &p, uint8_t *cache, float *scale, int64_t s_page,
                                          int64_t s_slot, int64_t s_head, int b, int hk, int col0) {
  constexpr int ROWS = kMoveThreads * kMoveItems / P;
  const int n = evict_keys(p, b);
  const int n_keep = min(n, p.budget);
  if (INPLACE && n <= p.budget) return;             // nothing moves
  const int32_t *kept = p.kept + ((int64_t)b * p.hkv + hk) * p.budget;
  const int32_t *bs = p.bt + (int64_t)b * p.bt_stride;
  const int32_t *bd = INPLACE ? bs : p.bt_out + (int64_t)b * p.bto_stride;
  uint8_t *head = cache + (int64_t)hk * s_head + col0;
  const int smask = p.page_size - 1;
  bool bad = false;
  for (int r0 = (INPLACE ? p.sink : (int)blockIdx.x * ROWS); r0 < n_keep; r0 += ROWS * (INPLACE ? 1 : gridDim.x)) {
    int j[kMoveItems], ps[kMoveItems], pd[kMoveItems];
    uint4 v[kMoveItems];
#pragma unroll
    for (int i = 0; i < kMoveItems; ++i) {
      const int rr = (threadIdx.x + i * kMoveThreads) / P, r = r0 + rr;
      j[i] = rr < ROWS && r < n_keep ? kept[r] : -1;
      if (INPLACE && j[i] == r) j[i] = -1;          // already there
    }
#pragma unroll
    for (int i = 0; i < kMoveItems; ++i) {
      const int r = r0 + (threadIdx.x + i * kMoveThreads) / P;
      ps[i] = pd[i] = -1;
      if (j[i] >= 0) {
        ps[i] = __ldg(bs + (j[i] >> p.page_shift));
        pd[i] = __ldg(bd + (r >> p.page_shift));
      }
    }
#pragma unroll
    for (int i = 0; i < kMoveItems; ++i) {
      const bool ok = (unsigned)ps[i] < (unsigned)p.n_pages && (unsigned)pd[i] < (unsigned)p.n_pages;
      bad = bad || (j[i] >= 0 && !ok);
      if (!ok) j[i] = -1;
      const int piece = ((threadIdx.x + i * kMoveThreads) % P) * 16;
      if (j[i] >= 0) v[i] = ld_row(head + (int64_t)ps[i] * s_page + (int64_t)(j[i] & smask) * s_slot + piece);
    }
    // the scales of the block's ranks go with a row's first piece
    float sv[kMoveItems];
    if (scale) {
#pragma unroll
      for (int i = 0; i < kMoveItems; ++i)
        if (j[i] >= 0 && (threadIdx.x + i * kMoveThreads) % P == 0)
          sv[i] = scale[((int64_t)ps[i] * p.page_size + (j[i] & smask)) * p.hkv + hk];
    }
    if (INPLACE) __syncthreads();                   // the block is read: its slots may be written
#pragma unroll
    for (int i = 0; i < kMoveItems; ++i) {
      const int e = threadIdx.x + i * kMoveThreads, r = r0 + e / P;
      if (j[i] < 0) continue;
      *reinterpret_cast<uint4 *>(head + (int64_t)pd[i] * s_page + (int64_t)(r & smask) * s_slot + (e % P) * 16) = v[i];
      if (scale && e % P == 0) scale[((int64_t)pd[i] * p.page_size + (r & smask)) * p.hkv + hk] = sv[i];
    }
  }
  if (bad) record_error(p.err, kErrBounds);
}

// Grid y: (kv head, column slice, K or V).  PK, PV: 16-byte pieces of a K and a
// V row slice; `slices` of them make a K row (a V row has at most as many).
template <int PK, int PV, bool INPLACE>
__global__ void __launch_bounds__(kMoveThreads) fa_evict_move_kernel(const EvictParams p, int slices) {
  const int is_v = blockIdx.y & 1, slice = (blockIdx.y >> 1) % slices, hk = (blockIdx.y >> 1) / slices, b = blockIdx.z;
  if (is_v) {
    if (slice * PV * 16 >= p.v_row) return;
    move_rows<PV, INPLACE>(p, p.v, slice == 0 ? p.v_scale : nullptr, p.v_page, p.v_slot, p.v_head, b, hk, slice * PV * 16);
  } else {
    move_rows<PK, INPLACE>(p, p.k, slice == 0 ? p.k_scale : nullptr, p.k_page, p.k_slot, p.k_head, b, hk, slice * PK * 16);
  }
}

template <int PK, int PV>
cudaError_t move_apart(const EvictLaunch &L) {
  const EvictParams &p = L.p;
  constexpr int ROWS = kMoveThreads * kMoveItems / (PK > PV ? PK : PV);
  const int64_t most = std::min<int64_t>(p.budget, p.max_keys);
  const unsigned x = (unsigned)std::max<int64_t>(1, (most + ROWS - 1) / ROWS);
  fa_evict_move_kernel<PK, PV, false><<<dim3(x, 2 * p.hkv, p.num_seqs), kMoveThreads, 0, L.stream>>>(p, 1);
  return cudaGetLastError();
}

cudaError_t launch_move(const EvictLaunch &L) {
  const EvictParams &p = L.p;
  if (!p.bt_out) {
    // In place a CTA walks its ranks alone; slices of 64 bytes make more CTAs.
    const int slices = p.k_row / 64;
    fa_evict_move_kernel<4, 4, true><<<dim3(1, 2 * p.hkv * slices, p.num_seqs), kMoveThreads, 0, L.stream>>>(p, slices);
    return cudaGetLastError();
  }
  switch (p.k_row) {
    case 64: return move_apart<4, 4>(L);
    case 128: return move_apart<8, 8>(L);
    case 192: return move_apart<12, 8>(L);
    case 256: return move_apart<16, 16>(L);
    case 384: return move_apart<24, 16>(L);
    default: return cudaErrorNotSupported;
  }
}

}  // namespace

cudaError_t launch_evict(const EvictLaunch &L) {
  cudaError_t e = launch_select(L);
  return e == cudaSuccess ? launch_move(L) : e;
}

}  // namespace fa
