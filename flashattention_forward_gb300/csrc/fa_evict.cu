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
// sort, and the weights are read once.  Bound by the latency of the passes (a
// barrier, 2048 bins to scan): 384 rows of 8192 weights 24 us, 12 of 100000 28.
//
// Moving (fa_evict_move_kernel, K and V in one launch): 16-byte copies, bound by
// HBM: 2048 rows of 384 (sequence, head)s, bf16, D 128, 114 us or 97% of the
// copy rate.  A lane finds one row's two addresses (two page look-ups) for the
// lanes that copy its pieces; with an address per 16-byte piece it took 168 us.
// In place, the row of rank r
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

constexpr int kBins = 2048;
constexpr int kSelThreads = 512;

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

// Exclusive prefix sum over the block's T threads; `total` gets the sum.
template <int T>
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *warp_sums, uint32_t &total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int NW = T / 32;
  auto warp_scan = [&](uint32_t x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const uint32_t incl = warp_scan(v);
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  const uint32_t sums = warp_scan(lane < NW ? warp_sums[lane] : 0u);
  total = __shfl_sync(0xffffffffu, sums, NW - 1);
  const uint32_t before = __shfl_sync(0xffffffffu, sums, max(warp - 1, 0));
  __syncthreads();
  return (warp ? before : 0u) + incl - v;
}

// Shared memory of the selection besides the cached weights.
struct SelShared {
  uint32_t hist[2][kBins];                          // passes alternate
  uint32_t warp_sums[32];
  uint32_t pick[2];                                 // digit, and what is still to be taken inside it
  uint32_t count;                                   // this CTA's (sure, equal) keys
};

// The new lengths' prefix sums, by one CTA.
template <int T>
__device__ __forceinline__ void evict_lengths(const EvictParams &p, uint32_t *warp_sums) {
  uint32_t run = 0, total;
  for (int base = 0; base < p.num_seqs; base += T) {
    const int x = base + threadIdx.x;
    const uint32_t n = x < p.num_seqs ? (uint32_t)min(evict_keys(p, x), p.budget) : 0u;
    const uint32_t before = block_scan<T>(n, warp_sums, total);
    if (x < p.num_seqs) p.cu_out[x + 1] = (int32_t)(run + before + n);
    run += total;
  }
  if (threadIdx.x == 0) p.cu_out[0] = 0;
}

// One CTA per (sequence, kv head) reads the weights again in every pass (they
// stay in L2) and writes a weight only behind those it has read, so that the
// update in place is safe.  Where such rows are few and long, CTAS CTAs (a
// cluster) share one: each reads a segment into shared memory, before any of
// them writes a weight, and the histograms and counts are read across the
// cluster.
template <int CTAS>
__global__ void __launch_bounds__(kSelThreads) fa_evict_select_kernel(const EvictParams p) {
  constexpr bool CACHED = CTAS > 1;
  constexpr int T = kSelThreads;
  constexpr int ITEMS = 8, CHUNK = T * ITEMS;       // consecutive keys per thread and step of the ordered pass
  extern __shared__ float cache[];
  __shared__ SelShared sh;
  namespace cg = cooperative_groups;
  const int tid = threadIdx.x, part = CTAS > 1 ? (int)(blockIdx.x % CTAS) : 0;
  const int hk = blockIdx.x / CTAS, b = blockIdx.y;
  if (hk == p.hkv) {
    if (b == 0 && part == 0) evict_lengths<T>(p, sh.warp_sums);
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
    for (int j = s0 + tid; j < s1; j += T) cache[j - s0] = w[j];
  }
  auto weight = [&](int j) { return CACHED ? cache[j - s0] : w[j]; };
  // Threshold: competitors above it stay, and of those equal to it the first `need`.
  uint32_t need = cut ? (uint32_t)(p.budget - p.sink - p.recent) : 0u;
  uint32_t thr = 0xFFFFFFFFu;
  for (int i = tid; i < kBins; i += T) sh.hist[0][i] = 0;
  __syncthreads();
  if (need > 0) {
    uint32_t prefix = 0, mask = 0;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : (pass == 1 ? 10 : 0);
      const uint32_t dmask = pass == 2 ? 1023u : 2047u;
      uint32_t *hist = sh.hist[pass & 1];
#pragma unroll 4
      for (int j = lo + tid; j < hi; j += T) {
        const uint32_t u = evict_order(weight(j));
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & dmask], 1u);
      }
      if (CTAS > 1) cg::this_cluster().sync();
      else __syncthreads();
      // bins from the highest: thread t owns B, counted from the top
      constexpr int B = kBins / T;
      uint32_t c[B], mine = 0, total;
      const int top = kBins - B - B * tid;
#pragma unroll
      for (int k = 0; k < B; ++k) c[k] = 0;
#pragma unroll
      for (int x = 0; x < CTAS; ++x) {
        const uint32_t *h = CTAS > 1 ? cg::this_cluster().map_shared_rank(hist, x) : hist;
#pragma unroll
        for (int q = 0; q < B / 4; ++q) {
          const uint4 v = *reinterpret_cast<const uint4 *>(h + top + 4 * q);
          c[B - 1 - 4 * q] += v.x;
          c[B - 2 - 4 * q] += v.y;
          c[B - 3 - 4 * q] += v.z;
          c[B - 4 - 4 * q] += v.w;
        }
      }
#pragma unroll
      for (int k = 0; k < B; ++k) mine += c[k];
      // the other buffer's readers passed the barrier above
      for (int i = tid; i < kBins; i += T) sh.hist[(pass + 1) & 1][i] = 0;
      uint32_t above = block_scan<T>(mine, sh.warp_sums, total);
#pragma unroll
      for (int k = 0; k < B; ++k) {
        if (above < need && need <= above + c[k]) {
          sh.pick[0] = (uint32_t)(top + B - 1 - k);
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
    for (int j = s0 + tid; j < s1; j += T) mine += classify(j, cache[j - s0]);
    block_scan<T>(mine, sh.warp_sums, total);
    if (tid == 0) sh.count = total;
    cg::this_cluster().sync();
    for (int x = 0; x < part; ++x) {
      const uint32_t v = *cg::this_cluster().map_shared_rank(&sh.count, x);
      sure_run += v & 0xFFFFu;
      eq_run += v >> 16;
    }
  }
  // One ordered pass, both counts in the halves of one word (a step has at
  // most CHUNK of each).
  for (int base = s0; base < s1; base += CHUNK) {
    const int j0 = base + tid * ITEMS;
    float wv[ITEMS];
    uint32_t flag[ITEMS], mine = 0;
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
      const int j = j0 + k;
      wv[k] = j < s1 ? weight(j) : 0.f;
      flag[k] = j < s1 ? classify(j, wv[k]) : 0u;
      mine += flag[k];
    }
    uint32_t total;
    const uint32_t before = block_scan<T>(mine, sh.warp_sums, total);   // its barriers also end this step's reads of w
    uint32_t sure = sure_run + (before & 0xFFFFu), eq = eq_run + (before >> 16);
#pragma unroll
    for (int k = 0; k < ITEMS; ++k) {
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
  for (int r = n_keep + part * T + tid; r < p.budget; r += CTAS * T) kept[r] = -1;
  for (int64_t r = n_keep + part * T + tid; r < p.extent_out; r += CTAS * T) wo[r] = 0.f;
  if (CTAS > 1) cg::this_cluster().sync();   // no CTA leaves while another may read its counts
}

template <int CTAS>
cudaError_t select_one(const EvictLaunch &L) {
  auto kern = fa_evict_select_kernel<CTAS>;
  const int64_t keys = std::min(L.p.max_keys, L.p.extent_in);
  const size_t smem = CTAS > 1 ? (size_t)((keys + CTAS - 1) / CTAS + 1) * sizeof(float) : 0;
  if (smem > 30 * 1024) {   // with the static part, past the 48 KB that need no opt-in
    static unsigned long long done = 0;
    cudaError_t e = ensure_smem_attr(kern, (kEvictSegKeys + 1) * (int)sizeof(float), &done);
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
  if (L.ctas == 8) return select_one<8>(L);
  if (L.ctas == 4) return select_one<4>(L);
  return select_one<1>(L);
}

constexpr int kMoveWarps = 8;
constexpr int kMoveRanks = kMoveWarps * 16;         // ranks of a block

__device__ __forceinline__ uint4 ld_row(const uint8_t *a) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a)
               : "memory");
  return v;
}

// One tensor's rows of one (sequence, kv head): P 16-byte pieces of each, from
// byte col0 on.  A warp moves 16 rows at a time: a lane finds one row's two
// addresses, and the lanes side by side copy its pieces.
template <int P, bool INPLACE>
__device__ __forceinline__ void move_rows(const EvictParams &p, uint8_t *cache, float *scale, int64_t s_page,
                                          int64_t s_slot, int64_t s_head, int b, int hk, int col0) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = evict_keys(p, b);
  const int n_keep = min(n, p.budget);
  if (INPLACE && n <= p.budget) return;             // nothing moves
  const int32_t *kept = p.kept + ((int64_t)b * p.hkv + hk) * p.budget;
  const int32_t *bs = p.bt + (int64_t)b * p.bt_stride;
  const int32_t *bd = INPLACE ? bs : p.bt_out + (int64_t)b * p.bto_stride;
  uint8_t *head = cache + (int64_t)hk * s_head + col0;
  const int smask = p.page_size - 1;
  bool bad = false;
  for (int r0 = (INPLACE ? p.sink : (int)blockIdx.x * kMoveRanks); r0 < n_keep;
       r0 += kMoveRanks * (INPLACE ? 1 : gridDim.x)) {
    const int r = r0 + warp * 16 + (lane & 15);
    int j = r < n_keep ? kept[r] : -1;
    if (INPLACE && j == r) j = -1;                  // already there
    const int ps = j >= 0 ? __ldg(bs + (j >> p.page_shift)) : -1, pd = j >= 0 ? __ldg(bd + (r >> p.page_shift)) : -1;
    const bool ok = (unsigned)ps < (unsigned)p.n_pages && (unsigned)pd < (unsigned)p.n_pages;
    bad = bad || (j >= 0 && !ok);
    const bool go = j >= 0 && ok;
    const uint8_t *src = go ? head + (int64_t)ps * s_page + (int64_t)(j & smask) * s_slot : nullptr;
    uint8_t *dst = go ? head + (int64_t)pd * s_page + (int64_t)(r & smask) * s_slot : nullptr;
    uint4 v[P / 2];
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const int e = i * 32 + lane;
      const uint8_t *a = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, (unsigned long long)src, e / P));
      if (a) v[i] = ld_row(a + (e % P) * 16);
    }
    float sv = 0.f;
    if (scale && go && lane < 16) sv = scale[((int64_t)ps * p.page_size + (j & smask)) * p.hkv + hk];
    if (INPLACE) __syncthreads();                   // the block is read: its slots may be written
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const int e = i * 32 + lane;
      uint8_t *a = reinterpret_cast<uint8_t *>(__shfl_sync(0xffffffffu, (unsigned long long)dst, e / P));
      if (a) *reinterpret_cast<uint4 *>(a + (e % P) * 16) = v[i];
    }
    if (scale && go && lane < 16) scale[((int64_t)pd * p.page_size + (r & smask)) * p.hkv + hk] = sv;
  }
  if (bad) record_error(p.err, kErrBounds);
}

// Grid y: (kv head, column slice, K or V).  PK, PV: 16-byte pieces of a K and a
// V row slice; `slices` of them make a K row (a V row has at most as many).
template <int PK, int PV, bool INPLACE>
__global__ void __launch_bounds__(kMoveWarps * 32) fa_evict_move_kernel(const EvictParams p, int slices) {
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
  const int64_t most = std::min<int64_t>(p.budget, p.max_keys);
  const unsigned x = (unsigned)std::max<int64_t>(1, (most + kMoveRanks - 1) / kMoveRanks);
  fa_evict_move_kernel<PK, PV, false><<<dim3(x, 2 * p.hkv, p.num_seqs), kMoveWarps * 32, 0, L.stream>>>(p, 1);
  return cudaGetLastError();
}

cudaError_t launch_move(const EvictLaunch &L) {
  const EvictParams &p = L.p;
  if (!p.bt_out) {
    // In place a CTA walks its ranks alone; slices of 64 bytes make more CTAs.
    const int slices = p.k_row / 64;
    fa_evict_move_kernel<4, 4, true><<<dim3(1, 2 * p.hkv * slices, p.num_seqs), kMoveWarps * 32, 0, L.stream>>>(p, slices);
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
  if (L.p.num_seqs == 0) return cudaMemsetAsync(L.p.cu_out, 0, sizeof(int32_t), L.stream);
  cudaError_t e = launch_select(L);
  return e == cudaSuccess ? launch_move(L) : e;
}

}  // namespace fa
