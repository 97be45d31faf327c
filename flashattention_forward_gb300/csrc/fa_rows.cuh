// fa_rows.cuh -- few query rows against cached keys that a warp streams through
// a ring of its own into MMA fragments (mma.sync as a dense FMA engine; the
// bound is HBM, and tcgen05's 128 rows would stand empty): what the rows form of the key weights (fa_key_weights.cuh) and the decode behind a shared
// prefix (fa_suffix.cuh) have in common.
//
// S^T = K Q^T with M = 16 keys, N = 8 query rows.  The contraction index is
// permuted: lane (g, t) = (lane / 4, lane % 4) holds the 16-byte pieces t, t + 4,
// ... of key rows g and g + 8 (A) and of query row g (B); each piece is two
// k-steps of bf16 or four of bytes.  The permutation is the same on both sides,
// so the sum is the product, and no ldmatrix is needed.
//
// The rows wait in shared memory, a few groups of 16 keys ahead, in a ring of
// the warp that uses them: pages of 16 or more keys (and packed keys) land as
// TMA boxes of 16 rows, smaller pages row by row with cp.async.  Measured over
// 64 sequences of 8192 keys (bf16, D = 128): whatever passes through the SM's
// load path (loads into registers, cp.async of fragment pieces or of whole
// rows) stops at 4.4 TB/s, and one cp.async.bulk per row at 3.4 TB/s, as an SM
// starts one only about every 23 cycles; the boxes reach 6.2 - 6.5 TB/s (5.1 at
// D = 64, where a box holds 2 KB, and 3.9 over int8, bound by the conversion).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_decode.cuh"
#include "sm103_ptx.cuh"

namespace fa {

__device__ __forceinline__ uint4 rows_ld_stream(const uint8_t *a) {
  uint4 v;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(a));
  return v;
}

__device__ __forceinline__ uint4 rows_lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ uint2 rows_lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ float rows_lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}
// 16 rows of ROW bytes in a ring slot: blocks of 128-byte columns, 128-byte
// swizzled, where the row is a multiple of that, else of 64-byte columns.
template <int ROW>
struct RowsBlocks {
  static constexpr bool kSw = ROW % 128 == 0;
  static constexpr int kCols = kSw ? 128 : 64;   // bytes
  static constexpr int NB = ROW / kCols;
  static constexpr int kBytes = 16 * ROW;
  // 16-byte piece p of row r
  static __device__ __forceinline__ uint32_t at(int p, int r) {
    if constexpr (kSw) return (uint32_t)((p >> 3) * 2048 + r * 128 + (((p ^ r) & 7) << 4));
    else return (uint32_t)((p >> 2) * 1024 + r * 64 + ((p & 3) << 4));
  }
  // The row (of 8) that stands at index i of a fragment.  A quarter warp reads
  // four pieces of the key rows of two lanes g, g + 1, and two pieces of the
  // value rows of four lanes' index 2t (or 2t + 1): with the swizzle this order
  // puts either in eight different chunks.
  static __device__ __forceinline__ int row(int i) { return kSw ? (0x37156240 >> (4 * i)) & 7 : i; }
};

// One warp's ring of S slots, each 16 key rows, 16 value rows (VROW 0: none)
// and, for byte caches, their scales.  All calls are warp-wide.
template <int KROW, int VROW, bool SCALES, int S>
struct RowsRing {
  using K = RowsBlocks<KROW>;
  using V = RowsBlocks<VROW ? VROW : 64>;
  static constexpr int kOffV = K::kBytes;
  static constexpr int kSlot = K::kBytes + (VROW ? V::kBytes : 0);   // multiples of 1024
  static constexpr int kOffScale = S * kSlot, kOffBar = kOffScale + (SCALES ? S * 128 : 0);
  static constexpr int kBytes = (kOffBar + S * 8 + 8 + 1023) / 1024 * 1024;
  static_assert(kSlot % 1024 == 0, "swizzle atoms");

  uint32_t base;
  volatile int *abort_flag;
  int use, fill;
  uint32_t phase;

  __device__ __forceinline__ void init(uint8_t *mem) {
    base = smem_u32(mem);
    abort_flag = reinterpret_cast<volatile int *>(mem + kOffBar + S * 8);
    use = 0;
    fill = 0;
    phase = 0;
    if ((threadIdx.x & 31) == 0) {
      for (int i = 0; i < S; ++i) mbar_init(base + kOffBar + 8 * i, 1);
      *abort_flag = 0;
      fence_mbar_init();
    }
    __syncwarp();
  }
  __device__ __forceinline__ uint32_t slot() const { return base + use * kSlot; }
  __device__ __forceinline__ uint32_t scales() const { return base + kOffScale + use * 128; }

  // Copies of ROW-byte rows by cp.async; lane src0 + r holds row r's address
  // (null: zeros).
  template <int ROW>
  static __device__ __forceinline__ void gather(uint32_t dst, const uint8_t *row, int src0) {
    constexpr int PIECES = ROW / 16;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < PIECES / 2; ++i) {
      const int e = i * 32 + lane, r = e / PIECES, c = e % PIECES;
      const uint8_t *src = reinterpret_cast<const uint8_t *>(__shfl_sync(0xffffffffu, (unsigned long long)row, src0 + r));
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + RowsBlocks<ROW>::at(c, r)), "l"(src + c * 16),
                   "r"(src ? 16u : 0u)
                   : "memory");
    }
  }
  // Starts the next group (if `any`) and ends its cp.async group; every lane is
  // done with the slot's last one.  Small pages: lane l < 16 has key row l at
  // `row`, lane 16 + l value row l.  Otherwise one box per block: `page` and
  // `slot0` (packed: page < 0 and slot0 the first row).  `scale`: of the lane's
  // row (null: 0).
  __device__ __forceinline__ void start(bool any, bool small, const CUtensorMap *tm_k, const CUtensorMap *tm_v, int hk,
                                        bool packed, int page, int slot0, const uint8_t *row, const float *scale) {
    if (any) {
      const uint32_t st = base + fill * kSlot;
      if (small) {
        gather<KROW>(st, row, 0);
        if constexpr (VROW != 0) gather<VROW>(st + kOffV, row, 16);
      } else if ((threadIdx.x & 31) == 0) {
        const uint32_t bar = base + kOffBar + 8 * fill;
        mbar_expect_tx(bar, kSlot);
#pragma unroll
        for (int c = 0; c < K::NB; ++c) {
          const int x = c * (K::kCols / (SCALES ? 1 : 2));
          if (packed) tma_load_3d(st + c * 16 * K::kCols, tm_k, bar, x, hk, slot0);
          else tma_load_4d(st + c * 16 * K::kCols, tm_k, bar, x, hk, slot0, page);
        }
        if constexpr (VROW != 0) {
#pragma unroll
          for (int c = 0; c < V::NB; ++c)
            tma_load_4d(st + kOffV + c * 16 * V::kCols, tm_v, bar, c * (V::kCols / (SCALES ? 1 : 2)), hk, slot0, page);
        }
      }
      if constexpr (SCALES)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(base + kOffScale + fill * 128 + (threadIdx.x & 31) * 4),
                     "l"(scale), "r"(scale ? 4u : 0u)
                     : "memory");
      fill = fill + 1 == S ? 0 : fill + 1;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // Waits for the group in slot `use`, S - 1 starts after its own; false: the
  // wait ran out.
  __device__ __forceinline__ bool wait(bool small, int *err) {
    bool ok = true;
    if (SCALES || small) asm volatile("cp.async.wait_group %0;" ::"n"(S - 1) : "memory");
    if (!small) ok = mbar_wait(base + kOffBar + 8 * use, phase, abort_flag, err);
    return __all_sync(0xffffffffu, ok);
  }
  __device__ __forceinline__ void next() {
    __syncwarp();   // every lane is done with the slot
    if (++use == S) {
      use = 0;
      phase ^= 1;
    }
  }
  // After a wait that ran out: what is still under way lands before the warp ends.
  __device__ __forceinline__ void drain() {
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    for (int i = 0; (threadIdx.x & 31) == 0 && i < S; ++i) mbar_drain(base + kOffBar + 8 * i, i < use ? phase ^ 1 : phase);
  }
};

// Row i' sees key j iff (unsigned)(i' - j + add) < range, for every mask; a row
// at kRowsHidden sees no key (positions stay below 2^30 in magnitude).
constexpr int kRowsHidden = -(1 << 30) - (1 << 29);
struct RowsVisible {
  int add;
  unsigned range;
};
__device__ __forceinline__ RowsVisible rows_visible(int causal, int window) {
  RowsVisible v;
  if (window > 0) {
    v.add = causal ? 0 : window - 1;
    v.range = causal ? (unsigned)window : 2u * (unsigned)window - 1u;
  } else {
    v.add = causal ? 0 : 1 << 30;
    v.range = 1u << 31;
  }
  return v;
}

// The prefix keys of group g: whole pages, inside the page table.  The suffix
// pass starts each sequence there, so both use this.
__device__ __forceinline__ int prefix_keys(const int32_t *prefix_lens, int g, int page_size, int64_t max_pages) {
  int64_t n = max(0, __ldg(prefix_lens + g));
  n = min(n, max_pages * page_size);
  return (int)(n & ~(int64_t)(page_size - 1));
}

// First index in [lo, hi) whose value exceeds x, of a sorted array.
__device__ __forceinline__ int upper_bound_i32(const int32_t *a, int lo, int hi, int x) {
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(a + mid) <= x) lo = mid + 1;
    else hi = mid;
  }
  return lo;
}

// B fragments of up to 8 NT query rows of kv head hk (row = token * group +
// head): bf16 as stored; for byte caches f16 with a power-of-two factor per
// row, max|q| 2^e in [2^14, 2^15), which is exact for bf16 values within 2^-24
// of the row's largest.  inv[nt] = 2^-e of row 8 nt + lane / 4.
template <int D, int KV, int NT>
__device__ __forceinline__ void rows_q_fragments(const __nv_bfloat16 *q, int64_t stride_t, int64_t stride_h, int qa, int hk,
                                                 int group, int rows, uint32_t (&qb)[D / 16][NT][2], float (&inv)[NT]) {
  constexpr int NP = D * (KV ? 1 : 2) / 64;   // 16-byte pieces of a key row per lane
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int r = nt * 8 + g;
    const bool live = r < rows;
    const __nv_bfloat16 *src = q;
    if (live) src = q + (int64_t)(qa + r / group) * stride_t + (int64_t)(hk * group + r % group) * stride_h;
    inv[nt] = 1.f;
    if constexpr (KV == 0) {
#pragma unroll
      for (int i = 0; i < NP; ++i) {
        const uint4 v = live ? __ldg(reinterpret_cast<const uint4 *>(src + 8 * (t + 4 * i))) : make_uint4(0, 0, 0, 0);
        qb[2 * i][nt][0] = v.x;
        qb[2 * i][nt][1] = v.y;
        qb[2 * i + 1][nt][0] = v.z;
        qb[2 * i + 1][nt][1] = v.w;
      }
    } else {
      uint4 v[2 * NP];
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          v[2 * i + u] =
              live ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * (t + 4 * i) + 8 * u)) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v[2 * i + u].x, v[2 * i + u].y, v[2 * i + u].z, v[2 * i + u].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int sh = 0;
      if (mx > 0.f && mx <= 3.0e38f) sh = min(141 - (int)((__float_as_uint(mx) >> 23) & 0xFF), 126);
      const float up = __uint_as_float((uint32_t)(sh + 127) << 23);
      inv[nt] = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
      for (int i = 0; i < 2 * NP; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = pack_f16x2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xFFFF0000u) * up);
        qb[2 * i][nt][0] = h[0];
        qb[2 * i][nt][1] = h[1];
        qb[2 * i + 1][nt][0] = h[2];
        qb[2 * i + 1][nt][1] = h[3];
      }
    }
  }
}

// S^T fragments of one 16-key group from the lane's key pieces (rows g, g + 8).
template <int D, int KV, int NT>
__device__ __forceinline__ void rows_qk(const uint4 *k0, const uint4 *k1, const uint32_t (&qb)[D / 16][NT][2],
                                        float (&c)[NT][4]) {
  constexpr int NP = D * (KV ? 1 : 2) / 64;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) c[nt][0] = c[nt][1] = c[nt][2] = c[nt][3] = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint32_t w0[4] = {k0[i].x, k0[i].y, k0[i].z, k0[i].w};
    const uint32_t w1[4] = {k1[i].x, k1[i].y, k1[i].z, k1[i].w};
    if constexpr (KV == 0) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const uint32_t a[4] = {w0[2 * s], w1[2 * s], w0[2 * s + 1], w1[2 * s + 1]};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_bf16_16816(c[nt], a, qb[2 * i + s][nt][0], qb[2 * i + s][nt][1]);
      }
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        uint32_t a[4];
        dec_bytes4_to_f16<KV>(w0[s], a[0], a[2]);
        dec_bytes4_to_f16<KV>(w1[s], a[1], a[3]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) mma_f16_16816(c[nt], a, qb[4 * i + s][nt][0], qb[4 * i + s][nt][1]);
      }
    }
  }
}

}  // namespace fa
