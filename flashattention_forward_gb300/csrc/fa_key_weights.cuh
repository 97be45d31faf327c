// fa_key_weights.cuh -- the attention weight that each cached key received:
//
//   w_out[b][hk][j] = beta * w_in[b][hk][j]
//                     + sum_{rows i of b, heads h of group hk} exp(s_ij - LSE[h][i])
//
// over the (i, j) that the masks allow, from the forward's saved LSE: the
// column sums of the attention matrix, which the forward itself never forms.
// V is not read, and the softmax needs no running statistics, so the keys can
// be cut anywhere without a merge.
//
// Rows form (few query rows per kv head: decode and drafts).  Bound by
// reading K once.  The keys go through per-warp rings into the A fragments of
// S^T = K Q^T (fa_rows.cuh): no barrier, and any page size costs one page-table
// read per key row.  The old weights are read a group ahead of their use (141
// against 115 us otherwise).  64 sequences of 512 to 8192 keys, 8 kv heads,
// bf16: 115 us, 5.4 TB/s; of one length, 6.2 - 6.5 TB/s.
//
// Tile form (prompts).  Bound by the QK product and one exponential per pair:
// S^T tiles of 128 keys x 128 query rows on tcgen05 with fp32 accumulators in
// TMEM.  A CTA keeps its 128 keys as the A operand and streams the query rows
// of its kv head -- (token, head of the group) packed into one tile by a
// three-dimensional TMA box -- as B.  A thread owns a key, so a column sum is a
// sum in one register: no shuffles, no atomics, the same result every run.
// Two CTAs per SM with two S^T buffers each, so that the products of one tile
// run under the exponentials of three; a tile takes 850 (D 64), 910 (128) and
// 1110 cycles (192) an SM, where the MMAs alone take 320, 576 and 832: 1330 and
// 1630 TFLOP/s at D 128 and 192 over 8192 x 8192, 16 heads.  A CTA's set-up
// (lengths, keys, TMEM, ~6 us) is what short sequences pay: 16 heads of 8
// sequences up to 2048 take 52 us.
//
// -LSE belongs to a column, i.e. every thread needs all 128 of a tile.  Read
// from shared memory they cost four cycles per 16 bytes and warp whatever the
// addresses (the register file takes 128 bytes a cycle), as much as the
// product's own operands: the kernel was bound by shared memory.  So they ride
// in the product instead: one more K=16 step adds sum of (parts of 1/k_scale of
// the key) x (parts of -LSE / scale of the row), each in three bf16 parts, and
// the exponent's argument is then the accumulator times one factor.  (Not under
// the soft-cap, which is not linear, nor with ALiBi, which needs the columns'
// positions in any case.)
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_rows.cuh"

namespace fa {

struct KeyWeightsParams {
  const __nv_bfloat16 *q;
  int64_t q_stride_t, q_stride_h;     // elements
  const int32_t *cu_q, *cu_k;
  const int32_t *block_table;         // null: packed
  int64_t bt_stride, max_pages;
  int32_t page_size, page_shift;
  int64_t n_pages;                    // pages in the pool (packed: rows of the cache)
  const uint8_t *k;
  int64_t s_page, s_slot, s_head;     // bytes: page (packed: token row), slot, kv head
  const float *k_scale;               // byte caches: per (token, kv head)
  const float *lse;                   // [Hq, T_q]
  int64_t total_q;
  const float *w_in;                  // null: beta is 0
  int64_t wi_stride_b, wi_stride_h;
  float *w_out;
  int64_t wo_stride_b, wo_stride_h;
  int64_t extent;                     // entries per (sequence, kv head) row of w_out
  int64_t max_keys;                   // the host's bound on a sequence's keys
  float beta;
  int32_t inplace;                    // w_out is w_in and beta is 1: entries that gain nothing stay untouched
  int32_t hq, hkv, group;
  int32_t kv;                         // 0 bf16, 1 e4m3, 2 int8
  int32_t mod, causal, window;
  float scale_log2, alibi_log2, softcap_arg, softcap_log2;
  int32_t keys_per_cta;               // rows form
  int32_t small_pages;                // rows form: pages of fewer than 16 keys, row copies instead of boxes
  int32_t tokens_per_tile;            // tile form: 128 / group
  int *err;
};

// The lengths of one sequence, with the key count held to what the weights
// and the page table cover (a longer sequence is flagged; one whose query rows
// lie outside q is flagged and adds nothing).
struct KwSeq {
  int qa, sq, ka, sk, shift;          // shift = Sk - Sq: i' = i + shift
};
__device__ __forceinline__ KwSeq kw_sequence(const KeyWeightsParams &p, int b) {
  KwSeq s;
  s.qa = __ldg(p.cu_q + b);
  s.sq = __ldg(p.cu_q + b + 1) - s.qa;
  s.ka = __ldg(p.cu_k + b);
  const int sk = __ldg(p.cu_k + b + 1) - s.ka;
  s.shift = sk - s.sq;
  int64_t cap = min(p.extent, p.max_keys);
  if (p.block_table) cap = min(cap, p.max_pages * p.page_size);
  if (sk > cap && threadIdx.x == 0) record_error(p.err, kErrBounds);
  s.sk = (int)min((int64_t)sk, cap);
  if (s.sq > 0 && (s.qa < 0 || (int64_t)s.qa + s.sq > p.total_q)) {
    if (threadIdx.x == 0) record_error(p.err, kErrBounds);
    s.sq = 0;
  }
  return s;
}

// Page of key j (packed: its row; page_size is then 1).  Looked up for several
// keys before any is used, so that the reads are in flight together; ids
// outside the cache are replaced by -1 and flagged by the caller's `bad`.
__device__ __forceinline__ int kw_page(const KeyWeightsParams &p, const int32_t *bt, int ka, int j, bool live, bool &bad) {
  if (!live) return -1;
  const int pg = bt ? __ldg(bt + (j >> p.page_shift)) : ka + j;
  const bool ok = pg >= 0 && pg < p.n_pages;
  bad = bad || !ok;
  return ok ? pg : -1;
}
__device__ __forceinline__ const uint8_t *kw_row(const KeyWeightsParams &p, int pg, int j, int hk) {
  return p.k + (int64_t)pg * p.s_page + (int64_t)(j & (p.page_size - 1)) * p.s_slot + (int64_t)hk * p.s_head;
}
__device__ __forceinline__ float kw_scale(const KeyWeightsParams &p, int pg, int j, int hk) {
  return __ldg(p.k_scale + ((int64_t)pg * p.page_size + (j & (p.page_size - 1))) * p.hkv + hk);
}

// Entries [lo, hi) that gain nothing: w_out = beta * w_in.
__device__ __forceinline__ void kw_carry(const KeyWeightsParams &p, int b, int hk, int64_t lo, int64_t hi) {
  if (p.inplace) return;
  const float *wi = p.w_in ? p.w_in + (int64_t)b * p.wi_stride_b + (int64_t)hk * p.wi_stride_h : nullptr;
  float *wo = p.w_out + (int64_t)b * p.wo_stride_b + (int64_t)hk * p.wo_stride_h;
  for (int64_t j = lo + threadIdx.x; j < hi; j += blockDim.x) wo[j] = wi ? p.beta * wi[j] : 0.f;
}

// --------------------------------------------------------------- rows form --
constexpr int kKwWarps = 8;

template <int D, int KV>
struct KwRowsCfg {
  static constexpr int kRow = D * (KV ? 1 : 2);
  static constexpr int NP = kRow / 64;                   // 16-byte pieces of a key row per lane
  // short rows are bound by the work on a group more than by its bytes: more warps
  static constexpr int kCtasPerSm = kRow <= 128 ? 3 : 2;
  // as many slots as these CTAs hold, up to six
  static constexpr int kFit = (222 * 1024 / (kCtasPerSm * kKwWarps) - 1200) / (16 * kRow + 160);
  static constexpr int kStages = kFit < 6 ? kFit : 6;
  using Ring = RowsRing<kRow, 0, KV != 0, kStages>;
  static constexpr int kSmemBytes = kKwWarps * Ring::kBytes + 1024;
  static_assert(kStages >= 2 && kCtasPerSm * (kSmemBytes + 1024) <= 233472, "shared memory");
};

// NT tiles of 8 query rows.
template <int D, int KV, int NT>
__global__ void __launch_bounds__(kKwWarps * 32, NT == 1 ? KwRowsCfg<D, KV>::kCtasPerSm : 2)
    fa_key_weights_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const KeyWeightsParams p) {
  using Cfg = KwRowsCfg<D, KV>;
  using Ring = typename Cfg::Ring;
  constexpr int NP = Cfg::NP, S = Cfg::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int hk = blockIdx.y, b = blockIdx.z;
  const KwSeq sq_ = kw_sequence(p, b);
  const int64_t lo64 = (int64_t)blockIdx.x * p.keys_per_cta;
  const int64_t hi64 = min(p.extent, lo64 + p.keys_per_cta);
  int rows = sq_.sq * p.group;
  if (rows > NT * 8) {
    if (threadIdx.x == 0) record_error(p.err, kErrBounds);
    rows = NT * 8;
  }
  if (rows <= 0 || lo64 >= sq_.sk) {
    kw_carry(p, b, hk, lo64, hi64);
    return;
  }
  const int lo = (int)lo64, hi = (int)min(hi64, (int64_t)sq_.sk);
  kw_carry(p, b, hk, hi, hi64);

  // The warp's groups are lo + 16 (warp + 8 i).  Lane l < 16 finds the row of
  // key base + l; S - 1 groups are under way while one is used, and the first
  // of them while the query rows are read.
  constexpr int STEP = kKwWarps * 16;
  const float *wi = p.w_in ? p.w_in + (int64_t)b * p.wi_stride_b + (int64_t)hk * p.wi_stride_h : nullptr;
  float *wo = p.w_out + (int64_t)b * p.wo_stride_b + (int64_t)hk * p.wo_stride_h;
  const int32_t *bt = p.block_table ? p.block_table + (int64_t)b * p.bt_stride : nullptr;
  bool bad = false;
  auto page_at = [&](int base) -> int {
    const int j = base + lane;
    return kw_page(p, bt, sq_.ka, j, lane < 16 && j < hi, bad);
  };
  const bool small = p.small_pages != 0;
  Ring ring;
  ring.init(smem + warp * Ring::kBytes);
  auto copy = [&](int base, int pg) {
    const int j = base + lane;
    const bool live = pg >= 0;
    ring.start(base < hi, small, &tm_k, nullptr, hk, bt == nullptr, pg, bt ? base & (p.page_size - 1) : sq_.ka + base,
               live && small ? kw_row(p, pg, j, hk) : nullptr,
               KV && live ? p.k_scale + ((int64_t)pg * p.page_size + (j & (p.page_size - 1))) * p.hkv + hk : nullptr);
  };
  const int first = lo + warp * 16;
  int pgn;
  {
    int pg[S - 1];
#pragma unroll
    for (int i = 0; i < S - 1; ++i) pg[i] = page_at(first + STEP * i);
    pgn = page_at(first + STEP * (S - 1));
#pragma unroll
    for (int i = 0; i < S - 1; ++i) copy(first + STEP * i, pg[i]);
  }

  uint32_t qb[D / 16][NT][2];
  float inv[NT];                              // byte caches: 2^-e of row 8 nt + g
  rows_q_fragments<D, KV, NT>(p.q, p.q_stride_t, p.q_stride_h, sq_.qa, hk, p.group, rows, qb, inv);
  // The rows of this lane's C columns, 8 nt + 2t + e: -LSE (log2 units), i'
  // (relative to key lo + kg, with the mask's offset) and the score factor.
  // Rows that see nothing (LSE -inf) weigh nothing.
  const RowsVisible vb = rows_visible(p.causal, p.window);
  const int kg = Ring::K::row(g);             // the lane's fragment rows: keys kg and kg + 8 of a group
  float nl[NT][2], sc[NT][2];
  int ip[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * t + e;
      const float f = __shfl_sync(0xffffffffu, inv[nt], (2 * t + e) * 4);
      sc[nt][e] = (p.mod == 2 ? 2.f * kLog2e * p.softcap_arg : p.scale_log2) * f;
      nl[nt][e] = -INFINITY;
      ip[nt][e] = kRowsHidden;
      if (r < rows) {
        const float l = __ldg(p.lse + (int64_t)(hk * p.group + r % p.group) * p.total_q + sq_.qa + r / p.group);
        nl[nt][e] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        ip[nt][e] = r / p.group + sq_.shift + vb.add - lo - kg;
      }
    }

  bool ok = true;
  // the old weights of keys kg and kg + 8, read one group ahead
  float w0[2] = {0.f, 0.f}, w1[2];
  auto old_weights = [&](int base, float (&w)[2]) {
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int j = base + 8 * x + kg;
      w[x] = wi && t == 0 && j < hi ? __ldcs(wi + j) : 0.f;
    }
  };
  old_weights(first, w1);
  for (int base = first; base < hi; base += STEP) {
    const int ahead = base + STEP * (S - 1);
    w0[0] = w1[0];
    w0[1] = w1[1];
    old_weights(base + STEP, w1);
    copy(ahead, pgn);
    pgn = page_at(ahead + STEP);
    ok = ring.wait(small, p.err);
    if (!ok) break;
    const uint32_t st = ring.slot();
    if (KV || small) __syncwarp();            // what other lanes copied
    float c[NT][4];
    {
      uint4 kr[2][NP];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < NP; ++i) kr[u][i] = rows_lds16(st + Ring::K::at(t + 4 * i, kg + 8 * u));
      rows_qk<D, KV, NT>(kr[0], kr[1], qb, c);
    }
    float ks[2] = {1.f, 1.f};
    if constexpr (KV != 0) {
      ks[0] = rows_lds4(ring.scales() + kg * 4);
      ks[1] = rows_lds4(ring.scales() + (kg + 8) * 4);
    }
    ring.next();
#pragma unroll
    for (int x = 0; x < 2; ++x) {             // keys base + 8 x + kg
      const int rel = base - lo + 8 * x, j = lo + rel + kg;
      float sum = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int d = ip[nt][e] - rel;      // i' - j + the mask's offset
          float y = c[nt][2 * x + e] * (KV ? sc[nt][e] * ks[x] : sc[nt][e]);
          if (p.mod == 2) {
            float r;
            y = softcap_log2_score(ex2(y), p.softcap_log2, r);
          } else if (p.mod == 1) {
            y = fmaf(-p.alibi_log2, fabsf((float)(d - vb.add)), y);
          }
          y = ex2(y + nl[nt][e]);
          sum += (unsigned)d < vb.range ? y : 0.f;
        }
      sum += __shfl_xor_sync(0xffffffffu, sum, 1);
      sum += __shfl_xor_sync(0xffffffffu, sum, 2);
      if (t == 0 && j < hi) wo[j] = fmaf(p.beta, w0[x], sum);
    }
  }
  if (!ok) ring.drain();
  if (bad) record_error(p.err, kErrBounds);
}

// --------------------------------------------------------------- tile form --
template <int D>
struct KwTileCfg {
  static constexpr int KC = D / 64;                 // 64-column blocks
  static constexpr int kChunkBytes = 128 * 128;
  static constexpr int NCH = D == 192 ? 3 : 4;      // Q ring, in blocks; two CTAs per SM
  static constexpr int kOffK = 0;
  static constexpr int kOffQ = KC * kChunkBytes;
  static constexpr int kOffCol = kOffQ + NCH * kChunkBytes;   // [2][128] -LSE, [128] tokens
  static constexpr int kOffSum = kOffCol + 3 * 128 * 4;       // [128] the second warpgroup's sums
  // K=16 operands of the LSE term, 32-byte swizzled: the keys', and the rows' of two tiles
  static constexpr int kAugBytes = 128 * 32;
  static constexpr int kOffAug = kOffSum + 128 * 4;
  static constexpr int kOffBar = kOffAug + 3 * kAugBytes;
  static constexpr int kSmemBytes = kOffBar + (2 * NCH + 5) * 8 + 16 + 1024;
  // two warpgroups take the tiles in turn, then the producer and the MMA warp
  static constexpr int kThreads = 10 * 32, kFill = 9 * 32;
  static constexpr int kProducerWarp = 8, kMmaWarp = 9;
  static constexpr uint32_t kTmemCols = 256;        // two S^T tiles
  static_assert(2 * (kSmemBytes + 1024) <= 233472, "two CTAs per SM");
};

// Eight e4m3 or int8 bytes -> eight bf16 (exact: both have at most 8
// significant bits).
template <int KV>
__device__ __forceinline__ uint4 kw_bytes8_to_bf16(uint2 w) {
  uint32_t h[4], o[4];
  dec_bytes4_to_f16<KV>(w.x, h[0], h[1]);
  dec_bytes4_to_f16<KV>(w.y, h[2], h[3]);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[e]));
    o[e] = pack_bf16x2(f.x, f.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// x = h + m + l to about 2^-24 relative, bf16 parts.
struct Bf16x3 {
  float h, m, l;
};
__device__ __forceinline__ Bf16x3 bf16_parts(float x) {
  Bf16x3 s;
  s.h = __bfloat162float(__float2bfloat16_rn(x));
  s.m = __bfloat162float(__float2bfloat16_rn(x - s.h));
  s.l = __bfloat162float(__float2bfloat16_rn(x - s.h - s.m));
  return s;
}
// Row r of a K=16 operand: six values, ten zeros; 16-byte chunk c of a row sits
// at chunk c ^ ((r >> 2) & 1).
__device__ __forceinline__ void aug_row(uint8_t *base, int r, float v0, float v1, float v2, float v3, float v4, float v5) {
  uint8_t *row = base + r * 32;
  const int sw = (r >> 2) & 1;
  *reinterpret_cast<uint4 *>(row + (sw << 4)) = make_uint4(pack_bf16x2(v0, v1), pack_bf16x2(v2, v3), pack_bf16x2(v4, v5), 0u);
  *reinterpret_cast<uint4 *>(row + ((1 ^ sw) << 4)) = make_uint4(0u, 0u, 0u, 0u);
}

// 16 bytes of shared memory, read where it stands (kept out of registers between uses).
__device__ __forceinline__ int4 kw_lds4(uint32_t a) {
  int4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}

// MOD 0: plain scores with a scale that LSE can be divided by; 1: ALiBi (or any
// scale, with slope 0); 2: soft-cap.
template <int D, int MOD>
__global__ void __launch_bounds__(KwTileCfg<D>::kThreads, 2)
    fa_key_weights_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const KeyWeightsParams p) {
  using Cfg = KwTileCfg<D>;
  constexpr int KC = Cfg::KC, NCH = Cfg::NCH;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // key tiles in the slowest grid dimension: under a causal mask the first
  // tiles of every sequence have the most queries, and so start first
  const int hk = blockIdx.x, b = blockIdx.y;
  const KwSeq s = kw_sequence(p, b);
  const int64_t j0_64 = (int64_t)blockIdx.z * 128;
  if (s.sq <= 0 || j0_64 >= s.sk) {
    kw_carry(p, b, hk, j0_64, min(p.extent, j0_64 + 128));
    return;
  }
  const int j0 = (int)j0_64;
  const int jl = min(j0 + 128, s.sk) - 1;           // last key of the tile
  // tokens [t_lo, t_hi) that see a key of the tile
  int t_lo = 0, t_hi = s.sq;
  if (p.causal) t_lo = max(t_lo, j0 - s.shift);
  if (p.window > 0) {
    t_hi = min(t_hi, jl + p.window - s.shift);                         // i' - j < window for some j
    if (!p.causal) t_lo = max(t_lo, j0 - p.window + 1 - s.shift);      // j - i' < window
  }
  const int tpt = p.tokens_per_tile;
  const int n_tiles = t_hi > t_lo ? (t_hi - t_lo + tpt - 1) / tpt : 0;
  if (n_tiles == 0) {
    kw_carry(p, b, hk, j0, min(p.extent, j0_64 + 128));
    return;
  }
  uint8_t *sK = smem + Cfg::kOffK, *sQ = smem + Cfg::kOffQ;
  float *col_nl = reinterpret_cast<float *>(smem + Cfg::kOffCol);      // [2][128]
  int *col_tok = reinterpret_cast<int *>(col_nl + 256);                // [128] token of a tile's column
  uint64_t *q_full = reinterpret_cast<uint64_t *>(smem + Cfg::kOffBar);
  uint64_t *q_empty = q_full + NCH, *s_full = q_empty + NCH, *s_empty = s_full + 2, *k_ready = s_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(k_ready + 1);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  const int rows_box = tpt * p.group;               // rows of a Q tile, at most 128
  if (threadIdx.x < 128) col_tok[threadIdx.x] = (int)threadIdx.x < rows_box ? (int)threadIdx.x / p.group : 1 << 20;
  if (threadIdx.x == 0) {
    for (int i = 0; i < NCH; ++i) {
      mbar_init(smem_u32(q_full + i), 1);
      mbar_init(smem_u32(q_empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(s_full + i), 1);
      mbar_init(smem_u32(s_empty + i), 128);
    }
    mbar_init(smem_u32(k_ready), Cfg::kFill);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == Cfg::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int32_t *bt = p.block_table ? p.block_table + (int64_t)b * p.bt_stride : nullptr;

  // Thread r of either warpgroup: key j0 + r and its scale (one too small to
  // divide by is raised to 2^-100, which leaves its products negligible), and
  // column r of the tiles: token t_lo + it * tpt + r / group, head r % group.
  const int r = threadIdx.x & 127, j = j0 + r;
  float key_factor = 1.f;
  if (p.kv && warp < 8) {
    bool bad = false;
    const int pg = kw_page(p, bt, s.ka, j, j < s.sk, bad);
    if (pg >= 0) key_factor = kw_scale(p, pg, j, hk);
  }
  if (MOD == 0 && fabsf(key_factor) < 0x1p-100f) key_factor = 0x1p-100f;
  const float *lse_r = p.lse + (int64_t)(hk * p.group + r % p.group) * p.total_q + s.qa;
  const int ctok = t_lo + r / p.group;
  // -LSE in log2 units of column r of tile it; -inf for a row that sees nothing
  auto column_nl = [&](int it) -> float {
    const int tok = ctok + it * tpt;
    if (it >= n_tiles || r >= rows_box || tok >= t_hi) return -INFINITY;
    const float l = __ldg(lse_r + tok);
    return l == -INFINITY ? -INFINITY : -l * kLog2e;
  };
  // Row r of tile it's operand of the LSE term: -LSE / scale.  Rows that see
  // nothing get a large finite value (0 * inf would be NaN) of the sign that
  // the scale turns negative.
  auto write_rows = [&](int it, float nl) {
    const float v = nl == -INFINITY ? copysignf(0x1p120f, -p.scale_log2) : nl / p.scale_log2;
    const Bf16x3 q = bf16_parts(v);
    aug_row(smem + Cfg::kOffAug + (1 + (it & 1)) * Cfg::kAugBytes, r, q.h, q.m, q.h, q.l, q.m, q.h);
  };
  auto row_operand = [&](int it) { write_rows(it, column_nl(it)); };

  if (warp != Cfg::kProducerWarp) {
    // The key tile as the K-major, 128-byte-swizzled A operand in bf16: any
    // page size, and byte caches exactly (their scale multiplies the key's sum
    // argument below).  Rows past the sequence are zero.  While the producer's
    // first query tiles are under way, the other nine warps read the keys,
    // every piece of a thread before it stores any.
    const int ft = warp == Cfg::kMmaWarp ? 256 + lane : (int)threadIdx.x;   // 0 ... kFill - 1
    constexpr int FT = Cfg::kFill;
    bool bad = false;
    if (p.kv == 0) {
      constexpr int PR = D / 8, N = (128 * PR + FT - 1) / FT;   // 16-byte pieces of a row, of a thread
      uint4 v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = ft + i * FT, r = e / PR, j = j0 + r;
        const int pg = kw_page(p, bt, s.ka, j, e < 128 * PR && j < s.sk, bad);
        v[i] = pg >= 0 ? rows_ld_stream(kw_row(p, pg, j, hk) + (e % PR) * 16) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = ft + i * FT, r = e / PR, c = e % PR;
        if (e < 128 * PR) *reinterpret_cast<uint4 *>(sK + (c >> 3) * Cfg::kChunkBytes + sw128(r, c & 7)) = v[i];
      }
    } else {
      constexpr int PR = D / 16, N = (128 * PR + FT - 1) / FT;
      uint4 v[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = ft + i * FT, r = e / PR, j = j0 + r;
        const int pg = kw_page(p, bt, s.ka, j, e < 128 * PR && j < s.sk, bad);
        v[i] = pg >= 0 ? rows_ld_stream(kw_row(p, pg, j, hk) + (e % PR) * 16) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int e = ft + i * FT, r = e / PR, c = e % PR;
        if (e >= 128 * PR) continue;
        const uint2 lo = make_uint2(v[i].x, v[i].y), hi = make_uint2(v[i].z, v[i].w);
        uint8_t *dst = sK + (c >> 2) * Cfg::kChunkBytes;
        const int c8 = (2 * c) & 7;
        *reinterpret_cast<uint4 *>(dst + sw128(r, c8)) = p.kv == 1 ? kw_bytes8_to_bf16<1>(lo) : kw_bytes8_to_bf16<2>(lo);
        *reinterpret_cast<uint4 *>(dst + sw128(r, c8 + 1)) =
            p.kv == 1 ? kw_bytes8_to_bf16<1>(hi) : kw_bytes8_to_bf16<2>(hi);
      }
    }
    if (bad) record_error(p.err, kErrBounds);
    // rows of the query tiles that no box writes (128 % group != 0) stay zero
    for (int e = ft; e < NCH * (128 - rows_box) * 8; e += FT) {
      const int ch = e / ((128 - rows_box) * 8), rest = e % ((128 - rows_box) * 8);
      *reinterpret_cast<uint4 *>(sQ + ch * Cfg::kChunkBytes + rows_box * 128 + rest * 16) = make_uint4(0, 0, 0, 0);
    }
    if (MOD == 0 && warp < 8) {
      // LSE term: the keys' operand, and the rows' of the first two tiles
      const int x = warp >> 2;
      if (x == 0) {
        const Bf16x3 a = bf16_parts(1.f / key_factor);
        aug_row(smem + Cfg::kOffAug, threadIdx.x, a.h, a.h, a.m, a.h, a.m, a.l);
      }
      row_operand(x);
    }
    fence_proxy_async_smem();
    mbar_arrive(smem_u32(k_ready));
  }

  if (warp == Cfg::kProducerWarp) {
    // ------------------------------------------------------- producer --
    if (lane == 0) {
      prefetch_tmap(&tm_q);
      const uint32_t bytes = (uint32_t)rows_box * 128u;
      int n = 0;
      bool ok = true;
      for (int it = 0; ok && it < n_tiles; ++it)
        for (int c = 0; c < KC; ++c, ++n) {
          const int slot = n % NCH;
          if (n >= NCH && !(ok = mbar_wait(smem_u32(q_empty + slot), ((n / NCH) - 1) & 1, abort_flag, p.err))) break;
          mbar_expect_tx(smem_u32(q_full + slot), bytes);
          tma_load_3d(smem_u32(sQ + slot * Cfg::kChunkBytes), &tm_q, smem_u32(q_full + slot), c * 64, hk * p.group,
                      s.qa + t_lo + it * tpt);
        }
      // the last loads have landed before the CTA ends, whatever the others do
      for (int i = max(0, n - NCH); i < n; ++i) mbar_drain(smem_u32(q_full + i % NCH), (i / NCH) & 1);
    }
  } else if (warp == Cfg::kMmaWarp) {
    // ----------------------------------------------------------- MMAs --
    if (elect_one()) {
      constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
      const uint64_t dk = smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint32_t hi = (uint32_t)(dk >> 32), lo_k = (uint32_t)dk;
      const uint32_t lo_q = (uint32_t)smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t aug = smem_desc_sw32(smem_u32(smem + Cfg::kOffAug));
      const uint32_t aug_lo = (uint32_t)aug, aug_hi = (uint32_t)(aug >> 32);
      int n = 0;
      bool ok = mbar_wait(smem_u32(k_ready), 0, abort_flag, p.err);
      for (int it = 0; ok && it < n_tiles; ++it) {
        const int x = it & 1;
        if (it >= 2 && !(ok = mbar_wait(smem_u32(s_empty + x), ((it >> 1) - 1) & 1, abort_flag, p.err))) break;
        const uint32_t d = tmem + x * 128u;
        for (int c = 0; c < KC; ++c, ++n) {
          const int slot = n % NCH;
          if (!(ok = mbar_wait(smem_u32(q_full + slot), (n / NCH) & 1, abort_flag, p.err))) break;
          tc_fence_after();
          uint32_t a = lo_k + (uint32_t)(c * (Cfg::kChunkBytes >> 4)), q = lo_q + (uint32_t)(slot * (Cfg::kChunkBytes >> 4));
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            if (ks == 0 && c == 0) mma_ss_w<0>(d, a, hi, q, hi, idesc);
            else mma_ss_w<1>(d, a, hi, q, hi, idesc);
            a += 2;
            q += 2;
          }
          tc_commit(smem_u32(q_empty + slot));
        }
        if (!ok) break;
        if constexpr (MOD == 0)
          mma_ss_w<1>(d, aug_lo, aug_hi, aug_lo + (uint32_t)((1 + x) * (Cfg::kAugBytes >> 4)), aug_hi, idesc);
        tc_commit(smem_u32(s_full + x));
      }
    }
  } else {
    // --------------------------------------------- one key per thread --
    // Warpgroup x takes the tiles x, x + 2, ...: the tiles of S^T buffer x.
    const int x = warp >> 2;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c = (MOD == 2 ? 2.f * kLog2e * p.softcap_arg : p.scale_log2) * key_factor;
    const RowsVisible vb = rows_visible(p.causal, p.window);
    float *nl_buf = col_nl + x * 128;               // MOD 1, 2
    float nl_next = column_nl(MOD == 0 ? x + 2 : x);
    float total = 0.f;
    bool ok = true;
    for (int it = x; it < n_tiles; it += 2) {
      if constexpr (MOD != 0) {
        // this tile's column constants, between the barriers of its readers
        if (it >= 2) asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
        nl_buf[r] = nl_next;
        asm volatile("bar.sync %0, 128;" ::"r"(1 + x) : "memory");
        nl_next = column_nl(it + 2);
      }
      const int ta = t_lo + it * tpt, tb = min(ta + tpt, t_hi) - 1;    // first and last token of the tile
      const int n_tok = tb - ta + 1;
      bool mask = n_tok < tpt;                       // rows of other sequences may hold anything
      if (p.causal) mask = mask || ta + s.shift < jl;
      if (p.window > 0) mask = mask || tb + s.shift - j0 >= p.window || (!p.causal && jl - ta - s.shift >= p.window);
      ok = mbar_wait(smem_u32(s_full + x), (it >> 1) & 1, abort_flag, p.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      if constexpr (MOD == 0) {
        // the product has read this buffer's row operand: the next tile's
        write_rows(it + 2, nl_next);
        fence_proxy_async_smem();
        nl_next = column_nl(it + 4);
      }
      const int d0 = ta + s.shift - j;               // i' - j of the tile's first token
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float v[32];
        tmem_ld32(tmem + lane_base + x * 128u + q * 32u, v);
        tmem_wait_ld();
        if (q == 3) {
          tc_fence_before();
          mbar_arrive(smem_u32(s_empty + x));
        }
        const float4 *nl4 = reinterpret_cast<const float4 *>(nl_buf + q * 32);
        const uint32_t tok4 = smem_u32(col_tok + q * 32);
        if constexpr (MOD == 2) {
          // cap tanh(u) = cap - 2 cap / (1 + 2^x), x = 2 u log2 e.  Four scores
          // share a reciprocal (2.25 MUFU operations per score instead of 3):
          // with a = min(1, 2^-30 + 2^(x - 30)) the product of four stays above
          // 2^-121, and 2^-30 is below half a step of 1.  A NaN becomes a = 0, an
          // infinite reciprocal, and NaN in its neighbours: they are cleared of
          // hidden scores first, and a visible one marks the key itself.
          if (mask) {
            const int da = d0 + vb.add;
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const int4 i = kw_lds4(tok4 + 4 * e);
              const int tok[4] = {i.x, i.y, i.z, i.w};
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                const bool on = tok[u] < n_tok && (unsigned)(tok[u] + da) < vb.range;
                if (on && v[e + u] != v[e + u]) acc[0] = v[e + u];
                v[e + u] = on ? v[e + u] : 0.f;
              }
            }
          }
          const float cl = p.softcap_log2;
#pragma unroll
          for (int e = 0; e < 32; e += 2) fma2(v[e], v[e + 1], v[e], v[e + 1], c, -30.f);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = add_sat(ex2(v[e]), 0x1p-30f);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 n = nl4[e >> 2];
            float x0, x1, x2, x3;
            rcp4(v[e], v[e + 1], v[e + 2], v[e + 3], x0, x1, x2, x3);
            fma2v(x0, x1, -0x1p-29f * cl, n.x + cl, n.y + cl);
            fma2v(x2, x3, -0x1p-29f * cl, n.z + cl, n.w + cl);
            v[e] = x0;
            v[e + 1] = x1;
            v[e + 2] = x2;
            v[e + 3] = x3;
          }
        } else if constexpr (MOD == 1) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float4 n = nl4[e >> 2];
            const int4 i = kw_lds4(tok4 + 4 * e);
            n.x = fmaf(-p.alibi_log2, fabsf((float)(i.x + d0)), n.x);
            n.y = fmaf(-p.alibi_log2, fabsf((float)(i.y + d0)), n.y);
            n.z = fmaf(-p.alibi_log2, fabsf((float)(i.z + d0)), n.z);
            n.w = fmaf(-p.alibi_log2, fabsf((float)(i.w + d0)), n.w);
            fma2v(v[e], v[e + 1], c, n.x, n.y);
            fma2v(v[e + 2], v[e + 3], c, n.z, n.w);
          }
        } else {
#pragma unroll
          for (int e = 0; e < 32; e += 2) mul2(v[e], v[e + 1], c);
        }
        if (mask) {
          const int da = d0 + vb.add;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const int4 i = kw_lds4(tok4 + 4 * e);
            v[e] = (i.x < n_tok && (unsigned)(i.x + da) < vb.range) ? v[e] : -INFINITY;
            v[e + 1] = (i.y < n_tok && (unsigned)(i.y + da) < vb.range) ? v[e + 1] : -INFINITY;
            v[e + 2] = (i.z < n_tok && (unsigned)(i.z + da) < vb.range) ? v[e + 2] : -INFINITY;
            v[e + 3] = (i.w < n_tok && (unsigned)(i.w + da) < vb.range) ? v[e + 3] : -INFINITY;
          }
        }
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          add2(acc[0], acc[1], ex2(v[e]), ex2(v[e + 1]));
          add2(acc[2], acc[3], ex2(v[e + 2]), ex2(v[e + 3]));
        }
      }
      total += (acc[0] + acc[1]) + (acc[2] + acc[3]);   // a tile's sum first: shorter chains of roundings
    }
    // the second warpgroup's sums join the first's
    float *sums = reinterpret_cast<float *>(smem + Cfg::kOffSum);
    if (x == 1) sums[r] = total;
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (x == 0 && *abort_flag == 0 && j0_64 + r < p.extent) {
      total += sums[r];
      const float *wi = p.w_in ? p.w_in + (int64_t)b * p.wi_stride_b + (int64_t)hk * p.wi_stride_h : nullptr;
      float *wo = p.w_out + (int64_t)b * p.wo_stride_b + (int64_t)hk * p.wo_stride_h;
      const float gain = j < s.sk ? total : 0.f;
      if (!p.inplace || j < s.sk) wo[j] = wi ? fmaf(p.beta, wi[j], gain) : gain;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == Cfg::kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, Cfg::kTmemCols);
  }
}

}  // namespace fa
