// fa_prefix.cuh -- the shared part of a decode batch whose sequences begin
// with the same pages: one attention pass over the prefix keys of a group of
// sequences for all query rows of the group at once.
//
// Decode reads the cache once per sequence.  Where the sequences of a group
// hold the same first pages, those keys can be read once per group instead:
// the rows (query token, head of the kv head's group) of all its sequences are
// one matrix Q [tokens * Hq/Hkv, D], and the prefix part of the attention is
// the dense product of the prefill -- O = softmax(Q K^T) V, with the running
// maximum and sum -- whose partial (O, LSE) merges with the partials of each
// sequence's own keys by the split-KV rule
//   LSE = ln sum_s exp(LSE_s),  out = sum_s exp(LSE_s - LSE) O_s.
//
// CTA (key split, kv head, rows): S = Q K^T and O += P V on tcgen05 with S, P
// and O in TMEM.  A TMA box of {64 columns, Hq/Hkv heads, 128 / (Hq/Hkv)
// tokens} lands Q with the heads of a kv head beside each other, so a GQA group
// fills a tile's 128 rows and K/V are read once for all its heads.
//
// bf16 caches: one tile per CTA and two CTAs per SM, so that one CTA's softmax
// runs under the other's products; 64 KB of K and V are in flight per CTA.
// 6144 rows over 65536 keys, D 128: 169 us, 1220 TFLOP/s; the same with the
// products issued behind (lane == 0) instead of an elected lane, 188 us.
//
// Every row has its own interval of visible keys (its sequence's length,
// causal limit and window), so the result does not depend on the prefix lying
// left of all queries; key tiles that no row sees are not loaded.
//
// Byte caches (KV 1 e4m3, 2 int8): two tiles A and B per CTA, each with its
// softmax warpgroup, share every K/V tile, which halves the conversion per
// product:  QK_A(0) QK_B(0) | PV_A(0) QK_A(1) PV_B(0) QK_B(1) | ...  Six
// converter warps turn the staged bytes into f16 in place: K exactly (k_scale
// multiplies the scores in fp32), V times v_scale 2^-E, with E one per tile of
// 128 keys, so that f16 holds it whatever the magnitude of V; 2^E joins the
// exponent of the tile's weights.  (Scales that belong to a column cost every
// softmax warp 128 shared-memory cycles per tile; with both kept that way the
// kernel spent half its time on them.)  Bound by shared memory: per pair of
// tiles 1536 cycles of operands, 768 of conversion, 1024 of K scales and 256 of
// loads.  768 rows of 8 kv heads over 65536 int8 keys take 229 us, 900 TFLOP/s.
#pragma once
#include <climits>

#include "fa_prefill.cuh"
#include "fa_suffix.cuh"

namespace fa {

struct PrefixParams {
  const int32_t *cu_q, *cu_k;
  const int32_t *cu_groups;      // [num_groups + 1]: sequences of a group
  const int32_t *prefix_lens;    // [num_groups]
  int32_t num_groups, num_seqs;
  const int32_t *block_table;
  int64_t bt_stride, max_pages, n_pages;
  int32_t page_size, page_shift, rows_per_box;
  int32_t gather;
  KvGather gk, gv;
  const float *k_scale, *v_scale;
  int64_t total_q;
  int32_t hq, hkv, group, tokens_per_tile;
  int32_t num_splits, split_tiles;   // key ranges, and the 128-key tiles of one
  float *o_part;                 // [splits of the whole call][T_q][Hq][D]; this pass writes the first num_splits
  float *lse_part;               // [splits of the whole call][Hq][T_q]
  int32_t causal, window;
  float scale_log2, alibi_log2, softcap_arg, softcap_log2;
  int *err;
};

template <int D, int KV>
struct PrefixCfg {
  static constexpr int NT = KV ? 2 : 1;                // row tiles per CTA
  static constexpr int KC = D / 64;
  static constexpr int kChunkBytes = 128 * 128;        // one 64-column block of 128 rows, 16-bit
  static constexpr int kTileBytes = KC * kChunkBytes;
  static constexpr int NS = (D == 64 ? 2 : 1) * NT;    // K and V stages
  static constexpr int kOffQ = 0;
  static constexpr int kOffK = NT * kTileBytes;
  static constexpr int kOffV = kOffK + NS * kTileBytes;
  // byte caches: scales of NSS tiles, [128 of K, 128 of V (f16 pairs), E] each.  Tile j's take
  // the slot of tile j - NS - 1: its K bytes landed after the QKs of tile
  // j - NS, which were issued after the softmax of tile j - NS - 1.
  static constexpr int NSS = NS + 1;
  static constexpr int kOffSc = kOffV + NS * kTileBytes;
  static constexpr int kScWords = 260;
  static constexpr int kOffBar = kOffSc + (KV ? NSS * kScWords * 4 : 0);
  static constexpr int kNumBars = 1 + NT + 6 * NS + 3 * NT + NSS;
  static constexpr int kOffMisc = kOffBar + kNumBars * 8;
  static constexpr int kSmemBytes = kOffMisc + 64 + 1024;
  // warps: NT softmax warpgroups, producer, MMA, then the converters (bf16: two
  // idle warps that fill the warpgroup); the softmax warps take registers from
  // the others (setmaxnreg), within what the launch holds
  static constexpr int kCtasPerSm = KV ? 1 : 2;
  static constexpr int kThreads = (KV ? 16 : 8) * 32, kConverters = 6;
  static constexpr int kProducerWarp = 4 * NT, kMmaWarp = 4 * NT + 1, kFirstConverter = 4 * NT + 2;
  static constexpr int kRegsSoftmax = KV ? 168 : 200, kRegsOther = KV ? 88 : 56;
  static constexpr int kPoolNeeded = NT * 128 * kRegsSoftmax + (kThreads - NT * 128) * kRegsOther;
  static constexpr uint32_t kTmemCols = NT * 256;      // S (and P) of each tile, then O of each
  static_assert(kCtasPerSm * kPoolNeeded <= 65536, "register file");
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 233472, "shared memory");
};

__device__ __forceinline__ float4 prefix_lds16(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
  return v;
}

__device__ __forceinline__ void prefix_tmem_st16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
      "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

// MOD: 0 plain with a positive scale, 1 ALiBi (or any scale), 2 soft-cap.
template <int D, int KV, int MOD>
__global__ void __launch_bounds__(PrefixCfg<D, KV>::kThreads, PrefixCfg<D, KV>::kCtasPerSm)
    fa_prefix_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const PrefixParams p) {
  using Cfg = PrefixCfg<D, KV>;
  constexpr int KC = Cfg::KC, NS = Cfg::NS, NT = Cfg::NT;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = blockIdx.x, hk = blockIdx.y;
  pdl_launch();   // the sequences' own keys need nothing of this pass

  // ------------------------------------------------------------ work tile --
  // The CTAs' rows (NT tiles) of all groups in a row; every warp finds this one's group.
  const int tokens = NT * p.tokens_per_tile;
  int grp = -1, tile = 0, q0 = 0, nq = 0, s0 = 0, s1 = 0, plen = 0;   // of the group: tokens, sequences, prefix
  {
    int before = 0;
    for (int g0 = 0; g0 < p.num_groups && grp < 0; g0 += 32) {
      const int g = g0 + lane;
      int first = 0, cnt = 0, a = 0, e = 0, len = 0;
      if (g < p.num_groups) {
        len = prefix_keys(p.prefix_lens, g, p.page_size, p.max_pages);
        a = min(max(__ldg(p.cu_groups + g), 0), p.num_seqs);
        e = min(max(__ldg(p.cu_groups + g + 1), a), p.num_seqs);
        first = __ldg(p.cu_q + a);
        cnt = __ldg(p.cu_q + e) - first;
        if (cnt > 0 && (first < 0 || (int64_t)first + cnt > p.total_q)) {   // rows outside q
          record_error(p.err, kErrBounds);
          cnt = 0;
        }
      }
      int tiles = cnt > 0 ? (cnt + tokens - 1) / tokens : 0;
      int incl = tiles;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, before + incl > (int)blockIdx.z);
      if (hit) {
        const int l = __ffs(hit) - 1;
        grp = g0 + l;
        tile = (int)blockIdx.z - before - __shfl_sync(0xffffffffu, incl - tiles, l);
        q0 = __shfl_sync(0xffffffffu, first, l);
        nq = __shfl_sync(0xffffffffu, cnt, l);
        s0 = __shfl_sync(0xffffffffu, a, l);
        s1 = __shfl_sync(0xffffffffu, e, l);
        plen = __shfl_sync(0xffffffffu, len, l);
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  if (split == 0 && hk == 0 && blockIdx.z == 0 && threadIdx.x == 0 &&
      (__ldg(p.cu_groups) != 0 || __ldg(p.cu_groups + p.num_groups) != p.num_seqs))
    record_error(p.err, kErrBounds);   // some sequence is in no group
  if (grp < 0) return;
  // row tile X starts at token tok0 + X tokens_per_tile and has rows_of(X) rows
  const int tok0 = q0 + tile * tokens, n_tok = q0 + nq - tok0;
  auto rows_of = [&](int X) { return max(0, min(p.tokens_per_tile, n_tok - X * p.tokens_per_tile)) * p.group; };
  const bool two = NT == 2 && n_tok > p.tokens_per_tile;

  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Cfg::kOffBar);
  uint64_t *q_full = bars, *q_conv = bars + 1, *k_full = q_conv + NT, *k_empty = k_full + NS, *k_stage = k_empty + NS,
           *v_full = k_stage + NS, *v_empty = v_full + NS, *v_stage = v_empty + NS, *s_full = v_stage + NS,
           *p_full = s_full + NT, *o_done = p_full + NT, *sc_full = o_done + NT;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + Cfg::kOffMisc);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + Cfg::kOffMisc + 8);
  int *range = reinterpret_cast<int *>(smem + Cfg::kOffMisc + 16);   // keys that any row sees
  const bool ranged = p.window > 0;          // rows decide which key tiles are visited
  if (threadIdx.x == 0) {
    range[0] = INT_MAX;
    range[1] = 0;
    *abort_flag = 0;
    const uint32_t n_fill = p.gather ? 32u : 1u;
    mbar_init(smem_u32(q_full), 1);
    for (int i = 0; i < NS; ++i) {
      mbar_init(smem_u32(k_full + i), KV ? 4 * KC : n_fill);
      mbar_init(smem_u32(k_empty + i), 1);
      mbar_init(smem_u32(k_stage + i), n_fill);
      mbar_init(smem_u32(v_full + i), KV ? 4 * KC : n_fill);
      mbar_init(smem_u32(v_empty + i), 1);
      mbar_init(smem_u32(v_stage + i), n_fill);
    }
    for (int X = 0; X < NT; ++X) {
      mbar_init(smem_u32(q_conv + X), 128);
      mbar_init(smem_u32(s_full + X), 1);
      mbar_init(smem_u32(p_full + X), 128);
      mbar_init(smem_u32(o_done + X), 1);
    }
    for (int i = 0; i < Cfg::NSS; ++i) mbar_init(smem_u32(sc_full + i), 2);
    fence_mbar_init();
  }
  if (warp == Cfg::kMmaWarp && !ranged) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  // Softmax thread r of tile X: token tok0 + X tokens_per_tile + r / group, head
  // hk * group + r % group, and the keys [row_lo, row_hi) of the prefix it sees.
  // Rows past the last see everything (they are never stored and must force no
  // masking).  Without a window the rows are looked up while the first keys are
  // on their way; with one they decide the key tiles first.
  int row_lo = 0, row_hi = INT_MAX, ip = 0;
  auto look_up_rows = [&]() {
    const int X = threadIdx.x >> 7, r = threadIdx.x & 127, rows = rows_of(X);
    // the row's sequence: the last that starts at or before its token, counted
    // by the warp 32 sequences at a time
    const int tok = tok0 + X * p.tokens_per_tile + min(r, max(rows - 1, 0)) / p.group;
    int b = s0 - 1;
    for (int i0 = s0; i0 < s1; i0 += 32) {
      const int start = i0 + lane < s1 ? __ldg(p.cu_q + i0 + lane) : INT_MAX;
#pragma unroll 8
      for (int k = 0; k < 32; ++k) b += __shfl_sync(0xffffffffu, start, k) <= tok;
    }
    if (r < rows) {
      const int qa = __ldg(p.cu_q + b), sq = __ldg(p.cu_q + b + 1) - qa;
      const int sk = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
      ip = tok - qa + sk - sq;
      row_hi = min(plen, sk);
      if (p.causal) row_hi = min(row_hi, ip + 1);
      if (p.window > 0) {
        row_lo = max(0, ip - p.window + 1);
        if (!p.causal) row_hi = min(row_hi, ip + p.window);
      }
      if (row_hi <= row_lo) row_lo = row_hi = 0;
    }
  };
  int seen_lo = 0, seen_hi = plen;           // keys that any row sees
  if (ranged) {
    __syncthreads();
    if (threadIdx.x < NT * 128) {
      look_up_rows();
      const bool live = (int)(threadIdx.x & 127) < rows_of(threadIdx.x >> 7);
      const int lo = __reduce_min_sync(0xffffffffu, live && row_hi > row_lo ? row_lo : INT_MAX);
      const int hi = __reduce_max_sync(0xffffffffu, live ? row_hi : 0);
      if (lane == 0) {
        atomicMin(range, lo);
        atomicMax(range + 1, hi);
      }
    }
    __syncthreads();
    seen_lo = range[0];
    seen_hi = range[1];
  }
  // this split's key tiles, of those that some row may see
  int kt_lo, kt_hi;
  {
    const int a = seen_hi > 0 ? seen_lo / kBlockN : 0, e = (seen_hi + kBlockN - 1) / kBlockN;
    // ranges of the same length in every group, so that a long prefix gets more
    // of them than a short one; the last takes what is left
    kt_lo = a + split * p.split_tiles;
    kt_hi = split == p.num_splits - 1 ? e : min(e, kt_lo + p.split_tiles);
  }
  if (kt_hi <= kt_lo) {
    for (int r = threadIdx.x; r < min(n_tok, tokens) * p.group; r += Cfg::kThreads)
      p.lse_part[((int64_t)split * p.hq + hk * p.group + r % p.group) * p.total_q + tok0 + r / p.group] = -INFINITY;
    if (!ranged) {
      tc_fence_before();
      __syncthreads();
      if (warp == Cfg::kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(*tmem_slot, Cfg::kTmemCols);
      }
    }
    return;
  }
  const int n_tiles = kt_hi - kt_lo;
  if (warp == Cfg::kMmaWarp && ranged) {
    tmem_alloc(smem_u32(tmem_slot), Cfg::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  uint8_t *sQ = smem + Cfg::kOffQ, *sK = smem + Cfg::kOffK, *sV = smem + Cfg::kOffV;
  float *sSc = reinterpret_cast<float *>(smem + Cfg::kOffSc);
  const int32_t *bt = p.block_table + (int64_t)s0 * p.bt_stride;   // the group's first sequence
  // Page of prefix key `key`, looked up ahead of its use: nothing here waits for
  // the value.  checked(): -1 (rows of zeros) past the prefix, or outside the
  // pool, which sets `bad`.
  constexpr int kNoPage = INT_MIN;
  auto page_of = [&](int key) { return key < plen ? __ldg(bt + (key >> p.page_shift)) : kNoPage; };
  bool bad = false;
  auto checked = [&](int pg) {
    const bool ok = pg >= 0 && pg < p.n_pages;
    bad = bad || (!ok && pg != kNoPage);
    return ok ? pg : -1;
  };

  if (warp >= Cfg::kProducerWarp) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsOther));

  if (warp == Cfg::kProducerWarp) {
    // ------------------------------------------------ producer: Q, K, V --
    if (lane == 0) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_k);
      prefetch_tmap(&tm_v);
      mbar_expect_tx(smem_u32(q_full), (uint32_t)((two ? 2 : 1) * KC * p.tokens_per_tile * p.group * 128));
      for (int X = 0; X < (two ? 2 : 1); ++X)
        for (int c = 0; c < KC; ++c)
          tma_load_3d(smem_u32(sQ + X * Cfg::kTileBytes + c * Cfg::kChunkBytes), &tm_q, smem_u32(q_full), c * 64,
                      hk * p.group, tok0 + X * p.tokens_per_tile);
    }
    uint64_t *kb = KV ? k_stage : k_full, *vb = KV ? v_stage : v_full;
    bool ok = true;
    int j = 0;
    if (p.gather) {
      GatherPipe<1> gp;
      // One slot in flight.  Waiting to refill K's slot the newest is V(j-1):
      // QK(j-NS), which frees the slot, needs K up to j-NS and V up to
      // j-NS-1.  Waiting for V's slot the newest is K(j): PV(j-NS) needs K and
      // V up to j-NS.
      auto pages = [&](int kt, int (&pg)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) pg[u] = kt < kt_hi ? page_of(kt * kBlockN + lane + 32 * u) : kNoPage;
      };
      int pg[4], pgn[4];
      pages(kt_lo, pg);
#pragma unroll
      for (int u = 0; u < 4; ++u) pg[u] = checked(pg[u]);
      for (; ok && j < n_tiles; ++j) {
        const int st = j % NS, key0 = (kt_lo + j) * kBlockN;
        pages(kt_lo + j + 1, pgn);
        if (lane == 0 && j >= NS) ok = mbar_wait(smem_u32(k_empty + st), ((j / NS) - 1) & 1, abort_flag, p.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          uint8_t *dst = sK + st * Cfg::kTileBytes + c * Cfg::kChunkBytes;
          if constexpr (KV) gather_block<kBlockN, 64, kGatherStage>(dst, p.gk, hk, key0, p.page_size - 1, c * 64, pg, lane);
          else gather_block<kBlockN, 128, kGatherSw128>(dst, p.gk, hk, key0, p.page_size - 1, c * 128, pg, lane);
        }
        gp.commit(smem_u32(kb + st));
        if (lane == 0 && j >= NS) ok = mbar_wait(smem_u32(v_empty + st), ((j / NS) - 1) & 1, abort_flag, p.err);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          uint8_t *dst = sV + st * Cfg::kTileBytes + c * Cfg::kChunkBytes;
          if constexpr (KV) gather_block<kBlockN, 64, kGatherStage>(dst, p.gv, hk, key0, p.page_size - 1, c * 64, pg, lane);
          else gather_block<kBlockN, 128, kGatherSw128>(dst, p.gv, hk, key0, p.page_size - 1, c * 128, pg, lane);
        }
        gp.commit(smem_u32(vb + st));
#pragma unroll
        for (int u = 0; u < 4; ++u) pg[u] = checked(pgn[u]);
      }
      gp.drain();
    } else {
      // Lane l < 128 / rows_per_box lands the boxes of rows l * rows_per_box..;
      // page ids are read one tile ahead.
      const int rb = p.rows_per_box, r0 = lane * rb;
      const bool boxer = r0 < kBlockN;
      auto page_at = [&](int kt) { return (boxer && kt < kt_hi) ? page_of(kt * kBlockN + r0) : kNoPage; };
      constexpr uint32_t kBytes = KV ? 128u * D : (uint32_t)Cfg::kTileBytes;
      auto load = [&](const CUtensorMap *tm, uint8_t *dst, uint64_t *bar, int kt, int pg) {
        if (!boxer) return;
        const int slot = (kt * kBlockN + r0) & (p.page_size - 1);
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          uint8_t *at = dst + c * Cfg::kChunkBytes;
          // bytes: raw rows of 64 in the upper half of their 32-row slice
          at += KV ? (r0 >> 5) * 4096 + 2048 + (r0 & 31) * 64 : r0 * 128;
          tma_load_4d(smem_u32(at), tm, smem_u32(bar), c * 64, hk, slot, pg);
        }
      };
      int pg = checked(page_at(kt_lo));
      for (; ok && j < n_tiles; ++j) {
        const int st = j % NS, kt = kt_lo + j;
        const int pg_next = page_at(kt + 1);
        if (lane == 0) {
          if (j >= NS) ok = mbar_wait(smem_u32(k_empty + st), ((j / NS) - 1) & 1, abort_flag, p.err);
          if (ok) mbar_expect_tx(smem_u32(kb + st), kBytes);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        load(&tm_k, sK + st * Cfg::kTileBytes, kb + st, kt, pg);
        if (lane == 0) {
          if (j >= NS) ok = mbar_wait(smem_u32(v_empty + st), ((j / NS) - 1) & 1, abort_flag, p.err);
          if (ok) mbar_expect_tx(smem_u32(vb + st), kBytes);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) {
          if (lane == 0) mbar_drain(smem_u32(kb + st), (j / NS) & 1);
          break;
        }
        load(&tm_v, sV + st * Cfg::kTileBytes, vb + st, kt, pg);
        pg = checked(pg_next);
      }
      // copies in flight land before the CTA ends, whatever the others do
      if (lane == 0)
        for (int i = max(0, j - NS); i < j; ++i) {
          mbar_drain(smem_u32(kb + i % NS), (i / NS) & 1);
          mbar_drain(smem_u32(vb + i % NS), (i / NS) & 1);
        }
    }
    if (lane == 0) mbar_drain(smem_u32(q_full), 0);
    if (bad) record_error(p.err, kErrBounds);
  } else if (warp == Cfg::kMmaWarp) {
    // ------------------------------------------------------- MMA issuer --
    if (elect_one()) {
      constexpr uint32_t id_qk = KV ? idesc_f16_f32(128, 128, 0, 0) : idesc_bf16_f32(128, 128, 0, 0);
      constexpr uint32_t id_pv = KV ? idesc_f16_f32(128, D, 0, 1) : idesc_bf16_f32(128, D, 0, 1);
      const uint64_t dq = smem_desc_sw128(smem_u32(sQ), 16, 1024);
      const uint64_t dv = smem_desc_sw128(smem_u32(sV), 128 * 128, 1024);
      const uint32_t hi = (uint32_t)(dq >> 32), lo_q = (uint32_t)dq;
      const uint32_t lo_k = (uint32_t)smem_desc_sw128(smem_u32(sK), 16, 1024);
      const uint32_t lo_v = (uint32_t)dv, hi_v = (uint32_t)(dv >> 32);
      auto qk = [&](int X, int st) {
        uint32_t a = lo_q + (uint32_t)(X * (Cfg::kTileBytes >> 4)), b = lo_k + (uint32_t)(st * (Cfg::kTileBytes >> 4));
        const uint32_t d = tmem + X * 128u;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          if (ks == 0) mma_ss_w<0>(d, a, hi, b, hi, id_qk);
          else mma_ss_w<1>(d, a, hi, b, hi, id_qk);
          const uint32_t step = ((ks + 1) & 3) ? 2u : (uint32_t)((128 * 128 - 96) >> 4);
          a += step;
          b += step;
        }
        tc_commit(smem_u32(s_full + X));
      };
      auto pv = [&](int X, int st, int j) {
        uint32_t b = lo_v + (uint32_t)(st * (Cfg::kTileBytes >> 4));
        const uint32_t a = tmem + X * 128u, d = tmem + NT * 128u + X * 128u;
#pragma unroll
        for (int ks = 0; ks < kBlockN / 16; ++ks) {
          mma_ts_w(d, a + ks * 8, b, hi_v, id_pv, (ks > 0 || j > 0) ? 1u : 0u);
          b += (16 * 128) >> 4;
        }
        tc_commit(smem_u32(o_done + X));
      };
      bool ok = mbar_wait(smem_u32(KV ? q_conv : q_full), 0, abort_flag, p.err);
      if (ok && KV && two) ok = mbar_wait(smem_u32(q_conv + 1), 0, abort_flag, p.err);
      if (ok) ok = mbar_wait(smem_u32(k_full), 0, abort_flag, p.err);
      if (ok) {
        tc_fence_after();
        qk(0, 0);
        if (two) qk(1, 0);
        tc_commit(smem_u32(k_empty));
      }
      for (int j = 0; ok && j < n_tiles; ++j) {
        const int st = j % NS, sn = (j + 1) % NS;
        const bool more = j + 1 < n_tiles;
        if (!(ok = mbar_wait(smem_u32(v_full + st), (j / NS) & 1, abort_flag, p.err))) break;
        if (!(ok = mbar_wait(smem_u32(p_full), j & 1, abort_flag, p.err))) break;
        tc_fence_after();
        pv(0, st, j);
        if (!two) tc_commit(smem_u32(v_empty + st));
        if (more) {
          if (!(ok = mbar_wait(smem_u32(k_full + sn), ((j + 1) / NS) & 1, abort_flag, p.err))) break;
          tc_fence_after();
          qk(0, sn);
        }
        if (two) {
          if (!(ok = mbar_wait(smem_u32(p_full + 1), j & 1, abort_flag, p.err))) break;
          tc_fence_after();
          pv(1, st, j);
          tc_commit(smem_u32(v_empty + st));
          if (more) qk(1, sn);
        }
        if (more) tc_commit(smem_u32(k_empty + sn));
      }
    }
  } else if (warp >= Cfg::kFirstConverter) {
    // ---------------------------------------- converters (byte caches) --
    // Slices of 32 rows x 64 columns, K's then V's of a tile, in turn to the
    // six warps.  A slice's bytes lie in the upper half of its own f16 output.
    if constexpr (KV != 0) {
      const int cw = warp - Cfg::kFirstConverter;
      // the first two warps bring the K and the V scales of a tile, one tile ahead
      const float *sc_src = cw == 1 ? p.v_scale : p.k_scale;
      // (their pages two)
      auto pages = [&](int kt, int (&pg)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) pg[u] = cw < 2 && kt < kt_hi ? page_of(kt * kBlockN + lane + 32 * u) : kNoPage;
      };
      auto scales = [&](int kt, const int (&pg)[4], float (&s)[4]) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = kt * kBlockN + lane + 32 * u, at = checked(pg[u]);
          s[u] = at >= 0 ? __ldg(sc_src + ((int64_t)at * p.page_size + (key & (p.page_size - 1))) * p.hkv + hk) : 0.f;
        }
      };
      int pg[4];
      float sc[4], scn[4];
      pages(kt_lo, pg);
      scales(kt_lo, pg, sc);
      pages(kt_lo + 1, pg);
      bool ok = true;
      for (int j = 0; ok && j < n_tiles; ++j) {
        const int st = j % NS;
        scales(kt_lo + j + 1, pg, scn);
        pages(kt_lo + j + 2, pg);
        float *slot = sSc + (j % Cfg::NSS) * Cfg::kScWords;
        for (int half = 0; ok && half < 2; ++half) {
          uint64_t *stage = half ? v_stage : k_stage, *full = half ? v_full : k_full;
          ok = mbar_wait(smem_u32(stage + st), (j / NS) & 1, abort_flag, p.err);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (half == 0 && cw == 0) {
#pragma unroll
            for (int u = 0; u < 4; ++u) slot[lane + 32 * u] = sc[u];
          } else if (half == 0 && cw == 1) {
            // E: the largest |v_scale| is below 2^E (E held within +-40)
            float mv = fmaxf(fmaxf(fabsf(sc[0]), fabsf(sc[1])), fmaxf(fabsf(sc[2]), fabsf(sc[3])));
#pragma unroll
            for (int o = 16; o; o >>= 1) mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
            const int e = min(max((int)((__float_as_uint(mv) >> 23) & 0xFF) - 126, -40), 40);
            const float f = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
            for (int u = 0; u < 4; ++u) slot[128 + lane + 32 * u] = __uint_as_float(pack_f16x2(sc[u] * f, sc[u] * f));
            if (lane == 0) slot[256] = (float)e;
          }
          if (half == 0 && cw < 2) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(sc_full + j % Cfg::NSS));
          }
          if (half == 1) {   // every converter needs the V scales
            ok = mbar_wait(smem_u32(sc_full + j % Cfg::NSS), (j / Cfg::NSS) & 1, abort_flag, p.err);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
          }
          uint8_t *tile_base = (half ? sV : sK) + st * Cfg::kTileBytes;
          for (int sl = (cw + (half ? 4 * KC : 0)) % Cfg::kConverters; sl < 4 * KC; sl += Cfg::kConverters) {
            uint8_t *base = tile_base + (sl >> 2) * Cfg::kChunkBytes + (sl & 3) * 4096;
            const uint8_t *stg = base + 2048;
            // all rows are read before any is written, so that their latencies overlap
            const int part = lane & 3;
            uint4 raw[4];
            uint32_t f[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int rr = 8 * t + (lane >> 2);
              raw[t] = *reinterpret_cast<const uint4 *>(stg + rr * 64 + part * 16);
              f[t] = half ? __float_as_uint(slot[128 + (sl & 3) * 32 + rr]) : 0u;
            }
            __syncwarp();
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const int rr = 8 * t + (lane >> 2);
              uint32_t h[8];
              dec_bytes4_to_f16<KV>(raw[t].x, h[0], h[1]);
              dec_bytes4_to_f16<KV>(raw[t].y, h[2], h[3]);
              dec_bytes4_to_f16<KV>(raw[t].z, h[4], h[5]);
              dec_bytes4_to_f16<KV>(raw[t].w, h[6], h[7]);
              if (half) {
#pragma unroll
                for (int k = 0; k < 8; ++k) asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(h[k]) : "r"(f[t]));
              }
              *reinterpret_cast<uint4 *>(base + sw128(rr, 2 * part)) = make_uint4(h[0], h[1], h[2], h[3]);
              *reinterpret_cast<uint4 *>(base + sw128(rr, 2 * part + 1)) = make_uint4(h[4], h[5], h[6], h[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(full + st));
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) sc[u] = scn[u];
      }
    }
  } else {
    // ---------------------------------------------------------- softmax --
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg::kRegsSoftmax));
    const int X = warp >> 2, r = threadIdx.x & 127, rows = rows_of(X);
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t sa = tmem + lane_base + X * 128u, oa = tmem + lane_base + NT * 128u + X * 128u;
    bool ok = true;
    const int n_steps = rows > 0 ? n_tiles : 0;   // a second tile without rows takes no part
    if (!ranged) look_up_rows();
    float rowf = 1.f;
    if constexpr (KV != 0) {
      // Q to f16 in place, with a power-of-two factor per row (max|q| 2^e in
      // [2^14, 2^15)); row r owns 128 bytes of each block, visited from chunk
      // r mod 8 on so that a warp's accesses spread over all banks.
      ok = mbar_wait(smem_u32(q_full), 0, abort_flag, p.err);
      if (ok && rows > 0) {
        uint8_t *qrow = sQ + X * Cfg::kTileBytes + r * 128;
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const uint4 w = *reinterpret_cast<const uint4 *>(qrow + c * Cfg::kChunkBytes + ((u + r) & 7) * 16);
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(ww[k] << 16)), fabsf(__uint_as_float(ww[k] & 0xFFFF0000u))));
          }
        int sh = 0;
        if (amax > 0.f && amax <= 3.0e38f) sh = min(141 - (int)((__float_as_uint(amax) >> 23) & 0xFF), 126);
        const float up = __uint_as_float((uint32_t)(sh + 127) << 23);
        rowf = __uint_as_float((uint32_t)(127 - sh) << 23);
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            uint4 *ptr = reinterpret_cast<uint4 *>(qrow + c * Cfg::kChunkBytes + ((u + r) & 7) * 16);
            const uint4 w = *ptr;
            const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
            uint32_t hh[4];
#pragma unroll
            for (int k = 0; k < 4; ++k)
              hh[k] = pack_f16x2(__uint_as_float(ww[k] << 16) * up, __uint_as_float(ww[k] & 0xFFFF0000u) * up);
            *ptr = make_uint4(hh[0], hh[1], hh[2], hh[3]);
          }
        fence_proxy_async_smem();
      }
      mbar_arrive(smem_u32(q_conv + X));
    }
    const float sl2 = p.scale_log2 * rowf;
    const float c2u = 2.f * kLog2e * p.softcap_arg * rowf;
    // plain scores keep their scale for the exponent's FMA
    constexpr bool raw = MOD == 0;
    const float cexp = raw ? sl2 : 1.f;
    float m_ref = -INFINITY, l = 0.f;
    for (int j = 0; ok && j < n_steps; ++j) {
      const int j0 = (kt_lo + j) * kBlockN;
      const float *ks = sSc + (j % Cfg::NSS) * Cfg::kScWords;
      const uint32_t ks_at = smem_u32(ks);
      float E = 0.f;       // byte caches: V stands at 2^-E
      if constexpr (KV != 0) {
        ok = mbar_wait(smem_u32(sc_full + j % Cfg::NSS), (j / Cfg::NSS) & 1, abort_flag, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        E = ks[256];
      }
      const bool need_mask = __any_sync(0xffffffffu, j0 < row_lo || j0 + kBlockN > row_hi);
      ok = mbar_wait(smem_u32(s_full + X), j & 1, abort_flag, p.err);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      tc_fence_after();
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      float alpha_tile = 1.f;
      bool warp_need = false;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        // the K scales come while the scores do, half a tile's at once (each read
        // just before its use, the softmax waited for shared memory: 192 sequences
        // of 4 heads behind 65536 int8 keys 330 -> 314 us)
        float4 kk[KV ? 16 : 1];
        if constexpr (KV != 0) {
#pragma unroll
          for (int e = 0; e < 16; ++e) kk[e] = prefix_lds16(ks_at + hf * 256 + e * 16);
        }
        float v[64];
        tmem_ld32(sa + hf * 64, *reinterpret_cast<float(*)[32]>(v));
        tmem_ld32(sa + hf * 64 + 32, *reinterpret_cast<float(*)[32]>(v + 32));
        tmem_wait_ld();
        const int jc = j0 + hf * 64;
        if constexpr (KV != 0) {
#pragma unroll
          for (int e = 0; e < 64; e += 4) {
            const float4 k4 = kk[e >> 2];
            mul2p(v[e], v[e + 1], k4.x, k4.y);
            mul2p(v[e + 2], v[e + 3], k4.z, k4.w);
          }
        }
        if constexpr (!raw) {
          // cap tanh(u) = cap - 2 cap / (1 + 2^x), x = 2 u log2 e
          if constexpr (MOD == 2 && KV != 0) {
            const float cl = p.softcap_log2;
#pragma unroll
            for (int e = 0; e < 64; e += 2) mul2(v[e], v[e + 1], c2u);
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = ex2(v[e]);
#pragma unroll
            for (int e = 0; e < 64; e += 2) add2(v[e], v[e + 1], 1.f, 1.f);
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = rcp_approx(v[e]);
#pragma unroll
            for (int e = 0; e < 64; e += 2) fma2(v[e], v[e + 1], v[e], v[e + 1], -2.f * cl, cl);
          }
          if constexpr (MOD == 2 && KV == 0) {
            // Four scores share a reciprocal, since the MUFU (16 operations a
            // cycle and SM) takes 2.25 of them per score then instead of 3: over
            // 65536 keys, 6144 rows, 314 -> 284 us.  (Byte caches are bound by
            // shared memory: 362 us as above, 381 this way.)  With
            // a = min(1, 2^-30 + 2^(x - 30)) the product of four stays above
            // 2^-121, and 2^-30 is below half a step of 1.  A NaN becomes a = 0,
            // an infinite reciprocal, and NaN in its neighbours: they are cleared
            // of hidden scores first, and a visible one marks the row itself.
            if (need_mask) {
              const int elo = row_lo - jc, ehi = row_hi - jc;
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                const bool on = e >= elo && e < ehi;
                if (on && v[e] != v[e]) sum[0] = v[e];
                v[e] = on ? v[e] : 0.f;
              }
            }
            const float cl = p.softcap_log2;
#pragma unroll
            for (int e = 0; e < 64; e += 2) fma2(v[e], v[e + 1], v[e], v[e + 1], c2u, -30.f);
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = add_sat(ex2(v[e]), 0x1p-30f);
#pragma unroll
            for (int e = 0; e < 64; e += 4) {
              float x0, x1, x2, x3;
              rcp4(v[e], v[e + 1], v[e + 2], v[e + 3], x0, x1, x2, x3);
              fma2(v[e], v[e + 1], x0, x1, -0x1p-29f * cl, cl);
              fma2(v[e + 2], v[e + 3], x2, x3, -0x1p-29f * cl, cl);
            }
          }
          if constexpr (MOD == 1) {
#pragma unroll
            for (int e = 0; e < 64; e += 2) mul2(v[e], v[e + 1], sl2);
            const float dbase = (float)(ip - jc);
#pragma unroll
            for (int e = 0; e < 64; ++e) v[e] = fmaf(-p.alibi_log2, fabsf(dbase - (float)e), v[e]);
          }
        }
        if (need_mask) {
          const int elo = row_lo - jc, ehi = row_hi - jc;
#pragma unroll
          for (int e = 0; e < 64; ++e) v[e] = (e >= elo && e < ehi) ? v[e] : -INFINITY;
        }
        float t1[22];
#pragma unroll
        for (int k = 0; k < 21; ++k) t1[k] = max3(v[3 * k], v[3 * k + 1], v[3 * k + 2]);
        t1[21] = v[63];
        float t2[8];
#pragma unroll
        for (int k = 0; k < 7; ++k) t2[k] = max3(t1[3 * k], t1[3 * k + 1], t1[3 * k + 2]);
        t2[7] = t1[21];
        float hmax = fmaxf(max3(t2[0], t2[1], t2[2]), fmaxf(max3(t2[3], t2[4], t2[5]), fmaxf(t2[6], t2[7])));
        if (raw && hmax != -INFINITY) hmax *= sl2;
        if constexpr (KV != 0) hmax += E;
        const float m_new = fmaxf(m_ref, hmax);
        const bool need = m_new > m_ref + kRescaleThreshold;
        if (__any_sync(0xffffffffu, need)) {
          const float alpha = need ? ex2(m_ref - m_new) : 1.f;   // 0 when m_ref is -inf
          if (need) {
            m_ref = m_new;
            l *= alpha;
#pragma unroll
            for (int q = 0; q < 4; ++q) sum[q] *= alpha;
          }
          alpha_tile *= alpha;
          warp_need = true;
          if (hf == 1) {
            // P of the first half was taken against the old reference
            tmem_wait_st();
            float pw[32];
            tmem_ld32(sa, pw);
            tmem_wait_ld();
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const uint32_t u = __float_as_uint(pw[e]);
              if constexpr (KV != 0) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u));
                w[e] = pack_f16x2(f.x * alpha, f.y * alpha);
              } else {
                w[e] = pack_bf16x2(__uint_as_float(u << 16) * alpha, __uint_as_float(u & 0xFFFF0000u) * alpha);
              }
            }
            tmem_st32(sa, w);
          }
        }
        const float m_use = m_ref == -INFINITY ? 0.f : m_ref - E;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float t0, t1_, t2_, t3;
            fma2(t0, t1_, v[32 * c + e], v[32 * c + e + 1], cexp, -m_use);
            fma2(t2_, t3, v[32 * c + e + 2], v[32 * c + e + 3], cexp, -m_use);
            t0 = ex2(t0);
            t1_ = ex2(t1_);
            t2_ = ex2(t2_);
            t3 = ex2(t3);
            add2(sum[0], sum[1], t0, t1_);
            add2(sum[2], sum[3], t2_, t3);
            pk[e / 2] = KV ? pack_f16x2(t0, t1_) : pack_bf16x2(t0, t1_);
            pk[e / 2 + 1] = KV ? pack_f16x2(t2_, t3) : pack_bf16x2(t2_, t3);
          }
          prefix_tmem_st16(sa + hf * 32 + c * 16, pk);
        }
      }
      const float tile_sum = (sum[0] + sum[1]) + (sum[2] + sum[3]);
      // the weights carry 2^E, the row sum does not
      l += KV ? tile_sum * __uint_as_float((uint32_t)(127 - (int)E) << 23) : tile_sum;
      if (warp_need && j > 0) {
        ok = mbar_wait(smem_u32(o_done + X), (j - 1) & 1, abort_flag, p.err);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(oa + c * 32, o);
          tmem_wait_ld();
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(o[e] * alpha_tile);
          tmem_st32(oa + c * 32, w);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(smem_u32(p_full + X));
    }
    // -------------------------------------------------------- epilogue --
    if (ok && n_steps > 0) {
      ok = mbar_wait(smem_u32(o_done + X), (n_tiles - 1) & 1, abort_flag, p.err);
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        const bool has = l > 0.f;
        const float inv = has ? 1.f / l : 0.f;
        const int64_t t = (int64_t)tok0 + X * p.tokens_per_tile + r / p.group;
        const int h = hk * p.group + r % p.group;
        float *dst = p.o_part + (((int64_t)split * p.total_q + t) * p.hq + h) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_ld32(oa + c * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = has ? o[e] * inv : 0.f;
          if (r < rows) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) st_global_f8(dst + c * 32 + e, o + e);
          }
        }
        if (r < rows)
          p.lse_part[((int64_t)split * p.hq + h) * p.total_q + t] = has ? (m_ref + __log2f(l)) * kLn2 : -INFINITY;
      }
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
