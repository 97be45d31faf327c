// fa_suffix.cuh -- decode of each sequence's own keys behind a shared prefix.
//
// Behind a prefix the sequences are short and ragged (tens to a few thousand
// keys), so a CTA that stages keys in shared memory spends much of its life
// filling its pipeline and merging its warps.  Here a warp works alone on one
// (key range, kv head, sequence): keys and values come through a ring of its
// own into MMA fragments (fa_rows.cuh), the softmax state is the warp's, and its
// partial (O, LSE) goes to the merge that joins it with the prefix's.  No
// barriers, and any page size.  Bound by HBM: 64 sequences of up to 1024 own
// keys, bf16, 27 us (4.7 TB/s); 192 of up to 2048, int8, 87 us (4.6 TB/s).
//
//   S^T = K Q^T          M = 16 keys, N = 8 rows: lane (g, t) gets keys g, g + 8
//                        (in the order of RowsBlocks::row) of rows 2t, 2t + 1
//   P^T by movmatrix     to the B operand of
//   O^T += V^T P^T       M = 16 dims, N = 8 rows, contracted over the 16 keys.
//                        Lane (g, t) reads D / 8 dims of the keys 2t, 2t + 1,
//                        2t + 8, 2t + 9, and a byte permute of two keys' words
//                        makes each A register's key pair; dims 2m and 2m + 1
//                        of the lane's are rows g and g + 8 of m-tile m.
//
// The running maximum moves only when a score
// exceeds it by 2^8 (then all lanes agree by shuffles); a group's check is two
// compares and a vote.  Byte caches: k_scale multiplies the scores, v_scale
// the weights, and the reference includes log2 v_scale, so that the f16
// weights use their range whatever the magnitude of V.
#pragma once
#include "fa_rows.cuh"

namespace fa {

struct SuffixParams {
  const __nv_bfloat16 *q;
  int64_t q_stride_t, q_stride_h;     // elements
  const int32_t *cu_q, *cu_k, *cu_groups, *prefix_lens;
  int32_t num_groups;
  const int32_t *block_table;
  int64_t bt_stride, max_pages, n_pages;
  int32_t page_size, page_shift;
  int32_t small_pages;                // fewer than 16 keys: row copies instead of boxes
  const uint8_t *k, *v;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;   // bytes
  const float *k_scale, *v_scale;     // byte caches: [N_pg, P_s, Hkv]
  int32_t num_seqs, hq, hkv, group;
  int32_t split_keys, num_splits;     // the last range runs to the sequence's end
  float *o_part;                      // [num_splits][T_q][Hq][D]
  float *lse_part;                    // [num_splits][Hq][T_q]
  int64_t total_q;
  int32_t mod, causal, window;
  float scale_log2, alibi_log2, softcap_arg, softcap_log2;
  int *err;
};

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 32 bytes, one sector.
__device__ __forceinline__ void st_global_f8(float *dst, const float *v) {
  asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

constexpr int kSufWarps = 4;

// The ring, and what the fragments read of a value row: per lane D / 8 dims,
// bf16 pieces g and g + 8, bytes one piece of 16 or 8 bytes.
template <int D, int KV>
struct SufCfg {
  static constexpr int kRow = D * (KV ? 1 : 2);
  static constexpr int kStages = kRow >= 256 ? 2 : (kRow >= 128 ? 3 : 4);
  using Ring = RowsRing<kRow, kRow, KV != 0, kStages>;
  static constexpr int NP = kRow / 64;                   // 16-byte key pieces per row and lane
  static constexpr int WV = kRow / 32;                   // 32-bit words per value row and lane
  static constexpr int kSmemBytes = kSufWarps * Ring::kBytes + 1024;
  // what the registers of one row tile allow; shared memory allows as many
  static constexpr int kCtasPerSm = kRow >= 256 ? 3 : 4;
  static_assert(kCtasPerSm * (kSmemBytes + 1024) <= 233472, "shared memory");
};

// A registers (one key pair) of the lane's dims: word i of keys a and b ->
// bf16 dims 2i, 2i + 1; bytes dims 4i ... 4i + 3.
template <int KV>
__device__ __forceinline__ void suf_pairs(uint32_t a, uint32_t b, uint32_t *o) {
  if constexpr (KV == 0) {
    o[0] = __byte_perm(a, b, 0x5410);
    o[1] = __byte_perm(a, b, 0x7632);
  } else {
    dec_bytes4_to_f16<KV>(__byte_perm(a, b, 0x5140), o[0], o[1]);
    dec_bytes4_to_f16<KV>(__byte_perm(a, b, 0x7362), o[2], o[3]);
  }
}

template <int D, int KV, int NT>
__device__ __forceinline__ void suffix_warp(const CUtensorMap *tm_k, const CUtensorMap *tm_v, const SuffixParams &p) {
  using Cfg = SufCfg<D, KV>;
  using Ring = typename Cfg::Ring;
  constexpr int NP = Cfg::NP, WV = Cfg::WV, S = Cfg::kStages;
  constexpr int MT = D / 16;                  // m-tiles of the output
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // The warps of a CTA take neighbouring kv heads: the same keys' rows, side by
  // side in memory, and so the same amount of work.
  const int64_t unit = (int64_t)blockIdx.x * kSufWarps + warp;
  const int hk = (int)(unit % p.hkv);
  const int64_t sb = unit / p.hkv;
  const int split = (int)(sb / p.num_seqs), b = (int)(sb % p.num_seqs);
  if (split >= p.num_splits) return;
  const int qa = __ldg(p.cu_q + b), sq = __ldg(p.cu_q + b + 1) - qa;
  int sk = __ldg(p.cu_k + b + 1) - __ldg(p.cu_k + b);
  const int shift = sk - sq;
  int rows = sq * p.group;
  if (rows <= 0) return;
  if (qa < 0 || (int64_t)qa + sq > p.total_q) {   // rows outside q
    if (lane == 0) record_error(p.err, kErrBounds);
    return;
  }
  // lengths that the host's bounds or the page table do not cover
  if (rows > NT * 8 || sk > p.max_pages * p.page_size) {
    if (lane == 0) record_error(p.err, kErrBounds);
    rows = min(rows, NT * 8);
    sk = (int)min((int64_t)sk, p.max_pages * p.page_size);
  }
  int lo = split * p.split_keys;
  {
    const int grp = upper_bound_i32(p.cu_groups, 0, p.num_groups + 1, b) - 1;
    if (grp >= 0 && grp < p.num_groups) lo += prefix_keys(p.prefix_lens, grp, p.page_size, p.max_pages);
  }
  const int hi = split == p.num_splits - 1 ? sk : min(sk, lo + p.split_keys);
  // the first row's first key (the others see later ones), at the start of its group
  if (p.window > 0 && shift - p.window + 1 > lo) lo += (shift - p.window + 1 - lo) & ~15;
  const int64_t part = (int64_t)split * p.total_q;
  if (lo >= hi) {
    for (int r = lane; r < rows; r += 32)
      p.lse_part[((int64_t)split * p.hq + hk * p.group + r % p.group) * p.total_q + qa + r / p.group] = -INFINITY;
    return;
  }
  const int32_t *bt = p.block_table + (int64_t)b * p.bt_stride;
  const int smask = p.page_size - 1;
  // Lane l stands for the key row (l < 16) or the value row of key base + l % 16.
  const bool isv = lane >= 16, small = p.small_pages != 0;
  bool bad = false;
  auto page_at = [&](int base) -> int {
    const int j = base + (lane & 15);
    if (j >= hi) return -1;
    const int pg = __ldg(bt + (j >> p.page_shift));
    const bool ok = pg >= 0 && pg < p.n_pages;
    bad = bad || !ok;
    return ok ? pg : -1;
  };
  const uint8_t *head = isv ? p.v + (int64_t)hk * p.v_head : p.k + (int64_t)hk * p.k_head;
  const int64_t s_page = isv ? p.v_page : p.k_page, s_slot = isv ? p.v_slot : p.k_slot;
  const float *scales = isv ? p.v_scale : p.k_scale;
  Ring ring;
  ring.init(smem + warp * Ring::kBytes);
  auto copy = [&](int base, int pg) {
    const int at = (base + (lane & 15)) & smask;
    const bool live = pg >= 0;
    const uint8_t *row = live && small ? head + (int64_t)pg * s_page + (int64_t)at * s_slot : nullptr;
    const float *sc = KV && live ? scales + ((int64_t)pg * p.page_size + at) * p.hkv + hk : nullptr;
    ring.start(base < hi, small, tm_k, tm_v, hk, false, pg, base & smask, row, sc);
  };
  // the first S - 1 groups; then group i + S - 1 is copied while group i is used
  int pgn;
  {
    int pg[S - 1];
#pragma unroll
    for (int i = 0; i < S - 1; ++i) pg[i] = page_at(lo + 16 * i);
    pgn = page_at(lo + 16 * (S - 1));
#pragma unroll
    for (int i = 0; i < S - 1; ++i) copy(lo + 16 * i, pg[i]);
  }
  uint32_t qb[D / 16][NT][2];
  float inv[NT];
  rows_q_fragments<D, KV, NT>(p.q, p.q_stride_t, p.q_stride_h, qa, hk, p.group, rows, qb, inv);
  // rows 8 nt + 2t + e of this lane's columns
  const RowsVisible vb = rows_visible(p.causal, p.window);
  float sc[NT][2], m[NT][2], l[NT][2];
  int ip[NT][2];                              // i' - lo - g + the mask's offset
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = nt * 8 + 2 * t + e;
      const float f = __shfl_sync(0xffffffffu, inv[nt], (2 * t + e) * 4);
      sc[nt][e] = (p.mod == 2 ? 2.f * kLog2e * p.softcap_arg : p.scale_log2) * f;
      ip[nt][e] = r < rows ? r / p.group + shift + vb.add - lo - Ring::K::row(g) : kRowsHidden;
      m[nt][e] = -INFINITY;
      l[nt][e] = 0.f;
    }
  float o[NT][MT][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < MT; ++i) o[nt][i][0] = o[nt][i][1] = o[nt][i][2] = o[nt][i][3] = 0.f;

  // fragment rows: keys kg and kg + 8 of a group; values index 2t and 2t + 1
  const int kg = Ring::K::row(g), v0 = Ring::V::row(2 * t), v1 = Ring::V::row(2 * t + 1);
  bool ok = true;
  for (int base = lo; base < hi; base += 16) {
    const int ahead = base + 16 * (S - 1);
    copy(ahead, pgn);
    pgn = page_at(ahead + 16);
    ok = ring.wait(small, p.err);
    if (!ok) break;
    const uint32_t st = ring.slot();
    if (!small && base + 16 > hi) {
      // value rows behind the last key may hold anything (0 * NaN is NaN)
      for (int r = hi - base; r < 16; ++r)
        if (lane < Cfg::kRow / 16)
          asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(st + Ring::kOffV + Ring::V::at(lane, r)), "r"(0u) : "memory");
    }
    if (KV || small || base + 16 > hi) __syncwarp();   // what other lanes copied or cleared
    float c[NT][4];
    {
      uint4 kr[2][NP];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < NP; ++i) kr[u][i] = rows_lds16(st + Ring::K::at(t + 4 * i, kg + 8 * u));
      rows_qk<D, KV, NT>(kr[0], kr[1], qb, c);
    }
    float vsc[2] = {1.f, 1.f}, ksc[2] = {1.f, 1.f}, lv[2] = {0.f, 0.f};
    if constexpr (KV != 0) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        ksc[u] = rows_lds4(ring.scales() + (kg + 8 * u) * 4);
        vsc[u] = rows_lds4(ring.scales() + 64 + (kg + 8 * u) * 4);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) lv[u] = __log2f(fminf(fmaxf(fabsf(vsc[u]), 0x1p-40f), 0x1p40f));
    }
    // scores in log2 units, -inf where hidden
    bool over = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int x = 0; x < 4; ++x) {           // key kg + 8 (x / 2), row 2t + x % 2
        const int e = x & 1, u = x >> 1;
        const int d = ip[nt][e] - (base - lo) - 8 * u;
        float y = c[nt][x] * (KV ? sc[nt][e] * ksc[u] : sc[nt][e]);
        if (p.mod == 2) {
          float r;
          y = softcap_log2_score(ex2(y), p.softcap_log2, r);
        } else if (p.mod == 1) {
          y = fmaf(-p.alibi_log2, fabsf((float)(d - vb.add)), y);
        }
        const bool vis = (unsigned)d < vb.range && base + kg + 8 * u < hi;
        c[nt][x] = vis ? y : -INFINITY;
        over = over || c[nt][x] + lv[u] > m[nt][e] + 8.f;
      }
    if (__any_sync(0xffffffffu, over)) {
      // some row's reference moves: maxima over the 16 keys (the lanes of each t)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float mx = fmaxf(c[nt][e] + lv[0], c[nt][2 + e] + lv[1]);
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
          if (mx > m[nt][e] + 8.f) {
            const float a = ex2(m[nt][e] - mx);   // 0 when the row had none
            m[nt][e] = mx;
            l[nt][e] *= a;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
              o[nt][i][e] *= a;
              o[nt][i][2 + e] *= a;
            }
          }
        }
    }
    uint32_t pb[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float w[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const float mr = m[nt][x & 1] == -INFINITY ? 0.f : m[nt][x & 1];
        w[x] = ex2(c[nt][x] - mr);
        l[nt][x & 1] += w[x];
      }
#pragma unroll
      for (int u = 0; u < 2; ++u)
        pb[nt][u] = movmatrix_trans(KV ? pack_f16x2(w[2 * u] * vsc[u], w[2 * u + 1] * vsc[u]) : pack_bf16x2(w[2 * u], w[2 * u + 1]));
    }
    constexpr int NM = KV ? 2 : 1;            // m-tiles per value word
#pragma unroll
    for (int q = 0; q < (WV + 3) / 4; ++q) {
      uint32_t vr[4][4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = ((u & 1) ? v1 : v0) + 8 * (u >> 1);
        if constexpr (WV == 2) {
          const uint2 x = rows_lds8(st + Ring::kOffV + Ring::V::at(g >> 1, row) + 8 * (g & 1));
          vr[u][0] = x.x;
          vr[u][1] = x.y;
        } else {
          const uint4 x = rows_lds16(st + Ring::kOffV + Ring::V::at(g + 8 * q, row));
          vr[u][0] = x.x;
          vr[u][1] = x.y;
          vr[u][2] = x.z;
          vr[u][3] = x.w;
        }
      }
#pragma unroll
      for (int i = 0; i < (WV < 4 ? WV : 4); ++i) {
        uint32_t a01[2 * NM], a23[2 * NM];
        suf_pairs<KV>(vr[0][i], vr[1][i], a01);
        suf_pairs<KV>(vr[2][i], vr[3][i], a23);
#pragma unroll
        for (int k = 0; k < NM; ++k) {
          const uint32_t a[4] = {a01[2 * k], a01[2 * k + 1], a23[2 * k], a23[2 * k + 1]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) dec_mma<KV>(o[nt][NM * (4 * q + i) + k], a, pb[nt][0], pb[nt][1]);
        }
      }
    }
    ring.next();
  }
  if (!ok) {
    ring.drain();
    return;
  }
  if (bad) record_error(p.err, kErrBounds);
  // partial output and LSE
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float s = l[nt][e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      const int r = nt * 8 + 2 * t + e;
      if (r >= rows) continue;
      const bool has = s > 0.f;
      const float iv = has ? 1.f / s : 0.f;
      const int64_t tok = (int64_t)qa + r / p.group;
      const int h = hk * p.group + r % p.group;
      float *dst = p.o_part + ((part + tok) * p.hq + h) * D;
#pragma unroll
      for (int i = 0; i < MT / 4; ++i) {      // 8 consecutive dims at a time
        float v[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[2 * k] = o[nt][4 * i + k][e] * iv;
          v[2 * k + 1] = o[nt][4 * i + k][2 + e] * iv;
        }
        // bf16: pieces g and g + 8 of 8 dims; bytes: the lane's 16 (or 8) in a row
        st_global_f8(dst + (KV ? g * (D / 8) + 8 * i : 8 * (g + 8 * i)), v);
      }
      if (g == 0) p.lse_part[((int64_t)split * p.hq + h) * p.total_q + tok] = has ? (m[nt][e] + __log2f(s)) * kLn2 : -INFINITY;
    }
}

// Runs beside the prefix pass, which it does not depend on (launched behind it
// with launch_behind).  It ends after the prefix pass, so that whatever waits
// for this kernel also finds the prefix's partials.
template <int D, int KV, int NT>
__global__ void __launch_bounds__(kSufWarps * 32, SufCfg<D, KV>::kCtasPerSm / NT) fa_suffix_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const SuffixParams p) {
  pdl_launch();
  suffix_warp<D, KV, NT>(&tm_k, &tm_v, p);
  pdl_wait();
}

}  // namespace fa
