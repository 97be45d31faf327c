// Instantiations and launcher of the shared-prefix pass (fa_prefix.cuh), and
// the merge of its partials with those of the sequences' own keys.
#include "fa_internal.h"

namespace fa {
namespace {

template <int D, int KV, int MOD>
cudaError_t prefix_one(const PrefixLaunch &L) {
  using Cfg = PrefixCfg<D, KV>;
  static unsigned long long done = 0;
  auto kern = fa_prefix_kernel<D, KV, MOD>;
  // The softmax warps wait for registers that the others release: the launch
  // has to hold the whole split (the same for every device of a process).
  static int fits = -1;
  if (fits < 0) {
    cudaFuncAttributes a;
    fits = cudaFuncGetAttributes(&a, kern) == cudaSuccess && a.numRegs * Cfg::kThreads >= Cfg::kPoolNeeded;
  }
  if (fits != 1) return cudaErrorNotSupported;
  cudaError_t e = ensure_smem_attr(kern, Cfg::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  kern<<<L.grid, Cfg::kThreads, Cfg::kSmemBytes, L.stream>>>(L.tm_q, L.tm_k, L.tm_v, L.p);
  return cudaGetLastError();
}

template <int D, int KV>
cudaError_t prefix_mod(const PrefixLaunch &L) {
  if (L.mod == 1) return prefix_one<D, KV, 1>(L);
  if (L.mod == 2) return prefix_one<D, KV, 2>(L);
  return prefix_one<D, KV, 0>(L);
}

template <int D>
cudaError_t prefix_kv(const PrefixLaunch &L) {
  if (L.kv == 1) return prefix_mod<D, 1>(L);
  if (L.kv == 2) return prefix_mod<D, 2>(L);
  return prefix_mod<D, 0>(L);
}

// LSE = ln sum_s exp(LSE_s), out = sum_s exp(LSE_s - LSE) O_s.  One CTA of four
// warps per (row, head): every warp forms all weights (the lanes read the
// partial LSEs at once), each sums a quarter of the partial rows, in batches of
// four so that their latencies overlap, and the quarters meet in shared memory.
// A partial with LSE -inf was not written and is not read.
template <int D>
__global__ void __launch_bounds__(128) fa_prefix_merge_kernel(const float *__restrict__ o_part,
                                                              const float *__restrict__ lse_part,
                                                              const int32_t *__restrict__ cu_q, int num_seqs,
                                                              int num_splits, int64_t n_rows, int hq,
                                                              __nv_bfloat16 *__restrict__ out, float *__restrict__ lse) {
  constexpr int kPer = D / 32;
  __shared__ float part[4][D];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  const int64_t t = blockIdx.x / hq;
  const int h = (int)(blockIdx.x % hq);
  const int last = __ldg(cu_q + num_seqs);
  auto lse_of = [&](int s) { return s < num_splits ? lse_part[((int64_t)s * hq + h) * n_rows + t] : -INFINITY; };
  const float first = lse_of(lane);
  float m = first;
  for (int s0 = 32; s0 < num_splits; s0 += 32) m = fmaxf(m, lse_of(s0 + lane));
#pragma unroll
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (t >= last) return;   // rows behind the last sequence stay as they were
  float acc[kPer], den = 0.f;
#pragma unroll
  for (int e = 0; e < kPer; ++e) acc[e] = 0.f;
  if (m != -INFINITY) {
    for (int s0 = 0; s0 < num_splits; s0 += 32) {
      const float w = ex2(((s0 ? lse_of(s0 + lane) : first) - m) * kLog2e);   // 0 for an empty partial
      den += w;
      const int cnt = min(32, num_splits - s0);
      for (int s = warp; s < cnt; s += 16) {
        float v[4][kPer], ww[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          ww[u] = __shfl_sync(0xffffffffu, w, (s + 4 * u) & 31);
          const bool on = s + 4 * u < cnt && ww[u] > 0.f;
          if (!on) ww[u] = 0.f;
          const float *src = o_part + (((int64_t)(s0 + s + 4 * u) * n_rows + t) * hq + h) * D + lane * kPer;
#pragma unroll
          for (int e = 0; e < kPer; e += 2) {
            const float2 x = on ? __ldcs(reinterpret_cast<const float2 *>(src + e)) : make_float2(0.f, 0.f);
            v[u][e] = x.x;
            v[u][e + 1] = x.y;
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int e = 0; e < kPer; ++e) acc[e] = fmaf(ww[u], v[u][e], acc[e]);
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) part[warp][lane * kPer + e] = acc[e];
  __syncthreads();
  const float inv = den > 0.f ? 1.f / den : 0.f;
  if (threadIdx.x < D / 2) {
    const int d = 2 * threadIdx.x;
    float x = 0.f, y = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      x += part[w][d];
      y += part[w][d + 1];
    }
    *reinterpret_cast<uint32_t *>(out + (t * hq + h) * D + d) = pack_bf16x2(x * inv, y * inv);
  }
  if (lse && threadIdx.x == 0) lse[(int64_t)h * n_rows + t] = den > 0.f ? m + __log2f(den) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_prefix(int d, const PrefixLaunch &L) { return d == 64 ? prefix_kv<64>(L) : prefix_kv<128>(L); }

cudaError_t launch_prefix_merge(int d, const float *o_part, const float *lse_part, const int32_t *cu_q, int num_seqs,
                                int num_splits, int64_t n_rows, int hq, void *out, float *lse, cudaStream_t stream) {
  const int threads = 128;
  const unsigned blocks = (unsigned)(n_rows * hq);
  auto *o = reinterpret_cast<__nv_bfloat16 *>(out);
  auto kern = d == 64 ? fa_prefix_merge_kernel<64> : fa_prefix_merge_kernel<128>;
  return launch_behind(kern, dim3(blocks), threads, 0, stream, o_part, lse_part, cu_q, num_seqs, num_splits, n_rows, hq, o,
                       lse);
}

}  // namespace fa
