// Instantiations and launcher of the decode behind a shared prefix (fa_suffix.cuh).
#include "fa_internal.h"

namespace fa {
namespace {

template <int D, int KV, int NT>
cudaError_t suffix_one(const SuffixLaunch &L) {
  static unsigned long long done = 0;
  auto kern = fa_suffix_kernel<D, KV, NT>;
  constexpr int kSmem = SufCfg<D, KV>::kSmemBytes;
  cudaError_t e = ensure_smem_attr(kern, kSmem, &done);
  if (e != cudaSuccess) return e;
  return launch_behind(kern, L.grid, kSufWarps * 32, kSmem, L.stream, L.tm_k, L.tm_v, L.p);
}

template <int D, int KV>
cudaError_t suffix_rows(const SuffixLaunch &L) {
  return L.row_tiles <= 1 ? suffix_one<D, KV, 1>(L) : suffix_one<D, KV, 2>(L);
}

template <int D>
cudaError_t suffix_kv(const SuffixLaunch &L) {
  if (L.kv == 1) return suffix_rows<D, 1>(L);
  if (L.kv == 2) return suffix_rows<D, 2>(L);
  return suffix_rows<D, 0>(L);
}

}  // namespace

cudaError_t launch_suffix(int d, const SuffixLaunch &L) { return d == 64 ? suffix_kv<64>(L) : suffix_kv<128>(L); }

}  // namespace fa
