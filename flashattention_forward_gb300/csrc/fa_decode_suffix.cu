// Split-KV decode of the keys behind a shared prefix (fa_decode.cuh, SUFFIX):
// token-major pages, in a translation unit of its own.
#include "fa_internal.h"

namespace fa {

template <int D, int KV, bool R8>
static cudaError_t suffix_one(const DecodeLaunch &L) {
  static unsigned long long done = 0;
  auto kern = fa_decode_kernel<D, KV, false, R8, true>;
  constexpr bool kDirect = dec_direct<D, KV, false>();
  constexpr int kSmem = DecodeCfg<D, KV, kDirect, kDirect && R8>::kSmemBytes;
  cudaError_t e = ensure_smem_attr(kern, kSmem, &done);
  if (e != cudaSuccess) return e;
  kern<<<L.grid, kDecThreads, kSmem, L.stream>>>(L.tm_k, L.tm_v, L.p);
  return cudaGetLastError();
}

template <int KV>
static cudaError_t suffix_kv(int d, const DecodeLaunch &L) {
  if (d == 64) return suffix_one<64, KV, false>(L);
  if constexpr (KV != 0) {
    if (L.rows8) return suffix_one<128, KV, true>(L);
  }
  return suffix_one<128, KV, false>(L);
}

cudaError_t launch_decode_suffix(int d, const DecodeLaunch &L) {
  if (L.kv == 1) return suffix_kv<1>(d, L);
  if (L.kv == 2) return suffix_kv<2>(d, L);
  return suffix_kv<0>(d, L);
}

}  // namespace fa
