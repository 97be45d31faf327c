// Instantiations and launchers of the key-weight kernels (fa_key_weights.cuh).
#include "fa_key_weights.cuh"
#include "fa_internal.h"

namespace fa {
namespace {

template <int D, int KV, int NT>
cudaError_t rows_one(const KeyWeightsLaunch &L) {
  static unsigned long long done = 0;
  auto kern = fa_key_weights_rows_kernel<D, KV, NT>;
  constexpr int kSmem = KwRowsCfg<D, KV>::kSmemBytes;
  cudaError_t e = ensure_smem_attr(kern, kSmem, &done);
  if (e != cudaSuccess) return e;
  kern<<<L.grid, kKwWarps * 32, kSmem, L.stream>>>(L.tm_k, L.p);
  return cudaGetLastError();
}

template <int D, int KV>
cudaError_t rows_by_tiles(const KeyWeightsLaunch &L) {
  return L.row_tiles <= 1 ? rows_one<D, KV, 1>(L) : rows_one<D, KV, 2>(L);
}

template <int D>
cudaError_t rows_by_kv(const KeyWeightsLaunch &L) {
  if (L.p.kv == 1) return rows_by_tiles<D, 1>(L);
  if (L.p.kv == 2) return rows_by_tiles<D, 2>(L);
  return rows_by_tiles<D, 0>(L);
}

template <int D, int MOD>
cudaError_t tile_one(const KeyWeightsLaunch &L) {
  using Cfg = KwTileCfg<D>;
  static unsigned long long done = 0;
  auto kern = fa_key_weights_tile_kernel<D, MOD>;
  cudaError_t e = ensure_smem_attr(kern, Cfg::kSmemBytes, &done);
  if (e != cudaSuccess) return e;
  kern<<<L.grid, Cfg::kThreads, Cfg::kSmemBytes, L.stream>>>(L.tm_q, L.p);
  return cudaGetLastError();
}

template <int D>
cudaError_t tile_by_mod(const KeyWeightsLaunch &L) {
  if (L.p.mod == 1) return tile_one<D, 1>(L);
  if (L.p.mod == 2) return tile_one<D, 2>(L);
  return tile_one<D, 0>(L);
}

}  // namespace

cudaError_t launch_key_weights(int d, const KeyWeightsLaunch &L) {
  if (L.row_tiles > 0) {
    if (d == 64) return rows_by_kv<64>(L);
    if (d == 128) return rows_by_kv<128>(L);
    return rows_by_kv<192>(L);
  }
  if (d == 64) return tile_by_mod<64>(L);
  if (d == 128) return tile_by_mod<128>(L);
  return tile_by_mod<192>(L);
}

}  // namespace fa
