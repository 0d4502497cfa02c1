// Tiled kernel of the shared projection with adapters and of the grouped
// products: 128 x 128 tiles, four waves, two workgroups per compute unit.  Device code and
// design notes: sgmv_matmul_tiled.h.
#include "sgmv_matmul_tiled.h"

namespace sgmv {

TiledKernel matmul_tiled_medium(int wd, int mode) {
  using namespace dev;
  using S = TileShape<2, 2, 2, 2, 2>;
  static const void* const kernels[2][4] = {
      {(const void*)matmul_tiled<F16, kDense, S>, (const void*)matmul_tiled<F16, kGrouped, S>,
       (const void*)matmul_tiled<F16, kGated, S>, (const void*)matmul_tiled<F16, kAdapted, S>},
      {(const void*)matmul_tiled<BF16, kDense, S>, (const void*)matmul_tiled<BF16, kGrouped, S>,
       (const void*)matmul_tiled<BF16, kGated, S>, (const void*)matmul_tiled<BF16, kAdapted, S>}};
  const void* k = wd == F16 || wd == BF16 ? kernels[wd == BF16][mode] : nullptr;
  return TiledKernel{k, S::BM, mode == kGated ? S::HN : S::BN, S::kNT};
}

}  // namespace sgmv
