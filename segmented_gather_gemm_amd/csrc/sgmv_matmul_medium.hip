// Tiled kernel of the shared projection with adapters and of the grouped
// products: 128 x 128 tiles, four waves, two workgroups per compute unit.  Device code and
// design notes: sgmv_matmul_tiled.h.
#include "sgmv_matmul_tiled.h"

namespace sgmv {

TiledKernel matmul_tiled_medium(int wd, int mode) {
  using namespace dev;
  using S = TileShape<2, 2, 2, 2>;
  const void* k = nullptr;
  if (wd == BF16)
    k = mode == kDense     ? (const void*)matmul_tiled<BF16, kDense, S>
        : mode == kGrouped ? (const void*)matmul_tiled<BF16, kGrouped, S>
                           : (const void*)matmul_tiled<BF16, kGated, S>;
  else if (wd == F16)
    k = mode == kDense     ? (const void*)matmul_tiled<F16, kDense, S>
        : mode == kGrouped ? (const void*)matmul_tiled<F16, kGrouped, S>
                           : (const void*)matmul_tiled<F16, kGated, S>;
  return TiledKernel{k, S::BM, mode == kGated ? S::HN : S::BN, S::kNT};
}

}  // namespace sgmv
