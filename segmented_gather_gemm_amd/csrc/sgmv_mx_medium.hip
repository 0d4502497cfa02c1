// Tiled kernel of the shared projection with adapters and of the grouped
// products on microscaled 4-bit operands: 128 x 128 tiles, four waves, two workgroups per compute unit.  Device
// code and design notes: sgmv_matmul_tiled.h.
#include "sgmv_matmul_tiled.h"

namespace sgmv {

TiledKernel mx_tiled_medium(int wd, int mode) {
  using namespace dev;
  using S = TileShape<2, 2, 2, 2, 2>;
  // The 16-bit dtype is that of the bias and the adapters: grouped products have neither.
  static const void* const kernels[2][4] = {
      {(const void*)matmul_tiled<F16, kDense, S, true>, (const void*)matmul_tiled<BF16, kGrouped, S, true>,
       (const void*)matmul_tiled<BF16, kGated, S, true>, (const void*)matmul_tiled<F16, kAdapted, S, true>},
      {(const void*)matmul_tiled<BF16, kDense, S, true>, (const void*)matmul_tiled<BF16, kGrouped, S, true>,
       (const void*)matmul_tiled<BF16, kGated, S, true>, (const void*)matmul_tiled<BF16, kAdapted, S, true>}};
  return TiledKernel{kernels[wd == BF16][mode], S::BM, mode == kGated ? S::HN : S::BN, S::kNT};
}

}  // namespace sgmv
