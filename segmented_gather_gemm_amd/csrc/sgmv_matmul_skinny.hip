// Kernels of the shared projection with adapters and of the grouped products
// for few rows: 16, 32 or 64 of them a tile.  Device code and design notes:
// sgmv_matmul_skinny.h.
#include "sgmv_matmul_skinny.h"

namespace sgmv {

TiledKernel matmul_skinny_16(int wd, int mode) {
  return TiledKernel{wd == dev::BF16 ? dev::skinny_kernel<dev::BF16, 1, 1, 2>(mode)
                                : dev::skinny_kernel<dev::F16, 1, 1, 2>(mode),
                     16, 16, 64 * dev::kSkinnyWaves};
}

TiledKernel matmul_skinny_32(int wd, int mode) {
  return TiledKernel{wd == dev::BF16 ? dev::skinny_kernel<dev::BF16, 2, 1, 2>(mode)
                                : dev::skinny_kernel<dev::F16, 2, 1, 2>(mode),
                     32, 16, 64 * dev::kSkinnyWaves};
}

TiledKernel matmul_skinny_64(int wd, int mode) {
  constexpr int kThreads = 64 * dev::kSkinnyWaves;
  // The gated form has two weight blocks a column block and the partial sums
  // of both to keep in LDS: 16 columns.
  if (mode == dev::kGated)
    return TiledKernel{wd == dev::BF16 ? (const void*)dev::matmul_skinny<dev::BF16, dev::kGated, 4, 1, 1>
                                       : (const void*)dev::matmul_skinny<dev::F16, dev::kGated, 4, 1, 1>,
                       64, 16, kThreads};
  return TiledKernel{wd == dev::BF16 ? dev::skinny_kernel<dev::BF16, 4, 2, 1>(mode)
                                     : dev::skinny_kernel<dev::F16, 4, 2, 1>(mode),
                     64, 32, kThreads};
}

}  // namespace sgmv
