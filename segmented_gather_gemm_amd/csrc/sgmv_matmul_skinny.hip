// Kernels of the shared projection with adapters and of the grouped products
// for few rows: 16 of them a tile; dense calls also 32, and with adapters 64.
// Device code and design notes: sgmv_matmul_skinny.h.
#include "sgmv_matmul_skinny.h"

namespace sgmv {

namespace {
constexpr int kThreadsSkinny = 64 * dev::kSkinnyWaves;
}

TiledKernel matmul_skinny_16(int wd, int mode) {
  using namespace dev;
  static const void* const kernels[2][4] = {
      {(const void*)matmul_skinny<F16, kDense, 1, 1, 2>, (const void*)matmul_skinny<F16, kGrouped, 1, 1, 2>,
       (const void*)matmul_skinny<F16, kGated, 1, 1, 2>, (const void*)matmul_skinny<F16, kAdapted, 1, 1, 2>},
      {(const void*)matmul_skinny<BF16, kDense, 1, 1, 2>, (const void*)matmul_skinny<BF16, kGrouped, 1, 1, 2>,
       (const void*)matmul_skinny<BF16, kGated, 1, 1, 2>, (const void*)matmul_skinny<BF16, kAdapted, 1, 1, 2>}};
  return TiledKernel{kernels[wd == BF16][mode], 16, 16, kThreadsSkinny};
}

TiledKernel matmul_skinny_32(int wd, bool adapted) {
  using namespace dev;
  const void* k = wd == BF16 ? adapted ? (const void*)matmul_skinny<BF16, kAdapted, 2, 1, 2>
                                       : (const void*)matmul_skinny<BF16, kDense, 2, 1, 2>
                  : adapted  ? (const void*)matmul_skinny<F16, kAdapted, 2, 1, 2>
                             : (const void*)matmul_skinny<F16, kDense, 2, 1, 2>;
  return TiledKernel{k, 32, 16, kThreadsSkinny};
}

TiledKernel matmul_skinny_64_adapted(int wd) {
  using namespace dev;
  return TiledKernel{wd == BF16 ? (const void*)matmul_skinny<BF16, kAdapted, 4, 2, 1>
                                : (const void*)matmul_skinny<F16, kAdapted, 4, 2, 1>,
                     64, 32, kThreadsSkinny};
}

}  // namespace sgmv
