// Kernels of the shared projection with adapters and of the grouped products
// with microscaled 4-bit weights for few rows.  Device code and design notes:
// sgmv_matmul_skinny.h.
#include "sgmv_matmul_skinny.h"

namespace sgmv {

namespace {
constexpr int kThreadsSkinny = 64 * dev::kSkinnyWaves;

template <int MODE, int MB, int NB, int G, int MX>
const void* skinny_of(int wd) {
  using namespace dev;
  return wd == BF16 ? (const void*)matmul_skinny<BF16, MODE, MB, NB, G, MX>
                    : (const void*)matmul_skinny<F16, MODE, MB, NB, G, MX>;
}
}  // namespace

TiledKernel mx_skinny_16(int wd, int mode) {
  using namespace dev;
  const void* k = mode == kDense     ? skinny_of<kDense, 1, 1, 2, kMxQuantise>(wd)
                  : mode == kGrouped ? skinny_of<kGrouped, 1, 1, 2, kMxQuantise>(wd)
                  : mode == kGated   ? skinny_of<kGated, 1, 1, 2, kMxQuantise>(wd)
                                     : skinny_of<kAdapted, 1, 1, 2, kMxQuantise>(wd);
  return TiledKernel{k, 16, 16, kThreadsSkinny};
}

TiledKernel mx_skinny_32(int wd, bool adapted) {
  using namespace dev;
  return TiledKernel{adapted ? skinny_of<kAdapted, 2, 1, 2, kMxBoth>(wd)
                             : skinny_of<kDense, 2, 1, 2, kMxBoth>(wd),
                     32, 16, kThreadsSkinny};
}

TiledKernel mx_skinny_64(int wd, bool adapted) {
  using namespace dev;
  return TiledKernel{adapted ? skinny_of<kAdapted, 4, 1, 2, kMxBoth>(wd)
                             : skinny_of<kDense, 4, 1, 2, kMxBoth>(wd),
                     64, 16, kThreadsSkinny};
}

}  // namespace sgmv
