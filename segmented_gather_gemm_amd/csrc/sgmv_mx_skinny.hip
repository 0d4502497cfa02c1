// Kernels of the shared projection with adapters and of the grouped products
// with microscaled 4-bit weights for few rows.  Device code and design notes:
// sgmv_mx_skinny.h.
#include "sgmv_mx_skinny.h"

namespace sgmv {

namespace {

template <int WD, int MODE, int MB>
const void* of_chunks(int chunks) {
  using namespace dev;
  return chunks == 1   ? (const void*)mx_skinny_rows<WD, MODE, MB, 1>
         : chunks == 2 ? (const void*)mx_skinny_rows<WD, MODE, MB, 2>
         : chunks == 3 ? (const void*)mx_skinny_rows<WD, MODE, MB, 3>
                       : (const void*)mx_skinny_rows<WD, MODE, MB, 4>;
}

template <int WD>
const void* of_mode(int mode, int rows, int chunks) {
  using namespace dev;
  if (mode == kGrouped) return of_chunks<WD, kGrouped, 1>(chunks);
  if (mode == kGated) return of_chunks<WD, kGated, 1>(chunks);
  if (mode == kAdapted)
    return rows == 16   ? of_chunks<WD, kAdapted, 1>(chunks)
           : rows == 32 ? of_chunks<WD, kAdapted, 2>(chunks)
                        : of_chunks<WD, kAdapted, 4>(chunks);
  return rows == 16   ? of_chunks<WD, kDense, 1>(chunks)
         : rows == 32 ? of_chunks<WD, kDense, 2>(chunks)
                      : of_chunks<WD, kDense, 4>(chunks);
}

}  // namespace

TiledKernel mx_skinny(int wd, int mode, int rows, int64_t groups) {
  // Chunks of a wave, in sets of at most four.
  const int64_t need = (groups + 2 * kMxSkinnyWaves - 1) / (2 * kMxSkinnyWaves);
  const int64_t sets = (need + 3) / 4;
  const int chunks = (int)((need + sets - 1) / sets);
  const void* k = wd == dev::BF16 ? of_mode<dev::BF16>(mode, rows, chunks) : of_mode<dev::F16>(mode, rows, chunks);
  return TiledKernel{k, rows, 16, 64 * kMxSkinnyWaves};
}

}  // namespace sgmv
