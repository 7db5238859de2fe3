// The tiled dense products with fp16 operands.
#include "dense_tile.h"

namespace ftmoe {

hipError_t launch_dense_tile_f16(DenseForm form, int tile, const DenseLaunch& l, hipStream_t s) {
  typedef DenseF16 D;
  typedef D::elem E;
  switch (form) {
    case kDenseGated: return launch_tiles<D, kDenseGated, E>(tile, l, s);
    case kDenseRows: return launch_tiles<D, kDenseRows, E>(tile, l, s);
    case kDenseGrad: return launch_tiles<D, kDenseGrad, E>(tile, l, s);
    case kDenseCols: return launch_tiles<D, kDenseCols, E>(tile, l, s);
    case kDenseOuter: return launch_tiles<D, kDenseOuter, E>(tile, l, s);
    default: return hipErrorInvalidValue;
  }
}

hipError_t launch_dense_pair_f16(int tile, const DensePair& l, hipStream_t s) {
  return launch_pairs<DenseF16>(tile, l, s);
}

}  // namespace ftmoe
