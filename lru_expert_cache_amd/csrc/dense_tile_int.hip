// The tiled dense products of 8-bit codes.
#include "dense_tile.h"

namespace ftmoe {

hipError_t launch_dense_tile_int(DenseForm form, int dtype, int tile, const DenseLaunch& l, hipStream_t s) {
  if (form == kDenseIntGated) return launch_tiles<DenseI8, kDenseIntGated, float>(tile, l, s);
  if (form != kDenseInt) return hipErrorInvalidValue;
  if (dtype == FT_DT_F32) return launch_tiles<DenseI8, kDenseInt, float>(tile, l, s);
  if (dtype == FT_DT_F16) return launch_tiles<DenseI8, kDenseInt, _Float16>(tile, l, s);
  return launch_tiles<DenseI8, kDenseInt, __bf16>(tile, l, s);
}

}  // namespace ftmoe
