// paged_variants.cuh -- which kernel a call takes.
#pragma once

#include "paged_launch.h"
#include "paged_rows.cuh"
#include "paged_tile.cuh"

namespace specv {

template <typename S>
PagedVariant rows_variant() {
  return {reinterpret_cast<void*>(&paged_rows_kernel<S>), S::kRows, S::D, S::kWarps, S::kThreads, static_cast<int>(sizeof(RowsSmem<S>)), S::kRegs};
}
template <typename S>
PagedVariant tile_variant() {
  return {reinterpret_cast<void*>(&paged_tile_kernel<S>), S::kRows, S::D, 1, kTileThreads, static_cast<int>(sizeof(TileSmem<S>)), kTileRegs};
}

// Blocks of 16 rows up to 16, of 32 up to 32, tiles of 128 beyond (heads up to 128).  Measured with 17 to 32 rows, few
// rows' kernel against tiles, us: 8 lanes x 8 columns, e4m3 75 / 89, bf16 76 / 72; 64 lanes, e4m3 355 / 516, bf16
// 366 / 375; 2 lanes, e4m3 53 / 33; 64 x 1 to 4 through a window, heads of 64, 36 / 40.
template <int TYPE>
PagedVariant paged_variant(int dim, int64_t rows, bool tiles) {
  if (dim > 128) return rows_variant<RowsShape<TYPE, 256, 1>>();
  if (rows > 32 && tiles) return dim > 64 ? tile_variant<TileShape<TYPE, 128>>() : tile_variant<TileShape<TYPE, 64>>();
  if (dim > 64) return rows > 16 ? rows_variant<RowsShape<TYPE, 128, 2>>() : rows_variant<RowsShape<TYPE, 128, 1>>();
  return rows > 16 ? rows_variant<RowsShape<TYPE, 64, 2>>() : rows_variant<RowsShape<TYPE, 64, 1>>();
}

}  // namespace specv
