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

template <int TYPE>
PagedVariant paged_variant(int dim, int64_t rows, bool tiles) {
  if (dim > 128) return rows_variant<RowsShape<TYPE, 256, 1>>();
  if (rows > 32 && tiles) return dim > 64 ? tile_variant<TileShape<TYPE, 128>>() : tile_variant<TileShape<TYPE, 64>>();
  if (dim > 64) return rows > 16 ? rows_variant<RowsShape<TYPE, 128, 2>>() : rows_variant<RowsShape<TYPE, 128, 1>>();
  return rows > 16 ? rows_variant<RowsShape<TYPE, 64, 2>>() : rows_variant<RowsShape<TYPE, 64, 1>>();
}

}  // namespace specv
