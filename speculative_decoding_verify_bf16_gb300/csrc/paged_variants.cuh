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

// Blocks of 16 rows up to 16, of 32 up to 32, tiles of 128 beyond (heads up to 128); tiles from 17 rows on
// where there are few lanes and cache heads: an item's parts are then fewer.  Measured with 32 rows, 8 cache heads of 128, few rows' kernel against tiles, us:
//   lanes behind 1,500 tokens      1       2       4
//     e4m3                      28/20   28/22   30/25
//     bf16                      23/18   24/20   26/23
//   behind 2,000 to 16,000         1       2       4       8        64
//     e4m3                      53/31   49/34   55/52   75/89   355/516
//     bf16                      44/28   44/31   53/46   76/72   366/375
template <int TYPE>
PagedVariant paged_variant(int dim, int64_t rows, bool tiles, bool few) {
  if (dim > 128) return rows_variant<RowsShape<TYPE, 256, 1>>();
  if (rows > (few ? 16 : 32) && tiles) return dim > 64 ? tile_variant<TileShape<TYPE, 128>>() : tile_variant<TileShape<TYPE, 64>>();
  if (dim > 64) return rows > 16 ? rows_variant<RowsShape<TYPE, 128, 2>>() : rows_variant<RowsShape<TYPE, 128, 1>>();
  return rows > 16 ? rows_variant<RowsShape<TYPE, 64, 2>>() : rows_variant<RowsShape<TYPE, 64, 1>>();
}

}  // namespace specv
