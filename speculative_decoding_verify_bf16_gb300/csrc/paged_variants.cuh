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
// where there are few lanes and cache heads (their product is `few` up to 38 on this GPU): an item's parts are then
// fewer.  Measured, few rows' kernel against tiles, us:
//   lanes x cache heads             1 x 8   2 x 8   4 x 8   8 x 8   8 x 1  32 x 1  16 x 2
//   heads of 128, 32 rows, behind 1,500
//     e4m3                          28/20   29/22   30/26   34/32   34/20   35/26   36/26
//     bf16                          24/18   25/20   27/23   29/28   27/18   31/23   31/23
//   behind 2,000 to 16,000
//     e4m3                          51/32   50/34   58/52   77/92   37/29   51/45   54/48
//     bf16                          44/28   44/31   57/46   78/73   34/26   57/43   59/44
//   through a window of 1,000
//     e4m3                          28/20   29/22   30/23   30/30   34/20   35/24   36/24
//     bf16                          21/18   23/20   23/21   31/27   28/18   29/22   30/22
//   heads of 64, behind 2,000 to 16,000
//     e4m3                          34/26   33/28   36/39   48/70   29/24   38/36   41/38
//     bf16                          30/23   30/25   32/34   45/55   27/22   35/32   37/33
//   heads of 64, through a window
//     e4m3                          20/17   20/19   21/20   21/25   27/17   28/20   30/21
//     bf16                          18/16   18/18   19/19   20/23   26/16   26/19   28/19
//   20 rows: 2 to 11 % less on both sides, the same order
template <int TYPE>
PagedVariant paged_variant(int dim, int64_t rows, bool tiles, bool few) {
  if (dim > 128) return rows_variant<RowsShape<TYPE, 256, 1>>();
  if (rows > (few ? 16 : 32) && tiles) return dim > 64 ? tile_variant<TileShape<TYPE, 128>>() : tile_variant<TileShape<TYPE, 64>>();
  if (dim > 64) return rows > 16 ? rows_variant<RowsShape<TYPE, 128, 2>>() : rows_variant<RowsShape<TYPE, 128, 1>>();
  return rows > 16 ? rows_variant<RowsShape<TYPE, 64, 2>>() : rows_variant<RowsShape<TYPE, 64, 1>>();
}

}  // namespace specv
