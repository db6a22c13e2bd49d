// paged_schedule.cuh -- how the attention over a paged cache is shared out to thread blocks.
//
// The query heads of one cache head and a lane's columns make up its rows: row r is column
// r / group, query head r % group of the group.  An item is a block of rows of a lane and cache
// head, a unit an item's step over a tile of positions.  All units stand in one order (lanes, heads, row blocks,
// tiles), and thread block c of g takes units total * c / g up to total * (c + 1) / g: every one has the
// same work to within a unit (and, of few units, one), however ragged the lanes are.  An item whose
// units fall to several blocks leaves partial sums, which a second launch joins; without scratch memory for
// them the borders move up to the next item.  Lanes' lengths are read on the device, so
// that a captured launch serves every round.
#pragma once

#include <cstdint>

#include "cache_params.h"

namespace specv {

// What a thread block leaves of an item that goes on in the next one: how many blocks hold parts of
// it, this one the first.
struct PartRecord {
  int32_t lane, head, block, parts;
};

struct AttendParams {
  CacheParams c;
  const __nv_bfloat16* q;  // strides in elements
  __nv_bfloat16* out;
  int64_t q_row, q_head, out_row, out_head;
  float* lse;
  int64_t lse_row;
  int32_t group, window;
  float scale;          // times log2(e)
  float* parts;         // two places for each thread block, part_floats() each; NULL: items stay whole
  PartRecord* records;  // one for each thread block
};

// Partial sums of a block of rows: the outputs' numerators [rows][size], then (maximum, sum) of
// each row.
__host__ __device__ constexpr int64_t part_floats(int rows, int size) {
  return static_cast<int64_t>(rows) * (size + 2);
}

// A place in the order of units.  (b == lanes: past the end.)
struct Cursor {
  int b, h, k, blocks;       // lane, cache head, block of rows, blocks of the lane
  int first, count, before;  // the lane's rows, and tokens before them
  int lo, hi;                // positions that the block's rows see
  int tile, t0, t1;          // tiles of positions
};

template <int ROWS, int TILE>
struct Schedule {
  static __device__ __forceinline__ void set_block(const AttendParams& p, Cursor& x) {
    const int i0 = x.k * ROWS / p.group, i1 = min(x.count - 1, (x.k * ROWS + ROWS - 1) / p.group);
    x.hi = x.before + i1 + 1;
    x.lo = p.window > 0 ? max(0, x.before + i0 - p.window + 1) : 0;
    x.t0 = x.lo / TILE;
    x.t1 = (x.hi + TILE - 1) / TILE;
    x.tile = x.t0;
  }
  // The lane at x.b or the first one after it that has work.
  static __device__ __forceinline__ void set_lane(const AttendParams& p, Cursor& x) {
    x.h = x.k = 0;
    for (; x.b < p.c.lanes; ++x.b)
      if (cache_lane(p.c, x.b, x.first, x.count, x.before) && x.count > 0) {
        x.blocks = (x.count * p.group + ROWS - 1) / ROWS;
        set_block(p, x);
        return;
      }
  }
  static __device__ __forceinline__ void next_item(const AttendParams& p, Cursor& x) {
    if (++x.k < x.blocks) {
      set_block(p, x);
    } else if (++x.h < p.c.kv_heads) {
      x.k = 0;
      set_block(p, x);
    } else {
      ++x.b;
      set_lane(p, x);
    }
  }
  static __device__ __forceinline__ void next_unit(const AttendParams& p, Cursor& x) {
    if (++x.tile == x.t1) next_item(p, x);
  }
  // Units of one head of the lane at x (its other fields are set on the way).
  static __device__ __forceinline__ int64_t head_units(const AttendParams& p, Cursor& x) {
    int64_t n = 0;
    for (x.k = 0; x.k < x.blocks; ++x.k) {
      set_block(p, x);
      n += x.t1 - x.t0;
    }
    return n;
  }
  static __device__ __forceinline__ int64_t lane_units(const AttendParams& p, int b) {
    Cursor x;
    x.b = b;
    if (!cache_lane(p.c, b, x.first, x.count, x.before) || x.count == 0) return 0;
    x.blocks = (x.count * p.group + ROWS - 1) / ROWS;
    return head_units(p, x) * p.c.kv_heads;
  }

  struct Shared {
    int64_t warp_sum[32];
    int64_t begin, end, total;
    Cursor from;
  };

  // The whole thread block: its range of units and the cursor at the first of them.
  static __device__ void plan(const AttendParams& p, Shared& sh) {
    const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.c.lanes + threads - 1) / threads;
    const int b0 = min(p.c.lanes, static_cast<int>(threadIdx.x) * per), b1 = min(p.c.lanes, b0 + per);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += lane_units(p, b);
    int64_t run = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t up = __shfl_up_sync(0xFFFFFFFFu, run, d);
      run += lane >= d ? up : 0;
    }
    if (lane == 31) sh.warp_sum[warp] = run;
    if (threadIdx.x == 0) {
      sh.begin = sh.end = 0;
      sh.from.b = p.c.lanes;
    }
    __syncthreads();
    int64_t total = 0, before = run - sum;
    for (int w = 0; w < threads / 32; ++w) {
      before += w < warp ? sh.warp_sum[w] : 0;
      total += sh.warp_sum[w];
    }
    if (threadIdx.x == 0) sh.total = total;
    const int64_t g = blocks_for(total, gridDim.x), c = blockIdx.x;
    if (c < g) {
#pragma unroll 1
      for (int i = 0; i < 2; ++i) {
        const int64_t u = total * (c + i) / g;
        if (u == total) {
          if (threadIdx.x == 0) sh.end = total;
        } else if (u >= before && u < before + sum) {  // the border lies in one of this thread's lanes
          Cursor x;
          const int64_t at = u + find(p, b0, u - before, x);
          if (i == 0) {
            sh.begin = at;
            sh.from = x;
          } else {
            sh.end = at;
          }
        }
      }
    }
    __syncthreads();
  }
  // Unit `left` of those of lanes b0 and after: the cursor there or, where items stay whole,
  // at the first item that begins there or later; how many units later that is.
  static __device__ __forceinline__ int64_t find(const AttendParams& p, int b0, int64_t left, Cursor& x) {
    x.b = b0;
    set_lane(p, x);
    for (int64_t n; left >= (n = lane_units(p, x.b));) {
      left -= n;
      ++x.b;
      set_lane(p, x);
    }
    const int64_t per_head = head_units(p, x);
    x.h = static_cast<int>(left / per_head);
    left -= x.h * per_head;
    for (x.k = 0;; ++x.k) {
      set_block(p, x);
      if (left < x.t1 - x.t0) break;
      left -= x.t1 - x.t0;
    }
    if (p.parts == nullptr && left > 0) {
      const int64_t later = x.t1 - x.t0 - left;
      next_item(p, x);
      return later;
    }
    x.tile = x.t0 + static_cast<int>(left);
    return 0;
  }
  // Thread blocks that get units: each at least one.
  static __device__ __forceinline__ int64_t blocks_for(int64_t total, int64_t grid) { return total < grid ? total : grid; }
  // The thread block that unit u falls to.
  static __device__ __forceinline__ int block_of(int64_t u, int64_t total) {
    return static_cast<int>(((u + 1) * blocks_for(total, gridDim.x) - 1) / total);
  }
};

}  // namespace specv
