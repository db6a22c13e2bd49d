// paged_schedule.cuh -- how the attention over a paged cache is shared out to thread blocks.
//
// The query heads of one cache head and a lane's columns make up its rows: row r is column
// r / group, query head r % group of the group.  An item is a block of rows of a lane and of some cache heads,
// a unit an item's step over a tile of positions.  All units stand in one order (lanes, heads,
// row blocks, tiles); an item costs its units and EXTRA for what it takes to begin and to end it, and
// worker c of g (a thread block, or some of its warps) takes what lies between total * c / g
// and total * (c + 1) / g of the costs: all have the same work to within a unit, however ragged the
// lanes are.  An item whose units fall to several workers leaves partial sums, which a second launch
// joins; without scratch memory for them the borders move up to the next item.  Lanes' lengths are
// read on the device, so that a captured launch serves every round.
#pragma once

#include <cstdint>

#include "cache_params.h"

namespace specv {

// What a worker leaves of an item that goes on in the next one: how many workers hold parts of
// it, this one the first.  (parts 0: nothing.)  The parts of a thread block's workers are joined at its
// end, into the place of the first of them.
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
  int32_t heads, head_groups;  // cache heads of an item (a power of two), and how many such groups there are
  int32_t workers;             // of a thread block
  float scale;                 // times log2(e)
  float* parts;                // two places for each worker, part_floats() each; NULL: items stay whole
  PartRecord* records;         // one for each worker
};
constexpr int kMostWorkers = 8;  // of a thread block

// Partial sums of an item (rows: of all its heads): the outputs' numerators [rows][size], then
// (maximum, sum) of each row.
__host__ __device__ constexpr int64_t part_floats(int rows, int size) {
  return static_cast<int64_t>(rows) * (size + 2);
}

// A place in the order of units.  (b == lanes: past the end.)
struct Cursor {
  int b, h, k, blocks;       // lane, group of cache heads, block of rows, blocks of the lane
  int first, count, before;  // the lane's rows, and tokens before them
  int lo, hi;                // positions that the block's rows see
  int tile, t0, t1;          // tiles of positions
};

// n / d for 0 <= n < 2^62, d > 0; most are small, and take a fraction of the time then.
__device__ __forceinline__ int64_t quotient(int64_t n, int64_t d) {
  if (static_cast<uint64_t>(n | d) >> 32 == 0) return static_cast<uint32_t>(n) / static_cast<uint32_t>(d);
  return n / d;
}

// LEAST: costs that a worker takes at least (more workers leave more parts to join).
template <int ROWS, int TILE, int EXTRA, int LEAST>
struct Schedule {
  static __device__ __forceinline__ void set_block(const AttendParams& p, Cursor& x) {
    const int i0 = x.k * ROWS / p.group, i1 = min(x.count - 1, (x.k * ROWS + ROWS - 1) / p.group);
    x.hi = x.before + i1 + 1;
    x.lo = p.window > 0 ? max(0, x.before + i0 - p.window + 1) : 0;
    x.t0 = x.lo / TILE;
    x.t1 = (x.hi + TILE - 1) / TILE;
    x.tile = x.t0;
  }
  // The lane at x.b, if it has work, at its first item.
  static __device__ __forceinline__ bool try_lane(const AttendParams& p, Cursor& x) {
    if (!cache_lane(p.c, x.b, x.first, x.count, x.before) || x.count == 0) return false;
    x.blocks = (x.count * p.group + ROWS - 1) / ROWS;
    x.h = x.k = 0;
    set_block(p, x);
    return true;
  }
  static __device__ __forceinline__ void next_item(const AttendParams& p, Cursor& x) {
    if (++x.k < x.blocks) {
      set_block(p, x);
    } else if (++x.h < p.head_groups) {
      x.k = 0;
      set_block(p, x);
    } else {
      while (++x.b < p.c.lanes && !try_lane(p, x)) {
      }
    }
  }
  static __device__ __forceinline__ void next_unit(const AttendParams& p, Cursor& x) {
    if (++x.tile == x.t1) next_item(p, x);
  }
  // Units of one head of the lane at x (whose block moves on the way).
  static __device__ __forceinline__ int64_t head_units(const AttendParams& p, Cursor& x) {
    int64_t n = 0;
    for (x.k = 0; x.k < x.blocks; ++x.k) {
      set_block(p, x);
      n += x.t1 - x.t0;
    }
    return n;
  }
  // Units and costs of lane b.
  static __device__ __forceinline__ void lane_sums(const AttendParams& p, int b, int64_t& units, int64_t& cost) {
    Cursor x;
    x.b = b;
    units = cost = 0;
    if (!try_lane(p, x)) return;
    units = head_units(p, x) * p.head_groups;
    cost = units + static_cast<int64_t>(EXTRA) * x.blocks * p.head_groups;
  }

  struct Shared {
    int64_t units[32], cost[32];
    int64_t begin[kMostWorkers], end[kMostWorkers];  // units of this thread block's workers
    Cursor from[kMostWorkers];                       // at the first of them
    PartRecord record[kMostWorkers];
  };

  // Workers that get work.
  static __device__ __forceinline__ int64_t workers_for(int64_t total, int64_t most) {
    const int64_t n = (total + LEAST - 1) / LEAST;
    return n < most ? n : most;
  }
  // The worker that a cost falls to.
  static __device__ __forceinline__ int worker_of(int64_t u, int64_t total, int64_t g) {
    return static_cast<int>(quotient((u + 1) * g - 1, total));
  }

  // What lies `left` costs behind the beginning of lane b0: the cursor there (in an item's EXTRA: at its
  // first unit; where items stay whole and one has begun: at the next), and the units
  // before it.  `in`: costs of the item up to there, `all`: its costs.
  static __device__ __forceinline__ int64_t find(const AttendParams& p, int b0, int64_t left, Cursor& x, int64_t& in,
                                                 int64_t& all) {
    int64_t before = 0;
    x.b = b0;
    for (;; ++x.b) {
      int64_t units, cost;
      lane_sums(p, x.b, units, cost);
      if (left < cost) break;
      left -= cost;
      before += units;
    }
    try_lane(p, x);
    const int64_t per_units = head_units(p, x), per_cost = per_units + static_cast<int64_t>(EXTRA) * x.blocks;
    x.h = static_cast<int>(quotient(left, per_cost));
    left -= x.h * per_cost;
    before += x.h * per_units;
    for (x.k = 0;; ++x.k) {
      set_block(p, x);
      all = x.t1 - x.t0 + EXTRA;
      if (left < all) break;
      left -= all;
      before += all - EXTRA;
    }
    in = left;
    if (left <= EXTRA) return before;
    if (p.parts == nullptr) {
      next_item(p, x);
      return before + all - EXTRA;
    }
    x.tile = x.t0 + static_cast<int>(left - EXTRA);
    return before + left - EXTRA;
  }

  // The whole thread block: its workers' ranges of units and the cursors at the first of them.
  static __device__ void plan(const AttendParams& p, Shared& sh) {
    const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int per = (p.c.lanes + threads - 1) / threads;
    const int b0 = min(p.c.lanes, static_cast<int>(threadIdx.x) * per), b1 = min(p.c.lanes, b0 + per);
    int64_t units = 0, cost = 0;
    for (int b = b0; b < b1; ++b) {
      int64_t u, n;
      lane_sums(p, b, u, n);
      units += u;
      cost += n;
    }
    int64_t run_units = units, run_cost = cost;
    if (warp * 32 * per < p.c.lanes)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int64_t u = __shfl_up_sync(0xFFFFFFFFu, run_units, d), n = __shfl_up_sync(0xFFFFFFFFu, run_cost, d);
        run_units += lane >= d ? u : 0;
        run_cost += lane >= d ? n : 0;
      }
    if (lane == 31) {
      sh.units[warp] = run_units;
      sh.cost[warp] = run_cost;
    }
    if (threadIdx.x < kMostWorkers) {
      sh.begin[threadIdx.x] = sh.end[threadIdx.x] = 0;
      sh.record[threadIdx.x].parts = 0;
    }
    __syncthreads();
    int64_t total = 0, all_units = 0, before = run_cost - cost, before_units = run_units - units;
    for (int w = 0; w < threads / 32; ++w) {
      before += w < warp ? sh.cost[w] : 0;
      before_units += w < warp ? sh.units[w] : 0;
      total += sh.cost[w];
      all_units += sh.units[w];
    }
    const int64_t g = workers_for(total, static_cast<int64_t>(gridDim.x) * p.workers);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * p.workers;
    int64_t last = 0;
#pragma unroll 1
    for (int i = 0; i <= p.workers && c + i <= g && c < g; ++i) {
      const int64_t u = quotient(total * (c + i), g);  // where worker i begins and the one before it ends
      if (u == total) {
        if (threadIdx.x == 0 && i > 0) sh.end[i - 1] = all_units;
      } else if (u >= before && u < before + cost) {  // in one of this thread's lanes
        Cursor x;
        int64_t in, all;
        const int64_t at = before_units + find(p, b0, u - before, x, in, all);
        if (i < p.workers) {
          sh.begin[i] = at;
          sh.from[i] = x;
        }
        if (i > 0) {
          sh.end[i - 1] = at;
          // An item that goes on, and that worker i - 1 begins.
          if (p.parts != nullptr && in > EXTRA && last <= u - in + EXTRA)
            sh.record[i - 1] = {x.b, x.h, x.k, worker_of(u - in + all - 1, total, g) - static_cast<int>(c + i - 1) + 1};
        }
      }
      last = u;
    }
    __syncthreads();
  }
};

}  // namespace specv
