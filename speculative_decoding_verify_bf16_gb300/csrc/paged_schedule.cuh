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
  int32_t first, count;  // the lane's rows
  int32_t unused[2];
};

struct AttendParams {
  CacheParams c;
  const __nv_bfloat16* q;  // strides in elements
  __nv_bfloat16* out;
  int64_t q_row, q_head, out_row, out_head;
  float* lse;
  int64_t lse_row;
  int32_t group, window;
  uint32_t group_magic, group_shift;
  int32_t heads, head_groups;  // cache heads of an item (a power of two), and how many such groups there are
  int32_t workers;             // of a thread block
  float scale;                 // times log2(e)
  float* parts;                // two places for each worker, part_floats() each; NULL: items stay whole
  PartRecord* records;         // one for each worker
};
__device__ __forceinline__ int column_of(const AttendParams& p, int row) { return by_magic(row, p.group_magic, p.group_shift); }
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

// LEAST: costs that a worker takes at least (more workers leave more parts to join).  WORKERS: of a thread
// block, at most.
template <int ROWS, int TILE, int EXTRA, int LEAST, int WORKERS = kMostWorkers>
struct Schedule {
  static __device__ __forceinline__ void set_block(const AttendParams& p, Cursor& x) {
    const int i0 = column_of(p, x.k * ROWS), i1 = min(x.count - 1, column_of(p, x.k * ROWS + ROWS - 1));
    x.hi = x.before + i1 + 1;
    x.lo = p.window > 0 ? max(0, x.before + i0 - p.window + 1) : 0;
    x.t0 = x.lo / TILE;
    x.t1 = (x.hi + TILE - 1) / TILE;
    x.tile = x.t0;
  }
  // The lane at x.b, if it has work and had not failed before the launch, at its first item.
  static __device__ __forceinline__ bool try_lane(const AttendParams& p, Cursor& x) {
    const bool failed = failed_before(p.c, x.b);
    if (!cache_lane(p.c, x.b, x.first, x.count, x.before) || x.count == 0 || failed) return false;
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
  struct Shared {
    int64_t units[32], cost[32];
    int64_t begin[WORKERS], end[WORKERS];  // units of this thread block's workers
    Cursor from[WORKERS];                       // at the first of them
    PartRecord record[WORKERS];
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

  // What lies `left` costs behind the beginning of the lane at x (at its first item; `units` and `cost`: all of
  // the lane's): the cursor there (in an item's EXTRA: at its first unit; where items stay whole and one has
  // begun: at the next), and the units before it.  `in`: costs of the item up to there, `all`: its costs.
  static __device__ __forceinline__ int64_t find(const AttendParams& p, int64_t left, int64_t units, int64_t cost, Cursor& x,
                                                 int64_t& in, int64_t& all) {
    all = x.t1 - x.t0 + EXTRA;
    const bool one = x.blocks == 1;
    const int64_t per_cost = one ? all : quotient(cost, p.head_groups);
    x.h = static_cast<int>(quotient(left, per_cost));
    left -= x.h * per_cost;
    int64_t before = x.h * (one ? all - EXTRA : quotient(units, p.head_groups));
    for (; !one && left >= all; all = x.t1 - x.t0 + EXTRA) {
      left -= all;
      before += all - EXTRA;
      ++x.k;
      set_block(p, x);
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

  // The borders of this block's workers that lie in the lane at x, which begins at `before`.
  static __device__ __forceinline__ void mark(const AttendParams& p, Shared& sh, const Cursor& lane, bool on, int64_t before,
                                              int64_t before_units, int64_t units, int64_t cost, int64_t total) {
    if (!on || cost == 0) return;
    const int64_t g = workers_for(total, static_cast<int64_t>(gridDim.x) * p.workers);
    const int64_t c = static_cast<int64_t>(blockIdx.x) * p.workers;
    int64_t last = 0;
#pragma unroll 1
    for (int i = 0; i <= p.workers && c + i <= g && c < g; ++i) {
      const int64_t u = quotient(total * (c + i), g);  // where worker i begins and the one before it ends
      if (u >= before && u < before + cost) {
        Cursor x = lane;
        int64_t in, all;
        const int64_t at = before_units + find(p, u - before, units, cost, x, in, all);
        if (i < p.workers) {
          sh.begin[i] = at;
          sh.from[i] = x;
        }
        if (i > 0) {
          sh.end[i - 1] = at;
          // An item that goes on, and that worker i - 1 begins.
          if (p.parts != nullptr && in > EXTRA && last <= u - in + EXTRA)
            sh.record[i - 1] = {x.b, x.h, x.k, worker_of(u - in + all - 1, total, g) - static_cast<int>(c + i - 1) + 1, x.first, x.count, {0, 0}};
        }
      }
      last = u;
    }
  }

  // The whole thread block: its workers' ranges of units and the cursors at the first of them.  (One
  // launch's first instructions come from far: few of them, and each thread reads one lane.)
  static __device__ void plan(const AttendParams& p, Shared& sh) {
    const int threads = blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (threadIdx.x < WORKERS) {
      sh.begin[threadIdx.x] = sh.end[threadIdx.x] = 0;
      sh.record[threadIdx.x].parts = 0;
    }
    // Lanes in rounds of as many as there are threads: first all for the sums, then, unless that was
    // one round, again for the borders.
    int64_t total = 0, all_units = 0;
#pragma unroll 1
    for (int find_at = p.c.lanes <= threads ? 1 : 0, again = find_at; again < 2; find_at = 1, ++again) {
      int64_t base = 0, base_units = 0;
#pragma unroll 1
      for (int b0 = 0; b0 < p.c.lanes; b0 += threads) {
        Cursor x;
        x.b = b0 + threadIdx.x;
        int64_t units = 0, cost = 0, of_units = 0, of_cost = 0;  // of the lane; of the warp's lanes before it
        const int warps = min(threads, p.c.lanes - b0 + 31) / 32;  // that have lanes
        if (warp < warps) {
          if (x.b < p.c.lanes && try_lane(p, x)) {
            int64_t n = x.t1 - x.t0;
            if (x.blocks > 1) {
#pragma unroll 1
              while (++x.k < x.blocks) {
                set_block(p, x);
                n += x.t1 - x.t0;
              }
              x.k = 0;
              set_block(p, x);
            }
            units = n * p.head_groups;
            cost = units + static_cast<int64_t>(EXTRA) * x.blocks * p.head_groups;
          }
          int64_t run_units = units, run_cost = cost;
#pragma unroll 1
          for (int d = 1; d < 32; d <<= 1) {
            const int64_t u = __shfl_up_sync(0xFFFFFFFFu, run_units, d), n = __shfl_up_sync(0xFFFFFFFFu, run_cost, d);
            run_units += lane >= d ? u : 0;
            run_cost += lane >= d ? n : 0;
          }
          if (lane == 31) {
            sh.units[warp] = run_units;
            sh.cost[warp] = run_cost;
          }
          of_units = run_units - units;
          of_cost = run_cost - cost;
        }
        __syncthreads();
        int64_t before = base, before_units = base_units;
#pragma unroll 1
        for (int w = 0; w < warps; ++w) {
          before += w < warp ? sh.cost[w] : 0;
          before_units += w < warp ? sh.units[w] : 0;
          base += sh.cost[w];
          base_units += sh.units[w];
        }
        if (b0 + threads >= p.c.lanes) {
          total = base;
          all_units = base_units;
        }
        if (find_at == 1) mark(p, sh, x, warp < warps, before + of_cost, before_units + of_units, units, cost, total);
        if (p.c.lanes > threads) __syncthreads();  // (the sums have been read)
      }
    }
    // The last border is nobody's lane's.
    const int64_t most = static_cast<int64_t>(gridDim.x) * p.workers, g = workers_for(total, most);
    const int64_t last = g - static_cast<int64_t>(blockIdx.x) * p.workers;  // workers from this block's first on
    if (threadIdx.x == 0 && total > 0 && last >= 1 && last <= p.workers) sh.end[last - 1] = all_units;
    __syncthreads();
  }
};

}  // namespace specv
