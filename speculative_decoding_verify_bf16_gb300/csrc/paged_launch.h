// paged_launch.h -- the attention kernels of one cache type, each type compiled on its own.
#pragma once

#include "paged_schedule.cuh"

namespace specv {

// A kernel over blocks of rows and what it is launched with.
struct PagedVariant {
  void* kernel;
  int rows, size;  // rows of an item and cache head, head size that the kernel works with
  int heads;       // cache heads that a thread block can take at a time, a power of two
  int threads, smem;
  int regs;  // registers that the warpgroups share out, four of a thread each (0: none are shared out)
};

// The kernel for heads of `dim` and up to `rows` rows of a lane and cache head; `tiles`: the
// one of large tiles may be taken; `few`: there are few lanes and heads.
PagedVariant paged_bf16(int dim, int64_t rows, bool tiles, bool few);
PagedVariant paged_e4m3(int dim, int64_t rows, bool tiles, bool few);
PagedVariant paged_int8(int dim, int64_t rows, bool tiles, bool few);

}  // namespace specv
