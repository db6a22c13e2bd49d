// cache_params.h -- what the paged cache's kernels are launched with (the checked form of
// spec_cache.h's structures), and where a lane's tokens lie.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "spec_cache.h"

namespace specv {

// The cache; strides in bytes.
struct CacheParams {
  uint8_t* k;
  uint8_t* v;
  int64_t page, slot, head;
  // The same in units of 2^unit_shift bytes, 16 at least, which divide them all; no head lies
  // 2^32 units or more behind the first.
  uint32_t page_units, slot_units, head_units;
  int32_t unit_shift;
  uint8_t* k_exps;
  uint8_t* v_exps;
  int64_t exp_page, exp_slot, exp_head;
  const int32_t* tables;
  int64_t table_stride;
  const int32_t* cached;
  const int32_t* offsets;
  int32_t* status;
  const int32_t* entry;  // status, or any other words where there is none; the bits of a word that count
  uint32_t entry_bits;
  int32_t pages, page_size;
  uint32_t page_magic, page_shift;  // p / page_size, see page_of
  int32_t lanes, rows, max_len, kv_heads, dim;
  int32_t most;  // most positions of a lane
};

// n / d for 0 <= n < 2^31 by a product.  With 2^s < d < 2^(s + 1) and the magic number m =
// floor(2^(32 + s) / d) + 1, n m / 2^(32 + s) exceeds n / d by at most n / 2^(32 + s) < 1 / d, so
// its whole part is the same.  Powers of two have magic number 0.
__host__ __device__ inline int32_t by_magic(int32_t n, uint32_t magic, uint32_t shift) {
#ifdef __CUDA_ARCH__
  return magic == 0 ? n >> shift : static_cast<int32_t>(__umulhi(n, magic) >> shift);
#else
  return magic == 0 ? n >> shift : static_cast<int32_t>((static_cast<uint64_t>(static_cast<uint32_t>(n)) * magic >> 32) >> shift);
#endif
}
inline void set_magic(int32_t d, uint32_t& magic, uint32_t& shift) {
  shift = 0;
  while ((int64_t{2} << shift) <= d) ++shift;
  magic = (d & (d - 1)) == 0 ? 0u : static_cast<uint32_t>((uint64_t{1} << (32 + shift)) / static_cast<uint32_t>(d)) + 1u;
}
__host__ __device__ inline int32_t page_of(const CacheParams& c, int32_t p) { return by_magic(p, c.page_magic, c.page_shift); }
inline void set_page_size(CacheParams& c, int32_t page_size) {
  c.page_size = page_size;
  set_magic(page_size, c.page_magic, c.page_shift);
}

// A lane's rows and the tokens before them; false for a lane that is laid out wrongly.
__device__ __forceinline__ bool cache_lane(const CacheParams& c, int b, int& first, int& count, int& before) {
  const int o0 = __ldg(c.offsets + b), o1 = __ldg(c.offsets + b + 1), n = __ldg(c.cached + b);
  first = o0;
  count = o1 - o0;
  before = n;
  return o0 >= 0 && o1 >= o0 && o1 <= c.rows && count <= c.max_len && n >= 0 && n <= c.most - count;
}

// Where a token's head begins, in units.
__device__ __forceinline__ uint32_t head_at(const CacheParams& c, int page, int slot, int head) {
  return page * c.page_units + slot * c.slot_units + head * c.head_units;
}
constexpr uint32_t kNowhere = 0xFFFFFFFFu;

__device__ __forceinline__ int lane_status(const CacheParams& c, int b) {
  return c.status != nullptr ? *static_cast<volatile int32_t*>(c.status + b) : SPEC_OK;
}
// The first error of a lane stays.
__device__ __forceinline__ void lane_failed(const CacheParams& c, int b, int code) {
  if (c.status != nullptr && lane_status(c, b) == SPEC_OK) c.status[b] = code;
}
// The attention's thread blocks, which may not all begin at once, have to agree on the lanes that had failed before
// the launch.  An error of its own stands in the status' highest four bits until its last launch moves it down.
constexpr int kFreshShift = 28;
constexpr uint32_t kEntryBits = (1u << kFreshShift) - 1;
__device__ __forceinline__ void lane_fails_now(const CacheParams& c, int b, int code) { lane_failed(c, b, code << kFreshShift); }
__device__ __forceinline__ bool failed_before(const CacheParams& c, int b) { return (c.entry[b] & c.entry_bits) != 0; }
// Moves all lanes' errors down (a thread block's threads).
__device__ __forceinline__ void settle_errors(const CacheParams& c) {
  if (c.status == nullptr) return;
  for (int b = threadIdx.x; b < c.lanes; b += blockDim.x) {
    const int status = lane_status(c, b);
    if (status != SPEC_OK && (status & kEntryBits) == 0) c.status[b] = static_cast<uint32_t>(status) >> kFreshShift;
  }
}

}  // namespace specv
