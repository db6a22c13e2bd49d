// paged_cache.cu -- host side of include/spec_cache.h: argument checks, the choice of kernel
// and the launches.
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "cache_rows.cuh"
#include "paged_launch.h"
#include "paged_rows.cuh"

namespace {

using specv::AttendParams;
using specv::CacheParams;
using specv::CacheRowsParams;
using specv::PagedVariant;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Positions end here, so that sums of a position and a tile fit 32 bits.
constexpr int64_t kMostPositions = INT32_MAX - 65536;

int check_cache(const spec_paged_cache& a, CacheParams* c) {
  if (a.type != SPEC_CACHE_BF16 && a.type != SPEC_CACHE_E4M3 && a.type != SPEC_CACHE_INT8) return SPEC_ERR_INVALID_ARG;
  if (a.lanes < 0 || a.rows < 0 || a.max_len < 0 || a.table_width < 0 || a.table_stride < a.table_width)
    return SPEC_ERR_INVALID_ARG;
  if (a.pages <= 0 || a.page_size <= 0 || a.kv_heads <= 0) return SPEC_ERR_INVALID_ARG;
  if (a.dim < 16 || a.dim > SPEC_CACHE_MAX_DIM || a.dim % 16 != 0) return SPEC_ERR_INVALID_ARG;
  const int size = a.type == SPEC_CACHE_BF16 ? 2 : 1;
  for (int64_t s : {a.page_stride, a.slot_stride, a.head_stride})
    if (s < 0 || s * size % 16 != 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(a.k_pages) || !aligned16(a.v_pages)) return SPEC_ERR_INVALID_ARG;
  if (a.type != SPEC_CACHE_BF16)
    for (int64_t s : {a.exp_page_stride, a.exp_slot_stride, a.exp_head_stride})
      if (s < 0) return SPEC_ERR_INVALID_ARG;
  if (a.lanes > 0) {
    if (a.k_pages == nullptr || a.v_pages == nullptr || a.cached_lens == nullptr || a.row_offsets == nullptr ||
        (a.table_width > 0 && a.block_tables == nullptr))
      return SPEC_ERR_INVALID_ARG;
    if (a.type != SPEC_CACHE_BF16 && (a.k_exps == nullptr || a.v_exps == nullptr)) return SPEC_ERR_INVALID_ARG;
  }
  c->k = static_cast<uint8_t*>(a.k_pages);
  c->v = static_cast<uint8_t*>(a.v_pages);
  c->page = a.page_stride * size;
  c->slot = a.slot_stride * size;
  c->head = a.head_stride * size;
  c->unit_shift = 4;
  while (c->unit_shift < 16 && ((c->page | c->slot | c->head) >> c->unit_shift & 1) == 0) ++c->unit_shift;
  // (by way of 64-bit floats: the products themselves could overflow)
  const double last = (a.pages - 1.0) * static_cast<double>(c->page) + (a.page_size - 1.0) * static_cast<double>(c->slot) +
                      (a.kv_heads - 1.0) * static_cast<double>(c->head);
  if (last / static_cast<double>(int64_t{1} << c->unit_shift) >= 4294967295.0) return SPEC_ERR_INVALID_ARG;
  c->page_units = static_cast<uint32_t>(c->page >> c->unit_shift);
  c->slot_units = static_cast<uint32_t>(c->slot >> c->unit_shift);
  c->head_units = static_cast<uint32_t>(c->head >> c->unit_shift);
  c->k_exps = a.k_exps;
  c->v_exps = a.v_exps;
  c->exp_page = a.exp_page_stride;
  c->exp_slot = a.exp_slot_stride;
  c->exp_head = a.exp_head_stride;
  c->tables = a.block_tables;
  c->table_stride = a.table_stride;
  c->cached = a.cached_lens;
  c->offsets = a.row_offsets;
  c->status = a.lane_status;
  c->entry = a.lane_status != nullptr ? a.lane_status : a.row_offsets;
  c->entry_bits = a.lane_status != nullptr ? specv::kEntryBits : 0u;
  c->pages = a.pages;
  specv::set_page_size(*c, a.page_size);
  c->lanes = a.lanes;
  c->rows = a.rows;
  c->max_len = a.max_len;
  c->kv_heads = a.kv_heads;
  c->dim = a.dim;
  const int64_t most = static_cast<int64_t>(a.table_width) * a.page_size;
  c->most = static_cast<int32_t>(most < kMostPositions ? most : kMostPositions);
  return SPEC_OK;
}

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
int g_sms[kMaxDevices];

int device_sms(int* dev, int* sms) {
  if (cudaGetDevice(dev) != cudaSuccess || *dev < 0 || *dev >= kMaxDevices) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  std::lock_guard<std::mutex> lock(g_mutex);
  int& n = g_sms[*dev];
  if (n == 0 && cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
    return SPEC_ERR_CUDA;
  }
  *sms = n;
  return SPEC_OK;
}

int launch(void* kernel, dim3 grid, unsigned block, size_t smem, void** args, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelExC(&cfg, kernel, args) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}

// Shared memory beyond 48 KB is asked for once for each kernel and device (and then the kernel's
// registers are looked at).
struct Granted {
  void* kernel;
  int dev;
};
Granted g_granted[256];
int g_granted_count = 0;

int grant_smem(const PagedVariant& v, int dev) {
  void* const kernel = v.kernel;
  std::lock_guard<std::mutex> lock(g_mutex);
  for (int i = 0; i < g_granted_count; ++i)
    if (g_granted[i].kernel == kernel && g_granted[i].dev == dev) return SPEC_OK;
  // The warpgroups' shares of registers must not add up to more than the launch brings.
  cudaFuncAttributes fa;
  if (v.regs > 0 && (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs * (v.threads / 128) < v.regs)) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  if (g_granted_count < 256) g_granted[g_granted_count++] = {kernel, dev};
  return SPEC_OK;
}

// ---------------------------------------------------------------------------
// Rows to slots and back
// ---------------------------------------------------------------------------
template <typename T, int TYPE, bool WRITE>
void* rows_kernel_for(int dim, int* group) {
  if (dim <= 64) {
    *group = 8;
    return reinterpret_cast<void*>(&specv::cache_rows_kernel<T, TYPE, 8, WRITE>);
  }
  if (dim <= 128) {
    *group = 16;
    return reinterpret_cast<void*>(&specv::cache_rows_kernel<T, TYPE, 16, WRITE>);
  }
  *group = 32;
  return reinterpret_cast<void*>(&specv::cache_rows_kernel<T, TYPE, 32, WRITE>);
}
template <typename T, bool WRITE>
void* rows_kernel_for(spec_cache_type type, int dim, int* group) {
  if (type == SPEC_CACHE_BF16) return rows_kernel_for<T, SPEC_CACHE_BF16, WRITE>(dim, group);
  if (type == SPEC_CACHE_E4M3) return rows_kernel_for<T, SPEC_CACHE_E4M3, WRITE>(dim, group);
  return rows_kernel_for<T, SPEC_CACHE_INT8, WRITE>(dim, group);
}

template <bool WRITE>
int cache_rows(const spec_cache_rows_args* a, void* stream) {
  if (a == nullptr) return SPEC_ERR_INVALID_ARG;
  CacheRowsParams p{};
  int rc = check_cache(a->cache, &p.c);
  if (rc != SPEC_OK) return rc;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  const int size = a->dtype == SPEC_F32 ? 4 : 2;
  for (int64_t s : {a->k_row_stride, a->k_head_stride, a->v_row_stride, a->v_head_stride})
    if (s < (WRITE ? 0 : 1) || s * size % 16 != 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(a->k) || !aligned16(a->v)) return SPEC_ERR_INVALID_ARG;
  if (p.c.lanes == 0) return SPEC_OK;
  if (p.c.rows > 0 && (a->k == nullptr || a->v == nullptr)) return SPEC_ERR_INVALID_ARG;
  p.k = static_cast<uint8_t*>(a->k);
  p.v = static_cast<uint8_t*>(a->v);
  p.k_row = a->k_row_stride * size;
  p.k_head = a->k_head_stride * size;
  p.v_row = a->v_row_stride * size;
  p.v_head = a->v_head_stride * size;
  int dev, sms, group;
  if ((rc = device_sms(&dev, &sms)) != SPEC_OK) return rc;
  void* const kernel = a->dtype == SPEC_F32 ? rows_kernel_for<float, WRITE>(a->cache.type, p.c.dim, &group)
                                            : rows_kernel_for<__nv_bfloat16, WRITE>(a->cache.type, p.c.dim, &group);
  // Four rounds of a CTA's threads where there are rows enough for all SMs, one row at least.
  const int64_t per_round = specv::kRowThreads / group;
  int64_t rows = (4 * per_round + p.c.kv_heads - 1) / p.c.kv_heads;
  const int64_t spread = (p.c.rows + 4 * static_cast<int64_t>(sms) - 1) / (4 * static_cast<int64_t>(sms));
  rows = rows < spread ? rows : spread;
  rows = rows < 1 ? 1 : rows > specv::kRowsMost ? specv::kRowsMost : rows;
  p.rows_per_cta = static_cast<int32_t>(rows);
  const int64_t grid = p.c.rows == 0 ? 1 : (p.c.rows + rows - 1) / rows;  // (lanes are checked even without rows)
  void* args[] = {&p};
  return launch(kernel, dim3(static_cast<unsigned>(grid)), specv::kRowThreads, 0, args, stream);
}

// ---------------------------------------------------------------------------
// Attention
// ---------------------------------------------------------------------------
// The last launch where no item was split.
constexpr int kStatusThreads = 128;
__global__ void __launch_bounds__(kStatusThreads) paged_status_kernel(const CacheParams c) {
  specv::griddep_wait();
  specv::griddep_launch_dependents();
  specv::settle_errors(c);
}

PagedVariant variant_for(spec_cache_type type, int dim, int64_t rows, bool tiles, bool few) {
  if (type == SPEC_CACHE_BF16) return specv::paged_bf16(dim, rows, tiles, few);
  if (type == SPEC_CACHE_E4M3) return specv::paged_e4m3(dim, rows, tiles, few);
  return specv::paged_int8(dim, rows, tiles, few);
}

uint64_t scratch_bytes(const PagedVariant& v, int sms) {
  // A thread block's workers times the heads that each takes are v.heads.  (Records for the most workers, so
  // that more columns never want less.)
  return static_cast<uint64_t>(sms) *
         (2 * specv::part_floats(v.rows * v.heads, v.size) * sizeof(float) + specv::kMostWorkers * sizeof(specv::PartRecord));
}

void* join_kernel(int size) {
  if (size == 64) return reinterpret_cast<void*>(&specv::paged_join_kernel<64>);
  if (size == 128) return reinterpret_cast<void*>(&specv::paged_join_kernel<128>);
  return reinterpret_cast<void*>(&specv::paged_join_kernel<256>);
}

}  // namespace

extern "C" {

int spec_cache_write(const spec_cache_rows_args* a, void* stream) { return cache_rows<true>(a, stream); }
int spec_cache_read(const spec_cache_rows_args* a, void* stream) { return cache_rows<false>(a, stream); }

uint64_t spec_paged_attention_workspace(int32_t q_heads, int32_t kv_heads, int32_t dim, int32_t max_len) {
  if (q_heads <= 0 || kv_heads <= 0 || q_heads % kv_heads != 0 || dim < 16 || dim > SPEC_CACHE_MAX_DIM || dim % 16 != 0 ||
      max_len <= 0)
    return 0;
  int dev, sms;
  if (device_sms(&dev, &sms) != SPEC_OK) return 0;
  const int64_t rows = static_cast<int64_t>(max_len) * (q_heads / kv_heads);
  uint64_t most = 0;
  for (spec_cache_type type : {SPEC_CACHE_BF16, SPEC_CACHE_E4M3, SPEC_CACHE_INT8}) {
    for (const bool few : {false, true}) {
      const uint64_t n = scratch_bytes(variant_for(type, dim, rows, true, few), sms);
      most = n > most ? n : most;
    }
  }
  return most;
}

int spec_paged_attention(const spec_paged_attention_args* a, void* stream) {
  if (a == nullptr) return SPEC_ERR_INVALID_ARG;
  AttendParams p{};
  int rc = check_cache(a->cache, &p.c);
  if (rc != SPEC_OK) return rc;
  if (a->q_heads <= 0 || a->q_heads % p.c.kv_heads != 0 || a->window < 0 || a->max_context < 0) return SPEC_ERR_INVALID_ARG;
  if (a->q_row_stride < 0 || a->q_head_stride < 0 || a->out_row_stride <= 0 || a->out_head_stride <= 0) return SPEC_ERR_INVALID_ARG;
  for (int64_t s : {a->q_row_stride, a->q_head_stride, a->out_row_stride, a->out_head_stride})
    if (s % 8 != 0) return SPEC_ERR_INVALID_ARG;
  if (a->lse != nullptr && a->lse_row_stride < a->q_heads) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(a->q) || !aligned16(a->out) || !aligned16(a->workspace)) return SPEC_ERR_INVALID_ARG;
  const int64_t rows = static_cast<int64_t>(p.c.max_len) * (a->q_heads / p.c.kv_heads);
  if (rows > (1 << 30)) return SPEC_ERR_INVALID_ARG;
  if (p.c.lanes == 0) return SPEC_OK;
  if (p.c.rows > 0 && (a->q == nullptr || a->out == nullptr)) return SPEC_ERR_INVALID_ARG;
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.q_row = a->q_row_stride;
  p.q_head = a->q_head_stride;
  p.out_row = a->out_row_stride;
  p.out_head = a->out_head_stride;
  p.lse = a->lse;
  p.lse_row = a->lse_row_stride;
  p.group = a->q_heads / p.c.kv_heads;
  specv::set_magic(p.group, p.group_magic, p.group_shift);
  p.window = a->window;
  p.scale = a->scale * 1.44269504088896f;
  if (a->max_context > 0 && a->max_context < p.c.most) p.c.most = a->max_context;
  int dev, sms;
  if ((rc = device_sms(&dev, &sms)) != SPEC_OK) return rc;
  // The tiles' kernel takes its maxima from unscaled scores: not for a scale of 0 or below (or NaN, or
  // infinite), nor for one that is nothing beside the largest numbers.
  const bool few = static_cast<int64_t>(p.c.lanes) * p.c.kv_heads <= sms / 4;
  const PagedVariant v = variant_for(a->cache.type, p.c.dim, rows, p.scale >= 0x1p-100f && p.scale <= 0x1.fffffep127f, few);
  if ((rc = grant_smem(v, dev)) != SPEC_OK) return rc;
  const bool split = a->workspace != nullptr && a->workspace_bytes >= scratch_bytes(v, sms);
  p.heads = v.heads;
  while (p.c.kv_heads % p.heads != 0) p.heads /= 2;
  p.head_groups = p.c.kv_heads / p.heads;
  p.workers = v.heads / p.heads;
  if (split) {
    p.records = static_cast<specv::PartRecord*>(a->workspace);
    p.parts = reinterpret_cast<float*>(p.records + sms * specv::kMostWorkers);
  }
  const char* const withhold = std::getenv("SPEC_PAGED_TEST_WITHHOLD_COPY");
  int test_withhold = withhold != nullptr && std::atoi(withhold) != 0;
  void* args[] = {&p, &test_withhold};
  rc = launch(v.kernel, dim3(static_cast<unsigned>(sms)), static_cast<unsigned>(v.threads), static_cast<size_t>(v.smem), args, stream);
  if (rc != SPEC_OK || (!split && p.c.status == nullptr)) return rc;
  if (!split) {
    void* status_args[] = {&p.c};
    return launch(reinterpret_cast<void*>(&paged_status_kernel), dim3(1), kStatusThreads, 0, status_args, stream);
  }
  // Rows of a thread block of the join: one, and more where that would be too many blocks, most of
  // which find nothing to do.
  int of_item = v.rows, used = static_cast<int>(rows < v.rows ? rows : v.rows);
  const int workers = sms * p.workers, tasks = used * p.heads;
  int per_block = (tasks * p.workers + 31) / 32;
  void* join_args[] = {&p, &of_item, &used, &per_block};
  return launch(join_kernel(v.size), dim3(static_cast<unsigned>(workers), static_cast<unsigned>((tasks + per_block - 1) / per_block)),
                specv::kJoinThreads, 0, join_args, stream);
}

}  // extern "C"
