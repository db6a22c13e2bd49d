// linear.cu -- host side of include/spec_linear.h: argument checks, the choice of
// kernel and the launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "linear_chunk.cuh"
#include "linear_params.h"
#include "linear_recurrent.cuh"

namespace {

using specv::LinearParams;

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Checks the arguments and lays them out for the kernels.  `empty` is set when
// there is nothing to do.
int check_args(const spec_linear_args* a, LinearParams* p, bool* empty) {
  *empty = false;
  if (a == nullptr) return SPEC_ERR_INVALID_ARG;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (a->lanes < 0 || a->rows < 0 || a->max_len < 0) return SPEC_ERR_INVALID_ARG;
  if (a->k_heads <= 0 || a->v_heads <= 0 || a->v_heads % a->k_heads != 0) return SPEC_ERR_INVALID_ARG;
  if (a->dk <= 0 || a->dk > SPEC_LINEAR_MAX_DIM || a->dv <= 0 || a->dv > SPEC_LINEAR_MAX_DIM || a->dv % 4 != 0)
    return SPEC_ERR_INVALID_ARG;
  const int64_t strides[] = {a->q_row_stride,   a->q_head_stride,   a->k_row_stride,     a->k_head_stride,
                             a->v_row_stride,   a->v_head_stride,   a->decay_row_stride, a->decay_head_stride,
                             a->out_row_stride, a->out_head_stride};
  for (int64_t s : strides)
    if (s < 0) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(a->state_in) || !aligned16(a->state_out)) return SPEC_ERR_INVALID_ARG;
  if (a->state_in != nullptr && (a->state_in_lane_stride % 4 != 0 || a->state_in_head_stride % 4 != 0))
    return SPEC_ERR_INVALID_ARG;
  if (a->state_out != nullptr && (a->state_out_lane_stride % 4 != 0 || a->state_out_head_stride % 4 != 0 ||
                                  a->state_out_col_stride % 4 != 0))
    return SPEC_ERR_INVALID_ARG;
  // One CTA for each lane, head and 32 columns of the state.
  const int64_t ctas = static_cast<int64_t>(a->lanes) * a->v_heads * ((a->dv + specv::kRecCols - 1) / specv::kRecCols);
  if (ctas > INT32_MAX) return SPEC_ERR_INVALID_ARG;
  if (a->lanes == 0) {
    *empty = true;
    return SPEC_OK;
  }
  if (a->row_offsets == nullptr) return SPEC_ERR_INVALID_ARG;
  if (a->rows > 0 && (a->q == nullptr || a->k == nullptr || a->v == nullptr || a->out == nullptr ||
                      a->log_decay == nullptr))
    return SPEC_ERR_INVALID_ARG;
  p->q = a->q;
  p->k = a->k;
  p->v = a->v;
  p->out = a->out;
  p->q_row = a->q_row_stride;
  p->q_head = a->q_head_stride;
  p->k_row = a->k_row_stride;
  p->k_head = a->k_head_stride;
  p->v_row = a->v_row_stride;
  p->v_head = a->v_head_stride;
  p->out_row = a->out_row_stride;
  p->out_head = a->out_head_stride;
  p->log_decay = a->log_decay;
  p->decay_row = a->decay_row_stride;
  p->decay_head = a->decay_head_stride;
  p->row_offsets = a->row_offsets;
  p->state_in = a->state_in;
  p->state_in_lane = a->state_in_lane_stride;
  p->state_in_head = a->state_in_head_stride;
  p->state_out = a->state_out;
  p->state_out_lane = a->state_out_lane_stride;
  p->state_out_col = a->state_out_col_stride;
  p->state_out_head = a->state_out_head_stride;
  p->lane_status = a->lane_status;
  p->lanes = a->lanes;
  p->rows = a->rows;
  p->max_len = a->max_len;
  p->v_heads = a->v_heads;
  p->group = a->v_heads / a->k_heads;
  p->dk = a->dk;
  p->dv = a->dv;
  p->scale = a->scale;
  return SPEC_OK;
}

template <typename T, bool STAGED>
void* recurrent_kernel_for(int dk) {
  if (dk <= 64) return reinterpret_cast<void*>(&specv::linear_recurrent_kernel<T, 4, STAGED>);
  if (dk <= 128) return reinterpret_cast<void*>(&specv::linear_recurrent_kernel<T, 8, STAGED>);
  return reinterpret_cast<void*>(&specv::linear_recurrent_kernel<T, 16, STAGED>);
}

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
struct DeviceCache {
  int sms = 0;
  bool chunk_attr = false;
};
DeviceCache g_cache[kMaxDevices];

int device_cache(DeviceCache** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPEC_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_mutex);
  DeviceCache& c = g_cache[dev];
  if (c.sms == 0 && cudaDeviceGetAttribute(&c.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return SPEC_ERR_CUDA;
  *out = &c;
  return SPEC_OK;
}

int launch(void* kernel, unsigned grid, unsigned block, size_t smem, void** args, void* stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
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

int launch_recurrent(const LinearParams& p, spec_dtype dtype, bool staged, void* stream) {
  void* kernel;
  if (dtype == SPEC_BF16)
    kernel = staged ? recurrent_kernel_for<__nv_bfloat16, true>(p.dk) : recurrent_kernel_for<__nv_bfloat16, false>(p.dk);
  else
    kernel = staged ? recurrent_kernel_for<float, true>(p.dk) : recurrent_kernel_for<float, false>(p.dk);
  const unsigned grid = static_cast<unsigned>(p.lanes) * p.v_heads * ((p.dv + specv::kRecCols - 1) / specv::kRecCols);
  void* args[] = {const_cast<LinearParams*>(&p)};
  return launch(kernel, grid, specv::kRecThreads, 0, args, stream);
}

// ---------------------------------------------------------------------------
// Chunked prefill
// ---------------------------------------------------------------------------
// Shorter prompts run token after token.  Measured, 16 heads of 128, chunked against token
// after token, in us: 8 tokens, 7.7 / 5.5 with 1 lane, 9.1 / 8.9 with 8, 48 / 60 with 64;
// 16 tokens, 7.9 / 8.8, 9.3 / 14.5 and 49 / 98; 4 tokens, 7.7 / 4.1, 8.9 / 6.6 and 47 / 42.
constexpr int kChunkMinLen = 8;

// Segments a lane's chunks are split into: with fewer (lane, head) pairs than half the
// SMs, as many as occupy them, of two chunks at least.  A split lane's k and v are read
// twice, by two launches, so short lanes do not pay, and short halves little.  Measured with
// 16 heads, whole against split, in us: 512 tokens, 19.0 / 24.4; 1024, 32.8 / 26.3; 2048,
// 60 / 32; 16384, 436 / 99; with 64 pairs, in halves: 1024 tokens, 33.6 / 39.1; 2048, 63 / 58;
// 4096, 117 / 94.
// At most as many as `most`, for which there is scratch memory.
int prefill_segments(int64_t pairs, int64_t chunks, int sms, int64_t most) {
  if (pairs <= 0 || 2 * pairs > sms || chunks < 8 || most < 2) return 1;
  const int64_t want = sms / pairs < most ? sms / pairs : most;
  const int64_t per = (chunks + want - 1) / want < 2 ? 2 : (chunks + want - 1) / want;
  const int64_t n = (chunks + per - 1) / per;
  return n > 2 || chunks > 16 ? static_cast<int>(n) : 1;
}

int64_t chunks_of(int max_len) { return (static_cast<int64_t>(max_len) + specv::kChunk - 1) / specv::kChunk; }

// Scratch memory of a segment of a (lane, head) pair: its state and its decay.
constexpr uint64_t kSegmentBytes = (128 * 128 + 4) * sizeof(float);

typedef CUresult (*EncodeTiled)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
  static const EncodeTiled f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeTiled>(p);
  }();
  return f;
}

// Whether a tensor map can describe bf16 activations with these strides.
bool mappable(const void* base, int64_t row_stride, int64_t head_stride, int heads) {
  if (!aligned16(base) || row_stride % 8 != 0 || row_stride <= 0 || row_stride >= (int64_t{1} << 38)) return false;
  return heads == 1 || (head_stride % 8 == 0 && head_stride > 0 && head_stride < (int64_t{1} << 38));
}

// [rows][heads][size] bf16, copied in boxes of 128 rows of 64 elements of one head (zeros
// past the head's size).
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int size, int64_t row_stride,
              int64_t head_stride) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(size), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads == 1 ? row_stride : head_stride) * 2,
                                 static_cast<cuuint64_t>(row_stride) * 2};
  const cuuint32_t box[3] = {64, 1, specv::kChunk}, step[3] = {1, 1, 1};
  return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// States [lanes][heads][dk][dv], copied in boxes of 128 rows of 32 numbers.
bool mappable_state(const void* base, int64_t lane_stride, int64_t head_stride, int lanes, int heads) {
  auto fits = [](int64_t s, int n) { return n == 1 || (s > 0 && s < (int64_t{1} << 37)); };
  return base == nullptr || (fits(lane_stride, lanes) && fits(head_stride, heads));
}

bool make_state_map(CUtensorMap* map, const void* base, int64_t lanes, int heads, int dk, int dv, int64_t lane_stride,
                    int64_t head_stride) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(dv), static_cast<cuuint64_t>(dk), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(lanes)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(dv) * 4,
                                 static_cast<cuuint64_t>(heads == 1 ? dk * dv : head_stride) * 4,
                                 static_cast<cuuint64_t>(lanes == 1 ? dk * dv : lane_stride) * 4};
  const cuuint32_t box[4] = {32, 128, 1, 1}, step[4] = {1, 1, 1, 1};
  return encode_tiled()(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4, const_cast<void*>(base), dims, strides, box, step,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool chunkable(const LinearParams& p, spec_dtype dtype) {
  const int k_heads = p.v_heads / p.group;
  return dtype == SPEC_BF16 && p.dk <= 128 && p.dv <= 128 && p.rows > 0 && p.max_len >= kChunkMinLen &&
         mappable(p.q, p.q_row, p.q_head, k_heads) && mappable(p.k, p.k_row, p.k_head, k_heads) &&
         mappable(p.v, p.v_row, p.v_head, p.v_heads) && mappable(p.out, p.out_row, p.out_head, p.v_heads) &&
         mappable_state(p.state_in, p.state_in_lane, p.state_in_head, p.lanes, p.v_heads) &&
         mappable_state(p.state_out, p.state_out_lane, p.state_out_head, p.lanes, p.v_heads) &&
         encode_tiled() != nullptr;
}

int launch_chunk(const LinearParams& p, DeviceCache* dc, const spec_linear_args* a, void* stream) {
  const int64_t pairs = static_cast<int64_t>(p.lanes) * p.v_heads;
  void* const states = reinterpret_cast<void*>(&specv::linear_chunk_kernel<true>);
  void* const full = reinterpret_cast<void*>(&specv::linear_chunk_kernel<false>);
  const int smem = static_cast<int>(sizeof(specv::ChunkSmem));
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (!dc->chunk_attr) {
      for (void* k : {states, full}) {
        // The warpgroups' shares must not add up to more than the launch brings.
        cudaFuncAttributes fa;
        if (cudaFuncGetAttributes(&fa, k) != cudaSuccess || fa.numRegs * (specv::kChunkThreads / 128) < specv::kChunkRegs)
          return SPEC_ERR_CUDA;
        if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
          cudaGetLastError();
          return SPEC_ERR_CUDA;
        }
      }
      dc->chunk_attr = true;
    }
  }
  specv::ChunkParams cp{};
  cp.p = p;
  const uint64_t held = a->workspace == nullptr ? 0 : a->workspace_bytes / (kSegmentBytes * pairs);
  cp.segments = prefill_segments(pairs, chunks_of(p.max_len), dc->sms, static_cast<int64_t>(held));
  if (cp.segments > 1 && !aligned16(a->workspace)) return SPEC_ERR_INVALID_ARG;
  cp.local = static_cast<float*>(a->workspace);
  cp.local_decay = cp.local + static_cast<int64_t>(cp.segments) * pairs * (128 * 128);
  const int k_heads = p.v_heads / p.group;
  CUtensorMap q, k, v, out, local, begin, end;
  if (!make_map(&q, p.q, p.rows, k_heads, p.dk, p.q_row, p.q_head) || !make_map(&k, p.k, p.rows, k_heads, p.dk, p.k_row, p.k_head) ||
      !make_map(&v, p.v, p.rows, p.v_heads, p.dv, p.v_row, p.v_head) ||
      !make_map(&out, p.out, p.rows, p.v_heads, p.dv, p.out_row, p.out_head))
    return SPEC_ERR_CUDA;
  const bool split = cp.segments > 1;
  if (split && !make_state_map(&local, cp.local, static_cast<int64_t>(cp.segments) * p.lanes, p.v_heads, 128, 128,
                               static_cast<int64_t>(p.v_heads) * 128 * 128, 128 * 128))
    return SPEC_ERR_CUDA;
  begin = split ? local : q;  // (where nothing is read or written, any map will do)
  end = q;
  if (!split && p.state_in != nullptr &&
      !make_state_map(&begin, p.state_in, p.lanes, p.v_heads, p.dk, p.dv, p.state_in_lane, p.state_in_head))
    return SPEC_ERR_CUDA;
  if (p.state_out != nullptr &&
      !make_state_map(&end, p.state_out, p.lanes, p.v_heads, p.dk, p.dv, p.state_out_lane, p.state_out_head))
    return SPEC_ERR_CUDA;
  void* args[] = {&cp, &q, &k, &v, &out, &begin, &end};
  void* states_args[] = {&cp, &q, &k, &v, &out, &begin, &local};
  cp.sort = p.lanes > 1 && p.lanes <= specv::kSortLanes && static_cast<int64_t>(p.lanes) * p.max_len != p.rows;
  const char* withhold = std::getenv("SPEC_LINEAR_TEST_WITHHOLD_COPY");
  cp.test_withhold = withhold != nullptr && std::atoi(withhold) != 0;
  if (split) {
    const int rc = launch(states, static_cast<unsigned>(pairs * (cp.segments - 1)), specv::kChunkThreads, smem, states_args, stream);
    if (rc != SPEC_OK) return rc;
  }
  return launch(full, static_cast<unsigned>(pairs * cp.segments), specv::kChunkThreads, smem, args, stream);
}

}  // namespace

extern "C" {

uint64_t spec_linear_workspace(int32_t lanes, int32_t v_heads, int32_t dk, int32_t dv, int32_t max_len) {
  if (lanes <= 0 || v_heads <= 0 || dk <= 0 || dk > 128 || dv <= 0 || dv > 128 || max_len < kChunkMinLen)
    return 0;
  DeviceCache* dc = nullptr;
  if (device_cache(&dc) != SPEC_OK) return 0;
  // The most that any call of up to this many lanes and tokens cuts.  (Fewer lanes may be cut
  // into more segments each, and shorter ones too: segments have two chunks at least.)
  const int64_t chunks = chunks_of(max_len);
  int64_t most = 0;
  for (int64_t pairs = v_heads; pairs <= static_cast<int64_t>(lanes) * v_heads && 2 * pairs <= dc->sms; pairs += v_heads) {
    const int64_t n = dc->sms / pairs < (chunks + 1) / 2 ? dc->sms / pairs : (chunks + 1) / 2;
    if (chunks >= 8 && (n > 2 || chunks > 16) && n * pairs > most) most = n * pairs;
  }
  return static_cast<uint64_t>(most) * kSegmentBytes;
}

int spec_linear_prefill(const spec_linear_args* a, void* stream) {
  LinearParams p{};
  bool empty = false;
  const int rc = check_args(a, &p, &empty);
  if (rc != SPEC_OK || empty) return rc;
  if (!chunkable(p, a->dtype)) return launch_recurrent(p, a->dtype, false, stream);
  DeviceCache* dc = nullptr;
  if (device_cache(&dc) != SPEC_OK) return SPEC_ERR_CUDA;
  return launch_chunk(p, dc, a, stream);
}

int spec_linear_verify(const spec_linear_args* a, void* stream) {
  LinearParams p{};
  bool empty = false;
  const int rc = check_args(a, &p, &empty);
  if (rc != SPEC_OK) return rc;
  if (a->lanes > 0 && a->state_out == nullptr) return SPEC_ERR_INVALID_ARG;
  if (empty) return SPEC_OK;
  return launch_recurrent(p, a->dtype, true, stream);
}

}  // extern "C"
