// linear.cu -- host side of include/spec_linear.h: argument checks, the choice of
// kernel and the launches.
#include <cuda_runtime.h>

#include <cstdint>

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

}  // namespace

extern "C" {

uint64_t spec_linear_workspace(int32_t, int32_t, int32_t, int32_t, int32_t) { return 0; }

int spec_linear_prefill(const spec_linear_args* a, void* stream) {
  LinearParams p{};
  bool empty = false;
  const int rc = check_args(a, &p, &empty);
  if (rc != SPEC_OK || empty) return rc;
  return launch_recurrent(p, a->dtype, false, stream);
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
