// linear_params.h -- what the linear-attention kernels are launched with (the checked
// form of spec_linear_args; strides in elements).
#pragma once

#include <cstdint>

#include "spec_linear.h"

namespace specv {

struct LinearParams {
  const void* q;
  const void* k;
  const void* v;
  void* out;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, out_row, out_head;
  const float* log_decay;
  int64_t decay_row, decay_head;
  const int32_t* row_offsets;
  const float* state_in;
  int64_t state_in_lane, state_in_head;
  float* state_out;
  int64_t state_out_lane, state_out_col, state_out_head;
  int32_t* lane_status;
  int32_t lanes, rows, max_len;
  int32_t v_heads, group;  // group: value heads of one key head
  int32_t dk, dv;
  float scale;
};

}  // namespace specv
