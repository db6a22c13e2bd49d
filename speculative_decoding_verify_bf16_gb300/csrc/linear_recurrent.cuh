// linear_recurrent.cuh -- linear attention with decay, token after token:
//   S_t = exp(g_t) S_(t-1) + k_t v_t^T,   o_t = scale * S_t^T q_t.
//
// The columns of S (over dv) are independent, so a CTA takes 32 of them for one
// (lane, head) and keeps its dk x 32 piece of the fp32 state in registers: four
// warps, each thread a float4 of one row out of sixteen.  A row access of a warp
// is then four full 128-byte lines.  q and k of a block of tokens are staged in
// shared memory as (k, q) pairs, so that one 8-byte broadcast read feeds the
// update and the product.  o needs a sum over dk: in the thread, then across the
// four row groups of a warp (two shuffles), then across the warps through shared
// memory, once a block of tokens.
//
// With snapshots most of the kernel's bytes are their writes: dk * dv * 4 bytes a column
// and head against 5 * dk * dv operations.  Stored around L2 (nothing here reads them again)
// they leave it to the states: 8 lanes x 8 columns of 16 fp32 heads of 128 (78 MB) take 15.2
// us instead of 18.1; a plain fill of 64 MiB takes 12.4.  64 lanes x up to 4 columns (238 MB)
// take 43.0 us, 5.5 TB/s of reads and writes together, 0.82 of the copy rate: a CTA waits for
// its piece of the state before its first column, and there are 4.5 CTAs for each place on
// an SM.  A single token of a single lane takes 3.3 us: one latency of the loads, the sums
// over dk and a launch.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "device_ptx.cuh"
#include "linear_params.h"

namespace specv {

constexpr int kRecThreads = 128;
constexpr int kRecCols = 32;   // columns of S (over dv) a CTA holds
constexpr int kRecBlock = 8;   // tokens staged at a time

template <typename T>
__device__ __forceinline__ float linear_load(const void* base, int64_t i) {
  return static_cast<float>(static_cast<const T*>(base)[i]);
}

// Rows of lane b, or the status that leaves the lane out.
__device__ __forceinline__ int linear_lane_rows(const LinearParams& p, int b, int& first, int& count) {
  const int o0 = p.row_offsets[b], o1 = p.row_offsets[b + 1];
  first = o0;
  count = o1 - o0;
  if (o0 < 0 || o1 < o0 || o1 > p.rows || count > p.max_len) return SPEC_ERR_LAYOUT;
  return SPEC_OK;
}

// RPT: rows of S a thread holds, dk <= 16 * RPT.  STAGED: the state goes out
// after every token, not after the last one.
template <typename T, int RPT, bool STAGED>
__global__ void __launch_bounds__(kRecThreads) linear_recurrent_kernel(const LinearParams p) {
  __shared__ float2 kq[kRecBlock][16 * RPT];
  __shared__ float vs[kRecBlock][kRecCols];
  __shared__ float decay[kRecBlock];
  __shared__ float part[kRecBlock][4][kRecCols];
  griddep_wait();
  griddep_launch_dependents();
  const int slices = (p.dv + kRecCols - 1) / kRecCols;
  const int slice = blockIdx.x % slices;
  const int h = (blockIdx.x / slices) % p.v_heads;
  const int b = blockIdx.x / slices / p.v_heads;
  // (the warps agree on a status that another head's CTA may be writing)
  if (p.lane_status != nullptr && __syncthreads_or(p.lane_status[b] != SPEC_OK)) return;
  int first, count;
  const int rc = linear_lane_rows(p, b, first, count);
  if (rc != SPEC_OK) {
    if (threadIdx.x == 0 && p.lane_status != nullptr) p.lane_status[b] = rc;
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = slice * kRecCols + (lane & 7) * 4;
  const int row0 = warp * 4 + (lane >> 3);  // rows row0 + 16 i
  const bool col_in = col < p.dv;

  float4 S[RPT];
  const float* in = p.state_in == nullptr ? nullptr
                                          : p.state_in + b * p.state_in_lane + h * p.state_in_head;
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    S[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    const int r = row0 + 16 * i;
    if (in != nullptr && col_in && r < p.dk)
      S[i] = *reinterpret_cast<const float4*>(in + static_cast<int64_t>(r) * p.dv + col);
  }
  float* snap = p.state_out == nullptr ? nullptr : p.state_out + b * p.state_out_lane + h * p.state_out_head;
  auto put = [&](float* dst) {
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      const int r = row0 + 16 * i;
      if (col_in && r < p.dk) __stcs(reinterpret_cast<float4*>(dst + static_cast<int64_t>(r) * p.dv + col), S[i]);
    }
  };

  const int hk = h / p.group;
  for (int t0 = 0; t0 < count; t0 += kRecBlock) {
    const int n = min(kRecBlock, count - t0);
    for (int i = threadIdx.x; i < n * 16 * RPT; i += kRecThreads) {
      const int t = i / (16 * RPT), r = i % (16 * RPT);
      const int64_t row = first + t0 + t;
      float2 x = make_float2(0.f, 0.f);
      if (r < p.dk) {
        x.x = linear_load<T>(p.k, row * p.k_row + hk * p.k_head + r);
        x.y = linear_load<T>(p.q, row * p.q_row + hk * p.q_head + r);
      }
      kq[t][r] = x;
    }
    for (int i = threadIdx.x; i < n * kRecCols; i += kRecThreads) {
      const int t = i / kRecCols, c = i % kRecCols;
      const int64_t row = first + t0 + t;
      vs[t][c] = slice * kRecCols + c < p.dv ? linear_load<T>(p.v, row * p.v_row + h * p.v_head + slice * kRecCols + c) : 0.f;
    }
    if (threadIdx.x < n) {
      const float g = p.log_decay[(first + t0 + static_cast<int64_t>(threadIdx.x)) * p.decay_row + h * p.decay_head];
      decay[threadIdx.x] = expf(g);
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float a = decay[t];
      const float4 v = *reinterpret_cast<const float4*>(&vs[t][(lane & 7) * 4]);
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float2 x = kq[t][row0 + 16 * i];
        S[i].x = fmaf(x.x, v.x, a * S[i].x);
        S[i].y = fmaf(x.x, v.y, a * S[i].y);
        S[i].z = fmaf(x.x, v.z, a * S[i].z);
        S[i].w = fmaf(x.x, v.w, a * S[i].w);
        o.x = fmaf(x.y, S[i].x, o.x);
        o.y = fmaf(x.y, S[i].y, o.y);
        o.z = fmaf(x.y, S[i].z, o.z);
        o.w = fmaf(x.y, S[i].w, o.w);
      }
      if (STAGED) put(snap + (t0 + t) * p.state_out_col);
#pragma unroll
      for (int d = 8; d < 32; d <<= 1) {
        o.x += __shfl_xor_sync(0xFFFFFFFFu, o.x, d);
        o.y += __shfl_xor_sync(0xFFFFFFFFu, o.y, d);
        o.z += __shfl_xor_sync(0xFFFFFFFFu, o.z, d);
        o.w += __shfl_xor_sync(0xFFFFFFFFu, o.w, d);
      }
      if (lane < 8) *reinterpret_cast<float4*>(&part[t][warp][lane * 4]) = o;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * kRecCols; i += kRecThreads) {
      const int t = i / kRecCols, c = i % kRecCols;
      if (slice * kRecCols + c >= p.dv) continue;
      const float s = p.scale * ((part[t][0][c] + part[t][1][c]) + (part[t][2][c] + part[t][3][c]));
      static_cast<T*>(p.out)[(first + t0 + static_cast<int64_t>(t)) * p.out_row + h * p.out_head + slice * kRecCols + c] =
          static_cast<T>(s);
    }
    // The next block's staging writes kq, vs and decay only, whose readers are past
    // the barrier above; `part` is written again behind the next block's barrier.
  }
  if (!STAGED && snap != nullptr) put(snap);
  // An infinity or NaN in k, v or g stays in the state (0 * inf is NaN): x - x is
  // 0 for finite x only.
  float bad = 0.f;
#pragma unroll
  for (int i = 0; i < RPT; ++i) bad += (S[i].x - S[i].x) + (S[i].y - S[i].y) + (S[i].z - S[i].z) + (S[i].w - S[i].w);
  if (bad != 0.f && p.lane_status != nullptr) p.lane_status[b] = SPEC_ERR_NONFINITE;
}

}  // namespace specv
