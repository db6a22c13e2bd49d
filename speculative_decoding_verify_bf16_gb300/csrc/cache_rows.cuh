// cache_rows.cuh -- rows of keys and values into the slots of a paged cache, and back.
//
// A group of 8, 16 or 32 threads takes a token's head, eight numbers a thread, keys and
// values of it one after the other; the largest number is a few shuffles away.  A CTA takes
// a run of rows, whose slots its threads look up first, one row each.
//
// It is bound by HBM.  Measured (device time): a lane of 40,001 tokens from int8 to fp32, 410 MB, 65
// us, 6.3 TB/s, 0.93 of the copy rate (83 us with each thread's fp32 numbers side by side: stores of 16
// bytes at every 32); 24 prompts of 0 to 3000 tokens in bf16 into e4m3 slots and back, 496 MB in two calls,
// 94 us, 5.3 TB/s (4 % more with CTAs of 256 threads, two rounds of loads at a time; 60 % with four,
// whose registers cost too many CTAs), into bf16 slots and back, 660 MB, 107 us, 6.2 TB/s; one row there
// and back 5.1 us, two launches.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "cache_params.h"
#include "device_ptx.cuh"

namespace specv {

constexpr int kRowThreads = 128;
constexpr int kRowsMost = 32;  // rows of a CTA

struct CacheRowsParams {
  CacheParams c;
  uint8_t* k;  // strides in bytes
  uint8_t* v;
  int64_t k_row, k_head, v_row, v_head;
  int32_t rows_per_cta;
};

// The row's lane, by bisection of offsets that ascend.
__device__ __forceinline__ int lane_of_row(const CacheParams& c, int row) {
  int lo = 0, hi = c.lanes;  // offsets[lo] <= row < offsets[hi], in good order
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(c.offsets + mid) <= row)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// Two e4m3 numbers as fp16 (exact), and two fp32 numbers rounded to e4m3.
__device__ __forceinline__ uint32_t e4m3_to_half2(uint32_t two) {
  uint32_t d;
  asm("{\n\t.reg .b16 s;\n\tcvt.u16.u32 s, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, s;\n\t}" : "=r"(d) : "r"(two));
  return d;
}
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t to_bf16x2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// The exponent's byte of a head whose largest magnitude is `top_bits` (of an fp32 number), 255
// if it cannot be held: the least e with top * 2^e >= 2^x m (1 <= m < 2), x - whole or one more.
template <int TYPE>
__device__ __forceinline__ uint32_t exponent_byte(uint32_t top_bits) {
  constexpr int kWhole = TYPE == SPEC_CACHE_E4M3 ? 8 : 6;                        // 448 = 1.75 * 2^8, 127 = 1.984375 * 2^6
  constexpr uint32_t kFraction = TYPE == SPEC_CACHE_E4M3 ? 0x600000u : 0x7E0000u;
  const int e = static_cast<int>(top_bits >> 23) - kWhole + ((top_bits & 0x7FFFFFu) > kFraction ? 1 : 0);
  if (e > 127 + SPEC_CACHE_MOST_EXP) return 255u;  // (NaN and infinities among them)
  return e < 127 + SPEC_CACHE_LEAST_EXP ? 127 + SPEC_CACHE_LEAST_EXP : e;
}

// A thread has eight numbers of a head in two fours, at `d` and `e`: in bf16 rows side by side, 16 bytes; in
// fp32 rows so that each four, 16 bytes too, lies beside the next thread's.
template <typename T>
__device__ __forceinline__ void load_fours(float (&x)[8], const uint8_t* from, int d, int e, bool on_d, bool on_e) {
  if constexpr (sizeof(T) == 4) {
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = on_d ? __ldcs(reinterpret_cast<const float4*>(from + 4 * d)) : zero;
    const float4 b = on_e ? __ldcs(reinterpret_cast<const float4*>(from + 4 * e)) : zero;
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 a = on_d ? __ldcs(reinterpret_cast<const uint4*>(from + 2 * d)) : make_uint4(0u, 0u, 0u, 0u);
    x[0] = bf16_lo(a.x), x[1] = bf16_hi(a.x), x[2] = bf16_lo(a.y), x[3] = bf16_hi(a.y);
    x[4] = bf16_lo(a.z), x[5] = bf16_hi(a.z), x[6] = bf16_lo(a.w), x[7] = bf16_hi(a.w);
  }
}
template <typename T>
__device__ __forceinline__ void store_fours(uint8_t* to, const float (&x)[8], int d, int e, bool on_d, bool on_e) {
  if constexpr (sizeof(T) == 4) {
    if (on_d) *reinterpret_cast<float4*>(to + 4 * d) = make_float4(x[0], x[1], x[2], x[3]);
    if (on_e) *reinterpret_cast<float4*>(to + 4 * e) = make_float4(x[4], x[5], x[6], x[7]);
  } else if (on_d) {
    *reinterpret_cast<uint4*>(to + 2 * d) =
        make_uint4(to_bf16x2(x[0], x[1]), to_bf16x2(x[2], x[3]), to_bf16x2(x[4], x[5]), to_bf16x2(x[6], x[7]));
  }
}

// GROUP threads a head (dim <= 8 * GROUP).  WRITE: rows to slots; otherwise slots to rows.  (Registers as for one
// pass over the rows: the loop over lanes alone would take 48 instead of 40, and a write 6 % longer.)
template <typename T, int TYPE, int GROUP, bool WRITE>
__global__ void __launch_bounds__(kRowThreads, WRITE ? 12 : 16) cache_rows_kernel(const CacheRowsParams p) {
  const CacheParams& c = p.c;
  __shared__ int64_t slot_at[kRowsMost], exp_at[kRowsMost];
  __shared__ int lane_at[kRowsMost];  // -1: nothing to do
  __shared__ volatile int turn;       // the next lane, where lanes take turns; -1: they do not
  if (threadIdx.x == 0) turn = -1;
  griddep_wait();
  griddep_launch_dependents();
  const int row0 = blockIdx.x * p.rows_per_cta;
  const int mine = min(p.rows_per_cta, c.rows - row0);
  // A row has one lane at most where offsets ascend.  Where some descend, the lanes are gone through one after
  // the other, each by its own.
  bool descend = false;
  if (threadIdx.x >= kRowsMost)  // (by the threads that look no row up)
#pragma unroll 1
    for (int b = threadIdx.x - kRowsMost; b < c.lanes; b += kRowThreads - kRowsMost)
      descend |= __ldg(c.offsets + b) > __ldg(c.offsets + b + 1);
  auto look_up = [&](int row, int b) {
    int first, count, before, lane = -1;
    int64_t at = 0, ea = 0;
    if (cache_lane(c, b, first, count, before) && row >= first && row < first + count &&
        (c.status == nullptr || c.status[b] == SPEC_OK)) {
      const int pos = before + row - first, page = page_of(c, pos);
      const int id = __ldg(c.tables + b * c.table_stride + page), in = pos - page * c.page_size;
      if (static_cast<uint32_t>(id) < static_cast<uint32_t>(c.pages)) {
        lane = b;
        at = id * c.page + in * c.slot;
        ea = id * c.exp_page + in * c.exp_slot;
      } else {
        lane_failed(c, b, SPEC_ERR_LAYOUT);
      }
    }
    lane_at[threadIdx.x] = lane;
    slot_at[threadIdx.x] = at;
    exp_at[threadIdx.x] = ea;
  };
  if (static_cast<int>(threadIdx.x) < mine) look_up(row0 + threadIdx.x, lane_of_row(c, row0 + threadIdx.x));
  // Lanes laid out wrongly own no row for certain: the first CTA looks at all of them.
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b < c.lanes; b += kRowThreads) {
      int first, count, before;
      if (!cache_lane(c, b, first, count, before)) lane_failed(c, b, SPEC_ERR_LAYOUT);
    }
  if (__syncthreads_or(descend)) {
    if (threadIdx.x < kRowsMost) lane_at[threadIdx.x] = -1;
    if (threadIdx.x == 0) turn = 0;
    __syncthreads();
  }
  const int unit = threadIdx.x % GROUP, heads = mine * c.kv_heads;
  const int d = sizeof(T) == 4 ? 4 * unit : 8 * unit, e = sizeof(T) == 4 ? d + 4 * GROUP : d + 4;
#pragma unroll 1
  for (;;) {
#pragma unroll 1
    for (int base = 0; base < heads; base += kRowThreads / GROUP) {
      const int i = base + threadIdx.x / GROUP;
      const int r = i / c.kv_heads, h = i - r * c.kv_heads;
      const int b = i < heads ? lane_at[r] : -1;
      const bool on_d = b >= 0 && d < c.dim, on_e = b >= 0 && e < c.dim;
      const int64_t at = b < 0 ? 0 : slot_at[r] + h * c.head;
      const int64_t ea = b < 0 ? 0 : exp_at[r] + h * c.exp_head;
      uint8_t* const kr = p.k + (row0 + r) * p.k_row + h * p.k_head;
      uint8_t* const vr = p.v + (row0 + r) * p.v_row + h * p.v_head;
      float x[2][8];
      if constexpr (WRITE) {
        load_fours<T>(x[0], kr, d, e, on_d, on_e);
        load_fours<T>(x[1], vr, d, e, on_d, on_e);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint8_t* const to = (s ? c.v : c.k) + at;
          // Magnitudes order as their bits, NaN above all.
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(x[s][j]) & 0x7FFFFFFFu);
          bool bad;
          if constexpr (TYPE == SPEC_CACHE_BF16) {
            bad = top > 0x7F7F7FFFu;  // rounds to an infinity in bf16, or is one or NaN (what is not there is 0)
            const uint2 lo = make_uint2(to_bf16x2(x[s][0], x[s][1]), to_bf16x2(x[s][2], x[s][3]));
            const uint2 hi = make_uint2(to_bf16x2(x[s][4], x[s][5]), to_bf16x2(x[s][6], x[s][7]));
            if constexpr (sizeof(T) == 4) {
              if (on_d) *reinterpret_cast<uint2*>(to + 2 * d) = lo;
              if (on_e) *reinterpret_cast<uint2*>(to + 2 * e) = hi;
            } else if (on_d) {
              *reinterpret_cast<uint4*>(to + 2 * d) = make_uint4(lo.x, lo.y, hi.x, hi.y);
            }
          } else {
#pragma unroll
            for (int z = 1; z < GROUP; z <<= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, z));
            const uint32_t byte = exponent_byte<TYPE>(top);
            const float inverse = __uint_as_float((254u - (byte == 255u ? 127u : byte)) << 23);
            uint32_t w[2];
            if constexpr (TYPE == SPEC_CACHE_E4M3) {
#pragma unroll
              for (int j = 0; j < 2; ++j)
                w[j] = to_e4m3x2(x[s][4 * j] * inverse, x[s][4 * j + 1] * inverse) |
                       to_e4m3x2(x[s][4 * j + 2] * inverse, x[s][4 * j + 3] * inverse) << 16;
            } else {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint32_t y[4];
#pragma unroll
                for (int z = 0; z < 4; ++z) y[z] = static_cast<uint32_t>(__float2int_rn(x[s][4 * j + z] * inverse)) & 255u;
                w[j] = y[0] | y[1] << 8 | y[2] << 16 | y[3] << 24;
              }
            }
            if constexpr (sizeof(T) == 4) {
              if (on_d) *reinterpret_cast<uint32_t*>(to + d) = w[0];
              if (on_e) *reinterpret_cast<uint32_t*>(to + e) = w[1];
            } else if (on_d) {
              *reinterpret_cast<uint2*>(to + d) = make_uint2(w[0], w[1]);
            }
            if (on_d && unit == 0) (s ? c.v_exps : c.k_exps)[ea] = static_cast<uint8_t>(byte);
            bad = byte == 255u && b >= 0 && unit == 0;
          }
          if (bad) lane_failed(c, b, SPEC_ERR_NONFINITE);
        }
      } else {
        if constexpr (TYPE == SPEC_CACHE_BF16) {
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint8_t* const from = (s ? c.v : c.k) + at;
            uint4 a = make_uint4(0u, 0u, 0u, 0u);
            if constexpr (sizeof(T) == 4) {
              if (on_d) *reinterpret_cast<uint2*>(&a.x) = __ldcs(reinterpret_cast<const uint2*>(from + 2 * d));
              if (on_e) *reinterpret_cast<uint2*>(&a.z) = __ldcs(reinterpret_cast<const uint2*>(from + 2 * e));
            } else if (on_d) {
              a = __ldcs(reinterpret_cast<const uint4*>(from + 2 * d));
            }
            x[s][0] = bf16_lo(a.x), x[s][1] = bf16_hi(a.x), x[s][2] = bf16_lo(a.y), x[s][3] = bf16_hi(a.y);
            x[s][4] = bf16_lo(a.z), x[s][5] = bf16_hi(a.z), x[s][6] = bf16_lo(a.w), x[s][7] = bf16_hi(a.w);
          }
        } else {
          uint2 w[2] = {};
          uint32_t byte[2] = {};
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const uint8_t* const from = (s ? c.v : c.k) + at;
            if constexpr (sizeof(T) == 4) {
              if (on_d) w[s].x = __ldcs(reinterpret_cast<const uint32_t*>(from + d));
              if (on_e) w[s].y = __ldcs(reinterpret_cast<const uint32_t*>(from + e));
            } else {
              w[s] = on_d ? __ldcs(reinterpret_cast<const uint2*>(from + d)) : make_uint2(0u, 0u);
            }
            byte[s] = on_d ? (s ? c.v_exps : c.k_exps)[ea] : 0u;
          }
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const float scale = byte[s] == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(byte[s] << 23);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t two = ((j < 2 ? w[s].x : w[s].y) >> (16 * (j & 1))) & 0xFFFFu;
              if constexpr (TYPE == SPEC_CACHE_E4M3) {
                const uint32_t hh = e4m3_to_half2(two);
                const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hh));
                x[s][2 * j] = f.x * scale;
                x[s][2 * j + 1] = f.y * scale;
              } else {
                x[s][2 * j] = static_cast<float>(static_cast<int8_t>(two & 255u)) * scale;
                x[s][2 * j + 1] = static_cast<float>(static_cast<int8_t>(two >> 8)) * scale;
              }
            }
          }
        }
        store_fours<T>(kr, x[0], d, e, on_d, on_e);
        store_fours<T>(vr, x[1], d, e, on_d, on_e);
      }
    }
    const int next = turn;
    if (next < 0) break;
    __syncthreads();
    if (next == c.lanes) break;
    if (static_cast<int>(threadIdx.x) < mine) look_up(row0 + threadIdx.x, next);
    if (threadIdx.x == 0) turn = next + 1;
    __syncthreads();
  }
}

}  // namespace specv
