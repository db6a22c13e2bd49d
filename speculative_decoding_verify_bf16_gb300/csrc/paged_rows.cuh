// paged_rows.cuh -- attention of a few rows (decoding, a verify round) over a paged cache.
//
// o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(x_j - M),  x_j = scale * log2(e) * q . k_j, with the running maximum M
// of a row: one pass over keys and values.  Scores, sums of weights and numerators are fp32; for the
// second product a weight is rounded to the operands' type, bf16 (an error like that of the output's own
// rounding, and independent of it) or, with an 8-bit cache, fp16 (an eighth of that).
//
// What bounds it is reading the cache: 2 * dim numbers a token and head, for the rows of all query
// heads and columns of that head together.  A thread block's computing warps take a cache head each (of
// a group of heads; where there are fewer heads than warps, of the next worker's units), keep maxima,
// sums and the outputs' numerators of all its rows in registers, and wait for no other warp.  To each
// belongs a warp that does nothing but look up where tokens lie, one by one (any page size and order will
// do), and copy them through a ring in shared memory, 16 bytes a thread: q of an item, then keys
// and values by turns.  (Bulk copies of whole heads, 128 or 256 bytes each, are fewer instructions, but one
// took some 19 cycles of an SM.)  Products are 16 x 8 x 16 ones of a warp: 16 rows are a fraction of
// a 128-row tile of the large tensor cores, and what they save is not short.
//
// Measured (device time, heads of 128): one lane of 131,000 tokens, 8 cache heads in bf16, 537 MB,
// 92 us, 5.8 TB/s, 0.86 of the copy rate; 64 lanes of up to 8,192 tokens in int8, 514 MB, 109 us, 4.7 TB/s
// (in bf16 162 us, 6.3 TB/s): without the arithmetic 92, 92 and 160 us are left.  8
// lanes x 8 columns of 4 heads a cache head (32 rows) in e4m3 77 us (56 without arithmetic: 32 rows' products
// and conversions take 5,300 cycles a unit, its copies at the HBM rate 2,800), in bf16 78; 64 lanes x 1 to 4 columns
// of 8 heads of 64 through a window of 1,000 37 us (31): ten of copies, the rest begins, ends and joins items; one
// lane of 1,500 tokens 12 us: a chain of latencies, and of fetching code (some 110 cycles for each 128
// bytes that a launch runs first), which is why inner loops are short.
// Four copying warps for eight that compute, sums joined through shared memory at each item's end:
// 105, 143 and 85 us for the first, second and third.
//
// 8-bit caches: numbers become fp16 in registers, exactly, and products are fp16.  q is
// taken times a power of two for each row into fp16's range (exactly, but for what is below
// 2^-38 of the row's largest).  The key's power of two multiplies its scores; the value's, 2^e,
// goes into the weight's exponent, w = 2^(x + e - M), and out of the sum of weights again.  M stays seven
// below the running maximum of x + e, so that fp16's 2^-25, below which a weight is lost, is 2^-32 of the
// largest: many small ones together count.  (Weights stay below 2^15; exponents lie within -48..48, so sums
// are within fp32.)  The components' order is free in both products: a thread takes sixteen neighbouring
// bytes of a token at a time.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>
#include <type_traits>

#include "cache_rows.cuh"
#include "device_ptx.cuh"
#include "paged_schedule.cuh"
#include "tcgen05_ptx.cuh"

namespace specv {

constexpr float kRowsSlack = 8.f;  // a maximum is raised when a score, in powers of two, exceeds it by more
// M, from which scores are taken, lies so far below the maximum: fp16 weights use the type's upper range.
template <bool EIGHT>
constexpr float kRowsBelow = EIGHT ? 7.f : 0.f;

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// 16-byte copy of a thread; zeros if not `on`.
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(void* dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
// One arrival (of those that the barrier was set up for) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
template <bool HALF>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (HALF)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t to_halfx2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// Whether four numbers are finite in bf16.
__device__ __forceinline__ bool finite4(float4 a) {
  constexpr float kEnd = 3.3961775e38f;  // from here on numbers round to an infinity
  return fabsf(a.x) < kEnd && fabsf(a.y) < kEnd && fabsf(a.z) < kEnd && fabsf(a.w) < kEnd;
}

// 2^-e of a whole number e within -126..126.
__device__ __forceinline__ float power_of_minus(float e) {
  return __uint_as_float(__float_as_uint(12582912.f + 127.f - e) << 23);  // (the sum's lowest byte is 127 - e)
}

// Bytes 2 i and 2 i + 1 of four 8-bit numbers (int8: with the top bits flipped) as fp16.
template <int TYPE>
__device__ __forceinline__ uint32_t eight_to_half2(uint32_t w, int i) {
  if constexpr (TYPE == SPEC_CACHE_E4M3) {
    return e4m3_to_half2(i == 0 ? w & 0xFFFFu : w >> 16);
  } else {
    // 0x6400 + u is 1024 + u in fp16; u = y + 128.
    const uint32_t m = __byte_perm(w, 0x64646464u, i == 0 ? 0x4140 : 0x4342);
    uint32_t d;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(m), "r"(0x64806480u));
    return d;
  }
}

constexpr int kUnseen = INT32_MIN;  // in a page's place: no row sees the token

template <int TYPE_, int D_, int MT_>
struct RowsShape {
  static constexpr int TYPE = TYPE_, D = D_, MT = MT_;  // cache type, head size (at most), blocks of 16 rows
  static constexpr bool kEight = TYPE != SPEC_CACHE_BF16;
  static constexpr int kRows = 16 * MT;
  static constexpr int kWarps = D > 128 ? 4 : 8;  // that compute; as many copy
  static constexpr int kThreads = 64 * kWarps;
  // Registers a thread, and what a launch must bring (0: they are not shared out).
  // (8 x 8 columns: over e4m3 83 us with 192 and 64, 77 with 200 and 56; over bf16 78 and 77, but 8 x 4 64.6
  // and 65.1, one lane 11.9 and 12.1)
  static constexpr int kRegsRows = kWarps != 8 ? 0 : kEight ? 200 : 192, kRegsCopy = kWarps != 8 ? 0 : kEight ? 56 : 64;
  static constexpr int kRegs = kWarps / 4 * (kRegsRows + kRegsCopy);
  static constexpr int kTokens = kEight || D <= 64 ? 32 : 16;  // of a unit
  static constexpr int kRowBytes = D * (kEight ? 1 : 2);
  // A place of the ring: the keys or the values of a unit, or 16 rows of q; with 8 bits also each token's
  // exponents (words that hold the key's and the value's, and where in them).
  static constexpr int kNumbers = kTokens * kRowBytes > 32 * D ? kTokens * kRowBytes : 32 * D;
  static constexpr int kPlace = kNumbers + (kEight ? kTokens * 9 : 0);
  // Where registers are short, q's operands lie in shared memory.
  static constexpr bool kShared = MT > 1 || D > 128;
  static constexpr int kOperands = kShared ? MT * (D / 16) * 32 : 1;
  static constexpr int kFit = (223 * 1024 / kWarps - kOperands * 16) / kPlace;
  static constexpr int kPlaces = kFit > 12 ? 12 : kFit;
  static constexpr int kExtra = 1;  // an item's beginning and end, in units
  static_assert(kPlaces >= 4, "the ring holds two units at least");
  // (a worker takes two units at least: one lane of 1,500 tokens 11.9 us, with four 14.2; 8 x 8 columns of e4m3
  // behind 1,000 tokens 30 us against 40)
  using Plan = Schedule<kRows, kTokens, kExtra, 2>;
};

template <typename S>
struct RowsSmem {
  uint8_t ring[S::kWarps][S::kPlaces][S::kPlace];
  uint4 q[S::kWarps][S::kOperands];
  typename S::Plan::Shared plan;
  uint64_t full[S::kWarps][S::kPlaces], empty[S::kWarps][S::kPlaces];
  int abort;
};

// Which 16-byte unit of row r a unit u goes to, so that neighbouring rows' equal units lie on
// other banks (8 bits: also those of rows two apart, together with the next unit).
template <bool EIGHT>
__device__ __forceinline__ uint32_t mixed(uint32_t r, uint32_t u) {
  return EIGHT ? u ^ ((r & 2) | (((r >> 2) ^ r) & 1) << 2) : u ^ (r & 7);
}
// (heads of 64 numbers of 8 bits: four units a row)
template <int BYTES, bool EIGHT>
__device__ __forceinline__ uint32_t unit_at(uint32_t r, uint32_t u) {
  return r * BYTES + (BYTES > 64 ? mixed<EIGHT>(r, u) : u ^ ((r >> 1) & 3)) * 16;
}
__device__ __forceinline__ uint4 load_shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

constexpr float kLn2 = 0.693147180559945f;

// A row's parts, joined by a warp: a lane has components 4 lane .. 4 lane + 3 (heads of 64: of every
// other part; of 256: also those 128 later).  take(i): part i's numerators of the row, its
// maximum and sum.
template <int D>
struct RowSum {
  static constexpr int kWide = D > 128 ? 2 : 1, kAcross = D / 4 / kWide, kSubs = 32 / kAcross;
  float top, sum;
  float4 a[kWide];

  // Parts i0, i0 + step, .. of n, lane j's weight the j-th's; BATCH of them on their way at a time.
  template <int BATCH, typename Rows>
  __device__ __forceinline__ void add(int i0, int n, int step, float f, const Rows& rows) {
    const int lane = threadIdx.x & 31, sub = lane / kAcross, at = lane % kAcross;
#pragma unroll 1
    for (int j0 = 0; j0 < n; j0 += BATCH * kSubs) {
      float4 b[BATCH][kWide];
#pragma unroll
      for (int j = 0; j < BATCH; ++j)  // (those past the end weigh 0: the last one again)
#pragma unroll
        for (int z = 0; z < kWide; ++z)
          b[j][z] = __ldcg(reinterpret_cast<const float4*>(rows(i0 + min(j0 + j * kSubs + sub, n - 1) * step)) + at + z * 32);
#pragma unroll
      for (int j = 0; j < BATCH; ++j) {
        const int x = j0 + j * kSubs + sub;
        const float from = __shfl_sync(0xFFFFFFFFu, f, x & 31), w = x < n ? from : 0.f;
#pragma unroll
        for (int z = 0; z < kWide; ++z) {
          a[z].x = fmaf(b[j][z].x, w, a[z].x), a[z].y = fmaf(b[j][z].y, w, a[z].y);
          a[z].z = fmaf(b[j][z].z, w, a[z].z), a[z].w = fmaf(b[j][z].w, w, a[z].w);
        }
      }
    }
  }
  template <int BATCH, typename Rows, typename Stats>
  __device__ __forceinline__ void take(int first, int parts, int step, const Rows& rows, const Stats& stats) {
    const int lane = threadIdx.x & 31;
    top = -INFINITY;
    sum = 0.f;
#pragma unroll
    for (int z = 0; z < kWide; ++z) a[z] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
    for (int i0 = first; i0 < parts; i0 += 32 * step) {  // 32 parts at a time
      const int mine = i0 + lane * step, n = min(32, (parts - i0 + step - 1) / step);
      float2 ms = make_float2(-INFINITY, 0.f);
      if (mine < parts) ms = __ldcg(stats(mine));
      const float most = warp_max_f32(ms.x), raise = fmaxf(most, top), down = top == -INFINITY ? 0.f : ex2_approx(top - raise);
      const float f = ms.x == -INFINITY ? 0.f : ex2_approx(ms.x - raise);
      float s = ms.y * f;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, d);
      sum = fmaf(sum, down, s);
      top = raise;
#pragma unroll
      for (int z = 0; z < kWide; ++z) a[z].x *= down, a[z].y *= down, a[z].z *= down, a[z].w *= down;
      if (BATCH > 4 && n > 8)
        add<BATCH>(i0, n, step, f, rows);
      else
        add<4>(i0, n, step, f, rows);
    }
    if constexpr (kSubs == 2) {
      a[0].x += __shfl_xor_sync(0xFFFFFFFFu, a[0].x, 16);
      a[0].y += __shfl_xor_sync(0xFFFFFFFFu, a[0].y, 16);
      a[0].z += __shfl_xor_sync(0xFFFFFFFFu, a[0].z, 16);
      a[0].w += __shfl_xor_sync(0xFFFFFFFFu, a[0].w, 16);
    }
  }
  // The finished row, of query head `head` and packed row `row`.  (SHIFT: of the errors, 0 in the last launch.)
  template <int SHIFT>
  __device__ __forceinline__ void finish(const AttendParams& p, int lane_of, int64_t row, int head) const {
    const int lane = threadIdx.x & 31, at = lane % kAcross;
    if (lane >= kAcross) return;
    const float inv = 1.f / sum;
#pragma unroll
    for (int z = 0; z < kWide; ++z) {
      const float4 b = make_float4(a[z].x * inv, a[z].y * inv, a[z].z * inv, a[z].w * inv);
      const int d = 4 * at + 128 * z;
      if (d < p.c.dim) {
        *reinterpret_cast<uint2*>(p.out + row * p.out_row + head * p.out_head + d) =
            make_uint2(to_bf16x2(b.x, b.y), to_bf16x2(b.z, b.w));
        if (!finite4(b)) lane_failed(p.c, lane_of, SPEC_ERR_NONFINITE << SHIFT);
      }
    }
    if (p.lse != nullptr && lane == 0) p.lse[row * p.lse_row + head] = (top + log2f(sum)) * kLn2;
  }
};

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1) paged_rows_kernel(const AttendParams p, const int test_withhold) {
  using Plan = typename S::Plan;
  constexpr int TYPE = S::TYPE, D = S::D, MT = S::MT, kTokens = S::kTokens, kPlaces = S::kPlaces;
  constexpr bool kEight = S::kEight;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RowsSmem<S>& sm = *reinterpret_cast<RowsSmem<S>*>(smem_raw);
  const CacheParams& c = p.c;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x < S::kWarps * kPlaces) {
    // (a full place: each copying thread's copies and, with 8 bits, what its warp wrote itself)
    mbar_init(&sm.full[0][0] + threadIdx.x, kEight ? 33 : 32);
    mbar_init(&sm.empty[0][0] + threadIdx.x, 1);
  }
  if (threadIdx.x == 0) sm.abort = 0;
  fence_mbar_init();
  griddep_wait();
  griddep_launch_dependents();
  Plan::plan(p, sm.plan);  // (its barriers publish the above)
  if (blockIdx.x == 0)  // lanes laid out wrongly have no units
    for (int b = threadIdx.x; b < c.lanes; b += S::kThreads) {
      int first, count, before;
      if (!cache_lane(c, b, first, count, before)) lane_fails_now(c, b, SPEC_ERR_LAYOUT);
    }
  const int pair = warp % S::kWarps, worker = pair / p.heads, head_in = pair - worker * p.heads;
  const int64_t begin = sm.plan.begin[worker], end = sm.plan.end[worker];
  int64_t left = end - begin;
  Cursor at = sm.plan.from[worker];
  uint8_t(&ring)[kPlaces][S::kPlace] = sm.ring[pair];
  uint64_t(&full)[kPlaces] = sm.full[pair];
  uint64_t(&empty)[kPlaces] = sm.empty[pair];
  int place = 0, phase = 0;
  auto next_place = [&] {
    if (++place == kPlaces) {
      place = 0;
      phase ^= 1;
    }
  };

  if (warp >= S::kWarps) {
    // ------------------------------------------------------------------ copies
    if constexpr (S::kRegsCopy > 0) registers_shrink<S::kRegsCopy>();
    constexpr int kUnits = S::kRowBytes / 16, kAtOnce = 32 / kUnits;  // 16-byte units of a token; tokens of an access
    const int unit = lane % kUnits, sub = lane / kUnits;
    const bool in_head = unit * 16 < c.dim * (kEight ? 1 : 2);
    const uint32_t by = 1u << c.unit_shift;
    // Pages are looked up two units ahead, within the item: with the memory busy, a load takes as long as
    // that.
    auto look_up = [&](int ahead) {
      const int pos = (at.tile + ahead) * kTokens + lane;
      int page = kUnseen;
      if (ahead < left && at.tile + ahead < at.t1 && lane < kTokens && pos >= at.lo && pos < at.hi)
        page = __ldg(c.tables + at.b * c.table_stride + page_of(c, pos));
      return page;
    };
    const bool withhold = test_withhold != 0 && begin == 0 && head_in == 0;
    bool ok = true, again = false, fresh = true;  // again: the ring has been gone through
    auto acquire = [&] { return ok = !again || warp_wait(&empty[place], phase ^ 1, &sm.abort); };
    auto hand_on = [&] {
      if (!withhold) cp_async_arrive(&full[place]);
      if constexpr (kEight) warp_arrive(&full[place]);
      next_place();
      again = again || place == 0;
    };
    int page0 = kUnseen, page1 = kUnseen;
#pragma unroll 1
    for (; left > 0; --left) {
      if (fresh) {
        page0 = look_up(0);
        page1 = look_up(1);
      }
      const int page2 = look_up(2);
      if (fresh) {  // the item's rows of q, 16 at a time
#pragma unroll 1
        for (int m = 0; m < MT && acquire(); ++m) {
          constexpr int kQUnits = D / 8, kQAtOnce = kQUnits > 32 ? 1 : 32 / kQUnits;
          const int r = at.k * S::kRows + m * 16 + (lane & 15), col = column_of(p, r);
          int64_t row = -1;
          if (col < at.count)
            row = (at.first + col) * p.q_row + ((at.h * p.heads + head_in) * p.group + r - col * p.group) * p.q_head;
          const uint32_t to = smem_addr(ring[place]);
#pragma unroll 4
          for (int j = 0; j < 16 / kQAtOnce; ++j) {
            const int i = j * kQAtOnce + lane / kQUnits, u = lane % kQUnits;
            const int64_t f = __shfl_sync(0xFFFFFFFFu, row, i);
            const bool on = f >= 0 && u * 8 < c.dim;
            cp_async16_or_zero(to + unit_at<2 * D, false>(i, u), p.q + (on ? f + u * 8 : 0), on);
          }
          hand_on();
        }
        if (!ok) break;
      }
      uint32_t from = kNowhere;
      uint8_t where = 255;  // of the exponents in their words: two bits each
      if (!acquire()) break;
      if (page0 != kUnseen) {
        if (static_cast<uint32_t>(page0) >= static_cast<uint32_t>(c.pages)) {
          lane_fails_now(c, at.b, SPEC_ERR_LAYOUT);
        } else {
          const int pos = at.tile * kTokens + lane, in = pos - page_of(c, pos) * c.page_size, head = at.h * p.heads + head_in;
          from = head_at(c, page0, in, head);
          if constexpr (kEight) {
            const int64_t e = page0 * c.exp_page + in * c.exp_slot + head * c.exp_head;
            const uintptr_t ke = reinterpret_cast<uintptr_t>(c.k_exps + e), ve = reinterpret_cast<uintptr_t>(c.v_exps + e);
            cp_async4(&ring[place][S::kNumbers + lane * 4], reinterpret_cast<const void*>(ke & ~uintptr_t{3}));
            cp_async4(&ring[place][S::kNumbers + (kTokens + lane) * 4], reinterpret_cast<const void*>(ve & ~uintptr_t{3}));
            where = static_cast<uint8_t>((ke & 3) | (ve & 3) << 2);
          }
        }
      }
      if (kEight && lane < kTokens) ring[place][S::kNumbers + kTokens * 8 + lane] = where;
#pragma unroll 1
      for (int v = 0; v < 2; ++v) {
        if (v == 1 && !acquire()) break;
        const uint32_t to = smem_addr(ring[place]);
        const uint8_t* const base = (v ? c.v : c.k) + unit * 16;
#pragma unroll
        for (int j = 0; j < kTokens / kAtOnce; ++j) {
          const int tok = j * kAtOnce + sub;
          const uint32_t f = __shfl_sync(0xFFFFFFFFu, from, tok);
          const bool on = f != kNowhere && in_head;
          cp_async16_or_zero(to + unit_at<S::kRowBytes, kEight>(tok, unit), base + (on ? static_cast<uint64_t>(f) * by : 0), on);
        }
        hand_on();
      }
      if (!ok) break;
      page0 = page1;
      page1 = page2;
      if (left > 1) {
        Plan::next_unit(p, at);
        fresh = at.tile == at.t0;
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // copies end before the thread does
  } else {
    // ------------------------------------------------------- scores and outputs
    if constexpr (S::kRegsRows > 0) registers_grow<S::kRegsRows>();
    const int g = lane >> 2, t = lane & 3;
    const uint32_t ring_at = smem_addr(&ring[0][0]);
    uint4* const operands = sm.q[pair];
    auto release = [&](int which) { warp_arrive(&empty[which]); };
    bool ok = true;
    while (ok && left > 0) {
      const int n_units = static_cast<int>(min(static_cast<int64_t>(at.t1 - at.tile), left));
      const bool started = at.tile == at.t0, ends = at.tile + n_units == at.t1;
      // q as left operands: of each 16 components a thread has four of rows g and g + 8.
      uint32_t qf[S::kShared ? 1 : D / 16][4];
      float qs[MT][2], o[MT][D / 8][4], top[MT][2], sum[MT][2];  // (top: M)
      int last[MT][2];  // one past the last position that a row sees
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (!(ok = ok && warp_wait(&full[place], phase, &sm.abort))) break;
        const uint32_t rows = ring_at + place * S::kPlace;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          last[m][i] = at.before + column_of(p, at.k * S::kRows + m * 16 + g + 8 * i) + 1;
          top[m][i] = -INFINITY;
          sum[m][i] = 0.f;
        }
        if constexpr (!kEight) {
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            uint32_t a[4];  // rows 0-7 and 8-15 of components 0-7, then of 8-15
            ldmatrix_x4(a, rows + unit_at<2 * D, false>(lane & 15, 2 * s + (lane >> 4)));
            if constexpr (S::kShared) {
              operands[(m * (D / 16) + s) * 32 + lane] = make_uint4(a[0], a[1], a[2], a[3]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) qf[s][j] = a[j];
            }
          }
        } else {
          // Components 16 (t + 4 (s / 4)) + 4 (s % 4) + 0..3 of each row, as fp16; the row's largest comes
          // to lie in 2^14 .. 2^15.  (Rows of tiny numbers are left smaller.)
          uint32_t f[2][D / 8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t most = 0;
#pragma unroll
            for (int u = 0; u < D / 32; ++u) {
              const uint4 v = load_shared16(rows + unit_at<2 * D, false>(g + 8 * i, 2 * (t + 4 * (u / 2)) + u % 2));
              f[i][4 * u] = v.x, f[i][4 * u + 1] = v.y, f[i][4 * u + 2] = v.z, f[i][4 * u + 3] = v.w;
            }
#pragma unroll
            for (int j = 0; j < D / 8; ++j) most = max(most, max(f[i][j] & 0x7FFFu, (f[i][j] >> 16) & 0x7FFFu));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            const int up = max(min(127 + 14 - static_cast<int>(most >> 7), 126), -126);
            const float by = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
            qs[m][i] = p.scale / by;
#pragma unroll
            for (int j = 0; j < D / 8; ++j) f[i][j] = to_halfx2(bf16_lo(f[i][j]) * by, bf16_hi(f[i][j]) * by);
          }
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            if constexpr (S::kShared) {
              operands[(m * (D / 16) + s) * 32 + lane] = make_uint4(f[0][2 * s], f[1][2 * s], f[0][2 * s + 1], f[1][2 * s + 1]);
            } else {
              qf[s][0] = f[0][2 * s], qf[s][1] = f[1][2 * s], qf[s][2] = f[0][2 * s + 1], qf[s][3] = f[1][2 * s + 1];
            }
          }
        }
        release(place);
        next_place();
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
      }
      if (!ok) break;
      const int seen_first = at.before + column_of(p, at.k * S::kRows);  // the block's first column's position
#pragma unroll 1
      for (int unit = 0; unit < n_units; ++unit, ++at.tile) {
        const int k_place = place;
        if (!(ok = warp_wait(&full[place], phase, &sm.abort))) break;
        next_place();
        const int v_place = place;
        if (!(ok = warp_wait(&full[place], phase, &sm.abort))) break;
        next_place();
        const int p0 = at.tile * kTokens;
        const uint32_t ks = ring_at + k_place * S::kPlace, vs = ring_at + v_place * S::kPlace;
        if constexpr (kEight) {
          // Each lane takes a token's exponents out of their words: 2^e of the key, e of the value.
          uint32_t* const f = reinterpret_cast<uint32_t*>(&ring[k_place][S::kNumbers]);
          const uint32_t where = ring[k_place][S::kNumbers + kTokens * 8 + lane];
          const uint32_t kb = where == 255u ? 127u : (f[lane] >> (where & 3) * 8) & 255u;
          const uint32_t vb = where == 255u ? 127u : (f[kTokens + lane] >> (where >> 2) * 8) & 255u;
          f[lane] = kb == 255u ? 0x7FC00000u : kb << 23;
          f[kTokens + lane] = vb == 255u ? 0x7FC00000u : __float_as_uint(static_cast<float>(static_cast<int>(vb) - 127));
          __syncwarp();
        }
        const bool whole = p0 + kTokens <= seen_first + 1 && (p.window == 0 || p0 > at.hi - 1 - p.window);
#pragma unroll 1
        for (int t0 = 0; t0 < kTokens; t0 += 16) {
          float x[MT][2][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[m][n][i] = 0.f;
          auto q_of = [&](int m, int s, uint32_t (&a)[4]) {
            if constexpr (S::kShared) {
              const uint4 v = operands[(m * (D / 16) + s) * 32 + lane];
              a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) a[j] = qf[s][j];
            }
          };
          if constexpr (!kEight) {
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              uint32_t b[4];
              ldmatrix_x4(b, ks + t0 * S::kRowBytes + unit_at<S::kRowBytes, false>((lane >> 4) * 8 + (lane & 7), 2 * s + ((lane >> 3) & 1)));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                uint32_t a[4];
                q_of(m, s, a);
                mma_16816<false>(x[m][0], a, b[0], b[1]);
                mma_16816<false>(x[m][1], a, b[2], b[3]);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              uint4 w[2];
#pragma unroll
              for (int n = 0; n < 2; ++n) w[n] = load_shared16(ks + t0 * S::kRowBytes + unit_at<S::kRowBytes, true>(n * 8 + g, t + 4 * i));
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t b[2][2];
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                  uint32_t v = (&w[n].x)[j];
                  if constexpr (TYPE == SPEC_CACHE_INT8) v ^= 0x80808080u;
                  b[n][0] = eight_to_half2<TYPE>(v, 0);
                  b[n][1] = eight_to_half2<TYPE>(v, 1);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                  uint32_t a[4];
                  q_of(m, 4 * i + j, a);
                  mma_16816<true>(x[m][0], a, b[0][0], b[0][1]);
                  mma_16816<true>(x[m][1], a, b[1][0], b[1][1]);
                }
              }
            }
          }
          // Scores in powers of two (8 bits: with the value's exponent), hidden ones -inf.
          const float* const exps = reinterpret_cast<const float*>(&ring[k_place][S::kNumbers]) + t0 + 2 * t;
          float2 ve[2];
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float2 kf;
            if constexpr (kEight) {
              kf = *reinterpret_cast<const float2*>(exps + n * 8);
              ve[n] = *reinterpret_cast<const float2*>(exps + kTokens + n * 8);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (kEight)
                  x[m][n][i] = fmaf(x[m][n][i] * ((i & 1) ? kf.y : kf.x), qs[m][i >> 1], (i & 1) ? ve[n].y : ve[n].x);
                else
                  x[m][n][i] *= p.scale;
              }
          }
          if (!whole) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int pos = p0 + t0 + n * 8 + 2 * t + (i & 1), lim = last[m][i >> 1];
                  const bool seen = pos < lim && pos >= at.lo && (p.window == 0 || pos >= lim - p.window);
                  x[m][n][i] = seen ? x[m][n][i] : -INFINITY;
                }
          }
          float raise[MT][2];
          bool any = false;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float most = fmaxf(fmaxf(x[m][0][2 * i], x[m][0][2 * i + 1]), fmaxf(x[m][1][2 * i], x[m][1][2 * i + 1]));
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
              raise[m][i] = most > top[m][i] + (kRowsSlack + kRowsBelow<kEight>) ? most - kRowsBelow<kEight> : top[m][i];
              any |= raise[m][i] != top[m][i];
            }
          if (__any_sync(0xFFFFFFFFu, any)) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float f = raise[m][i] == top[m][i] ? 1.f : ex2_approx(top[m][i] - raise[m][i]);
                sum[m][i] *= f;
#pragma unroll
                for (int n = 0; n < D / 8; ++n) {
                  o[m][n][2 * i] *= f;
                  o[m][n][2 * i + 1] *= f;
                }
                top[m][i] = raise[m][i];
              }
          }
          uint32_t w[MT][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float from = top[m][i] == -INFINITY ? 0.f : top[m][i];
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const float e0 = ex2_approx(x[m][n][2 * i] - from), e1 = ex2_approx(x[m][n][2 * i + 1] - from);
                if constexpr (kEight) {
                  sum[m][i] = fmaf(e0, power_of_minus(ve[n].x), fmaf(e1, power_of_minus(ve[n].y), sum[m][i]));
                  w[m][n * 2 + i] = to_halfx2(e0, e1);
                } else {
                  sum[m][i] += e0 + e1;
                  w[m][n * 2 + i] = to_bf16x2(e0, e1);
                }
              }
            }
          // Outputs' numerators: tokens are the products' inner dimension.
          if constexpr (!kEight) {
#pragma unroll
            for (int n = 0; n < D / 16; ++n) {
              uint32_t b[4];
              ldmatrix_x4_trans(b, vs + t0 * S::kRowBytes + unit_at<S::kRowBytes, false>(((lane >> 3) & 1) * 8 + (lane & 7), 2 * n + (lane >> 4)));
#pragma unroll
              for (int m = 0; m < MT; ++m) {
                mma_16816<false>(o[m][2 * n], w[m], b[0], b[1]);
                mma_16816<false>(o[m][2 * n + 1], w[m], b[2], b[3]);
              }
            }
          } else {
            constexpr int kBytes = D >= 128 ? 16 : 8;  // neighbouring components of a thread
#pragma unroll
            for (int i = 0; i < D / (8 * kBytes); ++i) {
              uint32_t y[4][kBytes / 4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {  // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
                const uint32_t r = 2 * t + (k & 1) + (k >> 1) * 8, d = (g + 8 * i) * kBytes;
                const uint32_t from = vs + t0 * S::kRowBytes + unit_at<S::kRowBytes, true>(r, d / 16) + d % 16;
                if constexpr (kBytes == 16) {
                  const uint4 v = load_shared16(from);
                  y[k][0] = v.x, y[k][1] = v.y, y[k][2] = v.z, y[k][3] = v.w;
                } else {
                  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(y[k][0]), "=r"(y[k][1]) : "r"(from) : "memory");
                }
                if constexpr (TYPE == SPEC_CACHE_INT8)
#pragma unroll
                  for (int j = 0; j < kBytes / 4; ++j) y[k][j] ^= 0x80808080u;
              }
#pragma unroll
              for (int j = 0; j < kBytes / 4; ++j)
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const uint32_t a = __byte_perm(y[0][j], y[1][j], z ? 0x7362 : 0x5140);
                  const uint32_t b = __byte_perm(y[2][j], y[3][j], z ? 0x7362 : 0x5140);
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    const uint32_t b0 = eight_to_half2<TYPE>(a, e), b1 = eight_to_half2<TYPE>(b, e);
#pragma unroll
                    for (int m = 0; m < MT; ++m) mma_16816<true>(o[m][i * kBytes + j * 4 + z * 2 + e], w[m], b0, b1);
                  }
                }
            }
          }
        }
        release(k_place);
        release(v_place);
      }
      if (!ok) break;
      // The item ends here, or goes on with the next worker.
      const int head = at.h * p.heads + head_in;
      float* const part = p.parts + (2 * (static_cast<int64_t>(blockIdx.x) * p.workers + worker) + (started ? 1 : 0)) *
                                        part_floats(S::kRows * p.heads, D);
      const bool direct = started && ends;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float s = sum[m][i];
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
          s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
          const int r = m * 16 + g + 8 * i, row = at.k * S::kRows + r, col = column_of(p, row);
          if (col >= at.count) continue;
          const int q_head = head * p.group + row - col * p.group;
          __nv_bfloat16* const out = p.out + (at.first + col) * p.out_row + q_head * p.out_head;
          float* const to = part + (head_in * S::kRows + r) * D;
          const float f = direct ? 1.f / s : 1.f;
          bool fine = true;
          constexpr int kBytes = D >= 128 ? 16 : 8;
          // (8 bits: four by four, components of the head that lie side by side)
#pragma unroll
          for (int n = 0; n < D / 8; n += kEight ? 4 : 1)
#pragma unroll
            for (int e = 0; e < (kEight ? 2 : 1); ++e) {
              const int d = kEight ? (2 * t + e + 8 * (n / kBytes)) * kBytes + n % kBytes : n * 8 + 2 * t;
              float4 a;
              if constexpr (kEight)
                a = make_float4(o[m][n][2 * i + e] * f, o[m][n + 1][2 * i + e] * f, o[m][n + 2][2 * i + e] * f, o[m][n + 3][2 * i + e] * f);
              else
                a = make_float4(o[m][n][2 * i] * f, o[m][n][2 * i + 1] * f, 0.f, 0.f);
              if (direct) {
                if (d < c.dim) {
                  if constexpr (kEight)
                    *reinterpret_cast<uint2*>(out + d) = make_uint2(to_bf16x2(a.x, a.y), to_bf16x2(a.z, a.w));
                  else
                    *reinterpret_cast<uint32_t*>(out + d) = to_bf16x2(a.x, a.y);
                  fine = fine && finite4(a);
                }
              } else if constexpr (kEight) {
                *reinterpret_cast<float4*>(to + d) = a;
              } else {
                *reinterpret_cast<float2*>(to + d) = make_float2(a.x, a.y);
              }
            }
          if (direct) {
            if (!fine) lane_fails_now(c, at.b, SPEC_ERR_NONFINITE);
            if (p.lse != nullptr && t == 0) p.lse[(at.first + col) * p.lse_row + q_head] = (top[m][i] + log2f(s)) * kLn2;
          } else if (t == 0) {
            *reinterpret_cast<float2*>(part + S::kRows * p.heads * D + 2 * (head_in * S::kRows + r)) = make_float2(top[m][i], s);
          }
        }
      left -= n_units;
      --at.tile;
      Plan::next_unit(p, at);
    }
  }
  __syncthreads();
  const int64_t worker0 = static_cast<int64_t>(blockIdx.x) * p.workers;
  if (sm.abort) {  // a wait gave up: all lanes of the block's units (and nothing to join)
    if (threadIdx.x < p.workers && c.status != nullptr) {
      Cursor x = sm.plan.from[threadIdx.x];
      for (int64_t u = sm.plan.begin[threadIdx.x]; u < sm.plan.end[threadIdx.x]; ++u, Plan::next_unit(p, x))
        lane_fails_now(c, x.b, SPEC_ERR_TIMEOUT);
    }
  } else if (p.parts != nullptr && p.workers > 1) {
    // Parts of one item that several of the block's workers hold become one part (or the output).
    const int64_t size = part_floats(S::kRows * p.heads, D);
    auto goes_on = [&](int w) {  // worker w begins inside an item
      return w < p.workers && sm.plan.begin[w] < sm.plan.end[w] && sm.plan.from[w].tile != sm.plan.from[w].t0;
    };
#pragma unroll 1
    for (int run = -1; run < p.workers; ++run) {
      // An item that goes on from before the block, then those that its workers begin: workers w0 to w1,
      // the first one's part in its first or later place.
      const int w0 = max(run, 0), later = run < 0 ? 0 : 1, parts = later ? sm.plan.record[w0].parts : 0;
      int w1 = w0;
      if (later) {
        w1 += min(parts, p.workers - w0) - 1;
      } else if (goes_on(0)) {
        while (sm.plan.record[w1].parts == 0 && goes_on(w1 + 1)) ++w1;
      }
      if (w1 <= w0) continue;
      const Cursor x = sm.plan.from[w1];
      float* const first = p.parts + (2 * (worker0 + w0) + later) * size;
      const float* const rest = p.parts + 2 * worker0 * size;
      const int used = min(S::kRows, x.count * p.group - x.k * S::kRows);
      const bool done = later && w1 - w0 + 1 == parts;
      auto part = [&](int i) { return i == 0 ? static_cast<const float*>(first) : rest + 2 * (w0 + i) * size; };
#pragma unroll 1
      for (int y = warp; y < used * p.heads; y += 2 * S::kWarps) {
        const int h = y / used, r = y - h * used, in = h * S::kRows + r;
        RowSum<D> sum;
        sum.template take<4>(0, w1 - w0 + 1, 1, [&](int i) { return part(i) + static_cast<int64_t>(in) * D; },
                 [&](int i) { return reinterpret_cast<const float2*>(part(i) + S::kRows * p.heads * D + 2 * in); });
        __syncwarp();  // (the first part's numbers have been read)
        if (done) {
          const int row = x.k * S::kRows + r, col = column_of(p, row);
          sum.template finish<kFreshShift>(p, x.b, x.first + col, (x.h * p.heads + h) * p.group + row - col * p.group);
        } else if (lane < RowSum<D>::kAcross) {
#pragma unroll
          for (int z = 0; z < RowSum<D>::kWide; ++z)
            reinterpret_cast<float4*>(first + static_cast<int64_t>(in) * D)[lane + z * 32] = sum.a[z];
          if (lane == 0)
            *reinterpret_cast<float2*>(first + S::kRows * p.heads * D + 2 * in) = make_float2(sum.top, sum.sum);
        }
      }
    }
  }
  if (p.parts != nullptr && threadIdx.x < p.workers) {
    // How many thread blocks hold parts.
    PartRecord record = sm.plan.record[threadIdx.x];
    if (record.parts > 0) record.parts = (static_cast<int>(threadIdx.x) + record.parts - 1) / p.workers + 1;
    p.records[worker0 + threadIdx.x] = record;
  }
}

// Joins the parts of items that were split over thread blocks.  blockIdx.x: the worker that an item
// begins with; blockIdx.y: some of its rows, of which there are `rows` for a head, at most `used` of
// them in use.  A warp takes a row; of many parts, and where a block has one row, all warps a share each.
constexpr int kJoinThreads = 128, kJoinAlone = 32;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const AttendParams p, int rows, int used, int per_block) {
  constexpr int kWarps = kJoinThreads / 32;
  using Sum = RowSum<D>;
  __shared__ float4 sums[kWarps][D / 4];
  __shared__ float2 stats[kWarps];
  griddep_wait();
  griddep_launch_dependents();
  if (blockIdx.x == 0 && blockIdx.y == 0) settle_errors(p.c);
  const PartRecord record = p.records[blockIdx.x];
  if (record.parts < 2) return;
  const int first = record.first, count = record.count;
  const int64_t size = part_floats(rows * p.heads, D);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Part 0: the first worker's later place; the others: the first place of the next thread blocks' first
  // worker.
  const float* const part0 = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + 1) * size;
  const float* const others = p.parts + 2 * static_cast<int64_t>(blockIdx.x / p.workers) * p.workers * size;
  auto part = [&](int i) { return i == 0 ? part0 : others + 2 * static_cast<int64_t>(i) * p.workers * size; };
  const int y1 = min(static_cast<int>(blockIdx.y + 1) * per_block, used * p.heads);
  const bool alone = record.parts <= kJoinAlone || per_block > 1;
#pragma unroll 1
  for (int y = blockIdx.y * per_block + (alone ? warp : 0); y < y1; y += alone ? kWarps : 1) {
    const int h = y / used, r = y - h * used, row = record.block * rows + r, col = column_of(p, row), in = h * rows + r;
    if (col >= count) continue;  // (the same for all threads that go on together)
    const int head = (record.head * p.heads + h) * p.group + row - col * p.group;
    Sum sum;
    sum.template take<D <= 128 ? 16 : 8>(alone ? 0 : warp, record.parts, alone ? 1 : kWarps, [&](int i) { return part(i) + static_cast<int64_t>(in) * D; },
             [&](int i) { return reinterpret_cast<const float2*>(part(i) + rows * p.heads * D + 2 * in); });
    if (!alone) {
      if (lane < Sum::kAcross)
#pragma unroll
        for (int z = 0; z < Sum::kWide; ++z) sums[warp][lane + z * 32] = sum.a[z];
      if (lane == 0) stats[warp] = make_float2(sum.top, sum.sum);
      __syncthreads();
      if (warp == 0) {
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) top = fmaxf(top, stats[w].x);
        Sum all{};
        all.top = top;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          const float f = stats[w].x == -INFINITY ? 0.f : ex2_approx(stats[w].x - top);
          all.sum = fmaf(stats[w].y, f, all.sum);
          if (lane < Sum::kAcross)
#pragma unroll
            for (int z = 0; z < Sum::kWide; ++z) {
              const float4 b = sums[w][lane + z * 32];
              all.a[z].x = fmaf(b.x, f, all.a[z].x), all.a[z].y = fmaf(b.y, f, all.a[z].y);
              all.a[z].z = fmaf(b.z, f, all.a[z].z), all.a[z].w = fmaf(b.w, f, all.a[z].w);
            }
        }
        all.template finish<0>(p, record.lane, first + col, head);
      }
      __syncthreads();  // (sums and stats have been read)
    } else {
      sum.template finish<0>(p, record.lane, first + col, head);
    }
  }
}

}  // namespace specv
