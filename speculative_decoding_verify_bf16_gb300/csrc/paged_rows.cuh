// paged_rows.cuh -- attention of a few rows (decoding, a verify round) over a paged cache.
//
// o = sum_j w_j v_j / sum_j w_j,  w_j = 2^(x_j - M),  x_j = scale * log2(e) * q . k_j, with the running maximum M
// of a row: one pass over keys and values.
//
// What bounds it is reading the cache: 2 * dim numbers a token and head, for the rows of all query
// heads and columns of that head together.  Every computing warp has tokens of its own, which come
// through a ring of its own in shared memory, and keeps maxima, sums and the outputs' numerators of
// all rows in registers: warps wait for nobody until an item ends, when their sums are joined
// in the ring's last place.  Four warps do nothing but look up where tokens lie, one by one (any page
// size and order will do), and copy them, 16 bytes a thread.  (Bulk copies of whole heads, 128 or 256 bytes
// each, are fewer instructions, but one took some 19 cycles of an SM: 142 us for 131,000 tokens
// where these took 109 from within the computing warps.)  Products are 16 x 8 x 16 ones of a warp: 16 rows are
// a fraction of a 128-row tile of the large tensor cores, and what they save is not short.
//
// 8-bit caches: numbers become fp16 in registers, exactly, and products are fp16.  q is
// taken times a power of two for each row into fp16's range (exactly, but for what is below
// 2^-38 of the row's largest).  The key's power of two multiplies its scores; the value's, 2^e,
// goes into the weight's exponent, w = 2^(x + e - M), and out of the sum of weights again.  (Exponents lie
// within -48..48, so a weight that vanishes beside the largest is below 2^-30 of it in the
// sum.)  The components' order is free in both products: a thread takes sixteen neighbouring
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

constexpr float kRowsSlack = 8.f;           // a maximum is raised when it is exceeded by more: weights stay below 2^8

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

constexpr int kCopyWarps = 4;
constexpr int kUnseen = INT32_MIN;  // in a page's place: no row sees the token

template <int TYPE_, int D_, int MT_>
struct RowsShape {
  static constexpr int TYPE = TYPE_, D = D_, MT = MT_;  // cache type, head size (at most), blocks of 16 rows
  static constexpr bool kEight = TYPE != SPEC_CACHE_BF16;
  static constexpr int kRows = 16 * MT;
  static constexpr int kWarps = D > 128 ? 4 : 8;  // that compute
  static constexpr int kThreads = 32 * (kWarps + kCopyWarps);
  // Registers a thread, and what a launch must bring (0: they are not shared out).
  static constexpr int kRegsRows = kWarps == 8 ? 208 : 0, kRegsCopy = kWarps == 8 ? 88 : 0;
  static constexpr int kRegs = kWarps / 4 * kRegsRows + kRegsCopy;
  static constexpr int kRowBytes = D * (kEight ? 1 : 2);
  static constexpr int kPitch = kRowBytes + 16;  // rows on other banks each
  static constexpr int kTokens = (kEight ? MT > 1 : kRowBytes >= 256) ? 16 : 32;  // tokens of a warp's step
  static constexpr int kSub = MT == 1 ? kTokens : 16;                             // of them, scores held at a time
  static constexpr int kTile = kTokens * kWarps;
  // A place: keys, values and, with 8 bits, each token's exponents (words that hold them, and where).
  static constexpr int kExps = 2 * kTokens * kPitch;
  static constexpr int kStage = kExps + (kEight ? kTokens * 9 : 0);
  // With 32 rows q is read from shared memory for each product (registers are short).
  static constexpr int kFragments = MT > 1 ? MT * (D / 16) * 32 : 0;
  static constexpr int kRing = (MT == 1 ? 223 : D > 64 ? 214 : 218) * 1024;  // shared memory of all rings
  static constexpr int kFit = kRing / kWarps / kStage;
  static constexpr int kStages = kFit > 8 ? 8 : kFit;
  static constexpr int kOutCols = 16 * (D + 4) * 4 <= kStage ? D : D / 2;  // columns of sums joined at a time
  static constexpr int kOutPitch = kOutCols + 4;
  static constexpr int kExtra = 1;  // an item's beginning and end, in units
  static_assert(kStages >= 3, "the ring has three places at least");
  static_assert(16 * kOutPitch * 4 <= kStage, "16 rows of sums fit a place of the ring");
  using Plan = Schedule<kRows, kTile, kExtra>;
};

template <typename S>
struct RowsSmem {
  uint8_t ring[S::kWarps][S::kStages][S::kStage];
  uint4 q[S::kFragments + 1];
  float top[S::kWarps][S::kRows], sum[S::kWarps][S::kRows];
  typename S::Plan::Shared plan;
  uint64_t full[S::kWarps][S::kStages], empty[S::kWarps][S::kStages];
  int abort;
};

constexpr float kLn2 = 0.693147180559945f;

template <typename S>
__global__ void __launch_bounds__(S::kThreads, 1) paged_rows_kernel(const AttendParams p, const int test_withhold) {
  using Plan = typename S::Plan;
  constexpr int TYPE = S::TYPE, D = S::D, MT = S::MT, kTokens = S::kTokens, kSub = S::kSub, kStages = S::kStages;
  constexpr bool kEight = S::kEight;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  RowsSmem<S>& sm = *reinterpret_cast<RowsSmem<S>*>(smem_raw);
  const CacheParams& c = p.c;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  if (threadIdx.x < S::kWarps * kStages) {
    // (a full place: each copying thread's copies and, with 8 bits, its warp's exponents)
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
      if (!cache_lane(c, b, first, count, before)) lane_failed(c, b, SPEC_ERR_LAYOUT);
    }
  const int64_t begin = sm.plan.begin, end = sm.plan.end;

  if (warp >= S::kWarps) {
    // ------------------------------------------------------------------ copies
    if constexpr (S::kRegsCopy > 0) registers_shrink<S::kRegsCopy>();
    constexpr int kUnits = S::kRowBytes / 16, kAtOnce = 32 / kUnits;  // 16-byte units of a token; tokens of an access
    constexpr int kMine = S::kWarps / kCopyWarps;                     // computing warps of this one
    const int unit = lane % kUnits, sub = lane / kUnits, first_warp = warp - S::kWarps;
    const bool in_head = unit * 16 < c.dim * (kEight ? 1 : 2);
    const uint32_t by = 1u << c.unit_shift;
    const uint8_t* const k_base = c.k + unit * 16;
    const uint8_t* const v_base = c.v + unit * 16;
    Cursor ld = sm.plan.from;
    int64_t left = begin < end ? end - begin : 0;
    // Pages are looked up two units ahead: with the memory busy, a load takes as long as that.
    Cursor ahead = ld;
    int64_t left_ahead = left;
    int id[3][kMine];  // of the unit and the next two: the page of this lane's token, kUnseen: none
    auto look_up = [&](int (&to)[kMine]) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int pos = ahead.tile * S::kTile + (first_warp + i * kCopyWarps) * kTokens + lane;
        if (left_ahead > 0 && lane < kTokens && pos >= ahead.lo && pos < ahead.hi)
          to[i] = __ldg(c.tables + ahead.b * c.table_stride + page_of(c, pos));
        else
          to[i] = kUnseen;
      }
      if (--left_ahead > 0) Plan::next_unit(p, ahead);
    };
    int stage[kMine] = {}, round[kMine] = {};  // of each warp's ring
    bool ok = true;
    look_up(id[0]);
    look_up(id[1]);
#pragma unroll 1
    for (; ok && left > 0; --left) {
      look_up(id[2]);
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int w = first_warp + i * kCopyWarps, p0 = ld.tile * S::kTile + w * kTokens;
        const bool seen_some = p0 < ld.hi && p0 + kTokens > ld.lo;  // (if not, a place goes by empty)
        if (!ok || (round[i] > 0 && !(ok = warp_wait(&sm.empty[w][stage[i]], (round[i] - 1) & 1, &sm.abort)))) continue;
        uint8_t* const place = sm.ring[w][stage[i]];
        const int page = id[0][i];
        uint32_t at = kNowhere;
        uint8_t where = 255;  // of the exponents in their words: two bits each
        if (page != kUnseen && static_cast<uint32_t>(page) >= static_cast<uint32_t>(c.pages)) {
          lane_failed(c, ld.b, SPEC_ERR_LAYOUT);
        } else if (page != kUnseen) {
          const int pos = p0 + lane, in = pos - page_of(c, pos) * c.page_size;
          at = head_at(c, page, in, ld.h);
          if constexpr (kEight) {
            const int64_t e = page * c.exp_page + in * c.exp_slot + ld.h * c.exp_head;
            const uintptr_t ke = reinterpret_cast<uintptr_t>(c.k_exps + e), ve = reinterpret_cast<uintptr_t>(c.v_exps + e);
            cp_async4(place + S::kExps + lane * 4, reinterpret_cast<const void*>(ke & ~uintptr_t{3}));
            cp_async4(place + S::kExps + (kTokens + lane) * 4, reinterpret_cast<const void*>(ve & ~uintptr_t{3}));
            where = static_cast<uint8_t>((ke & 3) | (ve & 3) << 2);
          }
        }
        if (kEight && lane < kTokens) place[S::kExps + kTokens * 8 + lane] = where;
        const uint32_t to = smem_addr(place + sub * S::kPitch + unit * 16);
#pragma unroll
        for (int j = 0; j < kTokens / kAtOnce && seen_some; ++j) {
          const uint32_t from = __shfl_sync(0xFFFFFFFFu, at, j * kAtOnce + sub);
          const bool on = from != kNowhere && in_head;
          const uint64_t off = on ? static_cast<uint64_t>(from) * by : 0;
          if (!(test_withhold != 0 && begin == 0 && w == 0 && j == 0)) {
            cp_async16_or_zero(to + j * kAtOnce * S::kPitch, k_base + off, on);
            cp_async16_or_zero(to + (kTokens + j * kAtOnce) * S::kPitch, v_base + off, on);
          }
        }
        if (!(test_withhold != 0 && begin == 0 && w == 0)) cp_async_arrive(&sm.full[w][stage[i]]);
        if constexpr (kEight) warp_arrive(&sm.full[w][stage[i]]);
        if (++stage[i] == kStages) {
          stage[i] = 0;
          ++round[i];
        }
        id[0][i] = id[1][i];
        id[1][i] = id[2][i];
      }
      if (left > 1) Plan::next_unit(p, ld);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");  // copies end before the thread does
  } else if (begin < end) {
    // ------------------------------------------------------- scores and outputs
    if constexpr (S::kRegsRows > 0) registers_grow<S::kRegsRows>();
    Cursor at = sm.plan.from;
    bool dead = false;  // a wait gave up: the warp only goes along to the barriers
    uint8_t(&ring)[kStages][S::kStage] = sm.ring[warp];
    const uint32_t ring_at = smem_addr(&ring[0][0]);
    auto all_rows = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * S::kWarps) : "memory"); };
    uint32_t qf[MT == 1 ? D / 16 : 1][4];
    float o[MT][D / 8][4];
    float top[MT][2], sum[MT][2], qs[MT][2];
    int last[MT][2];  // one past the last position that a row sees
    bool fresh = true, started = false;
    int stage = 0, phase = 0;  // of the ring
#pragma unroll 1
    for (int64_t u = begin; u < end; ++u) {
      const int p0 = at.tile * S::kTile + warp * kTokens;
      const bool seen_some = p0 < at.hi && p0 + kTokens > at.lo;
      if (fresh) {
        // q as left operands: of each 16 components a thread has four of rows g and g + 8.
        fresh = false;
        started = at.tile == at.t0;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          uint32_t f[D / 16][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int r = at.k * S::kRows + m * 16 + g + 8 * i, col = r / p.group;
            last[m][i] = at.before + col + 1;
            top[m][i] = -INFINITY;
            sum[m][i] = 0.f;
            const bool on = col < at.count;
            const __nv_bfloat16* const from =
                p.q + (on ? (at.first + col) * p.q_row + (at.h * p.group + r - col * p.group) * p.q_head : 0);
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              // (8 bits: components 16 (t + 4 (s / 4)) + 4 (s % 4) + 0..3)
              const int d = kEight ? 16 * (t + 4 * (s / 4)) + 4 * (s % 4) : 16 * s + 2 * t;
              const int d2 = kEight ? d + 2 : d + 8;
              f[s][i] = on && d < c.dim ? __ldg(reinterpret_cast<const uint32_t*>(from + d)) : 0u;
              f[s][i + 2] = on && d2 < c.dim ? __ldg(reinterpret_cast<const uint32_t*>(from + d2)) : 0u;
            }
          }
          if constexpr (kEight) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t most = 0;
#pragma unroll
              for (int s = 0; s < D / 16; ++s) {
                most = max(most, max(f[s][i] & 0x7FFFu, (f[s][i] >> 16) & 0x7FFFu));
                most = max(most, max(f[s][i + 2] & 0x7FFFu, (f[s][i + 2] >> 16) & 0x7FFFu));
              }
              most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
              most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
              // The largest comes to lie in 2^14 .. 2^15.  (Rows of tiny numbers are left smaller.)
              const int up = min(127 + 14 - static_cast<int>(most >> 7), 126);
              const float by = __uint_as_float(static_cast<uint32_t>(127 + max(up, -126)) << 23);
              qs[m][i] = p.scale / by;
#pragma unroll
              for (int s = 0; s < D / 16; ++s)
#pragma unroll
                for (int j = i; j < 4; j += 2) f[s][j] = to_halfx2(bf16_lo(f[s][j]) * by, bf16_hi(f[s][j]) * by);
            }
          }
#pragma unroll
          for (int s = 0; s < D / 16; ++s) {
            if constexpr (MT == 1) {
#pragma unroll
              for (int j = 0; j < 4; ++j) qf[s][j] = f[s][j];
            } else if (s % S::kWarps == warp) {  // (all warps have the same)
              sm.q[(m * (D / 16) + s) * 32 + lane] = make_uint4(f[s][0], f[s][1], f[s][2], f[s][3]);
            }
          }
#pragma unroll
          for (int n = 0; n < D / 8; ++n)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[m][n][i] = 0.f;
        }
        if constexpr (MT > 1) all_rows();
      }
      if (!dead) dead = !warp_wait(&sm.full[warp][stage], phase, &sm.abort);
      const uint32_t ks = ring_at + stage * S::kStage, vs = ks + kTokens * S::kPitch;
      if constexpr (kEight) {
        // Each lane takes a token's exponents out of their words: 2^e of the key, e of the value.
        if (lane < kTokens && seen_some && !dead) {
          uint32_t* const f = reinterpret_cast<uint32_t*>(&ring[stage][S::kExps]);
          const uint32_t where = ring[stage][S::kExps + kTokens * 8 + lane];
          const uint32_t kb = where == 255u ? 127u : (f[lane] >> (where & 3) * 8) & 255u;
          const uint32_t vb = where == 255u ? 127u : (f[kTokens + lane] >> (where >> 2) * 8) & 255u;
          f[lane] = kb == 255u ? 0x7FC00000u : kb << 23;
          f[kTokens + lane] = vb == 255u ? 0x7FC00000u : __float_as_uint(static_cast<float>(static_cast<int>(vb) - 127));
        }
        __syncwarp();
      }
      if (seen_some && !dead) {
        const int seen_first = at.before + at.k * S::kRows / p.group;  // the block's first column's position
        const bool whole = p0 + kTokens <= seen_first + 1 && (p.window == 0 || p0 > at.hi - 1 - p.window);
#pragma unroll
        for (int half = 0; half < kTokens / kSub; ++half) {
          float x[MT][kSub / 8][4];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int n = 0; n < kSub / 8; ++n)
#pragma unroll
              for (int i = 0; i < 4; ++i) x[m][n][i] = 0.f;
          auto q_of = [&](int m, int s, uint32_t (&a)[4]) {
            if constexpr (MT == 1) {
#pragma unroll
              for (int j = 0; j < 4; ++j) a[j] = qf[s][j];
            } else {
              const uint4 v = sm.q[(m * (D / 16) + s) * 32 + lane];
              a[0] = v.x, a[1] = v.y, a[2] = v.z, a[3] = v.w;
            }
          };
          if constexpr (!kEight) {
            const uint32_t base = ks + (half * kSub + (lane >> 4) * 8 + (lane & 7)) * S::kPitch + ((lane >> 3) & 1) * 16;
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
              uint32_t a[MT][4];
#pragma unroll
              for (int m = 0; m < MT; ++m) q_of(m, s, a[m]);
#pragma unroll
              for (int n = 0; n < kSub / 16; ++n) {
                uint32_t b[4];
                ldmatrix_x4(b, base + n * 16 * S::kPitch + s * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                  mma_16816<false>(x[m][2 * n], a[m], b[0], b[1]);
                  mma_16816<false>(x[m][2 * n + 1], a[m], b[2], b[3]);
                }
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
              uint4 w[kSub / 8];
#pragma unroll
              for (int n = 0; n < kSub / 8; ++n) {
                asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(w[n].x), "=r"(w[n].y), "=r"(w[n].z), "=r"(w[n].w)
                             : "r"(ks + (half * kSub + n * 8 + g) * S::kPitch + (t + 4 * i) * 16)
                             : "memory");
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t a[MT][4];
#pragma unroll
                for (int m = 0; m < MT; ++m) q_of(m, 4 * i + j, a[m]);
#pragma unroll
                for (int n = 0; n < kSub / 8; ++n) {
                  uint32_t v = (&w[n].x)[j];
                  if constexpr (TYPE == SPEC_CACHE_INT8) v ^= 0x80808080u;
                  const uint32_t b0 = eight_to_half2<TYPE>(v, 0), b1 = eight_to_half2<TYPE>(v, 1);
#pragma unroll
                  for (int m = 0; m < MT; ++m) mma_16816<true>(x[m][n], a[m], b0, b1);
                }
              }
            }
          }
          // Scores in powers of two (8 bits: with the value's exponent), hidden ones -inf.
          const float* const exps = reinterpret_cast<const float*>(&ring[stage][S::kExps]) + half * kSub + 2 * t;
#pragma unroll
          for (int n = 0; n < kSub / 8; ++n) {
            float2 kf, ve;
            if constexpr (kEight) {
              kf = *reinterpret_cast<const float2*>(exps + n * 8);
              ve = *reinterpret_cast<const float2*>(exps + kTokens + n * 8);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if constexpr (kEight)
                  x[m][n][i] = fmaf(x[m][n][i] * ((i & 1) ? kf.y : kf.x), qs[m][i >> 1], (i & 1) ? ve.y : ve.x);
                else
                  x[m][n][i] *= p.scale;
                if (!whole) {
                  const int pos = p0 + half * kSub + n * 8 + 2 * t + (i & 1), lim = last[m][i >> 1];
                  const bool seen = pos < lim && pos >= at.lo && (p.window == 0 || pos >= lim - p.window);
                  x[m][n][i] = seen ? x[m][n][i] : -INFINITY;
                }
              }
          }
          float raise[MT][2];
          bool any = false;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float most = -INFINITY;
#pragma unroll
              for (int n = 0; n < kSub / 8; ++n) most = fmaxf(most, fmaxf(x[m][n][2 * i], x[m][n][2 * i + 1]));
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
              raise[m][i] = most > top[m][i] + kRowsSlack ? most : top[m][i];
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
          uint32_t w[MT][kSub / 16][4];
#pragma unroll
          for (int n = 0; n < kSub / 8; ++n) {
            float2 vi;  // 2^-e
            if constexpr (kEight) {
              const float2 ve = *reinterpret_cast<const float2*>(exps + kTokens + n * 8);
              vi = make_float2(power_of_minus(ve.x), power_of_minus(ve.y));
            }
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float from = top[m][i] == -INFINITY ? 0.f : top[m][i];
                const float e0 = ex2_approx(x[m][n][2 * i] - from), e1 = ex2_approx(x[m][n][2 * i + 1] - from);
                if constexpr (kEight) {
                  sum[m][i] = fmaf(e0, vi.x, fmaf(e1, vi.y, sum[m][i]));
                  w[m][n / 2][(n & 1) * 2 + i] = to_halfx2(e0, e1);
                } else {
                  sum[m][i] += e0 + e1;
                  w[m][n / 2][(n & 1) * 2 + i] = to_bf16x2(e0, e1);
                }
              }
          }
          // Outputs' numerators: tokens are the products' inner dimension.
#pragma unroll
          for (int k16 = 0; k16 < kSub / 16; ++k16) {
            const int tok = half * kSub + k16 * 16;
            if constexpr (!kEight) {
              const uint32_t base = vs + (tok + ((lane >> 3) & 1) * 8 + (lane & 7)) * S::kPitch + (lane >> 4) * 16;
#pragma unroll
              for (int n = 0; n < D / 16; ++n) {
                uint32_t b[4];
                ldmatrix_x4_trans(b, base + n * 32);
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                  mma_16816<false>(o[m][2 * n], w[m][k16], b[0], b[1]);
                  mma_16816<false>(o[m][2 * n + 1], w[m][k16], b[2], b[3]);
                }
              }
            } else {
              constexpr int kBytes = D >= 128 ? 16 : 8;  // neighbouring components of a thread
#pragma unroll
              for (int i = 0; i < D / (8 * kBytes); ++i) {
                uint32_t y[4][kBytes / 4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {  // tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9
                  const uint32_t from = vs + (tok + 2 * t + (k & 1) + (k >> 1) * 8) * S::kPitch + (g + 8 * i) * kBytes;
                  if constexpr (kBytes == 16)
                    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(y[k][0]), "=r"(y[k][1]), "=r"(y[k][2]), "=r"(y[k][3])
                                 : "r"(from)
                                 : "memory");
                  else
                    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(y[k][0]), "=r"(y[k][1]) : "r"(from) : "memory");
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
                      for (int m = 0; m < MT; ++m)
                        mma_16816<true>(o[m][i * kBytes + j * 4 + z * 2 + e], w[m][k16], b0, b1);
                    }
                  }
              }
            }
          }
        }
      }
      if (at.tile + 1 == at.t1 || u + 1 == end) {
        // The item ends here, or goes on in the next thread block: the warps' sums are joined, 16
        // rows at a time, in the places of the ring that the warps have just read.
        const bool ends = at.tile + 1 == at.t1;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float s = sum[m][i];
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 1);
            s += __shfl_xor_sync(0xFFFFFFFFu, s, 2);
            if (t == 0) {
              sm.top[warp][m * 16 + g + 8 * i] = top[m][i];
              sm.sum[warp][m * 16 + g + 8 * i] = s;
            }
          }
        all_rows();
        float* const part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (started ? 1 : 0)) * part_floats(S::kRows, D);
        constexpr int kCols = S::kOutCols;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          float factor[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float most = -INFINITY;
#pragma unroll
            for (int w = 0; w < S::kWarps; ++w) most = fmaxf(most, sm.top[w][m * 16 + g + 8 * i]);
            factor[i] = top[m][i] == -INFINITY ? 0.f : ex2_approx(top[m][i] - most);
          }
#pragma unroll
          for (int d0 = 0; d0 < D; d0 += kCols) {
            // (8 bits: a thread's numbers of n = 0, 8, .. go to components all over the head: those of
            // a half are the ones whose place in it is even or odd, n % 8 below 4 or not)
            float* const mine = reinterpret_cast<float*>(&ring[stage][0]);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float* const to = mine + (g + 8 * i) * S::kOutPitch;
              const float f = factor[i];
              if constexpr (!kEight) {
#pragma unroll
                for (int n = d0 / 8; n < (d0 + kCols) / 8; ++n)
                  *reinterpret_cast<float2*>(to + n * 8 - d0 + 2 * t) = make_float2(o[m][n][2 * i] * f, o[m][n][2 * i + 1] * f);
              } else {
                constexpr int kBytes = D >= 128 ? 16 : 8;
#pragma unroll
                for (int n = 0; n < D / 8; n += 4)
#pragma unroll
                  for (int e = 0; e < 2; ++e) {
                    // Components 4 y .. 4 y + 3 of the head; a half takes every other four.
                    const int y = (2 * t + e + 8 * (n / kBytes)) * (kBytes / 4) + n % kBytes / 4;
                    if (kCols == D || (n / 4) % 2 == d0 / kCols)
                      *reinterpret_cast<float4*>(to + (kCols == D ? y : y / 2) * 4) =
                          make_float4(o[m][n][2 * i + e] * f, o[m][n + 1][2 * i + e] * f, o[m][n + 2][2 * i + e] * f,
                                      o[m][n + 3][2 * i + e] * f);
                  }
              }
            }
            all_rows();
#pragma unroll 1
            for (int x = threadIdx.x; x < 16 * (kCols / 4); x += 32 * S::kWarps) {
              const int r = x / (kCols / 4), y = x % (kCols / 4);
              const int d = kCols == D ? y * 4 : kEight ? (2 * y + d0 / kCols) * 4 : d0 + y * 4;
              float most = -INFINITY, total = 0.f;
#pragma unroll
              for (int w = 0; w < S::kWarps; ++w) most = fmaxf(most, sm.top[w][m * 16 + r]);
              float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int w = 0; w < S::kWarps; ++w) {
                const float mw = sm.top[w][m * 16 + r];
                total += mw == -INFINITY ? 0.f : sm.sum[w][m * 16 + r] * ex2_approx(mw - most);
                const float4 b = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(&sm.ring[w][stage][0]) +
                                                                  r * S::kOutPitch + y * 4);
                a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
              }
              if (started && ends) {
                const int row = at.k * S::kRows + m * 16 + r, col = row / p.group, head = at.h * p.group + row - col * p.group;
                if (col < at.count && d < c.dim) {
                  const float inv = 1.f / total;
                  a.x *= inv, a.y *= inv, a.z *= inv, a.w *= inv;
                  *reinterpret_cast<uint2*>(p.out + (at.first + col) * p.out_row + head * p.out_head + d) =
                      make_uint2(to_bf16x2(a.x, a.y), to_bf16x2(a.z, a.w));
                  if (!finite4(a)) lane_failed(c, at.b, SPEC_ERR_NONFINITE);
                  if (p.lse != nullptr && d == 0)
                    p.lse[(at.first + col) * p.lse_row + head] = (most + log2f(total)) * kLn2;
                }
              } else {
                *reinterpret_cast<float4*>(part + (m * 16 + r) * D + d) = a;
                if (d == 0) {
                  part[S::kRows * D + 2 * (m * 16 + r)] = most;
                  part[S::kRows * D + 2 * (m * 16 + r) + 1] = total;
                }
              }
            }
            all_rows();
          }
        }
        fresh = true;
      }
      Plan::next_unit(p, at);
      warp_arrive(&sm.empty[warp][stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    if (p.parts != nullptr) p.records[blockIdx.x] = sm.plan.record;
    if (sm.abort && c.status != nullptr) {  // a wait gave up: all lanes of the block's range
      Cursor x = sm.plan.from;
      for (int64_t u = begin; u < end; ++u, Plan::next_unit(p, x)) c.status[x.b] = SPEC_ERR_TIMEOUT;
    }
  }
}

// Joins the parts of items that were split.  blockIdx.x: the thread block that an item begins in;
// blockIdx.y: a slice of its rows.
constexpr int kJoinThreads = 128;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const AttendParams p, int rows, int slice) {
  griddep_wait();
  griddep_launch_dependents();
  const PartRecord record = p.records[blockIdx.x];
  if (record.parts < 2) return;
  const CacheParams& c = p.c;
  int first, count, before;
  if (!cache_lane(c, record.lane, first, count, before)) return;
  const int64_t size = part_floats(rows, D);
  // Part i: the first block's later place, the others' first place.
  const float* const base = p.parts + 2 * static_cast<int64_t>(blockIdx.x) * size;
  auto part = [&](int i) { return base + (i == 0 ? size : 2 * i * size); };
  for (int x = threadIdx.x; x < slice * (D / 4); x += kJoinThreads) {
    const int r = blockIdx.y * slice + x / (D / 4), d = x % (D / 4) * 4;
    const int row = record.block * rows + r, col = row / p.group;
    if (r >= rows || col >= count || d >= c.dim) continue;
    const int head = record.head * p.group + row - col * p.group;
    float most = -INFINITY;
#pragma unroll 4
    for (int i = 0; i < record.parts; ++i) most = fmaxf(most, __ldcg(part(i) + rows * D + 2 * r));
    float total = 0.f;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int i = 0; i < record.parts; ++i) {
      const float2 ms = __ldcg(reinterpret_cast<const float2*>(part(i) + rows * D + 2 * r));
      const float4 b = __ldcg(reinterpret_cast<const float4*>(part(i) + r * D + d));
      const float f = ms.x == -INFINITY ? 0.f : ex2_approx(ms.x - most);
      total = fmaf(ms.y, f, total);
      a.x = fmaf(b.x, f, a.x), a.y = fmaf(b.y, f, a.y), a.z = fmaf(b.z, f, a.z), a.w = fmaf(b.w, f, a.w);
    }
    const float inv = 1.f / total;
    a.x *= inv, a.y *= inv, a.z *= inv, a.w *= inv;
    *reinterpret_cast<uint2*>(p.out + (first + col) * p.out_row + head * p.out_head + d) =
        make_uint2(to_bf16x2(a.x, a.y), to_bf16x2(a.z, a.w));
    if (!finite4(a)) lane_failed(c, record.lane, SPEC_ERR_NONFINITE);
    if (p.lse != nullptr && d == 0) p.lse[(first + col) * p.lse_row + head] = (most + log2f(total)) * kLn2;
  }
}

}  // namespace specv
