// paged_tile.cuh -- attention of many rows (prompts, wide verify rounds) over a paged cache, on the
// tensor cores: heads up to 128, two tiles of 128 rows a thread block, 128 positions a step.
//
//   S = q k^T (fp32, tensor memory)     P = 2^(scale log2(e) S - M), hidden ones 0     O += P v
//
// P is rounded to bf16 (8-bit caches: fp16) as the few rows' kernel's weights are, and M is taken as there.
// It is raised, and O in tensor memory rescaled, only where a score (in powers of two) exceeds the row's running
// maximum by more than 8; sums of weights are fp32, in the thread that has the row.
//
// Products of a step and tile take 2 x 512 cycles on the tensor cores (heads of 128), the two tiles'
// take turns: while one's run, the other's scores become weights.  Per step and tile a warp does 32 x 128
// exponentials and some three further operations a number.
//
// Tensor memory: scores of both tiles (2 x 128 columns; the weights overwrite their first half),
// O of both (2 x 128).  Shared memory: q of both tiles, and a ring of tiles of keys and values, in rows
// with the 128-byte swizzle, so that a tile serves along either dimension.
//
// Warps: 0-3 and 4-7 a tile's rows, a thread each (q into shared memory, weights, rescaling,
// outputs); 8-11 bring keys and 12-15 values, 32 positions of a step each, looked up one by one, so
// that any page size and order will do; 16 issues the products.  Scores are read from tensor memory half
// a row at a time, the second half twice, for its maximum and for its weights: that leaves registers
// for eight copying warps, which 8-bit caches need (four took 5,800 cycles a step).
//
// Measured (device time): 2,048 tokens behind 30,000, 32 heads of 128 for 8 of a bf16 cache, 730 to 745 us, 1.4
// PFLOP/s, 0.75 of a library product's rate (801 to 812, 0.69, in a row of calls that the power limit slows), in
// e4m3 890; 12 prompts of 0 to 1,500 tokens behind 0 to 3,000, 16 heads for 2 in e4m3, 255 us (in bf16
// 218): short items, whose beginnings and ends do not overlap as their steps do.  A step of two tiles
// takes 2,900 cycles (8-bit caches: 4,000) where the products take 2,048: waits between scores, weights and the
// second product, and 57 % of the issue slots in use.  Whole rows of scores in registers, and four copying
// warps, took 718 us in bf16, but 1,341 in e4m3 (868 then) and 304 for the 12 prompts (244).
//
// 8-bit caches become fp16 on the way to shared memory, times 2^(e - r) with r the largest of a warp's 32
// exponents, and q becomes fp16 times a power of two for each row.  2^r multiplies the keys' scores; the
// values' r goes into the weights' exponents and out of their sum.  All of it is exact: keys' exponents may be
// 15 below r (e4m3's least number is then fp16's, 2^-24), and values' 7, so that M, which r enters, takes no
// more than that off the small weights.  A group of 32 positions with larger differences is taken apart: its
// numbers come as they are, and each score gets its own position's exponents, as in the few rows' kernel.  (With
// every group taken apart 2,048 tokens behind 30,000 take 4,050 us; activations have hardly any such group.)
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "paged_rows.cuh"
#include "paged_schedule.cuh"
#include "tcgen05_ptx.cuh"

namespace specv {

constexpr int kTileThreads = 640;
// Registers a thread of each warpgroup; their sum is what a launch must bring (5 x 96).
constexpr int kTileRegsRows = 136, kTileRegsCopy = 80, kTileRegsIssue = 48;
constexpr int kTileRegs = 2 * kTileRegsRows + 2 * kTileRegsCopy + kTileRegsIssue;
static_assert(kTileRegs <= 5 * 96 && kTileRegsCopy <= 96 && kTileRegsIssue <= 96 && kTileRegsRows >= 96,
              "shares within what the launch brings; those that shrink are below it, those that grow above");
constexpr int kTileHalf = 128 * 128;  // bytes of 128 rows of 64 numbers
// Differences of exponents within 32 positions up to which these are taken together.
constexpr uint32_t kKeysTogether = 15, kValuesTogether = 7;

template <int TYPE_, int D_>
struct TileShape {
  static constexpr int TYPE = TYPE_, D = D_;
  static constexpr bool kEight = TYPE != SPEC_CACHE_BF16;
  static constexpr int kRows = 256, kTile = 128;
  static constexpr int kBytes = kTileHalf * (D / 64);
  static constexpr int kStages = D > 64 ? 5 : 8;
  static constexpr int kExtra = 4;  // an item's beginning and end, in units (12 e4m3 prompts: 323 us with 1, 282 with 2, 255 with 4, 257 with 7)
  using Plan = Schedule<kRows, kTile, kExtra, 1, 1>;
  // Steps whose exponents are held.  A step's are written when its keys' place in the ring is free: five places
  // before it lie the values of the third step back, eight before it the keys of the fourth, whose scores follow
  // the weights of the fifth.  What is older has been read.
  static constexpr int kHeld = kStages / 2 + 1;
};

template <typename S>
struct TileSmem {
  uint8_t q[2][S::kBytes];
  uint8_t ring[S::kStages][S::kBytes];
  Cursor cursor[17], ahead[8];  // of each warp (registers are short)
  // Of a step's 32 positions each: 2^r of the keys, r of the values, 2^-r of them; -1, 0, 0: taken apart.
  alignas(16) float refs[S::kHeld][3][4];
  alignas(8) uint8_t own[S::kEight ? S::kHeld : 1][2][S::kTile];  // exponents' bytes of positions taken apart
  typename S::Plan::Shared plan;
  uint64_t full[S::kStages], empty[S::kStages];
  uint64_t q_full[2], s_full[2], p_half[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int abort;
};

// Descriptor of products of fp16 numbers instead of bf16.
__host__ __device__ constexpr uint32_t mma_desc_of(bool half, int M, int N, bool b_rows) {
  return half ? mma_desc(M, N, b_rows) & ~((1u << 7) | (1u << 10)) : mma_desc(M, N, b_rows);
}

// Byte offset of 16-byte unit u of row r: pieces of 64 numbers one after the other.
__device__ __forceinline__ uint32_t swizzled(uint32_t r, uint32_t u) {
  return (u >> 3) * kTileHalf + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

// A row's scores of positions taken apart (32 each; those whose `refs` are negative): with the positions' own
// exponents, their bytes in `own`, back to tensor memory at `at`, and the sum of their weights into `sum`.
// The row sees positions first .. end - 1 of the tile; gives back M and the sum.  (A function of its own: in place,
// although it never ran, 2,048 tokens behind 30,000 in e4m3 took 987 us instead of 886, 12 ragged prompts 268
// instead of 253; without it 875 and 245.)
static __device__ __noinline__ float2 tile_apart(uint32_t at, const float* refs, const uint8_t (*own)[128], float qs, int first, int end,
                                          float top, float sum) {
  auto byte_of = [](uint2 bytes, int k) { return ((k < 4 ? bytes.x : bytes.y) >> (8 * (k & 3))) & 255u; };
  float most = -INFINITY;
#pragma unroll 1
  for (int i = 0; i < 128; i += 8) {
    if (!(refs[i / 32] < 0.f)) continue;
    const uint2 kb = *reinterpret_cast<const uint2*>(own[0] + i), vb = *reinterpret_cast<const uint2*>(own[1] + i);
    uint32_t x[8];
    tmem_ld8(x, at + i);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float s = fmaf(__uint_as_float(x[k]) * __uint_as_float(byte_of(kb, k) << 23), qs,
                           static_cast<float>(static_cast<int>(byte_of(vb, k)) - 127));
      x[k] = __float_as_uint(s);
      if (i + k >= first && i + k < end) most = fmaxf(most, s);
    }
    tmem_st8(at + i, x);
  }
  tmem_wait_st();
  if (most > top + (kRowsSlack + kRowsBelow<true>)) {
    sum *= ex2_approx(top - (most - kRowsBelow<true>));
    top = most - kRowsBelow<true>;
  }
  __syncwarp();
  const float from = top == -INFINITY ? 0.f : top;
#pragma unroll 1
  for (int i = 0; i < 128; i += 8) {
    if (!(refs[i / 32] < 0.f)) continue;
    const uint2 vb = *reinterpret_cast<const uint2*>(own[1] + i);
    uint32_t x[8];
    tmem_ld8(x, at + i);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k >= first && i + k < end)
        sum = fmaf(ex2_approx(__uint_as_float(x[k]) - from), power_of_minus(static_cast<float>(static_cast<int>(byte_of(vb, k)) - 127)), sum);
  }
  return make_float2(top, sum);
}

template <typename S>
__global__ void __launch_bounds__(kTileThreads, 1) paged_tile_kernel(const AttendParams p, const int test_withhold) {
  using Plan = typename S::Plan;
  constexpr int D = S::D, kStages = S::kStages;
  constexpr bool kEight = S::kEight;
  constexpr uint32_t kColS = 0, kColO = 256;  // columns of tensor memory, 128 a tile
  extern __shared__ __align__(1024) uint8_t smem_tiles[];
  TileSmem<S>& sm = *reinterpret_cast<TileSmem<S>*>(smem_tiles);
  const CacheParams& c = p.c;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 4);
      mbar_init(&sm.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_half[i], 4);
      mbar_init(&sm.p_full[i], 4);
      mbar_init(&sm.o_full[i], 1);
    }
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
  }
  if (warp == 16) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  griddep_launch_dependents();
  Plan::plan(p, sm.plan);  // (its barriers publish the above)
  tc_fence_after();
  if (blockIdx.x == 0)  // lanes laid out wrongly have no units
    for (int b = threadIdx.x; b < c.lanes; b += kTileThreads) {
      int first, count, before;
      if (!cache_lane(c, b, first, count, before)) lane_fails_now(c, b, SPEC_ERR_LAYOUT);
    }
  const uint32_t tm = sm.tmem;
  const int64_t begin = sm.plan.begin[0], end = sm.plan.end[0];
  int64_t left = begin < end ? end - begin : 0;
  // Where the warp is: its first lane moves on, after all have read.
  Cursor& at = sm.cursor[min(warp, 16)];
  auto place = [&](Cursor& x) {
    if (lane == 0) x = sm.plan.from[0];
    __syncwarp();
  };
  auto move_on = [&](Cursor& x, int units) {  // within the item, or to the next one's first
    __syncwarp();
    if (lane == 0) {
      x.tile += units - 1;
      Plan::next_unit(p, x);
    }
    __syncwarp();
  };
  if (warp < 17) place(at);

  if (warp < 8) {
    // ------------------------------------------------------------ rows of a tile
    registers_grow<kTileRegsRows>();
    const int w = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t tms = tm + (static_cast<uint32_t>(warp & 3) << 21) + kColS + w * 128, tmo = tms + (kColO - kColS);
    float qs = p.scale;  // what a score is multiplied with
    // This thread's row of q.  (A tile without rows is left out.)
    auto has_rows = [&] { return at.count * p.group - at.k * S::kRows > w * 128; };
    auto load_q = [&] {
      const int r = at.k * S::kRows + w * 128 + row, col = column_of(p, r);
      const bool on = col < at.count;
      const __nv_bfloat16* const from =
          p.q + (on ? (at.first + col) * p.q_row + (at.h * p.group + r - col * p.group) * p.q_head : 0);
      uint4 x[D / 8];
#pragma unroll
      for (int u = 0; u < D / 8; ++u)
        x[u] = on && u * 8 < c.dim ? __ldg(reinterpret_cast<const uint4*>(from + u * 8)) : make_uint4(0u, 0u, 0u, 0u);
      if constexpr (kEight) {
        uint32_t most = 0;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          const uint32_t* const v = &x[u].x;
#pragma unroll
          for (int i = 0; i < 4; ++i) most = max(most, max(v[i] & 0x7FFFu, (v[i] >> 16) & 0x7FFFu));
        }
        // The largest comes to lie in 2^14 .. 2^15.
        const int up = max(min(127 + 14 - static_cast<int>(most >> 7), 126), -126);
        const float f = __uint_as_float(static_cast<uint32_t>(127 + up) << 23);
        qs = p.scale / f;
#pragma unroll
        for (int u = 0; u < D / 8; ++u) {
          uint32_t* const v = &x[u].x;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = to_halfx2(bf16_lo(v[i]) * f, bf16_hi(v[i]) * f);
        }
      }
#pragma unroll
      for (int u = 0; u < D / 8; ++u) *reinterpret_cast<uint4*>(sm.q[w] + swizzled(row, u)) = x[u];
      fence_async_smem();
      warp_arrive(&sm.q_full[w]);
    };
    int steps = 0, items = 0, refs = 0;
    bool ok = true;
    if (left > 0 && has_rows()) load_q();
    while (ok && left > 0) {
      const int n = static_cast<int>(min(static_cast<int64_t>(at.t1 - at.tile), left));
      const bool starts = at.tile == at.t0, ends = at.tile + n == at.t1;
      if (!has_rows()) {
        refs += n;
        left -= n;
        move_on(at, n);
        if (left > 0 && has_rows()) load_q();
        continue;
      }
      const int r = at.k * S::kRows + w * 128 + row, col = column_of(p, r);
      const int lim = at.before + col + 1, low = p.window > 0 ? lim - p.window : 0;
      float top = -INFINITY, sum = 0.f;  // (top: M)
      int p0 = at.tile * S::kTile;
#pragma unroll 1
      for (int j = 0; j < n; ++j, p0 += S::kTile, ++refs) {
        if (!(ok = warp_wait(&sm.s_full[w], steps++ & 1, &sm.abort))) break;
        tc_fence_after();
        // Of 32 positions each: a score's factor, and what its exponent gets.  (The factor is kept above 0 and
        // finite: hidden scores, -inf, must stay that, and scores of 0 too.  Where it is kept at 2^-126, scores
        // are below 2^-60; where at the largest number, others are beyond fp32.)
        const int held = kEight ? refs % S::kHeld : 0;
        auto factor = [&](int i) {
          if (!kEight) return qs;
          const float ref = sm.refs[held][0][i];
          return ref < 0.f ? 1.f : fminf(fmaxf(qs * ref, 0x1p-126f), 0x1.fffffep127f);
        };
        auto addend = [&](int i) { return kEight ? sm.refs[held][1][i] : 0.f; };
        const float before = top;
        if constexpr (kEight) {
          const float4 r = *reinterpret_cast<const float4*>(sm.refs[held][0]);
          if (fminf(fminf(r.x, r.y), fminf(r.z, r.w)) < 0.f) {
            const float2 now = tile_apart(tms, sm.refs[held][0], sm.own[held], qs, low - p0, lim - p0, top, sum);
            top = now.x;
            sum = now.y;
          }
        }
        const bool part_hidden = __any_sync(0xFFFFFFFFu, p0 + S::kTile > lim || p0 < low);
        uint32_t x[2][32];
        auto load = [&](int half) {
          tmem_ld32(x[0], tms + half * 64);
          tmem_ld32(x[1], tms + half * 64 + 32);
          tmem_wait_ld();
          if (part_hidden) {
            const int i0 = low - p0 - half * 64, i1 = lim - p0 - half * 64;
#pragma unroll
            for (int i = 0; i < 64; ++i) x[i / 32][i % 32] = i >= i0 && i < i1 ? x[i / 32][i % 32] : 0xFF800000u;
          }
        };
        float most = -INFINITY;
#pragma unroll
        for (int half = 1; half >= 0; --half) {  // (the first half stays in registers)
          load(half);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) m[k] = fmaxf(__uint_as_float(x[i][k]), __uint_as_float(x[i][k + 4]));
#pragma unroll
            for (int k = 8; k < 32; k += 8)
#pragma unroll
              for (int l = 0; l < 4; ++l) m[l] = fmaxf(m[l], fmaxf(__uint_as_float(x[i][k + l]), __uint_as_float(x[i][k + l + 4])));
            const float mi = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
            most = fmaxf(most, kEight ? fmaf(mi, factor(half * 2 + i), addend(half * 2 + i)) : mi * qs);
          }
        }
        const float raise = most > top + (kRowsSlack + kRowsBelow<kEight>) ? most - kRowsBelow<kEight> : top;
        if (__any_sync(0xFFFFFFFFu, raise != before)) {
          const float f = raise == before ? 1.f : ex2_approx(before - raise);
          sum *= kEight ? raise == top ? 1.f : ex2_approx(top - raise) : f;
          top = raise;
          if (j > 0) {
#pragma unroll 1
            for (int i = 0; i < D / 32; ++i) {
              uint32_t o[32];
              tmem_ld32(o, tmo + i * 32);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 32; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
              tmem_st32(tmo + i * 32, o);
            }
          }
        }
        const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          // (the second half's weights come to lie where its scores are not: columns 32 to 63)
          if (half == 1) load(1);
          uint32_t y[32];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float by = factor(half * 2 + i), add = addend(half * 2 + i);
            const f32x2 mul = pair(by, by), off = pair(add - from, add - from);
            f32x2 part[2] = {0ull, 0ull};
#pragma unroll
            for (int k = 0; k < 32; k += 2) {
              const f32x2 e = fma2(pair(__uint_as_float(x[i][k]), __uint_as_float(x[i][k + 1])), mul, off);
              const float e0 = ex2_approx(first_of(e)), e1 = ex2_approx(second_of(e));
              part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], pair(e0, e1));
              y[i * 16 + k / 2] = kEight ? to_halfx2(e0, e1) : to_bf16x2(e0, e1);
            }
            part[0] = add2(part[0], part[1]);
            const float s = first_of(part[0]) + second_of(part[0]);
            sum = kEight ? fmaf(s, sm.refs[held][2][half * 2 + i], sum) : sum + s;
          }
          tmem_st32(tms + half * 32, y);
          tmem_wait_st();
          tc_fence_before();
          warp_arrive(half ? &sm.p_full[w] : &sm.p_half[w]);  // (products begin with the first half)
        }
      }
      if (!ok) break;
      // The last scores are there, so q's tile is free: the next item's comes while the last
      // products run.
      const bool whole = starts && ends, on = col < at.count;
      const int head = at.h * p.group + r - col * p.group, b_done = at.b;
      const int64_t row_done = at.first + col;
      left -= n;
      move_on(at, n);
      if (left > 0 && has_rows()) load_q();
      if (!(ok = warp_wait(&sm.o_full[w], items++ & 1, &sm.abort))) break;
      tc_fence_after();
      __nv_bfloat16* const out = p.out + (on ? row_done * p.out_row + head * p.out_head : 0);
      float* const part = p.parts + (2 * static_cast<int64_t>(blockIdx.x) + (starts ? 1 : 0)) * part_floats(S::kRows, D);
      const float inv = 1.f / sum;
      bool fine = true;
#pragma unroll 1
      for (int i = 0; i < D / 32; ++i) {
        uint32_t o[32];
        tmem_ld32(o, tmo + i * 32);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 32; k += 8) {
          float4 a = make_float4(__uint_as_float(o[k]), __uint_as_float(o[k + 1]), __uint_as_float(o[k + 2]), __uint_as_float(o[k + 3]));
          float4 b = make_float4(__uint_as_float(o[k + 4]), __uint_as_float(o[k + 5]), __uint_as_float(o[k + 6]), __uint_as_float(o[k + 7]));
          if (whole) {
            a.x *= inv, a.y *= inv, a.z *= inv, a.w *= inv;
            b.x *= inv, b.y *= inv, b.z *= inv, b.w *= inv;
            if (on && i * 32 + k < c.dim) {
              *reinterpret_cast<uint4*>(out + i * 32 + k) =
                  make_uint4(to_bf16x2(a.x, a.y), to_bf16x2(a.z, a.w), to_bf16x2(b.x, b.y), to_bf16x2(b.z, b.w));
              fine = fine && finite4(a) && finite4(b);
            }
          } else {
            float4* const to = reinterpret_cast<float4*>(part + (w * 128 + row) * D + i * 32 + k);
            to[0] = a;
            to[1] = b;
          }
        }
      }
      tc_fence_before();
      if (whole) {
        if (!fine) lane_fails_now(c, b_done, SPEC_ERR_NONFINITE);
        if (on && p.lse != nullptr) p.lse[row_done * p.lse_row + head] = (top + log2f(sum)) * kLn2;
      } else {
        part[S::kRows * D + 2 * (w * 128 + row)] = top;
        part[S::kRows * D + 2 * (w * 128 + row) + 1] = sum;
      }
    }
  } else if (warp < 16) {
    // ------------------------------------------------------------ keys and values
    registers_shrink<kTileRegsCopy>();
    constexpr int kUnits = D * (kEight ? 1 : 2) / 16;  // 16-byte units of a token in the cache
    constexpr int kAtOnce = 32 / kUnits;               // tokens of a warp's access
    const int mine = warp & 3, which = (warp - 8) >> 2;  // positions of a step; keys or values
    const int used = c.dim * (kEight ? 1 : 2) / 16;
    const int unit = lane % kUnits, sub = lane / kUnits;
    const bool in_head = unit < used;
    // Where this lane's position lies is looked up ahead: its page two units (`ahead`), the place of its
    // head and its exponents one unit before they are used.
    Cursor& ahead = sm.ahead[warp - 8];
    place(ahead);
    int64_t left_ahead = left;
    int page = kUnseen, next_page = kUnseen;
    uint32_t from = kNowhere, ek = 0, ev = 0;
    auto look_up = [&] {
      const int pos = ahead.tile * S::kTile + mine * 32 + lane;
      next_page = kUnseen;
      if (left_ahead > 0 && pos >= ahead.lo && pos < ahead.hi)
        next_page = __ldg(c.tables + ahead.b * c.table_stride + page_of(c, pos));
      if (--left_ahead > 0) move_on(ahead, 1);
    };
    // For the unit at the cursor, whose page is `page`.
    auto locate = [&] {
      from = kNowhere;
      ek = ev = 127 + SPEC_CACHE_LEAST_EXP;
      if (page != kUnseen) {
        if (static_cast<uint32_t>(page) < static_cast<uint32_t>(c.pages)) {
          const int pos = at.tile * S::kTile + mine * 32 + lane, in = pos - page_of(c, pos) * c.page_size;
          from = head_at(c, page, in, at.h);
          if constexpr (kEight) {
            const int64_t e = page * c.exp_page + in * c.exp_slot + at.h * c.exp_head;
            ek = c.k_exps[e];
            ev = c.v_exps[e];
          }
        } else {
          lane_fails_now(c, at.b, SPEC_ERR_LAYOUT);
        }
      }
    };
    const uint32_t by = 1u << c.unit_shift;
    look_up();
    page = next_page;
    look_up();
    const uint8_t* const base = (which ? c.v : c.k) + unit * 16;
    int slot = which, round = 0;  // every other place of the ring
    bool ok = true;
    auto advance = [&] {
      if ((slot += 2) >= kStages) {
        slot -= kStages;
        ++round;
      }
    };
    const bool withhold = test_withhold != 0 && begin == 0 && which == 0;
    if constexpr (!kEight) {
      // A tile on its way while the next is asked for.
      int open_slot = -1;
      bool withheld = withhold;
      auto hand_on = [&] {  // the open tile, whose copies have landed
        fence_async_smem();
        if (!withheld) warp_arrive(&sm.full[open_slot]);
        withheld = false;
        open_slot = -1;
      };
#pragma unroll 1
      for (; ok && left > 0; --left) {
        locate();
        page = next_page;
        look_up();
        if (round > 0 && !__all_sync(0xFFFFFFFFu, mbar_try_wait(&sm.empty[slot], (round - 1) & 1))) {
          cp_async_wait<0>();
          if (open_slot >= 0) hand_on();
          if (!(ok = warp_wait(&sm.empty[slot], (round - 1) & 1, &sm.abort))) break;
        }
        const uint32_t to = smem_addr(sm.ring[slot]);
#pragma unroll
        for (int i = 0; i < 32 / kAtOnce; ++i) {
          const int tok = i * kAtOnce + sub;
          const uint32_t f = __shfl_sync(0xFFFFFFFFu, from, tok);
          const bool on = f != kNowhere && in_head;
          cp_async16_or_zero(to + swizzled(mine * 32 + tok, unit), base + (on ? static_cast<uint64_t>(f) * by : 0), on);
        }
        cp_async_commit();
        if (open_slot >= 0) {
          cp_async_wait<1>();
          hand_on();
        }
        open_slot = slot;
        advance();
        if (left > 1) move_on(at, 1);
      }
      cp_async_wait<0>();
      if (open_slot >= 0) hand_on();
    } else {
      constexpr int kLoads = 32 / kAtOnce;  // of a thread and tile
      uint4 x[kLoads];
      auto fetch = [&](uint32_t here) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const uint32_t f = __shfl_sync(0xFFFFFFFFu, here, i * kAtOnce + sub);
          x[i] = f != kNowhere && in_head ? __ldg(reinterpret_cast<const uint4*>(base + static_cast<uint64_t>(f) * by))
                                          : make_uint4(0u, 0u, 0u, 0u);
        }
      };
      // A tile as fp16 into the ring; `byte`: this lane's position's exponent, `ref` the largest (or the same: the
      // numbers as they are).  `tell` leaves word of the exponents.
      auto store = [&](uint32_t byte, uint32_t ref, auto tell) {
        if (round > 0 && !(ok = warp_wait(&sm.empty[slot], (round - 1) & 1, &sm.abort))) return;
        tell();
        uint8_t* const to = sm.ring[slot];
        const float f = byte == 255u ? __uint_as_float(0x7FC00000u)
                                     : __uint_as_float(static_cast<uint32_t>(max(127 + static_cast<int>(byte) - static_cast<int>(ref), 0)) << 23);
        const uint32_t scale = to_halfx2(f, f);
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int tok = i * kAtOnce + sub;
          const uint32_t s = __shfl_sync(0xFFFFFFFFu, scale, tok);
          const uint32_t* const in = &x[i].x;
          uint32_t y[8];
          if constexpr (S::TYPE == SPEC_CACHE_E4M3) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(y[k]) : "r"(eight_to_half2<S::TYPE>(in[k / 2], k & 1)), "r"(s));
          } else {
            // y = u - 128 with u + 1024 in hand: s (u + 1024) - 1152 s, rounded once.
            uint32_t less;
            asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(less) : "r"(s), "r"(0xE480E480u));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint32_t m = __byte_perm(in[k / 2] ^ 0x80808080u, 0x64646464u, (k & 1) == 0 ? 0x4140 : 0x4342);
              asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y[k]) : "r"(m), "r"(s), "r"(less));
            }
          }
          *reinterpret_cast<uint4*>(to + swizzled(mine * 32 + tok, unit * 2)) = make_uint4(y[0], y[1], y[2], y[3]);
          *reinterpret_cast<uint4*>(to + swizzled(mine * 32 + tok, unit * 2 + 1)) = make_uint4(y[4], y[5], y[6], y[7]);
        }
        fence_async_smem();
        if (!withhold || round > 0 || slot > 0) warp_arrive(&sm.full[slot]);
        advance();
      };
      auto largest = [&](uint32_t byte) { return __reduce_max_sync(0xFFFFFFFFu, byte == 255u ? 0u : byte); };
      // A unit's places and exponents are found while the one before it is fetched.
      uint32_t kb = 0, vb = 0, here = 0;
      auto take = [&] {  // what has been located becomes the unit in hand; the next one is located
        kb = ek;
        vb = ev;
        here = from;
        if (left > 1) {
          move_on(at, 1);
          page = next_page;
          locate();
          look_up();
        }
      };
      if (left > 0) {
        locate();
        page = next_page;
      }
      int held = 0;
#pragma unroll 1
      for (; ok && left > 0; --left, held = held + 1 == S::kHeld ? 0 : held + 1) {
        take();
        fetch(here);
        const uint32_t kr = largest(kb), vr = largest(vb);
        // (positions that no row of the item sees hold zeros)
        const bool apart = __any_sync(0xFFFFFFFFu, here != kNowhere && (kb + kKeysTogether < kr || vb + kValuesTogether < vr));
        const uint32_t byte = which ? vb : kb;
        store(byte, apart ? byte : which ? vr : kr, [&] {
          if (which != 0) return;
          if (apart) {
            sm.own[held][0][mine * 32 + lane] = static_cast<uint8_t>(kb);
            sm.own[held][1][mine * 32 + lane] = static_cast<uint8_t>(vb);
          }
          if (lane == 0) {
            const float r = static_cast<float>(static_cast<int>(vr) - 127);
            sm.refs[held][0][mine] = apart ? -1.f : __uint_as_float(kr << 23);
            sm.refs[held][1][mine] = apart ? 0.f : r;
            sm.refs[held][2][mine] = apart ? 0.f : power_of_minus(r);
          }
        });
      }
    }
  } else {
    // ------------------------------------------------------------------ products
    registers_shrink<kTileRegsIssue>();
    if (warp == 16) {
      const uint32_t lead = elect_one();
      const uint32_t tmu = __shfl_sync(0xFFFFFFFFu, tm, 0);
      constexpr uint32_t kScores = mma_desc_of(kEight, 128, 128, false), kOuts = mma_desc_of(kEight, 128, D, true);
      const uint32_t ring = smem_desc(smem_addr(sm.ring[0]), kTileHalf), qd = smem_desc(smem_addr(sm.q[0]), kTileHalf);
      int slot = 0, phase = 0;
      uint32_t parity = 0;  // bits 0, 1: of p_full; 2, 3: of q_full
      bool ok = true;
      auto advance = [&] {
        if (++slot == kStages) {
          slot = 0;
          phase ^= 1;
        }
      };
      auto scores = [&](int w, uint32_t kd) {
#pragma unroll
        for (int s = 0; s < D / 16; ++s) {
          const uint32_t off = ((s >> 2) * kTileHalf + (s & 3) * 32) / 16;
          mma_ss(lead, tmu + kColS + w * 128, qd + w * (S::kBytes / 16) + off, kd + off, kScores, s > 0);
        }
        mma_commit(lead, &sm.s_full[w]);
      };
      while (ok && left > 0) {
        const int n = __shfl_sync(0xFFFFFFFFu, static_cast<int>(min(static_cast<int64_t>(at.t1 - at.tile), left)), 0);
        const int tiles = __shfl_sync(0xFFFFFFFFu, at.count * p.group - at.k * S::kRows > 128 ? 2 : 1, 0);
        if (!(ok = warp_wait(&sm.full[slot], phase, &sm.abort))) break;
#pragma unroll 1
        for (int w = 0; w < tiles && ok; ++w) {
          ok = warp_wait(&sm.q_full[w], (parity >> (2 + w)) & 1, &sm.abort);
          if (!ok) break;
          parity ^= 4u << w;
          tc_fence_after();
          scores(w, ring + slot * (S::kBytes / 16));
        }
        if (!ok) break;
        mma_commit(lead, &sm.empty[slot]);
        advance();
#pragma unroll 1
        for (int j = 0; j < n && ok; ++j) {
          const int sv = slot;
          if (!(ok = warp_wait(&sm.full[sv], phase, &sm.abort))) break;
          advance();
          const int sk = slot;
          const uint32_t vd = ring + sv * (S::kBytes / 16), kd = ring + sk * (S::kBytes / 16);
          if (j + 1 < n && !(ok = warp_wait(&sm.full[sk], phase, &sm.abort))) break;
#pragma unroll 1
          for (int w = 0; w < tiles; ++w) {
#pragma unroll 1
            for (int half = 0; half < 2 && ok; ++half) {
              if (!(ok = warp_wait(half ? &sm.p_full[w] : &sm.p_half[w], (parity >> w) & 1, &sm.abort))) break;
              tc_fence_after();
#pragma unroll
              for (int s = 0; s < 4; ++s)
                mma_ts(lead, tmu + kColO + w * 128, tmu + kColS + w * 128 + half * 32 + s * 8, vd + (half * 4 + s) * (2048 / 16),
                       kOuts, half + s + j > 0);
            }
            if (!ok) break;
            parity ^= 1u << w;
            if (w + 1 == tiles) mma_commit(lead, &sm.empty[sv]);
            if (j + 1 < n) {
              scores(w, kd);
              if (w + 1 == tiles) mma_commit(lead, &sm.empty[sk]);
            } else {
              mma_commit(lead, &sm.o_full[w]);
            }
          }
          if (ok && j + 1 < n) advance();
        }
        if (!ok) break;
        left -= n;
        move_on(at, n);
      }
      // Tensor memory is given back only after the last product.
      mma_commit(lead, &sm.drain);
      mbar_wait_bounded(&sm.drain, 0);
      __syncwarp();
      if (lane == 0 && p.parts != nullptr) p.records[blockIdx.x] = sm.plan.record[0];
    }
  }
  __syncthreads();
  // A wait gave up: all lanes of the block's range.
  if (sm.abort && threadIdx.x == 0 && c.status != nullptr) {
    Cursor x = sm.plan.from[0];
    for (int64_t u = begin; u < end; ++u, Plan::next_unit(p, x)) lane_fails_now(c, x.b, SPEC_ERR_TIMEOUT);
  }
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tm, 512);
}

}  // namespace specv
