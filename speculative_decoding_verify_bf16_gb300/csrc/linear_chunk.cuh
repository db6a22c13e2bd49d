// linear_chunk.cuh -- linear attention with decay over prompts, a chunk of 128 tokens at
// a time on the tensor cores (bf16 activations, dk and dv up to 128; smaller heads are
// filled up with zeros by the copies).
//
// With G_i the sum of the log decays of the chunk's tokens 0..i (base 2), S the state
// before the chunk and all sums over the chunk's tokens:
//
//   o_i = scale * ( 2^G_i  S^T q_i  +  sum_{j <= i} 2^(G_i - G_j) (q_i . k_j) v_j )
//   S'  = 2^G_last S + sum_j (2^(G_last - G_j) k_j) v_j^T
//
// A CTA takes (lane, head) pairs, or segments of their chunks, one after the other, longest
// lanes first, and walks their chunks; tiles of the next item load while the last one's
// products run.  A chunk's products:
//
//   QK  scores [token][token]  = q k^T
//   QS  D [token][dv]          = q S,     D rows then times 2^G_i
//   KV  U [dk][dv]             = k'^T v,  k' = 2^(G_last - G_j) k_j
//   PV  D                     += P v,     P = weighted scores, 0 above the diagonal
//
// S stays in fp32 in the registers of four warps from the first chunk to the last, and
// S' = 2^G_last S + U is formed there: the tensor cores truncate each addition to an
// accumulator, which into S itself cost ten times the precision of its fp32 sums.
// Operands are bf16, so fp32 numbers enter a product in parts.  k' comes in three parts that
// hold all its 24 bits: U is what stays.  P and S come in two, 16 bits, far below the rounding
// of a bf16 output: its rms error is that rounding's, 0.0017 of its size (0.0023 with P and S
// rounded to one part, which would save 1,024 cycles of products a chunk).  q, k and v are
// taken as they are.  States come out within 4e-7 of 64-bit ones, like those of fp32 sums.
//
// Tensor memory holds U (128 columns), scores and P (128; P overwrites the scores it came
// from), D (128) and two buffers of k' for 32 tokens (96).  Shared memory holds a ring of
// five 32 KB tiles (k, v, q of a chunk; 128-byte swizzled rows, so that a tile serves as
// an operand along either dimension) and S in two parts, whose room also takes the copies of
// states in and out.
//
// Warps: 0 copies tiles, 1 issues the products, 2 sums the decays, 3 hands out the items,
// and five groups of four do what lies between the products: scores to P (4-11), D (8-11),
// S (12-15), k' for every other 32 tokens (16-19 and 20-23).  Where only states are wanted
// (the first of two launches for a lane cut in segments), 4-11 make k', too, into the room
// of scores and P, and U has two places.
//
// The products of a chunk take 8 x 512 cycles on the tensor cores (k' counts three times,
// S and P twice),
// its 128 KB of q, k, v and o about 5,500 at an SM's share of the HBM rate: the groups work
// beside each other, and what counts is the chain from scores to outputs.  A chunk's
// products go in the order KV (first half), QK, KV (second half), QS, PV: P is made beside the three after
// QK, the next S beside QS and PV, k' of the next tokens beside whatever is not KV.
//
// Measured (device time, 16 heads of 128): 64 lanes of 2,048 tokens 412 to 433 us, 0.76 to
// 0.79 of the copy rate (470 where each call finds L2 full of another kernel's writes); 24
// grouped lanes of 0 to 3000 tokens 120 us against 68; one lane of 16,384 99 us in two
// launches, each SM with few chunks and little to overlap their starts with; 200 tokens
// 12.0 us.  A chunk takes 3.6 us (3.9 with every SM at work on heads of 128) where HBM
// would allow 3.1: a chain bounds it, scores to P, QS, D's scaling, PV, outputs.  PV behind
// the next KV, or QS before KV's second half (423 us against 417), shortens that chain but
// holds v or wants q longer than the ring has tiles for.  Outputs straight from registers,
// which would free q's tile earlier, scatter: 455.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include <cstdint>

#include "linear_params.h"
#include "linear_recurrent.cuh"
#include "tcgen05_ptx.cuh"

namespace specv {

constexpr int kChunk = 128;
constexpr int kChunkThreads = 768;
// Registers a thread of each warpgroup; their sum is what a launch must bring (6 x 80).
constexpr int kRegsMisc = 64, kRegsOut = 64, kRegsState = 168, kRegsKey = 56;
constexpr int kChunkRegs = kRegsMisc + 2 * kRegsOut + kRegsState + 2 * kRegsKey;
constexpr int kTile = 32 * 1024;      // 128 rows of 128 bf16: two halves of 64 columns
constexpr int kHalf = kTile / 2;
constexpr int kRing = 5;
constexpr uint32_t kColU = 0, kColP = 128, kColD = 256, kColK = 384;  // columns of tensor memory
constexpr uint32_t kColKBuf = 48;     // a k' buffer: three parts of 16 columns (32 tokens)
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f;    // log2(e) in two parts
// The clamp keeps resets (-inf) and lowest values out of the sums.  A factor is finite, below
// 2^128, so that no growth over the 127 other tokens of a chunk brings back what this took:
// 2^-65536 2^(127 * 128) is 0 in fp32.  Sums of 128 of them are exact (2^23).
constexpr float kDecayFloor = -65536.f;

constexpr int kSortLanes = 64;       // most lanes that are taken longest first

// What a CTA walks: chunks c0 .. c1 - 1 of a lane's head.
struct ChunkItem {
  int b, h, seg;
  int first, count;  // first row and rows of the lane (count -1: no more items)
  int c0, c1;
  int last;          // the lane's last segment
};

struct ChunkSmem {
  uint8_t ring[kRing][kTile];
  uint8_t s[2][kTile];    // S, upper and lower parts; states on their way in and out
  float g_hi[2][kChunk];  // -G in two parts, chunk c in c % 2
  float g_lo[2][kChunk];
  float to_end[8][16];    // the P groups' warps: 2^(G at the end of 16 tokens - G_j)
  ChunkItem item[2];
  uint8_t order[kSortLanes];
  uint64_t full[kRing], empty[kRing];
  uint64_t item_full[2], item_empty[2];
  uint64_t g_full[2], g_empty[2];
  uint64_t scores_full, p_ready, qs_full, d_scaled, o_full, d_free, s_ready, v_clean, o_staged, drain;
  uint64_t kv_full[2], u_free[2];
  uint64_t kp_full[4], kp_empty[4];
  uint64_t st_full[2], st_free[2], st_done;
  uint64_t wanted, stolen;
  uint32_t tmem;
  int abort;
};

struct ChunkParams {
  LinearParams p;
  float* local;       // [segments][lanes][heads][128][128]: 0, the lanes' states before the
                      // call; r + 1, the state after segment r begun from zero
  float* local_decay; // [segments][lanes][heads]: whole decay of segment r
  int32_t segments;
  int32_t sort;       // lanes differ in length: longest first
  int32_t test_withhold;  // tests only: the first CTA announces its first copy but never issues it
};

// Waits for a phase; gives up after some seconds (a try sleeps up to 1.3 us in the barrier,
// measured).  Few instructions, no clock: the roles' loops together have to stay within
// the instruction cache, some 32 KB, or every warp waits for its code.
constexpr uint32_t kTries = 1u << 21;
__device__ __forceinline__ bool chunk_wait(uint64_t* bar, uint32_t parity, int* abort) {
#pragma unroll 1
  for (uint32_t i = 0; i < kTries; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  *static_cast<volatile int*>(abort) = 1;
  return false;
}
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* abort) {
  return __all_sync(0xFFFFFFFFu, chunk_wait(bar, parity, abort));
}
// Registers of the calling warpgroup (four warps), within what the CTA was launched with.
template <int N>
__device__ __forceinline__ void registers_grow() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void registers_shrink() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// The upper halves of two fp32 numbers, which are their bf16 parts by truncation; what
// truncation leaves; and two numbers rounded to bf16.
__device__ __forceinline__ uint32_t upper(f32x2 v) {
  return __byte_perm(static_cast<uint32_t>(v), static_cast<uint32_t>(v >> 32), 0x7632);
}
__device__ __forceinline__ f32x2 rest(f32x2 v) {
  const uint32_t a = static_cast<uint32_t>(v), b = static_cast<uint32_t>(v >> 32);
  return add2(v, pair(__uint_as_float((a & 0xFFFF0000u) ^ 0x80000000u), __uint_as_float((b & 0xFFFF0000u) ^ 0x80000000u)));
}
__device__ __forceinline__ uint32_t rounded(f32x2 v) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(second_of(v)), "f"(first_of(v)));
  return d;
}

// Byte offset of 16-byte unit u (of 16) of row r in a tile.
__device__ __forceinline__ uint32_t tile_unit(uint32_t r, uint32_t u) {
  return (u >> 3) * kHalf + r * 128 + (((u & 7) ^ (r & 7)) << 4);
}

// The next item into registers; false when there is none.
__device__ __forceinline__ bool next_item(ChunkSmem& sm, int& turn, ChunkItem& item) {
  const int slot = turn & 1;
  if (!warp_wait(&sm.item_full[slot], (turn >> 1) & 1, &sm.abort)) return false;
  ++turn;
  item = sm.item[slot];
  warp_arrive(&sm.item_empty[slot]);
  return item.count >= 0;
}

// A dk x dv state by one warp, into rows of `ld` numbers of a state of `rows` rows (zeros
// beyond dk and dv; from == nullptr: zeros).
__device__ __forceinline__ void copy_state(float* to, int rows, int ld, const float* from, int dk, int dv) {
  const int wide = ld / 4, n = rows * wide;
  const bool same = rows == dk && ld == dv;
  for (int i0 = threadIdx.x & 31; i0 < n; i0 += 8 * 32) {
    float4 x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = i0 + 32 * j;
      int at = 4 * i;
      bool in = from != nullptr && i < n;
      if (!same) {
        const int r = i / wide, c = i % wide * 4;
        at = r * dv + c;
        in = in && r < dk && c < dv;
      }
      x[j] = in ? __ldcg(reinterpret_cast<const float4*>(from + at)) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (i0 + 32 * j < n) reinterpret_cast<float4*>(to)[i0 + 32 * j] = x[j];
  }
}

// map_begin holds the states before the items: state_in or, with segments, `local` (slot
// r of lane b in its lane r * lanes + b); map_end takes those after them: state_out or, with
// STATES, `local`.
// STATES: only the states of all segments but the last, begun from zero (the first of
// two launches when a lane is split); otherwise outputs and final states.
template <bool STATES>
__global__ void __launch_bounds__(kChunkThreads, 1)
    linear_chunk_kernel(const ChunkParams cp, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_begin,
                        const __grid_constant__ CUtensorMap map_end) {
  constexpr int kLoads = STATES ? 2 : 3;  // tiles of a chunk: k, v (, q)
  // Without outputs their groups make k', too: four buffers of it, and two of U.
  constexpr int kKeyGroups = STATES ? 4 : 2, kKeyWarps = 4 * kKeyGroups;
  constexpr uint32_t kColKeys = STATES ? kColP : kColK, kColU2 = STATES ? kColK : kColU;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem& sm = *reinterpret_cast<ChunkSmem*>(smem_raw);
  const LinearParams& p = cp.p;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 1 + kKeyWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], 23);
      mbar_init(&sm.g_full[i], 1);
      mbar_init(&sm.g_empty[i], 20);
      mbar_init(&sm.kv_full[i], 1);
      mbar_init(&sm.u_free[i], 4);
      mbar_init(&sm.st_full[i], 1);
      mbar_init(&sm.st_free[i], 4);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sm.kp_full[i], 4);
      mbar_init(&sm.kp_empty[i], 1);
    }
    mbar_init(&sm.scores_full, 1);
    mbar_init(&sm.p_ready, 8);
    mbar_init(&sm.qs_full, 1);
    mbar_init(&sm.d_scaled, 4);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.d_free, 4);
    mbar_init(&sm.s_ready, 4);
    mbar_init(&sm.v_clean, 4);
    mbar_init(&sm.o_staged, 4);
    mbar_init(&sm.st_done, 1);
    mbar_init(&sm.wanted, 1);
    mbar_init(&sm.stolen, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_mbar_init();
    tma_prefetch_map(&map_q);
    tma_prefetch_map(&map_k);
    tma_prefetch_map(&map_v);
  }
  if (warp == 1) {
    tmem_alloc(&sm.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm.tmem;
  const uint32_t quarter = static_cast<uint32_t>(warp & 3) * 32;  // this warp's lanes of tensor memory
  const uint32_t row = quarter + lane;
  const uint32_t tmq = tm + (quarter << 16);
  const int heads = p.lanes * p.v_heads;
  ChunkItem it;
  int turn = 0;  // items taken
  int gc = 0;    // chunks done in the items before

  if (warp < 4) registers_shrink<kRegsMisc>();
  if (warp == 3) {
    // ------------------------------------------------------------------- items
    if (cp.sort) {
      // A lane's place: how many are longer, or as long and before it.
      for (int i = lane; i < p.lanes; i += 32) {
        const int n = p.row_offsets[i + 1] - p.row_offsets[i];
        int place = 0;
#pragma unroll 4
        for (int j = 0; j < p.lanes; ++j) {
          const int m = __ldg(p.row_offsets + j + 1) - __ldg(p.row_offsets + j);
          place += m > n || (m == n && j < i) ? 1 : 0;
        }
        sm.order[place] = static_cast<uint8_t>(i);
      }
      __syncwarp();
    }
    auto slot_free = [&] {
      return turn < 2 || warp_wait(&sm.item_empty[turn & 1], ((turn >> 1) - 1) & 1, &sm.abort);
    };
    auto publish = [&](const ChunkItem& x) {
      if (lane == 0) sm.item[turn & 1] = x;
      __threadfence_block();
      warp_arrive(&sm.item_full[turn & 1]);
      ++turn;
    };
    // Items past the first are CTAs that the hardware has not launched yet, in order: a CTA
    // takes the next one when its copies have run out of work.
    int index = blockIdx.x;
    int asked = 0;
    bool ok = slot_free();
    while (ok && index >= 0) {
      it.h = index % p.v_heads;
      it.b = index / p.v_heads % p.lanes;
      if (cp.sort) it.b = sm.order[it.b];
      it.seg = index / heads;
      const int rc = linear_lane_rows(p, it.b, it.first, it.count);
      // (lanes agree on a status that another head's CTA may be writing)
      const int status = p.lane_status == nullptr ? SPEC_OK : __shfl_sync(0xFFFFFFFFu, p.lane_status[it.b], 0);
      if (status == SPEC_OK && rc != SPEC_OK) {
        if (lane == 0 && p.lane_status != nullptr) p.lane_status[it.b] = rc;
      } else if (status == SPEC_OK) {
        const int chunks = (it.count + kChunk - 1) / kChunk;
        const int per = (chunks + cp.segments - 1) / cp.segments;
        it.c0 = min(chunks, it.seg * per);
        it.c1 = min(chunks, it.c0 + per);
        it.last = it.c1 == chunks;
        const bool work = it.c0 < it.c1 && !(STATES && it.last);
        if (work) publish(it);
        if (it.seg == 0) {
          const float* in =
              p.state_in == nullptr ? nullptr : p.state_in + it.b * p.state_in_lane + it.h * p.state_in_head;
          // The last segment writes the final state while others may yet begin, and the two
          // may be one buffer: with segments the first launch keeps a copy of the initial one.
          if (STATES && in != nullptr)
            copy_state(cp.local + (it.b * p.v_heads + it.h) * int64_t{128 * 128}, 128, 128, in, p.dk, p.dv);
          // An empty lane's state passes through.
          if (!STATES && chunks == 0 && p.state_out != nullptr)
            copy_state(p.state_out + it.b * p.state_out_lane + it.h * p.state_out_head, p.dk, p.dv, in, p.dk, p.dv);
        }
        if (work && !(ok = warp_wait(&sm.wanted, (turn - 1) & 1, &sm.abort) && slot_free())) break;
      }
      // The response comes into the item's own place.
      if (lane == 0) {
        mbar_arrive_expect_tx(&sm.stolen, 16);
        steal_cta(&sm.item[turn & 1], &sm.stolen);
      }
      __syncwarp();
      if (!(ok = warp_wait(&sm.stolen, asked++ & 1, &sm.abort))) break;
      index = stolen_cta(&sm.item[turn & 1]);
      fence_async_smem();
      __syncwarp();
    }
    if (ok) {
      it.count = -1;
      publish(it);
    }
  } else if (warp == 0) {
    // ------------------------------------------------------------------ copies
    int slot = 0, round = 0, issued = 0;
    bool ok = true;
    while (ok && next_item(sm, turn, it)) {
      for (int c = it.c0; c < it.c1 && ok; ++c) {
#pragma unroll 1
        for (int j = 0; j < kLoads; ++j) {
          if (round > 0 && !(ok = warp_wait(&sm.empty[slot], (round - 1) & 1, &sm.abort))) break;
          if (lane == 0) {
            const CUtensorMap* map = j == 0 ? &map_k : (j == 1 ? &map_v : &map_q);
            const int hh = j == 1 ? it.h : it.h / p.group, z = it.first + c * kChunk;
            mbar_arrive_expect_tx(&sm.full[slot], kTile);
            if (!(cp.test_withhold && blockIdx.x == 0 && issued == 0)) {
              tma_load_3d(sm.ring[slot], map, 0, hh, z, &sm.full[slot]);
              tma_load_3d(sm.ring[slot] + kHalf, map, 64, hh, z, &sm.full[slot]);
            }
          }
          ++issued;
          if (++slot == kRing) {
            slot = 0;
            ++round;
          }
        }
      }
      warp_arrive(&sm.wanted);
    }
    // Every copy lands before the CTA ends (also when a wait gave up).
    for (int i = max(0, issued - kRing); i < issued; ++i) mbar_wait_bounded(&sm.full[i % kRing], (i / kRing) & 1);
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    // What follows from a shuffle is the same in all lanes also to the compiler, which
    // then keeps loop counters and descriptors in uniform registers: a product is a few
    // instructions, issued well within the 64 cycles it takes.
    const uint32_t lead = elect_one();
    const uint32_t tmu = __shfl_sync(0xFFFFFFFFu, tm, 0);
    constexpr uint32_t kSame = mma_desc(128, 128, false), kRows = mma_desc(128, 128, true);
    const uint32_t ring = smem_desc(smem_addr(sm.ring[0]), kHalf);  // (for K-major tiles the piece distance is not used)
    const uint32_t ds = smem_desc(smem_addr(sm.s[0]), kHalf);  // (the lower part a tile behind)
    uint32_t kphase = 0;     // bit i: phase of k' buffer i
    int slot = 0, phase = 0; // the ring's slot of this chunk's k and its phase
    int tails = 0;           // chunks that did not fill a tile
    bool ok = true;
    while (ok && next_item(sm, turn, it)) {
    const int loops = __shfl_sync(0xFFFFFFFFu, it.c1 - it.c0, 0);
    const int rows_left = __shfl_sync(0xFFFFFFFFu, it.count - it.c0 * kChunk, 0);
    ok = false;
    for (int c = 0; c < loops; ++c, ++gc) {
      const uint32_t ph = gc & 1;
      const int n = min(kChunk, rows_left - c * kChunk);
      const int bufs = (n + 31) / 32;  // products over the chunk's tokens stop at the last 32 that hold any
      const int sk = slot, pk = phase;
      auto advance = [&] {
        if (++slot == kRing) {
          slot = 0;
          phase ^= 1;
        }
      };
      advance();
      const int sv = slot, pv = phase;
      advance();
      const int sq = slot, pq = phase;
      if (!STATES) advance();
      const uint32_t dk = ring + sk * (kTile / 16), dv = ring + sv * (kTile / 16), dq = ring + sq * (kTile / 16);
      if (!warp_wait(&sm.full[sv], pv, &sm.abort)) break;
      if (n < kChunk && !warp_wait(&sm.v_clean, tails++ & 1, &sm.abort)) break;
      // U alternates between two places with STATES.
      const uint32_t ub = STATES ? gc & 1 : 0, uph = STATES ? (gc >> 1) & 1 : ph;
      if (gc > (STATES ? 1 : 0) && !warp_wait(&sm.u_free[ub], uph ^ 1, &sm.abort)) break;
      bool fine = true;
#pragma unroll 1
      for (int t = 0; t < bufs || t == 2; ++t) {
        if (t == 2) {  // QK between the halves of KV (and behind a short chunk's)
          if (!STATES) {
            if (!(fine = warp_wait(&sm.full[sq], pq, &sm.abort) && warp_wait(&sm.full[sk], pk, &sm.abort))) break;
            tc_fence_after();
#pragma unroll
            for (int s = 0; s < 8; ++s) {
              const uint32_t off = ((s >> 2) * kHalf + (s & 3) * 32) / 16;
              mma_ss(lead, tmu + kColP, dq + off, dk + off, kSame, s > 0);
            }
            mma_commit(lead, &sm.scores_full);
            mma_commit(lead, &sm.empty[sk]);
          } else if (lead) {
            mbar_arrive(&sm.empty[sk]);
          }
          if (bufs <= 2) break;
        }
        const uint32_t kb = t % kKeyGroups;
        if (!(fine = warp_wait(&sm.kp_full[kb], (kphase >> kb) & 1, &sm.abort))) break;
        tc_fence_after();
        const uint32_t parts = tmu + kColKeys + kb * kColKBuf, dvt = dv + t * (2 * 2048 / 16);
#pragma unroll
        for (int i = 0; i < 6; ++i)  // the least part first
          mma_ts(lead, tmu + (ub ? kColU2 : kColU), parts + 32 - (i >> 1) * 16 + (i & 1) * 8, dvt + (i & 1) * (2048 / 16), kRows, i + t > 0);
        mma_commit(lead, &sm.kp_empty[kb]);
        kphase ^= 1u << kb;
        if (t == 0 && bufs == 1) t = 1;  // on to QK
      }
      if (!fine) break;
      mma_commit(lead, &sm.kv_full[ub]);
      if (!STATES) {
        if (!warp_wait(&sm.s_ready, ph, &sm.abort)) break;
        if (gc > 0 && !warp_wait(&sm.d_free, ph ^ 1, &sm.abort)) break;
        tc_fence_after();
#pragma unroll 1
        for (int part = 1; part >= 0; --part)  // the lower part first
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_ss(lead, tmu + kColD, dq + ((s >> 2) * kHalf + (s & 3) * 32) / 16,
                   ds + part * (kTile / 16) + s * (2048 / 16), kRows, s > 0 || part == 0);
        mma_commit(lead, &sm.qs_full);
        if (!warp_wait(&sm.p_ready, ph, &sm.abort) || !warp_wait(&sm.d_scaled, ph, &sm.abort)) break;
        tc_fence_after();
#pragma unroll 1
        for (int t = 0; t < bufs; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_ts(lead, tmu + kColD, tmu + kColP + t * 32 + (i & 1) * 16 + 8 - (i >> 1) * 8,
                   dv + t * (2 * 2048 / 16) + (i & 1) * (2048 / 16), kRows, true);
        mma_commit(lead, &sm.o_full);
      }
      mma_commit(lead, &sm.empty[sv]);
      if (lead) mbar_arrive_n(&sm.empty[sv], kKeyWarps);
      ok = c + 1 == loops;  // the item is done
    }
    }
    // Tensor memory is given back only after the last product.
    mma_commit(lead, &sm.drain);
    mbar_wait_bounded(&sm.drain, 0);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ decays
    // Fixed point with 32 fractional bits: sums and differences are exact, whatever large
    // decays stand between two tokens.  A lane has four tokens of the chunk; it hands on
    // whole part and fraction.
    bool ok = true;
    while (ok && next_item(sm, turn, it)) {
      const int rows = it.count - it.c0 * kChunk, end = (it.c1 - it.c0) * kChunk;
      const float* src = p.log_decay + (it.first + it.c0 * static_cast<int64_t>(kChunk)) * p.decay_row + it.h * p.decay_head;
      float next[4];
      auto fetch = [&](int t) {
#pragma unroll
        for (int i = 0; i < 4; ++i) next[i] = t + i < rows ? __ldg(src + (t + i) * p.decay_row) : 0.f;
      };
      fetch(lane * 4);
#pragma unroll 1
      for (int t = 0; t < end; t += kChunk, ++gc) {
        const int buf = gc & 1;
        long long sum[4];
        bool bad = false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float hi = next[i] * kLog2eHi;
          float lo = fmaf(next[i], kLog2eHi, -hi) + next[i] * kLog2eLo;
          bad |= !(hi < 128.f);  // NaN, or a factor infinite in fp32
          lo = hi > kDecayFloor ? lo : 0.f;
          hi = fmaxf(hi, kDecayFloor);
          const float whole = rintf(hi);
          sum[i] = (static_cast<long long>(__float2int_rn(whole)) << 32) + __float2int_rn((hi - whole) * 0x1p32f) +
                   __float2int_rn(lo * 0x1p32f);
          if (i > 0) sum[i] += sum[i - 1];
        }
        if (t + kChunk < end) fetch(t + kChunk + lane * 4);
        long long run = sum[3];
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, run, d);
          run += lane >= d ? up : 0;
        }
        run -= sum[3];
        // A NaN makes all the chunk's sums NaN.
        const float poison = __any_sync(0xFFFFFFFFu, bad) ? __uint_as_float(0x7FC00000u) : 0.f;
        float4 hi, lo;
        float* const ph = &hi.x;
        float* const pl = &lo.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const long long g = -(run + sum[i]);
          ph[i] = static_cast<float>(static_cast<int>(g >> 32)) + poison;
          pl[i] = static_cast<float>(static_cast<uint32_t>(g)) * 0x1p-32f;
        }
        if (gc >= 2 && !(ok = warp_wait(&sm.g_empty[buf], ((gc >> 1) - 1) & 1, &sm.abort))) break;
        *reinterpret_cast<float4*>(&sm.g_hi[buf][lane * 4]) = hi;
        *reinterpret_cast<float4*>(&sm.g_lo[buf][lane * 4]) = lo;
        __threadfence_block();
        warp_arrive(&sm.g_full[buf]);
      }
    }
  } else if (!STATES && warp >= 4 && warp < 12) {
    // ------------------------------------------- scores to P; outputs (8-11)
    registers_shrink<kRegsOut>();
    const int group = (warp - 4) >> 2;  // which 16 of every 32 tokens
    float* const to_end = sm.to_end[warp - 4];
    int slot = 2;    // the ring's slot of the chunk's q
    int stores = 0;  // chunks that went out as tiles
    bool ok = true;
    while (ok && next_item(sm, turn, it)) {
      for (int c = it.c0; c < it.c1; ++c, ++gc) {
        const int buf = gc & 1;
        if (!(ok = warp_wait(&sm.g_full[buf], (gc >> 1) & 1, &sm.abort))) break;
        const float ghi = -sm.g_hi[buf][row], glo = -sm.g_lo[buf][row];
        if (!(ok = warp_wait(&sm.scores_full, gc & 1, &sm.abort))) break;
        tc_fence_after();
#pragma unroll 1
        for (int j0 = group * 16; j0 < kChunk; j0 += 32) {  // tokens j0 .. j0 + 15
          uint32_t hi[8], lo[8];
          if (j0 >= static_cast<int>(quarter) + 32) {  // all after this warp's rows
#pragma unroll
            for (int i = 0; i < 8; ++i) hi[i] = lo[i] = 0u;
          } else {
            uint32_t s[16];
            tmem_ld16(s, tmq + kColP + j0);
            if (j0 < static_cast<int>(quarter)) {
              // All before this warp's rows: 2^(G_i - G_j) in two factors, to the end of the
              // 16 tokens and from there, of which neither can overflow where the whole
              // does not.
              const float ehi = sm.g_hi[buf][j0 + 15], elo = sm.g_lo[buf][j0 + 15];
              const float from_end = ex2_approx((ghi + ehi) + (glo + elo));
              __syncwarp();
              if (lane < 16) to_end[lane] = ex2_approx((sm.g_hi[buf][j0 + lane] - ehi) + (sm.g_lo[buf][j0 + lane] - elo));
              __syncwarp();
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                const f32x2 x = mul2(mul2(pair(from_end, from_end), *reinterpret_cast<const f32x2*>(&to_end[i])),
                                     pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
                hi[i / 2] = upper(x);
                lo[i / 2] = rounded(rest(x));
              }
            } else {
              const int seen = static_cast<int>(row) - j0;  // the last of the tokens that this row sees
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; i += 2) {
                // (the arrays hold -G)
                const f32x2 d = add2(add2(pair(ghi, ghi), *reinterpret_cast<const f32x2*>(&sm.g_hi[buf][j0 + i])),
                                     add2(pair(glo, glo), *reinterpret_cast<const f32x2*>(&sm.g_lo[buf][j0 + i])));
                f32x2 x = mul2(pair(ex2_approx(first_of(d)), ex2_approx(second_of(d))),
                               pair(__uint_as_float(s[i]), __uint_as_float(s[i + 1])));
                // (a select: what is masked may be NaN)
                x = pair(i > seen ? 0.f : first_of(x), i + 1 > seen ? 0.f : second_of(x));
                hi[i / 2] = upper(x);
                lo[i / 2] = rounded(rest(x));
              }
            }
          }
          // For each 16 tokens 8 columns of upper and 8 of lower parts.
          tmem_st8(tmq + kColP + j0, hi);
          tmem_st8(tmq + kColP + j0 + 8, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&sm.p_ready);
        warp_arrive(&sm.g_empty[buf]);
        if (group == 0) continue;

        const float e = exp2f(ghi + glo);
        if (!(ok = warp_wait(&sm.qs_full, gc & 1, &sm.abort))) break;
        tc_fence_after();
#pragma unroll 1
        for (int piece = 0; piece < 4; ++piece) {
          uint32_t d[32];
          tmem_ld32(d, tmq + kColD + piece * 32);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const f32x2 x = mul2(pair(e, e), pair(__uint_as_float(d[i]), __uint_as_float(d[i + 1])));
            d[i] = static_cast<uint32_t>(x);
            d[i + 1] = static_cast<uint32_t>(x >> 32);
          }
          tmem_st32(tmq + kColD + piece * 32, d);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&sm.d_scaled);
        if (!(ok = warp_wait(&sm.o_full, gc & 1, &sm.abort))) break;
        tc_fence_after();
        // The chunk's q has been read: its tile takes the outputs on their way out.
        uint8_t* tile = sm.ring[slot];
        const int n = it.count - c * kChunk;
        const f32x2 scale = pair(p.scale, p.scale);
#pragma unroll 1
        for (int piece = 0; piece < 4; ++piece) {
          uint32_t d[32], o[16];
          tmem_ld32(d, tmq + kColD + piece * 32);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o[i] = rounded(mul2(scale, pair(__uint_as_float(d[2 * i]), __uint_as_float(d[2 * i + 1]))));
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<uint4*>(tile + tile_unit(row, piece * 4 + i / 4)) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
        }
        tc_fence_before();
        warp_arrive(&sm.d_free);
        fence_async_smem();
        // By a copy, unless it would go on into the next lane's rows or, as it ends in steps of 16
        // bytes, into what lies behind the head.
        if (n >= kChunk && p.dv % 8 == 0) {
          warp_arrive(&sm.o_staged);
          if (warp == 8) {
            if (!(ok = warp_wait(&sm.o_staged, stores++ & 1, &sm.abort))) break;
            if (lane == 0) {
              const int z = it.first + c * kChunk;
              tma_store_3d(&map_out, tile, 0, it.h, z);
              tma_store_3d(&map_out, tile + kHalf, 64, it.h, z);
              bulk_commit_group();
              bulk_wait_group_read<0>();
              mbar_arrive_n(&sm.empty[slot], 1 + kKeyWarps);
            }
            __syncwarp();
          }
        } else {
          __syncwarp();
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + it.h * p.out_head;
#pragma unroll 1
          for (int i = lane; i < 32 * 16; i += 32) {
            const int r = static_cast<int>(quarter) + i / 16, left = p.dv - (i % 16) * 8;
            if (r >= n || left <= 0) continue;
            __nv_bfloat16* const to = dst + (it.first + c * static_cast<int64_t>(kChunk) + r) * p.out_row + (i % 16) * 8;
            const uint8_t* const from = tile + tile_unit(r, i % 16);
            if (left >= 8)
              *reinterpret_cast<uint4*>(to) = *reinterpret_cast<const uint4*>(from);
            else  // (dv is a multiple of four)
              *reinterpret_cast<uint2*>(to) = *reinterpret_cast<const uint2*>(from);
          }
          fence_async_smem();  // the tile's next content comes by a copy
          __syncwarp();
          if (lane == 0) mbar_arrive_n(&sm.empty[slot], warp == 8 ? 6 : 1);
        }
        slot = slot >= 2 ? slot - 2 : slot + 3;  // three tiles on
      }
    }
    // (the last copies end before the CTA does)
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  } else if (warp >= 12 && warp < 16) {
    // ------------------------------------------------------------------ states
    registers_grow<kRegsState>();
    // States come and go by copies through sm.s (columns 0..63 in the first), which holds S in
    // parts only from a chunk's start to its QS; the group's first warp issues them.
    const bool has_in = !STATES && p.state_in != nullptr;
    int loads = 0;       // states loaded so far
    int frees[2] = {0, 0};  // phases of st_free
    int stored = 0;      // states stored so far
    bool ok = true;
    while (ok && next_item(sm, turn, it)) {
      const int64_t head = it.b * p.v_heads + it.h;
      f32x2 S[64];  // row `row` of S
#pragma unroll
      for (int i = 0; i < 64; ++i) S[i] = 0ull;
      if (!STATES && gc > 0 && !(ok = warp_wait(&sm.qs_full, (gc - 1) & 1, &sm.abort))) break;
      if (stored > 0 && !(ok = warp_wait(&sm.st_done, (stored - 1) & 1, &sm.abort))) break;
      if (!STATES) {
        // The state before the segment: the lane's, then every earlier segment's from zero
        // behind its decay.
        const int n = (has_in ? 1 : 0) + it.seg, slot0 = has_in ? 0 : 1;
        auto load = [&](int k, int half) {
          if (lane == 0) {
            uint8_t* dst = sm.s[half];
            const int z = (slot0 + k) * p.lanes + it.b;
            mbar_arrive_expect_tx(&sm.st_full[half], kTile);
            tma_load_4d(dst, &map_begin, half * 64, 0, it.h, z, &sm.st_full[half]);
            tma_load_4d(dst + kHalf, &map_begin, half * 64 + 32, 0, it.h, z, &sm.st_full[half]);
          }
          __syncwarp();
        };
        if (n > 0 && warp == 12) {
          load(0, 0);
          load(0, 1);
        }
#pragma unroll 1
        for (int k = 0; k < n && ok; ++k, ++loads) {
          const int r = slot0 + k - 1;
          const float a = r < 0 ? 0.f : __ldcg(cp.local_decay + r * static_cast<int64_t>(heads) + head);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!(ok = ok && warp_wait(&sm.st_full[half], loads & 1, &sm.abort))) break;
            const uint8_t* src = sm.s[half];
#pragma unroll
            for (int f = 0; f < 16; ++f) {
              const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(src + tile_unit(row, f));
              S[half * 32 + 2 * f] = fma2(S[half * 32 + 2 * f], pair(a, a), x.x);
              S[half * 32 + 2 * f + 1] = fma2(S[half * 32 + 2 * f + 1], pair(a, a), x.y);
            }
            warp_arrive(&sm.st_free[half]);
            ++frees[half];
            if (warp == 12 && k + 1 < n) {
              if (!(ok = warp_wait(&sm.st_free[half], (frees[half] - 1) & 1, &sm.abort))) break;
              load(k + 1, half);
            }
          }
        }
        if (!ok) break;
        if (n > 0 && !(ok = warp_wait(&sm.st_free[0], (frees[0] - 1) & 1, &sm.abort) &&
                            warp_wait(&sm.st_free[1], (frees[1] - 1) & 1, &sm.abort)))
          break;
      }
      float total = 1.f;  // the segment's whole decay
      for (int c = it.c0; c < it.c1; ++c, ++gc) {
        const int buf = gc & 1;
        if (!STATES) {
          // S in two parts to shared memory for the chunk's QS, the last chunk's done.
          if (c > it.c0 && !(ok = warp_wait(&sm.qs_full, (gc - 1) & 1, &sm.abort))) break;
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const uint32_t unit = tile_unit(row, i / 4);
            *reinterpret_cast<uint4*>(sm.s[0] + unit) =
                make_uint4(upper(S[i]), upper(S[i + 1]), upper(S[i + 2]), upper(S[i + 3]));
            *reinterpret_cast<uint4*>(sm.s[1] + unit) = make_uint4(rounded(rest(S[i])), rounded(rest(S[i + 1])),
                                                                   rounded(rest(S[i + 2])), rounded(rest(S[i + 3])));
          }
          fence_async_smem();
          warp_arrive(&sm.s_ready);
        }
        if (!(ok = warp_wait(&sm.g_full[buf], (gc >> 1) & 1, &sm.abort))) break;
        const float decay = exp2f(-(sm.g_hi[buf][kChunk - 1] + sm.g_lo[buf][kChunk - 1]));
        total *= decay;
        warp_arrive(&sm.g_empty[buf]);
        const uint32_t ub = STATES ? gc & 1 : 0, uph = STATES ? (gc >> 1) & 1 : gc & 1;
        if (!(ok = warp_wait(&sm.kv_full[ub], uph, &sm.abort))) break;
        tc_fence_after();
        uint32_t u[2][8];
        const uint32_t from = tmq + (ub ? kColU2 : kColU);
        tmem_ld8(u[0], from);
#pragma unroll
        for (int piece = 0; piece < 16; ++piece) {
          tmem_wait_ld();
          if (piece < 15) tmem_ld8(u[(piece + 1) & 1], from + (piece + 1) * 8);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            S[piece * 4 + i] = fma2(S[piece * 4 + i], pair(decay, decay),
                                    pair(__uint_as_float(u[piece & 1][2 * i]), __uint_as_float(u[piece & 1][2 * i + 1])));
        }
        tc_fence_before();
        warp_arrive(&sm.u_free[ub]);
      }
      if (!ok) break;
      f32x2 bad = 0ull;  // 0 times S: NaN where S is not finite
#pragma unroll
      for (int i = 0; i < 64; ++i) bad = fma2(S[i], 0ull, bad);
      if (!STATES && it.last && first_of(bad) + second_of(bad) != 0.f && p.lane_status != nullptr)
        p.lane_status[it.b] = SPEC_ERR_NONFINITE;
      if (STATES && row == 0) cp.local_decay[it.seg * static_cast<int64_t>(heads) + head] = total;
      if (!STATES && !(it.last && p.state_out != nullptr)) continue;
      if (!STATES && !(ok = warp_wait(&sm.qs_full, (gc - 1) & 1, &sm.abort))) break;
#pragma unroll
      for (int f = 0; f < 32; ++f)
        *reinterpret_cast<ulonglong2*>(sm.s[f < 16 ? 0 : 1] + tile_unit(row, f & 15)) =
            make_ulonglong2(S[2 * f], S[2 * f + 1]);
      fence_async_smem();
      warp_arrive(&sm.st_free[0]);
      ++frees[0];
      ++stored;
      if (warp == 12) {
        if (!(ok = warp_wait(&sm.st_free[0], (frees[0] - 1) & 1, &sm.abort))) break;
        if (lane == 0) {
          const int z = STATES ? (it.seg + 1) * p.lanes + it.b : it.b;
          for (int i = 0; i < 4; ++i)
            tma_store_4d(&map_end, sm.s[i < 2 ? 0 : 1] + (i & 1) * kHalf, i * 32, 0, it.h, z);
          bulk_commit_group();
          bulk_wait_group_read<0>();
          mbar_arrive(&sm.st_done);
        }
        __syncwarp();
      }
    }
    // Copies end before the CTA does (loads that a wait gave up on, too).
    if (warp == 12) {
      if (sm.abort && loads > 0) {
        mbar_wait_bounded(&sm.st_full[0], loads & 1);
        mbar_wait_bounded(&sm.st_full[1], loads & 1);
      }
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
    }
  } else {  // (warps 16 .. 23, with STATES also 4 .. 11)
    // ---------------------------------------------------------------------- k'
    // Lane i of k'^T is component i of k, along the tokens.  Transposing loads bring a
    // thread two tokens of one component, weighted pairs of which go out as they lie.
    registers_shrink<kRegsKey>();
    const int kb = warp >= 16 ? (warp - 16) >> 2 : (warp + 4) >> 2;  // this group's buffer of k'
    int step = 0;                     // times it has been filled
    int slot = 0, phase = 0;          // the ring's slot of the chunk's k and its phase
    bool ok = true;
    while (ok && next_item(sm, turn, it))
    for (int c = it.c0; c < it.c1; ++c, ++gc) {
      const int buf = gc & 1;
      const int n = min(kChunk, it.count - c * kChunk);
      const int sk = slot, pk = phase, sv = slot + 1 == kRing ? 0 : slot + 1, pv = slot + 1 == kRing ? phase ^ 1 : phase;
      slot += kLoads;
      if (slot >= kRing) {
        slot -= kRing;
        phase ^= 1;
      }
      if (!(ok = warp_wait(&sm.g_full[buf], (gc >> 1) & 1, &sm.abort))) break;
      if (n < kChunk && kb == 0) {  // rows past the lane take part in products (times 0): make them 0
        if (!(ok = warp_wait(&sm.full[sv], pv, &sm.abort))) break;
        uint8_t* vt = sm.ring[sv];
        if (static_cast<int>(row) >= n)
          for (uint32_t u = 0; u < 16; ++u)
            *reinterpret_cast<uint4*>(vt + tile_unit(row, u)) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        warp_arrive(&sm.v_clean);
      }
      const float last_hi = sm.g_hi[buf][kChunk - 1], last_lo = sm.g_lo[buf][kChunk - 1];
      if (!(ok = warp_wait(&sm.full[sk], pk, &sm.abort))) break;
      const uint32_t tile = smem_addr(sm.ring[sk]);
      const int used = (n + 31) / 32;
      for (int t0 = kb * 32; t0 < used * 32; t0 += kKeyGroups * 32, ++step) {
        // Each lane has the weight of one of the 32 tokens.
        const float weight = exp2f((sm.g_hi[buf][t0 + lane] - last_hi) + (sm.g_lo[buf][t0 + lane] - last_lo));
        const int pick = 2 * (lane & 3);
        if (t0 + lane >= n) {  // rows past the lane may hold NaN: what this warp reads of them becomes 0
          for (int u = 0; u < 4; ++u)
            *reinterpret_cast<uint4*>(sm.ring[sk] + tile_unit(t0 + lane, quarter / 8 + u)) = make_uint4(0u, 0u, 0u, 0u);
          fence_async_smem();  // the tile's next content comes by a copy
        }
        __syncwarp();
        f32x2 w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
          w[m] = pair(__shfl_sync(0xFFFFFFFFu, weight, 8 * m + pick), __shfl_sync(0xFFFFFFFFu, weight, 8 * m + pick + 1));
        const uint32_t dst = tmq + kColKeys + kb * kColKBuf;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          uint32_t hi[8], mid[8], lo[8];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t raw[4];
            ldmatrix_trans(raw, tile + tile_unit(t0 + lane, quarter / 8 + half * 2 + i));
#pragma unroll
            for (int m = 0; m < 4; ++m) {
              f32x2 x = mul2(w[m], pair(__uint_as_float(raw[m] << 16), __uint_as_float(raw[m] & 0xFFFF0000u)));
              hi[2 * m + i] = upper(x);
              x = rest(x);
              mid[2 * m + i] = upper(x);
              lo[2 * m + i] = upper(rest(x));
            }
          }
          if (half == 0) {
            if (step >= 1 && !(ok = warp_wait(&sm.kp_empty[kb], (step - 1) & 1, &sm.abort))) break;
            tc_fence_after();
          }
          tmem_st_16x16(dst + (half << 20), hi);
          tmem_st_16x16(dst + (half << 20) + 16, mid);
          tmem_st_16x16(dst + (half << 20) + 32, lo);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&sm.kp_full[kb]);
      }
      if (!ok) break;
      warp_arrive(&sm.g_empty[buf]);
      warp_arrive(&sm.empty[sk]);
    }
  }
  __syncthreads();
  // A wait gave up: the lanes of the items that were under way.  (No warp is more than one
  // item behind the copies, nor the copies behind the items' warp.)
  if (sm.abort && lane == 0 && (turn > 0 || warp == 3) && p.lane_status != nullptr)
    p.lane_status[it.b] = SPEC_ERR_TIMEOUT;
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tm, 512);
}

}  // namespace specv
