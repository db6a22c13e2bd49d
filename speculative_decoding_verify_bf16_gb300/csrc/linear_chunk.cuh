// linear_chunk.cuh -- linear attention with decay over prompts, a chunk of 128 tokens at
// a time on the tensor cores (bf16 activations, dk = dv = 128).
//
// With G_i the sum of the log decays of the chunk's tokens 0..i (base 2), S the state
// before the chunk and all sums over the chunk's tokens:
//
//   o_i = scale * ( 2^G_i  S^T q_i  +  sum_{j <= i} 2^(G_i - G_j) (q_i . k_j) v_j )
//   S'  = 2^G_last S + sum_j (2^(G_last - G_j) k_j) v_j^T
//
// One CTA walks the chunks of one (lane, head), or of a segment of them.  Its products:
//
//   QK  scores [token][token]  = q k^T
//   QS  D [token][dv]          = q S,     D rows then times 2^G_i
//   KV  U [dk][dv]             = k'^T v,  k' = 2^(G_last - G_j) k_j
//   PV  D                     += P v,     P = weighted scores, 0 above the diagonal
//
// S stays in fp32 in the registers of four warps from the first chunk to the last, and
// S' = 2^G_last S + U is formed there: the tensor cores truncate each addition to an
// accumulator, which into S itself cost ten times the precision of its fp32 sums.
// Operands are bf16, so fp32 numbers enter a product in parts: k' in three (all 24 bits),
// P and S in two (16 bits, far below the rounding of a bf16 output).  q, k and v are
// taken as they are.
//
// Tensor memory holds U (128 columns), scores and P (128; P overwrites the scores it came
// from), D (128) and two buffers of k' for 32 tokens (96).  Shared memory holds a ring of
// five 32 KB tiles (k, v, q of a chunk; 128-byte swizzled rows, so that a tile serves as
// an operand along either dimension) and S in two parts.
//
// Warps: 0 copies tiles, 1 issues the products, 2 sums the decays, and five groups of
// four do what lies between the products: scores to P (4-7), D (8-11), S (12-15), k' for
// every other 32 tokens (16-19 and 20-23).  The products of a chunk take 8 x 512 cycles on the tensor cores, its
// 128 KB of q, k, v and o about 5,500 at an SM's share of the HBM rate: the groups work
// beside each other so that the larger of the two counts.  A chunk's products go in the
// order KV (first half), QK, KV (second half), QS, PV: P is made beside the three after
// QK, the next S beside QS and PV, k' of the next tokens beside whatever is not KV.
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
constexpr int kRegsMisc = 64, kRegsScores = 72, kRegsOut = 64, kRegsState = 168, kRegsKey = 56;
constexpr int kChunkRegs = kRegsMisc + kRegsScores + kRegsOut + kRegsState + 2 * kRegsKey;
constexpr int kTile = 32 * 1024;      // 128 rows of 128 bf16: two halves of 64 columns
constexpr int kHalf = kTile / 2;
constexpr int kRing = 5;
constexpr uint32_t kColU = 0, kColP = 128, kColD = 256, kColK = 384;  // columns of tensor memory
constexpr uint32_t kColKBuf = 48;     // a k' buffer: three parts of 16 columns (32 tokens)
constexpr float kLog2eHi = 1.44269502f, kLog2eLo = 1.92596303e-8f;    // log2(e) in two parts
// A decay of 2^-160 is 0 in fp32 against everything a state can hold; the clamp keeps
// resets (-inf) and lowest values out of the sums.
constexpr float kDecayFloor = -160.f;

struct ChunkSmem {
  uint8_t ring[kRing][kTile];
  uint8_t s_hi[kTile];
  uint8_t s_lo[kTile];
  float g_hi[2][kChunk];  // -G in two parts, chunk c in c % 2
  float g_lo[2][kChunk];
  float to_end[4][32];    // the P group's warps: 2^(G at the end of 32 tokens - G_j)
  uint64_t full[kRing], empty[kRing];
  uint64_t g_full[2], g_empty[2];
  uint64_t scores_full, p_ready, qs_full, d_scaled, o_full, d_free, s_ready, kv_full, u_free, v_clean, o_staged, drain;
  uint64_t kp_full[2], kp_empty[2];
  uint32_t tmem;
  int abort;
  int status;             // the lane's status on entry
};

struct ChunkParams {
  LinearParams p;
  float* local;       // [segments][lanes][heads][128][128]: 0, the lanes' states before the
                      // call; r + 1, the state after segment r begun from zero
  float* local_decay; // [segments][lanes][heads]: whole decay of segment r
  int32_t segments;
};

// Waits for a phase; gives up after some seconds or when another warp has.  (Few
// instructions: the roles' code shares the instruction cache, and a warp that misses there
// holds up all that wait for it.)
constexpr uint32_t kPolls = 1u << 24;
__device__ __forceinline__ bool chunk_wait(uint64_t* bar, uint32_t parity, int* abort) {
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i)
    if (*static_cast<volatile int*>(abort) || i == kPolls) {
      *static_cast<volatile int*>(abort) = 1;
      return false;
    }
  return true;
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

// The chunks of a segment, and where they lie.
struct Segment {
  int b, h, seg, first, count;  // lane, head, segment, first row and rows of the lane
  int c0, c1;                   // chunks of the lane
  bool last;                    // the lane's last segment with rows
};

// STATES: only the states of all segments but the last, begun from zero (the first of
// two launches when a lane is split); otherwise outputs and final states.
template <bool STATES>
__global__ void __launch_bounds__(kChunkThreads, 1)
    linear_chunk_kernel(const ChunkParams cp, const __grid_constant__ CUtensorMap map_q,
                        const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                        const __grid_constant__ CUtensorMap map_out) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  ChunkSmem& sm = *reinterpret_cast<ChunkSmem*>(smem_raw);
  const LinearParams& p = cp.p;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  Segment sg;
  sg.h = blockIdx.x % p.v_heads;
  sg.b = blockIdx.x / p.v_heads % p.lanes;
  sg.seg = blockIdx.x / p.v_heads / p.lanes;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], 9);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.g_full[i], 1);
      mbar_init(&sm.g_empty[i], STATES ? 12 : 20);
      mbar_init(&sm.kp_full[i], 4);
      mbar_init(&sm.kp_empty[i], 1);
    }
    mbar_init(&sm.scores_full, 1);
    mbar_init(&sm.p_ready, 4);
    mbar_init(&sm.qs_full, 1);
    mbar_init(&sm.d_scaled, 4);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.d_free, 4);
    mbar_init(&sm.s_ready, 4);
    mbar_init(&sm.kv_full, 1);
    mbar_init(&sm.u_free, 4);
    mbar_init(&sm.v_clean, 4);
    mbar_init(&sm.o_staged, 4);
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
  // Read once: another head's CTA may write it meanwhile, and all warps must agree.
  if (threadIdx.x == 0) sm.status = p.lane_status == nullptr ? SPEC_OK : p.lane_status[sg.b];
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm.tmem;

  const int rc = linear_lane_rows(p, sg.b, sg.first, sg.count);
  const bool skip = rc != SPEC_OK || sm.status != SPEC_OK;
  const int chunks = (sg.count + kChunk - 1) / kChunk;
  const int per = (chunks + cp.segments - 1) / cp.segments;
  sg.c0 = min(chunks, sg.seg * per);
  sg.c1 = min(chunks, sg.c0 + per);
  sg.last = sg.c1 == chunks && (sg.c0 < chunks || sg.seg == 0);
  const bool active = !skip && sg.c0 < sg.c1 && !(STATES && sg.last);
  if (rc != SPEC_OK && threadIdx.x == 0 && p.lane_status != nullptr && sm.status == SPEC_OK) p.lane_status[sg.b] = rc;
  const int64_t head = static_cast<int64_t>(sg.b) * p.v_heads + sg.h;
  const int64_t heads = static_cast<int64_t>(p.lanes) * p.v_heads;
  const float* state_in =
      p.state_in == nullptr ? nullptr : p.state_in + sg.b * p.state_in_lane + sg.h * p.state_in_head;
  float* state_out =
      p.state_out == nullptr ? nullptr : p.state_out + sg.b * p.state_out_lane + sg.h * p.state_out_head;

  if (!STATES && !skip && chunks == 0 && sg.seg == 0 && state_out != nullptr) {  // an empty lane's state passes through
    for (int i = threadIdx.x; i < 128 * 128 / 4; i += kChunkThreads)
      reinterpret_cast<float4*>(state_out)[i] =
          state_in == nullptr ? make_float4(0.f, 0.f, 0.f, 0.f) : reinterpret_cast<const float4*>(state_in)[i];
  }

  // The last segment writes the final state while others may yet begin, and the two may
  // be one buffer: with segments the first launch keeps a copy of the initial state.
  if (STATES && !skip && sg.seg == 0 && state_in != nullptr) {
    for (int i = threadIdx.x; i < 128 * 128 / 4; i += kChunkThreads)
      reinterpret_cast<float4*>(cp.local + head * (128 * 128))[i] = reinterpret_cast<const float4*>(state_in)[i];
  }

  const uint32_t quarter = static_cast<uint32_t>(warp & 3) * 32;  // this warp's lanes of tensor memory
  const uint32_t row = quarter + lane;
  const uint32_t tmq = tm + (quarter << 16);
  const int n_chunks = active ? sg.c1 - sg.c0 : 0;
  constexpr int kLoads = STATES ? 2 : 3;  // tiles of a chunk: k, v (, q)

  if (warp < 4) registers_shrink<kRegsMisc>();
  if (warp == 0) {
    // ------------------------------------------------------------------ copies
    if (lane == 0) {
      int issued = 0;
      bool ok = true;
      for (int c = 0; c < n_chunks && ok; ++c) {
        const int z = sg.first + (sg.c0 + c) * kChunk;
#pragma unroll 1
        for (int j = 0; j < kLoads; ++j) {
          const int slot = issued % kRing, turn = issued / kRing;
          if (turn > 0 && !chunk_wait(&sm.empty[slot], (turn - 1) & 1, &sm.abort)) {
            ok = false;
            break;
          }
          const CUtensorMap* map = j == 0 ? &map_k : (j == 1 ? &map_v : &map_q);
          const int hh = j == 1 ? sg.h : sg.h / p.group;
          mbar_arrive_expect_tx(&sm.full[slot], kTile);
          tma_load_3d(sm.ring[slot], map, 0, hh, z, &sm.full[slot]);
          tma_load_3d(sm.ring[slot] + kHalf, map, 64, hh, z, &sm.full[slot]);
          ++issued;
        }
      }
      // Every copy lands before the CTA ends (also when a wait gave up).
      for (int i = max(0, issued - kRing); i < issued; ++i)
        mbar_wait_bounded(&sm.full[i % kRing], (i / kRing) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------------- products
    // What follows from a shuffle is the same in all lanes also to the compiler, which
    // then keeps loop counters and descriptors in uniform registers: a product is a few
    // instructions, issued well within the 64 cycles it takes.
    const uint32_t lead = elect_one();
    const int loops = __shfl_sync(0xFFFFFFFFu, n_chunks, 0);
    const int rows_left = __shfl_sync(0xFFFFFFFFu, sg.count - sg.c0 * kChunk, 0);
    const uint32_t tmu = __shfl_sync(0xFFFFFFFFu, tm, 0);
    constexpr uint32_t kSame = mma_desc(128, 128, false), kRows = mma_desc(128, 128, true);
    const uint32_t ring = smem_desc(smem_addr(sm.ring[0]), kHalf);  // (for K-major tiles the piece distance is not used)
    const uint32_t dlo = smem_desc(smem_addr(sm.s_lo), kHalf), dhi = smem_desc(smem_addr(sm.s_hi), kHalf);
    uint32_t kphase = 0;     // bit i: phase of k' buffer i
    int slot = 0, phase = 0; // the ring's slot of this chunk's k and its phase
    for (int c = 0; c < loops; ++c) {
      const uint32_t ph = c & 1;
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
      if (n < kChunk && !warp_wait(&sm.v_clean, 0, &sm.abort)) break;
      if (c > 0 && !warp_wait(&sm.u_free, ph ^ 1, &sm.abort)) break;
      bool ok = true;
#pragma unroll 1
      for (int t = 0; t < bufs || t == 2; ++t) {
        if (t == 2) {  // QK between the halves of KV (and behind a short chunk's)
          if (!STATES) {
            if (!(ok = warp_wait(&sm.full[sq], pq, &sm.abort) && warp_wait(&sm.full[sk], pk, &sm.abort))) break;
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
        const uint32_t kb = t & 1;
        if (!(ok = warp_wait(&sm.kp_full[kb], (kphase >> kb) & 1, &sm.abort))) break;
        tc_fence_after();
        const uint32_t parts = tmu + kColK + kb * kColKBuf, dvt = dv + t * (2 * 2048 / 16);
#pragma unroll
        for (int i = 0; i < 6; ++i)  // the least part first
          mma_ts(lead, tmu + kColU, parts + 32 - (i >> 1) * 16 + (i & 1) * 8, dvt + (i & 1) * (2048 / 16), kRows, i + t > 0);
        mma_commit(lead, &sm.kp_empty[kb]);
        kphase ^= 1u << kb;
        if (t == 0 && bufs == 1) t = 1;  // on to QK
      }
      if (!ok) break;
      mma_commit(lead, &sm.kv_full);
      if (!STATES) {
        if (!warp_wait(&sm.s_ready, ph, &sm.abort)) break;
        if (c > 0 && !warp_wait(&sm.d_free, ph ^ 1, &sm.abort)) break;
        tc_fence_after();
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const uint32_t ds = part == 0 ? dlo : dhi;
#pragma unroll
          for (int s = 0; s < 8; ++s)
            mma_ss(lead, tmu + kColD, dq + ((s >> 2) * kHalf + (s & 3) * 32) / 16, ds + s * (2048 / 16), kRows, part + s > 0);
        }
        mma_commit(lead, &sm.qs_full);
        if (!warp_wait(&sm.p_ready, ph, &sm.abort) || !warp_wait(&sm.d_scaled, ph, &sm.abort)) break;
        tc_fence_after();
#pragma unroll 1
        for (int t = 0; t < bufs; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mma_ts(lead, tmu + kColD, tmu + kColP + t * 32 + 16 - (i >> 1) * 16 + (i & 1) * 8,
                   dv + t * (2 * 2048 / 16) + (i & 1) * (2048 / 16), kRows, true);
        mma_commit(lead, &sm.o_full);
      }
      mma_commit(lead, &sm.empty[sv]);
      if (lead) mbar_arrive_n(&sm.empty[sv], 8);
    }
    // Tensor memory is given back only after the last product.
    mma_commit(lead, &sm.drain);
    mbar_wait_bounded(&sm.drain, 0);
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------------------ decays
    // Fixed point with 32 fractional bits: sums and differences are exact, whatever
    // large decays stand between two tokens.  32 tokens at a time, a lane each.
    auto fetch = [&](int t) {
      t += sg.c0 * kChunk + lane;
      return t < sg.count ? __ldg(p.log_decay + (sg.first + static_cast<int64_t>(t)) * p.decay_row + sg.h * p.decay_head)
                          : 0.f;
    };
    float next = n_chunks > 0 ? fetch(0) : 0.f;
    long long before = 0;
    float poison = 0.f;  // NaN once the chunk holds a NaN or a factor infinite in fp32
#pragma unroll 1
    for (int t = 0; t < n_chunks * kChunk; t += 32) {
      const int c = t / kChunk, buf = c & 1;
      const float g = next;
      if (t + 32 < n_chunks * kChunk) next = fetch(t + 32);
      if (t % kChunk == 0) {
        if (c >= 2 && !warp_wait(&sm.g_empty[buf], ((c >> 1) - 1) & 1, &sm.abort)) break;
        before = 0;
        poison = 0.f;
      }
      float hi = g * kLog2eHi;
      float lo = fmaf(g, kLog2eHi, -hi) + g * kLog2eLo;
      if (__any_sync(0xFFFFFFFFu, !(hi < 128.f))) poison = __uint_as_float(0x7FC00000u);
      if (!(hi > kDecayFloor)) {
        hi = kDecayFloor;
        lo = 0.f;
      }
      long long sum = __float2ll_rn(hi * 4294967296.f) + __float2ll_rn(lo * 4294967296.f);
#pragma unroll 1
      for (int d = 1; d < 32; d <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += up;
      }
      sum += before;
      before = __shfl_sync(0xFFFFFFFFu, sum, 31);
      hi = __ll2float_rn(sum);
      lo = __ll2float_rn(sum - __float2ll_rn(hi));
      sm.g_hi[buf][t % kChunk + lane] = fmaf(hi, -0x1p-32f, poison);
      sm.g_lo[buf][t % kChunk + lane] = lo * -0x1p-32f;
      if (t % kChunk == kChunk - 32) {
        // (every use of a chunk's sums takes in the last one, directly or by the state)
        __threadfence_block();
        warp_arrive(&sm.g_full[buf]);
      }
    }
  } else if (warp >= 4 && warp < 8) {
    // ------------------------------------------------------------- scores to P
    registers_shrink<kRegsScores>();
    if (!STATES) {
      for (int c = 0; c < n_chunks; ++c) {
        const int buf = c & 1;
        if (!warp_wait(&sm.g_full[buf], (c >> 1) & 1, &sm.abort)) break;
        const float ghi = -sm.g_hi[buf][row], glo = -sm.g_lo[buf][row];
        if (!warp_wait(&sm.scores_full, c & 1, &sm.abort)) break;
        tc_fence_after();
        float* const to_end = sm.to_end[warp - 4];
#pragma unroll 1
        for (int j0 = 0; j0 < kChunk; j0 += 32) {  // tokens j0 .. j0 + 31
          uint32_t hi[16], lo[16];
          if (j0 > static_cast<int>(quarter)) {  // all after this warp's rows
#pragma unroll
            for (int i = 0; i < 16; ++i) hi[i] = lo[i] = 0u;
          } else {
            uint32_t s[32];
            tmem_ld32(s, tmq + kColP + j0);
            if (j0 < static_cast<int>(quarter)) {
              // All before this warp's rows: 2^(G_i - G_j) in two factors, to the end of the
              // 32 tokens and from there, of which neither can overflow where the whole
              // does not.
              const float ehi = sm.g_hi[buf][j0 + 31], elo = sm.g_lo[buf][j0 + 31];
              const float from_end = ex2_approx((ghi + ehi) + (glo + elo));
              __syncwarp();
              to_end[lane] = ex2_approx((sm.g_hi[buf][j0 + lane] - ehi) + (sm.g_lo[buf][j0 + lane] - elo));
              __syncwarp();
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const ulonglong2 t = *reinterpret_cast<const ulonglong2*>(&to_end[i]);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  const f32x2 w = mul2(mul2(pair(from_end, from_end), e ? t.y : t.x),
                                       pair(__uint_as_float(s[i + e]), __uint_as_float(s[i + e + 1])));
                  hi[(i + e) / 2] = upper(w);
                  lo[(i + e) / 2] = rounded(rest(w));
                }
              }
            } else {
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                const ulonglong2 jh = *reinterpret_cast<const ulonglong2*>(&sm.g_hi[buf][j0 + i]);
                const ulonglong2 jl = *reinterpret_cast<const ulonglong2*>(&sm.g_lo[buf][j0 + i]);
#pragma unroll
                for (int e = 0; e < 4; e += 2) {
                  // (the arrays hold -G)
                  const f32x2 d = add2(add2(pair(ghi, ghi), e ? jh.y : jh.x), add2(pair(glo, glo), e ? jl.y : jl.x));
                  f32x2 w = mul2(pair(ex2_approx(first_of(d)), ex2_approx(second_of(d))),
                                 pair(__uint_as_float(s[i + e]), __uint_as_float(s[i + e + 1])));
                  // (a select: what is masked may be NaN)
                  w = pair(i + e > lane ? 0.f : first_of(w), i + e + 1 > lane ? 0.f : second_of(w));
                  hi[(i + e) / 2] = upper(w);
                  lo[(i + e) / 2] = rounded(rest(w));
                }
              }
            }
          }
          // Columns of P: for each 32 tokens 16 of upper and 16 of lower parts.
          tmem_st16(tmq + kColP + j0, hi);
          tmem_st16(tmq + kColP + j0 + 16, lo);
        }
        tmem_wait_st();
        tc_fence_before();
        warp_arrive(&sm.p_ready);
        warp_arrive(&sm.g_empty[buf]);
      }
    }
  } else if (warp >= 8 && warp < 12) {
    // ----------------------------------------------------------------- outputs
    registers_shrink<kRegsOut>();
    if (!STATES) {
      for (int c = 0; c < n_chunks; ++c) {
        const int buf = c & 1;
        if (!warp_wait(&sm.g_full[buf], (c >> 1) & 1, &sm.abort)) break;
        const float e = exp2f(-(sm.g_hi[buf][row] + sm.g_lo[buf][row]));
        warp_arrive(&sm.g_empty[buf]);
        if (!warp_wait(&sm.qs_full, c & 1, &sm.abort)) break;
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
        if (!warp_wait(&sm.o_full, c & 1, &sm.abort)) break;
        tc_fence_after();
        // The chunk's q has been read: its tile takes the outputs on their way out.
        const int slot = (kLoads * c + 2) % kRing;
        uint8_t* tile = sm.ring[slot];
        const int n = sg.count - (sg.c0 + c) * kChunk;
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
        if (n >= kChunk) {
          warp_arrive(&sm.o_staged);
          if (warp == 8) {
            if (!warp_wait(&sm.o_staged, c & 1, &sm.abort)) break;
            if (lane == 0) {
              const int z = sg.first + (sg.c0 + c) * kChunk;
              tma_store_3d(&map_out, tile, 0, sg.h, z);
              tma_store_3d(&map_out, tile + kHalf, 64, sg.h, z);
              bulk_commit_group();
              bulk_wait_group_read<0>();
              mbar_arrive_n(&sm.empty[slot], 9);
            }
            __syncwarp();
          }
        } else {  // (a copy would go on into the next lane's rows)
          __syncwarp();
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.out) + sg.h * p.out_head;
#pragma unroll 1
          for (int i = lane; i < 32 * 16; i += 32) {
            const int r = static_cast<int>(quarter) + i / 16;
            if (r < n)
              *reinterpret_cast<uint4*>(dst + (sg.first + (sg.c0 + c) * static_cast<int64_t>(kChunk) + r) * p.out_row + (i % 16) * 8) =
                  *reinterpret_cast<const uint4*>(tile + tile_unit(r, i % 16));
          }
        }
      }
      // (the last copies end before the CTA does)
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
    }
  } else if (warp >= 12 && warp < 16) {
    // ------------------------------------------------------------------ states
    registers_grow<kRegsState>();
    f32x2 S[64];  // row `row` of S
#pragma unroll
    for (int i = 0; i < 64; ++i) S[i] = 0ull;
    const int at = static_cast<int>(row) * 128;
    if (!STATES && n_chunks > 0) {
      // The state before the segment: the lane's, then every earlier segment's from
      // zero behind its decay.
      const float* begin = cp.segments > 1 ? cp.local + head * (128 * 128) : state_in;
      if (state_in != nullptr) {
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(begin + at + 2 * i));
          S[i] = pair(x.x, x.y);
          S[i + 1] = pair(x.z, x.w);
        }
      }
      for (int r = 0; r < sg.seg; ++r) {
        const float a = __ldcg(cp.local_decay + r * heads + head);
        const float* src = cp.local + ((r + 1) * heads + head) * (128 * 128) + at;
#pragma unroll
        for (int i = 0; i < 64; i += 2) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(src + 2 * i));
          S[i] = fma2(S[i], pair(a, a), pair(x.x, x.y));
          S[i + 1] = fma2(S[i + 1], pair(a, a), pair(x.z, x.w));
        }
      }
    }
    bool ok = true;
    float total = 1.f;  // the segment's whole decay
    for (int c = 0; c < n_chunks; ++c) {
      const int buf = c & 1;
      if (!STATES) {
        // S in two parts to shared memory for the chunk's QS, the last chunk's done.
        if (c > 0 && !(ok = warp_wait(&sm.qs_full, (c - 1) & 1, &sm.abort))) break;
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          const uint32_t unit = tile_unit(row, i / 4);
          *reinterpret_cast<uint4*>(sm.s_hi + unit) = make_uint4(upper(S[i]), upper(S[i + 1]), upper(S[i + 2]), upper(S[i + 3]));
          *reinterpret_cast<uint4*>(sm.s_lo + unit) = make_uint4(rounded(rest(S[i])), rounded(rest(S[i + 1])),
                                                                 rounded(rest(S[i + 2])), rounded(rest(S[i + 3])));
        }
        fence_async_smem();
        warp_arrive(&sm.s_ready);
      }
      if (!(ok = warp_wait(&sm.g_full[buf], (c >> 1) & 1, &sm.abort))) break;
      const float decay = exp2f(-(sm.g_hi[buf][kChunk - 1] + sm.g_lo[buf][kChunk - 1]));
      total *= decay;
      warp_arrive(&sm.g_empty[buf]);
      if (!(ok = warp_wait(&sm.kv_full, c & 1, &sm.abort))) break;
      tc_fence_after();
      uint32_t u[2][8];
      tmem_ld8(u[0], tmq + kColU);
#pragma unroll
      for (int piece = 0; piece < 16; ++piece) {
        tmem_wait_ld();
        if (piece < 15) tmem_ld8(u[(piece + 1) & 1], tmq + kColU + (piece + 1) * 8);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          S[piece * 4 + i] = fma2(S[piece * 4 + i], pair(decay, decay),
                                  pair(__uint_as_float(u[piece & 1][2 * i]), __uint_as_float(u[piece & 1][2 * i + 1])));
      }
      tc_fence_before();
      warp_arrive(&sm.u_free);
    }
    if (n_chunks > 0 && ok) {
      float* dst = STATES ? cp.local + ((sg.seg + 1) * heads + head) * (128 * 128) : (sg.last ? state_out : nullptr);
      if (STATES && row == 0) cp.local_decay[sg.seg * heads + head] = total;
      f32x2 bad = 0ull;  // 0 times S: NaN where S is not finite
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        bad = fma2(S[i], 0ull, fma2(S[i + 1], 0ull, bad));
        if (dst != nullptr)
          *reinterpret_cast<float4*>(dst + at + 2 * i) =
              make_float4(first_of(S[i]), second_of(S[i]), first_of(S[i + 1]), second_of(S[i + 1]));
      }
      if (!STATES && sg.last && first_of(bad) + second_of(bad) != 0.f && p.lane_status != nullptr) p.lane_status[sg.b] = SPEC_ERR_NONFINITE;
    }
  } else if (warp >= 16) {
    // ---------------------------------------------------------------------- k'
    // Lane i of k'^T is component i of k, along the tokens.  Transposing loads bring a
    // thread two tokens of one component, weighted pairs of which go out as they lie.
    registers_shrink<kRegsKey>();
    const int kb = (warp - 16) >> 2;  // this group's buffer of k'
    int step = 0;                     // times it has been filled
    bool ok = true;
    for (int c = 0; c < n_chunks && ok; ++c) {
      const int buf = c & 1;
      const int n = min(kChunk, sg.count - (sg.c0 + c) * kChunk);
      const int lk = kLoads * c, lv = lk + 1;
      if (!(ok = warp_wait(&sm.g_full[buf], (c >> 1) & 1, &sm.abort))) break;
      if (n < kChunk && kb == 0) {  // rows past the lane take part in products (times 0): make them 0
        if (!(ok = warp_wait(&sm.full[lv % kRing], (lv / kRing) & 1, &sm.abort))) break;
        uint8_t* vt = sm.ring[lv % kRing];
        if (static_cast<int>(row) >= n)
          for (uint32_t u = 0; u < 16; ++u)
            *reinterpret_cast<uint4*>(vt + tile_unit(row, u)) = make_uint4(0u, 0u, 0u, 0u);
        fence_async_smem();
        warp_arrive(&sm.v_clean);
      }
      const float last_hi = sm.g_hi[buf][kChunk - 1], last_lo = sm.g_lo[buf][kChunk - 1];
      if (!(ok = warp_wait(&sm.full[lk % kRing], (lk / kRing) & 1, &sm.abort))) break;
      const uint32_t tile = smem_addr(sm.ring[lk % kRing]);
      const int used = (n + 31) / 32;
      for (int t0 = kb * 32; t0 < used * 32; t0 += 64, ++step) {
        // Each lane has the weight of one of the 32 tokens.
        const float weight = exp2f((sm.g_hi[buf][t0 + lane] - last_hi) + (sm.g_lo[buf][t0 + lane] - last_lo));
        const int pick = 2 * (lane & 3);
        f32x2 w[4];
#pragma unroll
        for (int m = 0; m < 4; ++m)
          w[m] = pair(__shfl_sync(0xFFFFFFFFu, weight, 8 * m + pick), __shfl_sync(0xFFFFFFFFu, weight, 8 * m + pick + 1));
        const uint32_t dst = tmq + kColK + kb * kColKBuf;
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
              if (t0 + 32 > n)  // (rows past the lane may be NaN)
                x = pair(t0 + 8 * m + pick < n ? first_of(x) : 0.f, t0 + 8 * m + pick + 1 < n ? second_of(x) : 0.f);
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
      warp_arrive(&sm.empty[lk % kRing]);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && sm.abort && p.lane_status != nullptr) p.lane_status[sg.b] = SPEC_ERR_TIMEOUT;
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tm, 512);
}

}  // namespace specv
