// logprobs.cu -- log probabilities of given tokens, entropies and top alternatives:
// the C ABI of include/spec_logprobs.h.
//
// With z = x / T, m = max z, s = sum e^(z - m) and t = sum e^(z - m) (z - m):
//   log p(i) = z_i - m - log s,     entropy = log s - t / s.
// One pass over the row gives m, s and t (fp32, relative to the running maximum of a
// warp) and the largest logit of every block of 512.  The n likeliest tokens lie in the n
// blocks with the largest maxima (taken by maximum, then lower block: a block outside has
// n better tokens before it), so the alternatives cost the pass one maximum a block, and
// afterwards a second look at some n blocks, which L2 still holds.
//
// A row is one thread-block cluster's work; every CTA of it takes a contiguous range of
// blocks and hands its sums and block maxima to the first one through distributed shared
// memory.  The pass is bound by HBM, with the exponentials close behind (16 a cycle and
// SM).  Each warp streams for itself: bulk copies of up to 4 KB into its own ring of two
// slots, so that an SM keeps up to 192 KB on the way without holding registers for it
// and no barrier stands between warps.  Rows off 16-byte alignment take the same way, their
// copies from the last boundary before them.
//
// Measured (device time, bf16 rows, five alternatives and temperatures, nothing of them in
// L2): 576 rows of 262,144 at ragged temperatures with rows left out 41.5 us, where the bytes
// of those asked for take 26.0 at the measured copy rate; 64 of 151,936 with 20 alternatives
// 15.2 us, of which some 6 are the second look (the exchange, the selection, 20 blocks read
// again and sorted out: a chain of latencies that few rows leave exposed); one of 262,144
// 7.7 us; four of 1,024 in fp32 5.9 us.  576 fp32 rows of 151,937, none but the first aligned, are
// read at 5.5 TB/s (63 us), and in bf16 at 4.1 TB/s (43 us).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "device_ptx.cuh"
#include "spec_logprobs.h"
#include "tcgen05_ptx.cuh"

namespace {

using specv::add2;
using specv::bf16_hi;
using specv::bf16_lo;
using specv::cluster_arrive_relaxed;
using specv::cluster_ctarank;
using specv::cluster_map;
using specv::cluster_wait_acquire;
using specv::ex2_approx;
using specv::f32x2;
using specv::first_of;
using specv::fma2;
using specv::mul2;
using specv::pair;
using specv::second_of;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kCtasPerSm = 3;
constexpr int kBlock = 512;          // logits of a block: 16 a lane
constexpr int kPerLane = kBlock / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxGroups = 1024;     // block maxima one CTA keeps
static_assert(kMaxCluster * kMaxGroups <= 1 << 16, "groups are listed in 16 bits");
constexpr int kCandidates = 256;     // tokens the last selection holds
constexpr int kSlots = 2;            // a warp's ring
constexpr int kSlotBytes = 4096;
constexpr int kSlotStride = kSlotBytes + 16;  // (a row off 16-byte alignment starts inside a slot)
constexpr int kRingBytes = kWarps * kSlots * kSlotStride;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Exponents below this are 0 in fp32 (2^-126 is the smallest normal number and the
// exponential flushes); held there, a masked logit adds 0 * kLowExp to the entropy's sum
// and not 0 * (-inf).
constexpr float kLowExp = -140.f;
// Largest logits (times log2(e) / T) up to here take the plain form of the weights.
constexpr float kPlainExp = 0x1p22f;

struct Params {
  const uint8_t* logits;
  int64_t ld_bytes;
  int32_t V;
  const int32_t* tokens;
  const float* temps;
  float* logprobs;
  float* entropy;
  int32_t top;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* row_status;
  int32_t cluster;        // CTAs of a row
  int32_t subs_per_cta;   // blocks of 512 a CTA takes (a multiple of group)
  int32_t group;          // blocks that share one kept maximum, a power of two
  int32_t group_bits;     // its logarithm
  int32_t groups_total;   // kept maxima of a row
  int32_t chunk;          // blocks of one bulk copy
  int32_t test_withhold;  // tests only: the first row's first copy (1), or that of its second
                          // look (2), is announced but never issued
};

struct alignas(16) Sums {
  float m, s, t;  // largest logit, sum and weighted sum relative to it (log2 units)
  int status;
};

// A logit and where it stands: a token, or a group's largest.
struct alignas(8) Entry {
  float v;
  int i;
};
// Larger logits first, then lower indices (NaN comes before nothing).  (No || and &&: their
// branches diverge, and cost the search for a row's alternatives five times its time.)
__device__ __forceinline__ bool before(const Entry& a, const Entry& b) {
  return (a.v > b.v) | ((a.v == b.v) & (a.i < b.i));
}
constexpr int kNowhere = INT32_MAX;

// log p of logit v; -inf has probability 0 at an infinite temperature, too.
__device__ __forceinline__ float log_p(float v, float m, float T, float log_s) {
  return v > -INFINITY ? (v - m) / T - log_s : -INFINITY;
}

struct alignas(128) Head {
  union {
    Sums part[kMaxCluster * kWarps];
    Entry cand[kCandidates];  // (once the parts are summed)
  };
  alignas(16) Entry col[kWarps][32];
  alignas(16) Entry rank[kWarps][32];
  uint64_t full[kWarps][kSlots], again[kWarps];
  Sums all;
  float log_s;
  int nsel, ncand;
};

__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Places in a list for the lanes that want one; one atomic a warp.
__device__ __forceinline__ int reserve(int* total, bool want) {
  const uint32_t all = __ballot_sync(0xFFFFFFFFu, want);
  if (all == 0) return 0;
  int base = 0;
  if ((threadIdx.x & 31) == 0) base = atomicAdd(total, __popc(all));
  return __shfl_sync(0xFFFFFFFFu, base, 0) + __popc(all & ((1u << (threadIdx.x & 31)) - 1));
}

// This lane's 16 logits of block `sub`, as they are stored: element e of them is logit
// index_of(e) of the row.  Past the vocabulary: -inf.
template <bool BF16, bool VEC>
struct Block {
  static constexpr int kWords = BF16 ? kPerLane / 2 : kPerLane;
  static constexpr int kBytes = kBlock * (BF16 ? 2 : 4);
  static constexpr int kTogether = kSlotBytes / kBytes;
  uint32_t w[kWords];

  __device__ static __forceinline__ int64_t index_of(int sub, int lane, int e) {
    constexpr int n = VEC ? (BF16 ? 8 : 4) : 1;  // elements of a load
    return sub * static_cast<int64_t>(kBlock) + (e / n) * (32 * n) + lane * n + e % n;
  }
  __device__ static __forceinline__ float at(const uint8_t* row, int64_t i) {
    if (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[i]);
    return reinterpret_cast<const float*>(row)[i];
  }
  __device__ __forceinline__ float value(int e) const {
    if (!BF16) return __uint_as_float(w[e]);
    return e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
  }
  // A whole block from shared memory, 16-byte aligned if VEC.
  __device__ __forceinline__ void load_shared(const uint8_t* block, int lane) {
    if (VEC) {
#pragma unroll
      for (int j = 0; j < kWords / 4; ++j) {
        const uint4 u = *reinterpret_cast<const uint4*>(block + j * 512 + lane * 16);
        w[4 * j] = u.x;
        w[4 * j + 1] = u.y;
        w[4 * j + 2] = u.z;
        w[4 * j + 3] = u.w;
      }
    } else if (BF16) {
#pragma unroll
      for (int e = 0; e < kPerLane; e += 2)
        w[e / 2] = reinterpret_cast<const uint16_t*>(block)[e * 32 + lane] |
                   static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(block)[e * 32 + 32 + lane]) << 16;
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) w[e] = reinterpret_cast<const uint32_t*>(block)[e * 32 + lane];
    }
  }
  // A block that may end past the vocabulary, from the row itself.
  __device__ __forceinline__ void load(const uint8_t* row, int V, int sub, int lane) {
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const int64_t i = index_of(sub, lane, e);
      if (BF16) {
        const uint32_t x = i < V ? reinterpret_cast<const uint16_t*>(row)[i] : 0xFF80u;
        if (e % 2) w[e / 2] |= x << 16;
        else w[e / 2] = x;
      } else {
        w[e] = i < V ? reinterpret_cast<const uint32_t*>(row)[i] : 0xFF800000u;
      }
    }
  }
  // The largest, NaN if any is.
  __device__ __forceinline__ float top() const {
    if (BF16) {
      uint32_t m = w[0];
#pragma unroll
      for (int j = 1; j < kWords; ++j) m = specv::bf16x2_max_nan(m, w[j]);
      return specv::f32_max_nan(bf16_lo(m), bf16_hi(m));
    }
    float m = __uint_as_float(w[0]);
#pragma unroll
    for (int j = 1; j < kWords; ++j) m = specv::f32_max_nan(m, __uint_as_float(w[j]));
    return m;
  }
};

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) token_logprobs_kernel(const Params p) {
  using B = Block<BF16, VEC>;
  extern __shared__ __align__(128) uint8_t smem[];
  Head& hd = *reinterpret_cast<Head*>(smem);
  float* maxima = reinterpret_cast<float*>(smem + sizeof(Head));  // [groups_total], whole in the first CTA
  uint8_t* ring = smem + sizeof(Head) + (p.groups_total * 6 + 127) / 128 * 128;
  const uint32_t rank = p.cluster > 1 ? cluster_ctarank() : 0;
  const int r = blockIdx.x / p.cluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.cluster > 1) cluster_arrive_relaxed();
  if (lane == 0) {
    for (int i = 0; i < kSlots; ++i) specv::mbar_init(&hd.full[warp][i], 1);
    specv::mbar_init(&hd.again[warp], 1);
    specv::fence_mbar_init();
  }
  __syncwarp();
  specv::griddep_wait();
  specv::griddep_launch_dependents();

  const int tok = p.tokens[r];
  const bool asked = tok >= 0 && tok < p.V;
  const uint8_t* row = p.logits + r * p.ld_bytes;
  const float T = p.temps != nullptr && p.temps[r] > 0.f ? p.temps[r] : 1.f;
  const float c = fminf(kLog2e / T, FLT_MAX);
  const float given = asked && rank == 0 && threadIdx.x == kThreads - 32 ? B::at(row, tok) : 0.f;
  const int subs = (p.V - 1) / kBlock + 1;
  const int first = rank * p.subs_per_cta;
  const int last = min(subs, first + p.subs_per_cta);
  const int g0 = first >> p.group_bits;
  const int ngroups = last > first ? (last - first + p.group - 1) >> p.group_bits : 0;
  Sums acc{-INFINITY, 0.f, 0.f, SPEC_OK};
  if (asked) {
    float* mine = maxima + g0;  // kept at the same offsets in every CTA of the cluster
    if (p.group > 1) {
      for (int i = threadIdx.x; i < ngroups; i += kThreads) mine[i] = -INFINITY;
      __syncthreads();
    }
    f32x2 s2 = 0ull, t2 = 0ull;
    // Sums are relative to 2^ref (plain) or to 2^(c m): weights are 2^(c x - ref), where
    // ref = c m rounded once cancels in the end, or 2^((x - m) c).
    float ref = 0.f;
    bool plain = false;
    uint32_t low = 0;  // (plain) what is below it has weight 0
    auto keep = [&](float top, int sub) {  // block `sub`'s largest
      if (p.group == 1) {
        mine[sub - first] = top;
      } else {
        int* cell = reinterpret_cast<int*>(&mine[(sub - first) >> p.group_bits]);
        int old = *reinterpret_cast<volatile int*>(cell);
        while (__int_as_float(old) < top) {
          const int seen = atomicCAS(cell, old, __float_as_int(top));
          if (seen == old) break;
          old = seen;
        }
      }
    };
    // The running maximum raised to `top`; false where nothing counts.
    auto raise = [&](float top) {
      if (!(top < INFINITY)) acc.status = SPEC_ERR_NONFINITE;
      if (!(top > -INFINITY)) return false;
      if (top > acc.m) {
        const float next = top * c;
        // The plain form where ref's rounding (at most 2^-3, a factor of 1.1 on all weights) and
        // its bound on x are small numbers.  Otherwise (x - m) c, every exponent clamped: with
        // logits around 1e9, or divided by a small temperature, the rounding of ref would be an
        // exponent of hundreds.
        const float at = (next + kLowExp) / c;
        const bool was = plain;
        plain = fabsf(next) < kPlainExp && at > -0x1p126f;
        if (acc.m > -INFINITY) {
          // From the old reference to the new one, each as exact as it is.
          const float to = plain ? (was ? ref - next : fmaf(acc.m, c, -next)) : was ? fmaf(-top, c, ref) : (acc.m - top) * c;
          const float d = fmaxf(to, kLowExp), f = ex2_approx(d);
          t2 = mul2(pair(f, f), fma2(s2, pair(d, d), t2));
          s2 = mul2(pair(f, f), s2);
        }
        ref = next;
        acc.m = top;
        if (BF16) {
          low = __bfloat16_as_ushort(__float2bfloat16_rd(at));
          low |= low << 16;
        }
      }
      return true;
    };
    auto add = [&](const B& x) {
      const f32x2 c2 = pair(c, c);
      if (plain) {
        const f32x2 r2 = pair(-ref, -ref);
#pragma unroll
        for (int e = 0; e < kPerLane; e += 2) {
          f32x2 a;
          if (BF16) {
            const uint32_t w = specv::bf16x2_max_nan(x.w[e / 2], low);
            a = fma2(pair(bf16_lo(w), bf16_hi(w)), c2, r2);
          } else {
            a = fma2(pair(x.value(e), x.value(e + 1)), c2, r2);
            a = pair(fmaxf(first_of(a), kLowExp), fmaxf(second_of(a), kLowExp));
          }
          const f32x2 w = pair(ex2_approx(first_of(a)), ex2_approx(second_of(a)));
          s2 = add2(s2, w);
          t2 = fma2(w, a, t2);
        }
      } else {
        const f32x2 m2 = pair(-acc.m, -acc.m);
#pragma unroll
        for (int e = 0; e < kPerLane; e += 2) {
          f32x2 a = mul2(add2(pair(x.value(e), x.value(e + 1)), m2), c2);
          a = pair(fmaxf(first_of(a), kLowExp), fmaxf(second_of(a), kLowExp));
          const f32x2 w = pair(ex2_approx(first_of(a)), ex2_approx(second_of(a)));
          s2 = add2(s2, w);
          t2 = fma2(w, a, t2);
        }
      }
    };
    auto take = [&](const B& x, int sub) {
      const float top = warp_max_nan(x.top());
      if (lane == 0) keep(top, sub);
      if (raise(top)) add(x);
    };
    // Whole blocks through the ring, `chunk` of them a copy, the warps in turn.  Copies take
    // whole pieces of 16 aligned bytes: those of a row that starts inside such a piece begin
    // with it.  (Every piece holds a byte of the row, so that it lies in the same memory page.)
    uint8_t* slots = ring + warp * (kSlots * kSlotStride);
    const uint32_t shift = VEC ? 0u : static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row) & 15u);
    const int whole = min(last, p.V / kBlock);
    const int step = kWarps * p.chunk;
    auto issue = [&](int sub, int slot) {
      if (lane == 0 && sub < whole) {
        const uint32_t bytes = (shift + min(p.chunk, whole - sub) * B::kBytes + 15u) & ~15u;
        specv::mbar_arrive_expect_tx(&hd.full[warp][slot], bytes);
        if (!(p.test_withhold == 1 && blockIdx.x == 0 && sub == 0))
          specv::bulk_g2s(slots + slot * kSlotStride, row - shift + sub * static_cast<int64_t>(B::kBytes), bytes,
                          &hd.full[warp][slot]);
      }
    };
    int sub = first + warp * p.chunk;  // (blocks, at most 2^22 of them)
    for (int i = 0; i < kSlots; ++i) issue(sub + i * step, i);
    int slot = 0, phase = 0;
    for (; sub < whole; sub += step) {
      if (!specv::mbar_wait_bounded(&hd.full[warp][slot], phase)) {
        acc.status = SPEC_ERR_TIMEOUT;  // (what is on the way still lands before the CTA ends)
        for (int i = 0; i < kSlots && sub + i * step < whole; ++i) {
          specv::mbar_wait_bounded(&hd.full[warp][slot], phase);
          if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
          }
        }
        break;
      }
      const int n = min(p.chunk, whole - sub);
      const uint8_t* src = slots + slot * kSlotStride + shift;
      // A slot's blocks at once: their latencies overlap.  (Not where bf16 logits come two
      // bytes a load, whose addresses and halves spill: 576 x 151,937 89 us so, 43 one by one.)
      if ((VEC || !BF16) && n == B::kTogether) {
        B x[B::kTogether];
        float top[B::kTogether], most = -INFINITY, own = 0.f;
#pragma unroll
        for (int i = 0; i < B::kTogether; ++i) x[i].load_shared(src + i * B::kBytes, lane);
#pragma unroll
        for (int i = 0; i < B::kTogether; ++i) {
          top[i] = warp_max_nan(x[i].top());
          most = specv::f32_max_nan(most, top[i]);
          own = lane == i ? top[i] : own;
        }
        if (lane < B::kTogether) keep(own, sub + lane);
        if (raise(most)) {
#pragma unroll
          for (int i = 0; i < B::kTogether; ++i) add(x[i]);
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < n; ++i) {
          B x;
          x.load_shared(src + i * B::kBytes, lane);
          take(x, sub + i);
        }
      }
      __syncwarp();
      issue(sub + kSlots * step, slot);
      if (++slot == kSlots) {
        slot = 0;
        phase ^= 1;
      }
    }
    if (first < last && whole < last && warp == 0) {  // the row's last, partial block (a CTA may have none)
      B x;
      x.load(row, p.V, whole, lane);
      take(x, whole);
    }
    // The maximum is the warp's, so the lanes' sums add directly.
    acc.s = first_of(s2) + second_of(s2);
    acc.t = first_of(t2) + second_of(t2);
    if (plain) {  // handed on as sums of 2^(c (x - m)): ref is c m but for this rounding
      const float d = fmaf(-acc.m, c, ref), f = ex2_approx(d);
      acc.t = f * fmaf(acc.s, d, acc.t);
      acc.s *= f;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      acc.s += __shfl_xor_sync(0xFFFFFFFFu, acc.s, d);
      acc.t += __shfl_xor_sync(0xFFFFFFFFu, acc.t, d);
      acc.status = max(acc.status, __shfl_xor_sync(0xFFFFFFFFu, acc.status, d));
    }
  }
  if (p.cluster > 1) {
    cluster_wait_acquire();  // every CTA of the cluster has started
    if (asked && rank != 0) {
      __syncthreads();
      const uint32_t dst = cluster_map(maxima + g0, 0);
      for (int i = threadIdx.x; i < ngroups; i += kThreads)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 4 * i), "f"(maxima[g0 + i]) : "memory");
      if (lane == 0) {
        const uint32_t s = cluster_map(&hd.part[rank * kWarps + warp], 0);
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(s), "r"(__float_as_uint(acc.m)),
                     "r"(__float_as_uint(acc.s)), "r"(__float_as_uint(acc.t)), "r"(acc.status)
                     : "memory");
      }
    }
    if (rank == 0 && lane == 0) hd.part[warp] = acc;
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    if (rank != 0) return;  // (the first CTA waits for those that have not ended)
    cluster_wait_acquire();
  } else {
    if (lane == 0) hd.part[warp] = acc;
    __syncthreads();
  }
  const int n = p.top;
  int32_t* ids = p.top_ids + static_cast<int64_t>(r) * n;
  float* lps = p.top_logprobs + static_cast<int64_t>(r) * n;
  if (!asked) {
    const float none = tok < 0 ? 0.f : NAN;
    if (threadIdx.x == 0) {
      p.logprobs[r] = none;
      if (p.entropy != nullptr) p.entropy[r] = none;
      if (p.row_status != nullptr) p.row_status[r] = tok < 0 ? SPEC_OK : SPEC_ERR_TOKEN_RANGE;
    }
    if (threadIdx.x < n) {
      ids[threadIdx.x] = -1;
      lps[threadIdx.x] = none;
    }
    return;
  }
  // The last warp sums up while the others look for the alternatives' groups.
  if (threadIdx.x == 0) hd.nsel = hd.ncand = 0;
  Entry best{-INFINITY, kNowhere};
  if (n > 0) {  // the groups are dealt to 32 columns: this thread's part of its column's best
    for (int i = threadIdx.x; i < p.groups_total; i += kThreads) {
      const Entry x{maxima[i], i};
      if (before(x, best)) best = x;
    }
    hd.col[warp][lane] = best;
    __syncthreads();
  }
  // The n-th of the 32 columns' best: a lower bound of the n-th best of all, since n are no
  // worse.  A warp finds it for itself (col is filled, a barrier behind).
  auto bound = [&] {
    Entry v = hd.col[0][lane];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      const Entry x = hd.col[w][lane];
      const bool b = before(x, v);
      v.v = b ? x.v : v.v;
      v.i = b ? x.i : v.i;
    }
    Entry* const mine = hd.rank[warp];
    mine[lane] = v;
    __syncwarp();
    int pos = 0;
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      const float4 o = *reinterpret_cast<const float4*>(&mine[j]);
      const int i0 = __float_as_int(o.y), i1 = __float_as_int(o.w);
      // (columns without entries are alike)
      pos += (o.x > v.v) | ((o.x == v.v) & ((i0 < v.i) | ((i0 == v.i) & (j < lane))));
      pos += (o.z > v.v) | ((o.z == v.v) & ((i1 < v.i) | ((i1 == v.i) & (j + 1 < lane))));
    }
    __syncwarp();
    return mine[__ffs(__ballot_sync(0xFFFFFFFFu, pos == n - 1)) - 1];
  };
  uint16_t* const sel = reinterpret_cast<uint16_t*>(maxima + p.groups_total);
  Entry thr{0.f, 0};
  if (warp == kWarps - 1) {
    const int parts = p.cluster * kWarps;
    Sums a{-INFINITY, 0.f, 0.f, SPEC_OK};
    float m = -INFINITY;
    for (int i = lane; i < parts; i += 32) m = fmaxf(m, hd.part[i].m);
    a.m = specv::warp_max_f32(m);
    for (int i = lane; i < parts; i += 32) {
      const Sums x = hd.part[i];
      a.status = max(a.status, x.status);
      if (!(x.s == 0.f)) {  // (a NaN fails the row)
        const float d = fmaxf((x.m - a.m) * c, kLowExp), f = ex2_approx(d);
        a.s = fmaf(x.s, f, a.s);
        a.t = fmaf(f, fmaf(x.s, d, x.t), a.t);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      a.s += __shfl_xor_sync(0xFFFFFFFFu, a.s, d);
      a.t += __shfl_xor_sync(0xFFFFFFFFu, a.t, d);
    }
    a.status = __reduce_max_sync(0xFFFFFFFFu, a.status);
    if (a.status == SPEC_OK && !(a.s > 0.f)) a.status = SPEC_ERR_NONFINITE;
    const float log_s = logf(a.s);
    if (lane == 0) {
      hd.all = a;
      hd.log_s = log_s;
      const bool ok = a.status == SPEC_OK;
      p.logprobs[r] = ok ? log_p(given, a.m, T, log_s) : NAN;
      if (p.entropy != nullptr) p.entropy[r] = ok ? log_s - (a.t / a.s) * kLn2 : NAN;
      if (p.row_status != nullptr) p.row_status[r] = a.status;
    }
    if (n == 0) return;
  } else {
    if (n == 0) return;
    thr = bound();
    for (int i0 = 0; i0 < p.groups_total; i0 += kThreads - 32) {
      const int i = i0 + threadIdx.x;
      const bool want = i < p.groups_total && !before(thr, Entry{maxima[i], i});
      const int at = reserve(&hd.nsel, want);
      if (want) sel[at] = static_cast<uint16_t>(i);
    }
  }
  __syncthreads();
  const Sums all = hd.all;
  const float log_s = hd.log_s;
  if (all.status != SPEC_OK) {
    if (threadIdx.x < n) {
      ids[threadIdx.x] = -1;
      lps[threadIdx.x] = NAN;
    }
    return;
  }
  // The selected groups' blocks, each warp some of them, by way of its part of the ring (in
  // several batches if need be): f(block, where it lies).
  using S = Block<BF16, true>;  // (as they lie in the ring)
  const int nblocks = hd.nsel * p.group;
  constexpr int kHeld = kSlots * kSlotBytes / S::kBytes;
  uint8_t* const held = ring + warp * (kSlots * kSlotStride);
  int staged = -1, batch = 0;
  bool late = false;  // a copy did not come
  auto blocks = [&](auto f) {
    for (int i0 = warp; i0 < nblocks && !late; i0 += kWarps * kHeld) {
      auto block = [&](int j) {  // the j-th block of the batch, or one past the row
        const int i = i0 + j * kWarps;
        return i < nblocks ? (sel[i >> p.group_bits] << p.group_bits) + (i & (p.group - 1)) : subs;
      };
      if (staged != i0) {
        if (staged >= 0) specv::fence_async_smem();  // (plain stores may have filled what copies fill now)
        __syncwarp();
        staged = i0;
        uint32_t bytes = 0;
#pragma unroll 1
        for (int j = 0; j < kHeld; ++j) {
          const int sub = block(j);
          if (sub >= subs) continue;
          uint8_t* dst = held + j * S::kBytes;
          if (VEC && (sub + 1) * static_cast<int64_t>(kBlock) <= p.V) {
            bytes += S::kBytes;
          } else {  // NaN past the vocabulary
#pragma unroll 4
            for (int e = lane; e < kBlock; e += 32) {
              const int64_t id = sub * static_cast<int64_t>(kBlock) + e;
              if (BF16) reinterpret_cast<uint16_t*>(dst)[e] = id < p.V ? reinterpret_cast<const uint16_t*>(row)[id] : 0x7FC0u;
              else reinterpret_cast<uint32_t*>(dst)[e] = id < p.V ? reinterpret_cast<const uint32_t*>(row)[id] : 0x7FC00000u;
            }
          }
        }
        if (VEC && bytes > 0) {
          if (lane == 0) {
            specv::mbar_arrive_expect_tx(&hd.again[warp], bytes);
#pragma unroll 1
            for (int j = 0; j < kHeld; ++j) {
              const int sub = block(j);
              if (sub < subs && (sub + 1) * static_cast<int64_t>(kBlock) <= p.V &&
                  !(p.test_withhold == 2 && blockIdx.x == 0 && warp + batch + j == 0))
                specv::bulk_g2s(held + j * S::kBytes, row + sub * static_cast<int64_t>(S::kBytes), S::kBytes, &hd.again[warp]);
            }
          }
          late = !__all_sync(0xFFFFFFFFu, specv::mbar_wait_bounded(&hd.again[warp], batch & 1));
          if (late) {  // (what is on the way still lands before the CTA ends)
            specv::mbar_wait_bounded(&hd.again[warp], batch & 1);
            break;
          }
          ++batch;
        }
        __syncwarp();
      }
#pragma unroll 1
      for (int j = 0; j < kHeld; ++j) {
        const int sub = block(j);
        if (sub >= subs) continue;
        S x;
        x.load_shared(held + j * S::kBytes, lane);
        f(x, sub, held + j * S::kBytes);
      }
    }
  };
  // A barrier; the row fails as a whole where a copy did not come.
  auto gave_up = [&] {
    if (!__syncthreads_or(late)) return false;
    if (threadIdx.x == 0) {
      p.logprobs[r] = NAN;
      if (p.entropy != nullptr) p.entropy[r] = NAN;
      if (p.row_status != nullptr) p.row_status[r] = SPEC_ERR_TIMEOUT;
    }
    if (threadIdx.x < n) {
      ids[threadIdx.x] = -1;
      lps[threadIdx.x] = NAN;
    }
    return true;
  };
  // Once more the n-th of 32 columns, now of tokens, then all that are no worse.
  best = Entry{-INFINITY, kNowhere};
  blocks([&](const S& x, int sub, const uint8_t*) {
    float v = x.value(0);
    int at = 0;
#pragma unroll
    for (int e = 1; e < kPerLane; ++e) {  // (in the order of the tokens: the first of equals stays)
      const bool b = x.value(e) > v;  // (NaN, past the vocabulary, never is)
      v = b ? x.value(e) : v;
      at = b ? e : at;
    }
    const Entry k{v, static_cast<int>(S::index_of(sub, lane, at))};
    if (before(k, best)) best = k;
  });
  hd.col[warp][lane] = best;  // (a barrier after the groups' columns were read)
  if (gave_up()) return;
  const Entry low = bound();
  blocks([&](const S& x, int sub, const uint8_t* lies) {
    uint32_t mask = 0;
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) mask |= static_cast<uint32_t>(x.value(e) >= low.v) << e;
    while (mask != 0) {
      const int e = __ffs(mask) - 1;
      mask &= mask - 1;
      const int64_t id = S::index_of(sub, lane, e);
      const Entry k{B::at(lies, id - sub * static_cast<int64_t>(kBlock)), static_cast<int>(id)};
      if (before(low, k)) continue;
      const int at = atomicAdd(&hd.ncand, 1);
      if (at < kCandidates) hd.cand[at] = k;
    }
  });
  if (gave_up()) return;
  const int ncand = hd.ncand;
  auto emit = [&](int pos, const Entry& k) {
    ids[pos] = k.i;
    lps[pos] = log_p(k.v, all.m, T, log_s);
  };
  if (ncand <= kCandidates) {
    for (int i = threadIdx.x; i < ncand; i += kThreads) {
      const Entry k = hd.cand[i];
      int pos = 0;
#pragma unroll 4
      for (int j = 0; j < ncand; ++j) pos += before(hd.cand[j], k);
      if (pos < n) emit(pos, k);
    }
    if (threadIdx.x < n && threadIdx.x >= ncand) {
      ids[threadIdx.x] = -1;
      lps[threadIdx.x] = -INFINITY;
    }
    return;
  }
  // The best tokens crowd in few columns: one after the other, the best behind the last.
  Entry done{INFINITY, -1};
  for (int pos = 0; pos < n; ++pos) {
    Entry v{-INFINITY, kNowhere};
    blocks([&](const S&, int sub, const uint8_t*) {
#pragma unroll 1
      for (int e = 0; e < kBlock; e += 32) {  // (from memory: little code for what is rare)
        const int64_t id = sub * static_cast<int64_t>(kBlock) + e + lane;
        const Entry k{id < p.V ? B::at(row, id) : NAN, static_cast<int>(id)};
        if (before(done, k) && before(k, v)) v = k;
      }
    });
    const float wv = specv::warp_max_f32(v.v);
    const int wi = __reduce_min_sync(0xFFFFFFFFu, v.v == wv ? v.i : kNowhere);
    if (lane == 0) hd.col[warp][0] = Entry{wv, wi};
    if (gave_up()) return;
    done = hd.col[0][0];
    for (int w = 1; w < kWarps; ++w)
      if (before(hd.col[w][0], done)) done = hd.col[w][0];
    __syncthreads();
    if (threadIdx.x == 0) emit(pos, done);
  }
}

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
int g_sms[kMaxDevices] = {};
bool g_attr[kMaxDevices][4] = {};

constexpr int64_t round_up(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Dynamic shared memory: head, block maxima and the list of those selected, ring.
int64_t smem_bytes(int64_t groups) { return sizeof(Head) + round_up(groups * 6, 128) + kRingBytes; }

}  // namespace

extern "C" int spec_token_logprobs(const spec_logprobs_args* a, void* stream) {
  if (a == nullptr || a->rows < 0 || a->V <= 0 || a->ld < a->V || a->top < 0 || a->top > SPEC_LOGPROBS_MAX_TOP)
    return SPEC_ERR_INVALID_ARG;
  if (a->dtype != SPEC_F32 && a->dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (a->rows == 0) return SPEC_OK;
  if (a->logits == nullptr || a->tokens == nullptr || a->logprobs == nullptr) return SPEC_ERR_INVALID_ARG;
  if (a->top > 0 && (a->top_ids == nullptr || a->top_logprobs == nullptr)) return SPEC_ERR_INVALID_ARG;
  if (static_cast<int64_t>(a->rows) * kMaxCluster > INT32_MAX) return SPEC_ERR_INVALID_ARG;

  void* const kernels[4] = {reinterpret_cast<void*>(&token_logprobs_kernel<false, false>),
                            reinterpret_cast<void*>(&token_logprobs_kernel<false, true>),
                            reinterpret_cast<void*>(&token_logprobs_kernel<true, false>),
                            reinterpret_cast<void*>(&token_logprobs_kernel<true, true>)};
  const int esize = a->dtype == SPEC_BF16 ? 2 : 4;
  const bool vec = (reinterpret_cast<uintptr_t>(a->logits) & 15u) == 0 && (a->ld * esize) % 16 == 0;
  const int which = (a->dtype == SPEC_BF16 ? 2 : 0) + (vec ? 1 : 0);

  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return SPEC_ERR_CUDA;
  int sms;
  {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (g_sms[dev] == 0 &&
        cudaDeviceGetAttribute(&g_sms[dev], cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return SPEC_ERR_CUDA;
    sms = g_sms[dev];
    if (!g_attr[dev][which]) {
      if (cudaFuncSetAttribute(kernels[which], cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess ||
          cudaFuncSetAttribute(kernels[which], cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(smem_bytes(kMaxCluster * kMaxGroups))) != cudaSuccess) {
        cudaGetLastError();
        return SPEC_ERR_CUDA;
      }
      g_attr[dev][which] = true;
    }
  }
  const int subs = (a->V - 1) / kBlock + 1;
  // CTAs for most SMs, each with a block of 512 a warp at least.  More of them a row cost more
  // than they bring, by their start and the exchange: 64 rows of 151,936 take 18.5, 15.0,
  // 17.4 and 20.0 us with 1, 2, 4 and 8, a single row of 262,144 20.6 with one and 7.8 with 16.
  int cluster = 1;
  while (cluster < kMaxCluster && 4 * static_cast<int64_t>(a->rows) * cluster < 3 * sms && subs > cluster * kWarps)
    cluster *= 2;
  int group = 1;
  int per = (subs + cluster - 1) / cluster;
  while ((per + group - 1) / group > kMaxGroups) group *= 2;
  per = static_cast<int>(round_up(per, group));

  Params p{};
  p.logits = static_cast<const uint8_t*>(a->logits);
  p.ld_bytes = a->ld * esize;
  p.V = a->V;
  p.tokens = a->tokens;
  p.temps = a->temperatures;
  p.logprobs = a->logprobs;
  p.entropy = a->entropy;
  p.top = a->top;
  p.top_ids = a->top_ids;
  p.top_logprobs = a->top_logprobs;
  p.row_status = a->row_status;
  p.cluster = cluster;
  p.subs_per_cta = per;
  p.group = group;
  while ((1 << p.group_bits) < group) ++p.group_bits;
  p.groups_total = (subs + group - 1) / group;
  // Copies as large as a slot, or as leave every warp one.
  const int most = kSlotBytes / (kBlock * esize), share = (per + kWarps - 1) / kWarps;
  p.chunk = share < most ? share : most;

  const char* withhold = std::getenv("SPEC_LOGPROBS_TEST_WITHHOLD_COPY");
  p.test_withhold = withhold != nullptr ? std::atoi(withhold) : 0;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a->rows) * cluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem_bytes(p.groups_total));
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void* args[] = {&p};
  if (cudaLaunchKernelExC(&cfg, kernels[which], args) != cudaSuccess) {
    cudaGetLastError();
    return SPEC_ERR_CUDA;
  }
  return SPEC_OK;
}
