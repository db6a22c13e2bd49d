// logprobs.cu -- log probabilities of given tokens, entropies and top alternatives:
// the C ABI of include/spec_logprobs.h.
//
// With z = x / T, m = max z, s = sum e^(z - m) and t = sum e^(z - m) (z - m):
//   log p(i) = z_i - m - log s,     entropy = log s - t / s.
// One pass over the row gives m, s and t and the largest logit of every block of
// 512.  The n likeliest tokens lie in the n blocks with the largest maxima (taken
// by maximum, then lower block: a block outside has n better tokens before it), so
// the alternatives cost the pass one maximum a block, and afterwards a second look at
// some n blocks, which L2 still holds.
//
// A row is one thread-block cluster's work; every CTA of it takes a contiguous range
// of blocks and hands its sums and block maxima to the first one through distributed
// shared memory.  The pass is bound by HBM; 512 elements of a warp are two or four
// 16-byte loads a lane.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <mutex>

#include "device_ptx.cuh"
#include "spec_logprobs.h"

namespace {

using specv::bf16_hi;
using specv::bf16_lo;
using specv::cluster_arrive_relaxed;
using specv::cluster_ctarank;
using specv::cluster_map;
using specv::cluster_wait_acquire;
using specv::ex2_approx;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBlock = 512;          // logits of a block: 16 a lane
constexpr int kPerLane = kBlock / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxGroups = 1024;     // block maxima one CTA keeps
constexpr int kCandidates = 1024;    // tokens the last selection holds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// Exponents below this are 0 in fp32 (2^-126 is the smallest normal number and the
// exponential flushes): weights that far down are dropped, which also keeps
// 0 * (-inf) out of the entropy's sum.
constexpr float kLowExp = -140.f;

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
  int32_t group;          // blocks that share one kept maximum
  int32_t groups_total;   // kept maxima of a row
};

struct Sums {
  float m, s, t;  // largest logit, sum and weighted sum relative to it (log2 units)
  int bad;        // a NaN or +inf was seen
};

struct Head {
  Sums part[kMaxCluster];
  Sums warp[kWarps];
  float col_max[kWarps][32];
  int col_idx[kWarps][32];
  float thr;
  int thr_idx;
  int nsel, ncand;
  unsigned long long best[kWarps];
  float cand_val[kCandidates];
  int cand_idx[kCandidates];
};

// (a, i) before (b, j): larger value, then lower index.
__device__ __forceinline__ bool before(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Merge partial sums: both relative to their own maximum, c = log2(e) / T.
__device__ __forceinline__ Sums merge(const Sums& a, const Sums& b, float c) {
  Sums r;
  r.bad = a.bad | b.bad;
  r.m = fmaxf(a.m, b.m);
  r.s = r.t = 0.f;
  if (a.s > 0.f) {
    const float d = fmaxf((a.m - r.m) * c, kLowExp), f = ex2_approx(d);
    r.s += a.s * f;
    r.t += f * fmaf(a.s, d, a.t);
  }
  if (b.s > 0.f) {
    const float d = fmaxf((b.m - r.m) * c, kLowExp), f = ex2_approx(d);
    r.s += b.s * f;
    r.t += f * fmaf(b.s, d, b.t);
  }
  return r;
}

// The 16 logits of this lane of block `sub`: element e of them is logit
// index_of(e) of the row.  Past the vocabulary: -inf.
template <bool BF16, bool VEC>
struct Block {
  __device__ static __forceinline__ int64_t index_of(int sub, int lane, int e) {
    constexpr int w = VEC ? (BF16 ? 8 : 4) : 1;  // elements of a load
    return sub * static_cast<int64_t>(kBlock) + (e / w) * (32 * w) + lane * w + e % w;
  }
  __device__ static __forceinline__ float at(const uint8_t* row, int64_t i) {
    if (BF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(row)[i]);
    return reinterpret_cast<const float*>(row)[i];
  }
  __device__ static __forceinline__ void load(const uint8_t* row, int V, int sub, int lane, float (&x)[kPerLane]) {
    if (VEC && (sub + 1) * static_cast<int64_t>(kBlock) <= V) {
      constexpr int w = BF16 ? 8 : 4;
      constexpr int size = BF16 ? 2 : 4;
#pragma unroll
      for (int j = 0; j < kPerLane / w; ++j) {
        const uint4 u = __ldg(reinterpret_cast<const uint4*>(
            row + (static_cast<int64_t>(sub) * kBlock + j * (32 * w) + lane * w) * size));
        const uint32_t word[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if (BF16) {
            x[j * w + 2 * e] = bf16_lo(word[e]);
            x[j * w + 2 * e + 1] = bf16_hi(word[e]);
          } else {
            x[j * w + e] = __uint_as_float(word[e]);
          }
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        const int64_t i = index_of(sub, lane, e);
        x[e] = i < V ? at(row, i) : -INFINITY;
      }
    }
  }
};

template <bool BF16, bool VEC>
__global__ void __launch_bounds__(kThreads) token_logprobs_kernel(const Params p) {
  using B = Block<BF16, VEC>;
  extern __shared__ __align__(16) uint8_t smem[];
  Head& hd = *reinterpret_cast<Head*>(smem);
  float* maxima = reinterpret_cast<float*>(smem + sizeof(Head));       // [groups_total], the first CTA's
  int* sel = reinterpret_cast<int*>(maxima + p.groups_total);          // [groups_total]
  const uint32_t rank = p.cluster > 1 ? cluster_ctarank() : 0;
  const int r = blockIdx.x / p.cluster;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.cluster > 1) cluster_arrive_relaxed();
  specv::griddep_wait();
  specv::griddep_launch_dependents();

  const int tok = p.tokens[r];
  const bool asked = tok >= 0 && tok < p.V;
  const uint8_t* row = p.logits + r * p.ld_bytes;
  const float T = p.temps != nullptr && p.temps[r] > 0.f ? p.temps[r] : 1.f;
  const float c = kLog2e / T;
  const int subs = (p.V + kBlock - 1) / kBlock;
  const int first = rank * p.subs_per_cta;
  const int last = min(subs, first + p.subs_per_cta);
  const int g0 = first / p.group;
  const int ngroups = last > first ? (last - first + p.group - 1) / p.group : 0;
  Sums acc{-INFINITY, 0.f, 0.f, 0};
  if (asked) {
    float* mine = maxima + g0;  // kept at the same offsets in every CTA of the cluster
    if (p.group > 1) {
      for (int i = threadIdx.x; i < ngroups; i += kThreads) mine[i] = -INFINITY;
      __syncthreads();
    }
    for (int sub = first + warp; sub < last; sub += kWarps) {
      float x[kPerLane];
      B::load(row, p.V, sub, lane, x);
      float top = x[0];
#pragma unroll
      for (int e = 1; e < kPerLane; ++e) top = specv::f32_max_nan(top, x[e]);
      top = warp_max_nan(top);
      if (lane == 0) {
        if (p.group == 1) {
          mine[sub - first] = top;
        } else {  // float order as integer order
          int* cell = reinterpret_cast<int*>(&mine[(sub - first) / p.group]);
          int old = *reinterpret_cast<volatile int*>(cell);
          while (__int_as_float(old) < top) {
            const int seen = atomicCAS(cell, old, __float_as_int(top));
            if (seen == old) break;
            old = seen;
          }
        }
      }
      if (!(top < INFINITY)) acc.bad = 1;
      if (!(top > -INFINITY)) continue;
      if (top > acc.m) {
        if (acc.s > 0.f) {
          const float d = fmaxf((acc.m - top) * c, kLowExp), f = ex2_approx(d);
          acc.t = f * fmaf(acc.s, d, acc.t);
          acc.s *= f;
        }
        acc.m = top;
      }
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        const float a = fmaxf((x[e] - acc.m) * c, kLowExp);
        const float w = ex2_approx(a);
        acc.s += w;
        acc.t = fmaf(w, a, acc.t);
      }
    }
    // The maximum is the warp's, so the lanes' sums add directly.
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      acc.s += __shfl_xor_sync(0xFFFFFFFFu, acc.s, d);
      acc.t += __shfl_xor_sync(0xFFFFFFFFu, acc.t, d);
    }
    if (lane == 0) hd.warp[warp] = acc;
  }
  __syncthreads();
  if (asked && threadIdx.x == 0) {
    acc = hd.warp[0];
    for (int w = 1; w < kWarps; ++w) acc = merge(acc, hd.warp[w], c);
    hd.part[rank] = acc;
  }
  if (p.cluster > 1) {
    cluster_wait_acquire();  // every CTA of the cluster has started
    if (asked && rank != 0) {
      const uint32_t dst = cluster_map(maxima + g0, 0);
      for (int i = threadIdx.x; i < ngroups; i += kThreads)
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + 4 * i), "f"(maxima[g0 + i]) : "memory");
      if (threadIdx.x == 0) {
        const uint32_t s = cluster_map(&hd.part[rank], 0);
        asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(s), "r"(__float_as_uint(acc.m)),
                     "r"(__float_as_uint(acc.s)), "r"(__float_as_uint(acc.t)), "r"(acc.bad)
                     : "memory");
      }
    }
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    cluster_wait_acquire();
    if (rank != 0) return;
  }
  const int n = p.top;
  int32_t* ids = p.top_ids + static_cast<int64_t>(r) * n;
  float* lps = p.top_logprobs + static_cast<int64_t>(r) * n;
  __syncthreads();
  Sums all{-INFINITY, 0.f, 0.f, 0};
  if (asked)
    for (int i = 0; i < p.cluster; ++i) all = merge(all, hd.part[i], c);
  const bool ok = asked && !all.bad && all.s > 0.f;
  const float log_s = logf(all.s);
  if (threadIdx.x == 0) {
    float lp = 0.f, ent = 0.f;
    if (ok) {
      lp = (B::at(row, tok) - all.m) / T - log_s;
      ent = log_s - (all.t / all.s) * kLn2;
    } else if (tok >= 0) {
      lp = ent = NAN;
    }
    p.logprobs[r] = lp;
    if (p.entropy != nullptr) p.entropy[r] = ent;
    if (p.row_status != nullptr)
      p.row_status[r] = ok || tok < 0 ? SPEC_OK : (asked ? SPEC_ERR_NONFINITE : SPEC_ERR_TOKEN_RANGE);
  }
  if (n == 0) return;
  if (!ok) {
    if (threadIdx.x < n) {
      ids[threadIdx.x] = -1;
      lps[threadIdx.x] = tok < 0 ? 0.f : NAN;
    }
    return;
  }

  // A lower bound of the n-th likeliest token: the groups are dealt to 32 columns,
  // and the n-th of the columns' maxima has n tokens no worse than it.
  {
    float v = -INFINITY;
    int vi = INT32_MAX;
    for (int i = threadIdx.x; i < p.groups_total; i += kThreads)
      if (vi == INT32_MAX || maxima[i] > v) {
        v = maxima[i];
        vi = i;
      }
    hd.col_max[warp][lane] = v;
    hd.col_idx[warp][lane] = vi;
    if (threadIdx.x == 0) hd.nsel = hd.ncand = 0;
  }
  __syncthreads();
  if (warp == 0) {
    float v = hd.col_max[0][lane];
    int vi = hd.col_idx[0][lane];
    for (int w = 1; w < kWarps; ++w)
      if (before(hd.col_max[w][lane], hd.col_idx[w][lane], v, vi)) {
        v = hd.col_max[w][lane];
        vi = hd.col_idx[w][lane];
      }
    int pos = 0;
    for (int j = 0; j < 32; ++j) {
      const float ov = __shfl_sync(0xFFFFFFFFu, v, j);
      const int oi = __shfl_sync(0xFFFFFFFFu, vi, j);
      pos += before(ov, oi, v, vi) || (ov == v && oi == vi && j < lane) ? 1 : 0;
    }
    if (pos == n - 1) {
      hd.thr = v;
      hd.thr_idx = vi;
    }
  }
  __syncthreads();
  const float thr = hd.thr;
  const int thr_idx = hd.thr_idx;
  for (int i = threadIdx.x; i < p.groups_total; i += kThreads)
    if (!before(thr, thr_idx, maxima[i], i)) sel[atomicAdd(&hd.nsel, 1)] = i;
  __syncthreads();
  const int nsel = hd.nsel;
  // Tokens equal to the bound count up to the end of its group.
  const int64_t tie_end = thr_idx == INT32_MAX ? INT64_MAX : (static_cast<int64_t>(thr_idx) + 1) * p.group * kBlock;
  for (int i = warp; i < nsel * p.group; i += kWarps) {
    const int sub = sel[i / p.group] * p.group + i % p.group;
    if (sub >= subs) continue;
    float x[kPerLane];
    B::load(row, p.V, sub, lane, x);
#pragma unroll
    for (int e = 0; e < kPerLane; ++e) {
      const int64_t id = B::index_of(sub, lane, e);
      if (id < p.V && (x[e] > thr || (x[e] == thr && id < tie_end))) {
        const int at = atomicAdd(&hd.ncand, 1);
        if (at < kCandidates) {
          hd.cand_val[at] = x[e];
          hd.cand_idx[at] = static_cast<int>(id);
        }
      }
    }
  }
  __syncthreads();
  const int ncand = hd.ncand;
  auto emit = [&](int pos, float v, int id) {
    ids[pos] = id;
    lps[pos] = (v - all.m) / T - log_s;
  };
  if (ncand <= kCandidates) {
    for (int i = threadIdx.x; i < ncand; i += kThreads) {
      const float v = hd.cand_val[i];
      const int id = hd.cand_idx[i];
      int pos = 0;
      for (int j = 0; j < ncand; ++j) pos += before(hd.cand_val[j], hd.cand_idx[j], v, id) ? 1 : 0;
      if (pos < n) emit(pos, v, id);
    }
    if (threadIdx.x < n && threadIdx.x >= ncand) {
      ids[threadIdx.x] = -1;
      lps[threadIdx.x] = -INFINITY;
    }
    return;
  }
  // Many equal logits: one token after the other, the best behind the last.
  float lv = INFINITY;
  int li = -1;
  for (int pos = 0; pos < n; ++pos) {
    float v = -INFINITY;
    int vi = INT32_MAX;
    for (int i = warp; i < nsel * p.group; i += kWarps) {
      const int sub = sel[i / p.group] * p.group + i % p.group;
      if (sub >= subs) continue;
      float x[kPerLane];
      B::load(row, p.V, sub, lane, x);
#pragma unroll
      for (int e = 0; e < kPerLane; ++e) {
        const int64_t id = B::index_of(sub, lane, e);
        if (id < p.V && before(lv, li, x[e], static_cast<int>(id)) && before(x[e], static_cast<int>(id), v, vi)) {
          v = x[e];
          vi = static_cast<int>(id);
        }
      }
    }
    const float wv = specv::warp_max_f32(v);
    const int wi = __reduce_min_sync(0xFFFFFFFFu, v == wv ? vi : INT32_MAX);
    __syncthreads();
    if (lane == 0) {
      hd.col_max[warp][0] = wv;
      hd.col_idx[warp][0] = wi;
    }
    __syncthreads();
    lv = hd.col_max[0][0];
    li = hd.col_idx[0][0];
    for (int w = 1; w < kWarps; ++w)
      if (before(hd.col_max[w][0], hd.col_idx[w][0], lv, li)) {
        lv = hd.col_max[w][0];
        li = hd.col_idx[w][0];
      }
    if (threadIdx.x == 0) emit(pos, lv, li);
  }
}

constexpr int kMaxDevices = 64;
std::mutex g_mutex;
int g_sms[kMaxDevices] = {};
bool g_attr[kMaxDevices][4] = {};

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
                               static_cast<int>(sizeof(Head)) + 2 * kMaxCluster * kMaxGroups * 4) != cudaSuccess)
        return SPEC_ERR_CUDA;
      g_attr[dev][which] = true;
    }
  }
  const int subs = (a->V + kBlock - 1) / kBlock;
  // Enough CTAs for two on every SM, each with a block of 512 a warp at least.
  int cluster = 1;
  while (cluster < kMaxCluster && static_cast<int64_t>(a->rows) * cluster < 2 * sms && subs > cluster * kWarps) cluster *= 2;
  int group = 1;
  int per = (subs + cluster - 1) / cluster;
  while ((per + group - 1) / group > kMaxGroups) group *= 2;
  per = (per + group - 1) / group * group;

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
  p.groups_total = (subs + group - 1) / group;

  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a->rows) * cluster, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = sizeof(Head) + 2 * static_cast<size_t>(p.groups_total) * 4;
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
