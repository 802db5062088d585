// Verification of drafted tokens against the target's probabilities, from given
// random numbers (lynx_verify_drafts).
//
//   draft i is accepted while u_i q_i(x_i) < p_i(x_i)  (float32 product)
//   n = number of accepted drafts; the next token is drawn from
//   w = max(0, p_n - q_n) (float32) after a rejection, from p_n behind the last
//   draft; and from p_n too where w has no weight
//   weights are whole multiples of 2^-40 (rounded down, at most 1), so their
//   sums are exact in any order;  the token is the first k with
//   sum_{j <= k} w_j > floor(W floor(2^24 u_T) / 2^24),  W = sum_j w_j
//
// A thread-block cluster takes one request, each CTA a contiguous part of the
// vocabulary.  Every CTA tests the drafts itself (a gather of T values), then
// sums its part of the two rows that the outcome selects in runs of kRun
// values, one warp a run; the CTAs' sums are exchanged through distributed
// shared memory, and the CTA that holds the limit goes through its run sums
// and re-reads the one run in question.  One launch, no workspace, no atomics;
// every value of the two rows is read once.
//
// Bound by the reads of the two rows for a batch, by the chain draft -> gather
// -> row -> exchange for one request.

#include "lynx_internal.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>

namespace cg = cooperative_groups;

namespace lynx {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 512;                          // values per run, 16 a lane

__device__ __forceinline__ float prob(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

// whole multiples of 2^-40 of a weight, 0 for NaN
__device__ __forceinline__ unsigned long long units(float w) {
  w = fminf(fmaxf(w, 0.0f), 1.0f);
  return __float2ull_rz(w * 1099511627776.0f);
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
verify_drafts_kernel(const VerifyArgs a) {
  extern __shared__ unsigned long long s_run[];    // sums of this CTA's runs
  __shared__ unsigned s_ok[2];
  __shared__ unsigned long long s_part[kWarps];
  __shared__ unsigned long long s_sum;             // of this CTA's part, read by the whole cluster

  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int b = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* p = static_cast<const T*>(a.p) + (int64_t)b * a.p_stride_b;
  const T* q = a.q ? static_cast<const T*>(a.q) + (int64_t)b * a.q_stride_b : nullptr;
  const float* u = a.u + (int64_t)b * (a.T + 1);
  const int32_t* draft = a.draft + (int64_t)b * a.T;
  const int n_draft = a.n_draft ? min(max(a.n_draft[b], 0), a.T) : a.T;

  if (tid < 64) {
    bool ok = false;
    if (tid < n_draft) {
      const int x = draft[tid];
      if (x >= 0 && x < a.V) {
        const float qx = q ? prob(q + tid * a.q_stride_t, x) : 1.0f;
        ok = __fmul_rn(u[tid], qx) < prob(p + tid * a.p_stride_t, x);
      }
    }
    const unsigned m = __ballot_sync(0xffffffffu, ok);
    if (lane == 0) s_ok[warp] = m;
  }
  __syncthreads();
  const unsigned long long oks = s_ok[0] | ((unsigned long long)s_ok[1] << 32);
  const int n = __ffsll(~oks) - 1 < 0 ? 64 : __ffsll(~oks) - 1;   // leading accepted drafts
  const bool rejected = n < n_draft;
  const T* row = p + n * a.p_stride_t;
  const T* drafted = rejected && q ? q + n * a.q_stride_t : nullptr;
  // without draft probabilities a rejected draft had all of its row's
  const int out = rejected && !q ? draft[n] : -1;

  // this CTA's runs
  const int n_runs = (a.V + kRun - 1) / kRun;
  const int r0 = (int)((int64_t)n_runs * rank / C), r1 = (int)((int64_t)n_runs * (rank + 1) / C);

  bool residual = true;
  unsigned long long total = 0, before = 0;
  auto weight = [&](int64_t i) {
    float w = prob(row, i);
    if (residual) {
      if (drafted) w = __fsub_rn(w, prob(drafted, i));
      if (i == out) w = 0.0f;
    }
    return units(w);
  };
  for (int attempt = 0; attempt < 2; ++attempt) {
    unsigned long long mine = 0;
    for (int r = r0 + warp; r < r1; r += kWarps) {
      unsigned long long v = 0;
      const int64_t i0 = (int64_t)r * kRun + lane;
#pragma unroll
      for (int k = 0; k < kRun / 32; ++k)
        if (i0 + 32 * k < a.V) v += weight(i0 + 32 * k);
      v = warp_sum(v);
      if (lane == 0) s_run[r - r0] = v;
      mine += v;
    }
    if (lane == 0) s_part[warp] = mine;
    __syncthreads();
    if (tid == 0) {
      unsigned long long v = 0;
      for (int i = 0; i < kWarps; ++i) v += s_part[i];
      s_sum = v;
    }
    cluster.sync();
    total = before = 0;
    for (int c = 0; c < C; ++c) {
      const unsigned long long v = *cluster.map_shared_rank(&s_sum, c);
      if (c < rank) before += v;
      total += v;
    }
    cluster.sync();   // s_sum may change, or this CTA leave, only when all have read it
    if (total > 0 || !residual || !rejected) break;
    residual = false;
  }

  int32_t* tokens = a.tokens + (int64_t)b * (a.T + 1);
  if (rank == 0) {
    for (int i = tid; i <= a.T; i += kThreads)
      if (i != n) tokens[i] = i < n ? draft[i] : -1;
    if (tid == 0) {
      a.n_accept[b] = n;
      if (total == 0) tokens[n] = -1;
    }
  }
  if (total == 0) return;
  const float uf = u[a.T];
  const long long step = min(max((long long)(uf * 16777216.0f), 0ll), (1ll << 24) - 1);   // NaN: 0
  const unsigned long long limit =
      (total >> 24) * (unsigned long long)step + (((total & 0xFFFFFFull) * (unsigned long long)step) >> 24);
  if (warp != 0 || limit < before || limit >= before + s_sum) return;

  // the run that holds the limit: 32 runs at a time
  unsigned long long at = before;
  int found = r1 - 1;
  for (int base = 0; base < r1 - r0; base += 32) {
    unsigned long long v = base + lane < r1 - r0 ? s_run[base + lane] : 0, incl = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at + incl > limit);
    if (hit) {
      const int l = __ffs(hit) - 1;
      found = r0 + base + l;
      at += __shfl_sync(0xffffffffu, incl - v, l);
      break;
    }
    at += __shfl_sync(0xffffffffu, incl, 31);
  }
  for (int k = 0; k < kRun / 32; ++k) {
    const int64_t i = (int64_t)found * kRun + 32 * k + lane;
    unsigned long long incl = i < a.V ? weight(i) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at + incl > limit);
    if (hit) {
      if (lane == 0) tokens[n] = (int32_t)((int64_t)found * kRun + 32 * k + __ffs(hit) - 1);
      return;
    }
    at += __shfl_sync(0xffffffffu, incl, 31);
  }
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
  // CTAs per request: as many as the machine has room for, at most 8
  int C = 8;
  while (C > 1 && (int64_t)a.B * C > 2 * device_sm_count()) C >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)(((a.V + kRun - 1) / kRun + C - 1) / C) * 8;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace lynx
