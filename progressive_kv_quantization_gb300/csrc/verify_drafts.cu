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
// Bound by the chain draft -> gather -> row -> exchange -> search for few requests
// (4.8 us for one of 32,000 values) and by the reads of the two rows for many: 256 of
// 151,936 float32 values take 54.6 us (5.7 TB/s, 84% of a copy); 32 take 11.2 us (51%),
// of which some 5 are the chain.  A request's values are in flight three runs a warp
// deep, in shared memory: loads to registers held fewer.

#include "f32x2.cuh"
#include "lynx_internal.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>

namespace cg = cooperative_groups;

namespace lynx {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kRun = 256;                          // values per run, 8 a lane
constexpr int kStages = 3;                         // runs of a warp in flight or in hand
constexpr int kStageBytes = kStages * 4 * kThreads * 16;   // two pieces of each row a thread

__device__ __forceinline__ float prob(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float prob(const __nv_bfloat16* p, int64_t i) { return __bfloat162float(p[i]); }

// Sums of weights in whole multiples of 2^-40 (NaN and negative weights 0, at
// most 1 each).  A weight's two 20-bit halves come from float additions rounded
// down onto numbers whose last place is 2^-20 and 2^-40: the bits that the sum
// holds above those of 8 and 2^-17 are the whole multiples.  Two weights at a
// time, four instructions each; the conversion float -> uint64 took 39.5 us for
// 32 rows of 151,936.  A run's halves fit 32 bits over a whole warp.
struct Units {
  uint32_t hi = 0, lo = 0;
  // max(0, p - q), at most 1, 0 for NaN
  static __device__ __forceinline__ float weight(float p, float q) {
    float w;
    asm("sub.rn.sat.f32 %0, %1, %2;" : "=f"(w) : "f"(p), "f"(q));
    return w;
  }
  __device__ __forceinline__ void add2(float w0, float w1) {
    const uint64_t w = pair(w0, w1);
    const uint64_t h = add2_down(w, pair(8.0f, 8.0f));
    const uint64_t top = lynx::add2(h, pair(-8.0f, -8.0f));
    const uint64_t rest = fma2(top, pair(-1.0f, -1.0f), w);   // exact, below 2^-20
    const uint64_t l = add2_down(rest, pair(0x1p-17f, 0x1p-17f));
    hi += (uint32_t)h + (uint32_t)(h >> 32) - 2u * 0x41000000u;   // bits of 8
    lo += (uint32_t)l + (uint32_t)(l >> 32) - 2u * 0x37000000u;   // bits of 2^-17
  }
  static __device__ __forceinline__ unsigned long long join(uint32_t hi, uint32_t lo) {
    return ((unsigned long long)hi << 20) + lo;
  }
  __device__ __forceinline__ unsigned long long value() const { return join(hi, lo); }
  __device__ __forceinline__ unsigned long long over_warp() const {
    return join(__reduce_add_sync(0xffffffffu, hi), __reduce_add_sync(0xffffffffu, lo));
  }
  static __device__ __forceinline__ unsigned long long of(float w) {
    Units u;
    u.add2(w, 0.0f);
    return u.value();
  }
};

// value e of 16 bytes of a row
template <typename T>
__device__ __forceinline__ float value(const uint4& x, int e) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  if (sizeof(T) == 4) return __uint_as_float(w[e]);
  return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
}

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

__device__ __forceinline__ unsigned long long warp_sum(unsigned long long v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2)
verify_drafts_kernel(const VerifyArgs a) {
  constexpr int kVec = 16 / sizeof(T), kLoads = kRun / 32 / kVec;
  extern __shared__ __align__(16) uint8_t s_dyn[];
  uint4* s_stage = reinterpret_cast<uint4*>(s_dyn);                                          // [stage][piece][thread]
  unsigned long long* s_run = reinterpret_cast<unsigned long long*>(s_dyn + kStageBytes);    // sums of this CTA's runs
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
  allow_dependent_launch();
  wait_prerequisite_grids();
  // read ahead of their first use: the request's counts and numbers arrive together
  const float u_last = u[a.T];
  const int n_draft = a.n_draft ? min(max(a.n_draft[b], 0), a.T) : a.T;

  if (tid < 64) {
    bool ok = false;
    const int x = tid < a.T ? draft[tid] : -1;
    const float ux = tid < a.T ? u[tid] : 0.0f;
    if (x >= 0 && x < a.V) {
      const float qx = q ? prob(q + tid * a.q_stride_t, x) : 1.0f;
      ok = __fmul_rn(ux, qx) < prob(p + tid * a.p_stride_t, x) && tid < n_draft;
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
  const int drafted_id = rejected && !q ? draft[n] : -1;
  const int out = drafted_id < a.V ? drafted_id : -1;

  // this CTA's runs
  const int n_runs = (a.V + kRun - 1) / kRun;
  const int r0 = (int)((int64_t)n_runs * rank / C), r1 = (int)((int64_t)n_runs * (rank + 1) / C);

  bool residual = true;
  unsigned long long total = 0, before = 0;
  auto weight = [&](int64_t i) {
    const float w = Units::weight(prob(row, i), residual && drafted ? prob(drafted, i) : 0.0f);
    return residual && i == out ? 0.0f : w;
  };
  // both rows on 16-byte boundaries
  const bool wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0 &&
                    (!drafted || (reinterpret_cast<uintptr_t>(drafted) & 15) == 0);
  for (int attempt = 0; attempt < 2; ++attempt) {
    unsigned long long mine = 0;
    const bool minus = residual && drafted;
    // A thread's 16-byte pieces of the next kStages - 1 runs of its warp are on
    // their way to its own places in shared memory while it sums this run's.
    const int n_mine = r1 - r0 > warp ? (r1 - r0 - warp + kWarps - 1) / kWarps : 0;
    auto staged = [&](int r) { return wide && (int64_t)(r + 1) * kRun <= a.V; };
    auto fetch = [&](int k) {
      const int r = r0 + warp + k * kWarps;
      if (k < n_mine && staged(r)) {
        uint4* dst = s_stage + (k % kStages) * 4 * kThreads + tid;
        const int64_t i0 = (int64_t)r * kRun + lane * kVec;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          copy_async16(dst + x * kThreads, row + i0 + x * 32 * kVec);
          if (minus) copy_async16(dst + (2 + x) * kThreads, drafted + i0 + x * 32 * kVec);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int k = 0; k < kStages - 1; ++k) fetch(k);
    for (int k = 0; k < n_mine; ++k) {
      fetch(k + kStages - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
      const int r = r0 + warp + k * kWarps;
      Units sum;
      if (staged(r)) {
        const uint4* src = s_stage + (k % kStages) * 4 * kThreads + tid;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          const uint4 px = src[x * kThreads];
          uint4 qx = make_uint4(0u, 0u, 0u, 0u);
          if (minus) qx = src[(2 + x) * kThreads];
#pragma unroll
          for (int e = 0; e < kVec; e += 2)   // w - 0 is w
            sum.add2(Units::weight(value<T>(px, e), value<T>(qx, e)), Units::weight(value<T>(px, e + 1), value<T>(qx, e + 1)));
        }
      } else {
        const int64_t i0 = (int64_t)r * kRun + lane;
        float x[8], y[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          x[e] = i0 + 32 * e < a.V ? prob(row, i0 + 32 * e) : 0.0f;
          y[e] = minus && i0 + 32 * e < a.V ? prob(drafted, i0 + 32 * e) : 0.0f;
        }
#pragma unroll
        for (int e = 0; e < 8; e += 2) sum.add2(Units::weight(x[e], y[e]), Units::weight(x[e + 1], y[e + 1]));
      }
      unsigned long long v = sum.over_warp();
      if (residual && out >= 0 && out / kRun == r) v -= Units::of(Units::weight(prob(row, out), 0.0f));   // the certain draft's
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
    // one CTA's sum a lane (C <= 32)
    const unsigned long long part = lane < C ? *cluster.map_shared_rank(&s_sum, lane) : 0;
    total = warp_sum(part);
    before = warp_sum(lane < rank ? part : 0);
    if (total > 0 || !residual || !rejected) break;
    residual = false;
    cluster.sync();   // s_sum changes only when all have read it
  }
  // a CTA leaves only when all have read its sum
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");

  int32_t* tokens = a.tokens + (int64_t)b * (a.T + 1);
  if (rank == 0 && warp == 1) {   // the first warp looks for the token meanwhile
    for (int i = lane; i <= a.T; i += 32)
      if (i != n) tokens[i] = i < n ? draft[i] : -1;
    if (lane == 0) {
      a.n_accept[b] = n;
      if (total == 0) tokens[n] = -1;
    }
  }
  // ---- the CTA that holds the limit looks for the token; its first warp
  auto find = [&]() {
    if (total == 0) return;
    const long long step = min(max((long long)(u_last * 16777216.0f), 0ll), (1ll << 24) - 1);   // NaN: 0
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
    // 8 values a lane, one behind the other: the lane, then its value
    constexpr int kOwn = kRun / 32;
    const int64_t i0 = (int64_t)found * kRun + lane * kOwn;
    float w[kOwn];
#pragma unroll
    for (int k = 0; k < kOwn; ++k) w[k] = i0 + k < a.V ? weight(i0 + k) : 0.0f;
    Units own;
#pragma unroll
    for (int k = 0; k < kOwn; k += 2) own.add2(w[k], w[k + 1]);
    unsigned long long incl = own.value();
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long x = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += x;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, at + incl > limit);
    if (hit && lane == __ffs(hit) - 1) {
      at += incl - own.value();
      int k = 0;
#pragma unroll
      for (int e = 0; e < kOwn; ++e) {
        at += Units::of(w[e]);
        k += at <= limit;
      }
      tokens[n] = (int32_t)(i0 + k);
    }
  };
  find();
  __syncwarp();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, cudaStream_t s) {
  // CTAs per request: as many as run at once, at most 8 (the portable cluster).  us for
  // rows of 151,936: 32 requests 10.0 (8 CTAs) against 13.6 (4); 64: 14.7 (4) against
  // 18.6 (8); 256: 54.6 (1) against 69.5 (8).
  int C = 8;
  while (C > 1 && (int64_t)a.B * C > 2 * device_sm_count()) C >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.B * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kStageBytes + (size_t)(((a.V + kRun - 1) / kRun + C - 1) / C) * 8;
  static bool configured[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(verify_drafts_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kStageBytes + kVerifyMaxVocab / kRun * 8);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, verify_drafts_kernel<T>, a);
}

}  // namespace

cudaError_t launch_verify_drafts(const VerifyArgs& a, bool bf16, cudaStream_t s) {
  return bf16 ? launch_t<__nv_bfloat16>(a, s) : launch_t<float>(a, s);
}

}  // namespace lynx
