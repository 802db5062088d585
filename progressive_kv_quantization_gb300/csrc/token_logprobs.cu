// Log probabilities of given tokens under their logits, the entropies of the
// distributions, and their most likely tokens (lynx_token_logprobs), in one pass
// over the logits.
//
//   d_k = x_k - max x,  s = sum_k e^(d_k),  t = sum_k e^(d_k) d_k
//   log p_k = d_k - ln s,  entropy = ln s - t / s
// (in powers of two: d log2(e), and ln 2 times the result)
//
// A thread-block cluster takes a row, each CTA a contiguous part of it, a thread
// every 256th piece of 16 bytes.  s and t are kept against a reference that follows
// the thread's maximum at a distance of at most 6 (so that both are scaled again on few pieces),
// and are brought to the row's maximum at the end.  A thread may have 65,536 terms, whose roundings
// go one way where they are alike (4e-5 of s for 1,048,576 flat logits, 4.9e-4 for sixteen times as many):
// a batch's 12 to 32 are summed first, and the running sums keep what each addition lost.  (2,047 rows of
// 128,256 BF16 with 20 alternatives 109 us against 105, the others 1% at most; behind every fourth or eighth
// batch only, or with the running sums in shared memory, 111 to 118.)
//
// The n most likely tokens (equal ones: the lowest first) as 64-bit keys: the float's bits in
// an order of whole numbers, and under them the token's from behind.  While the first quarter
// of a CTA's part goes by, a thread only notes its largest value and the piece that it is in.  The
// n-th largest of the notes of 64 groups of 4 threads is a bound that at least n tokens
// reach; the pieces of threads whose own note reaches it (some n of 256) are gone
// through again, still in L2, and of the other three quarters what reaches the bound is kept as it
// goes by: some 5 n tokens, which are ranked by counting.  (Going through the whole part again
// at its end read lines of 16 bytes from DRAM: 1,000 rows of 128,256 float32 took 114 us against 93.)
// Parts of fewer than 8 batches a thread are still in L2 then, and noted as a whole.
//
// Bound by the reads of the logits for many rows: 2,047 rows of 128,256 BF16 take 83 us (6.35 TB/s,
// 93% of a copy), with 20 alternatives 109 us; 1,000 rows of as many float32 80 and 94 us.  By the
// chain (launch, one round trip of loads, the reductions, the bound, the ranks) for few: 64 rows of
// 151,936 float32 10.4 us without alternatives, 16.8 us with 20 (39 MB, 5.7 us at a copy's rate).
// Copies go into shared memory, three batches a thread deep: loads to registers held fewer (93 and
// 119 us for the BF16 rows; 88 us for the float32 rows with alternatives).

#include "f32x2.cuh"
#include "lynx_internal.cuh"

#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <math_constants.h>

namespace cg = cooperative_groups;

namespace lynx {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = kThreads / 4;
constexpr int kMaxTop = kLogprobsMaxTop;
constexpr int kFound = 2048;            // tokens that reach the bound, at most
constexpr int kKept = 256;              // pieces with such tokens, at most
constexpr int kMaxCluster = 8;
constexpr float kLag = 6.0f;            // of the reference behind the maximum
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLeast = -1024.0f;      // 2^kLeast is 0, and so is the product of the two
static_assert(kGroups >= kMaxTop && kFound >= kGroups * 4 * 8, "bounds on what reaches the bound");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// the larger one, NaN if one is NaN
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// floats in the order of whole numbers, -0 as 0; never 0
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t o) {
  return __uint_as_float(o ^ (o >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}
using Key = unsigned long long;   // 0: none
__device__ __forceinline__ Key key_of(float x, int token) {
  return (Key)ordered(x) << 32 | (0xFFFFFFFFu - (uint32_t)token);
}

// batches of pieces on their way to a thread
template <bool TOP>
struct Stream {
  static constexpr int kBatch = TOP ? 3 : 4, kStages = 3;
  static constexpr int kBytes = kStages * kBatch * kThreads * 16;
};

__device__ __forceinline__ void copy_async16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

template <typename T>
struct Piece {   // 16 bytes of a row
  static constexpr int kN = 16 / sizeof(T);
  uint4 raw;
  __device__ __forceinline__ float at(int e) const {
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    if (sizeof(T) == 4) return __uint_as_float(w[e]);
    return __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
  }
  __device__ __forceinline__ float largest() const {
    float m = fmaxf(at(0), at(1));
#pragma unroll
    for (int e = 2; e < kN; e += 2) m = max3(m, at(e), at(e + 1));
    return m;
  }
};

// sums against the reference `ref` (natural units): a batch's by themselves, and the running ones with
// what their roundings lost, to be taken off
struct Sums {
  float ref = -3.402823466e38f;
  float s = 0.0f, s_lost = 0.0f, t = 0.0f, t_lost = 0.0f;
  uint64_t s2 = 0, t2 = 0;   // of the batch, pairs

  // to a reference `to` >= ref, of one value each
  static __device__ __forceinline__ void move(float from, float to, float& s, float& t) {
    const float d = fmaxf((from - to) * kLog2e, kLeast), f = ex2(d);
    t = f * fmaf(d, s, t);
    s *= f;
  }
  // in front of a batch
  __device__ __forceinline__ void follow(float largest) {
    if (largest > ref + kLag) {
      move(ref, largest, s, t);
      move(ref, largest, s_lost, t_lost);
      ref = largest;
    }
  }
  __device__ __forceinline__ void add(float x0, float x1) {
    float d0, d1;
    unpair(mul2(add2(pair(x0, x1), pair(-ref, -ref)), pair(kLog2e, kLog2e)), d0, d1);
    d0 = max_nan(d0, kLeast);   // of a logit of -inf; NaN stays
    d1 = max_nan(d1, kLeast);
    const uint64_t e = pair(ex2(d0), ex2(d1));
    s2 = add2(s2, e);
    t2 = fma2(e, pair(d0, d1), t2);
  }
  static __device__ __forceinline__ void put(uint64_t more, float& sum, float& lost) {
    float m0, m1;
    unpair(more, m0, m1);
    const float m = __fadd_rn(__fadd_rn(m0, m1), -lost), next = __fadd_rn(sum, m);
    lost = __fadd_rn(__fadd_rn(next, -sum), -m);
    sum = next;
  }
  // behind a batch
  __device__ __forceinline__ void flush() {
    put(s2, s, s_lost);
    put(t2, t, t_lost);
    s2 = t2 = 0;
  }
};

// what a CTA has found, read by the cluster's first
struct Found {
  float top, s, t;   // largest logit, sums against it
  Key best[kMaxTop];
};

struct Yes { static constexpr bool value = true; };
struct No { static constexpr bool value = false; };

template <typename T, bool TOP>
__global__ void __launch_bounds__(kThreads, 4)
token_logprobs_kernel(const LogprobsArgs a) {
  using P = Piece<T>;
  using S = Stream<TOP>;
  constexpr int kBatch = S::kBatch, kStages = S::kStages;
  extern __shared__ __align__(16) uint4 s_stage[];   // [stage][piece of a batch][thread]
  __shared__ Found s_found;
  __shared__ float s_part[kWarps][2];
  __shared__ Key s_group[TOP ? kGroups : 1];
  __shared__ Key s_bound;
  __shared__ int s_count, s_n_again, s_n_kept;
  __shared__ uint4 s_kept[TOP ? kKept : 1];     // pieces that reach the bound, and which they are
  __shared__ int s_kept_k[TOP ? kKept : 1];
  __shared__ int s_again[TOP ? kThreads : 1];   // threads whose pieces are gone through again
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int64_t row = blockIdx.x / C;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* x = static_cast<const T*>(a.logits) + row * a.row_stride;
  // the row as whole pieces, and up to 2 (kN - 1) tokens in front of and behind them, which are rank 0's
  const int front = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T), a.V);
  const int pieces = (a.V - front) / P::kN, behind = front + pieces * P::kN;
  const int k0 = (int)((int64_t)pieces * rank / C), k1 = (int)((int64_t)pieces * (rank + 1) / C);
  const uint4* body = reinterpret_cast<const uint4*>(x + front);
  const int loose = front + a.V - behind;
  const int loose_at = rank == 0 && tid < loose ? (tid < front ? tid : behind + tid - front) : -1;
  auto value = [&](int i) { return static_cast<float>(x[i]); };

  wait_prerequisite_grids();
  float token_x = 0.0f;
  int token = -1;
  if (rank == 0 && tid == 0) {
    token = a.tokens[row];
    if (token >= 0 && token < a.V) token_x = value(token);
  }

  Sums sums;
  float top = -CUDART_INF_F;
  int top_k = -1;   // the piece that it is in
  Key bound = 0;
  float least = CUDART_INF_F;
  Key* s_keys = reinterpret_cast<Key*>(s_stage);   // when all pieces have been read
  auto look = [&](float v, int i) {
    if (!(v >= least)) return;
    const Key key = key_of(v, i);
    if (key >= bound) {
      const int at = atomicAdd(&s_count, 1);
      if (at < kFound) s_keys[at] = key;
    }
  };
  auto look_at = [&](const P& p, int k) {
#pragma unroll
    for (int e = 0; e < P::kN; ++e) look(p.at(e), front + k * P::kN + e);
  };
  // a piece with a value that reaches the bound, for the end
  auto keep = [&](const P& p, int k) {
    const int at = atomicAdd(&s_n_kept, 1);
    if (at < kKept) {
      s_kept[at] = p.raw;
      s_kept_k[at] = k;
    }
  };
  auto take = [&](const P& p, int k, float m, auto notes) {
    if (TOP && decltype(notes)::value && (m > top || top_k < 0)) top_k = k;
    top = fmaxf(top, m);
#pragma unroll
    for (int e = 0; e < P::kN; e += 2) sums.add(p.at(e), p.at(e + 1));
  };
  float loose_x = -CUDART_INF_F;
  if (loose_at >= 0) {
    loose_x = value(loose_at);
    sums.follow(loose_x);
    sums.add(loose_x, -CUDART_INF_F);
    sums.flush();
  }
  // The bound of what was noted, and what reaches it.  Every thread comes here once; others' pieces
  // are those up to `end`.
  auto set_bound = [&](int end) {
    // a thread's note: its largest value, and the last token of its piece
    Key note = top_k < 0 ? 0 : key_of(top, front + top_k * P::kN + P::kN - 1);
    note = max(note, __shfl_xor_sync(0xffffffffu, note, 1));
    note = max(note, __shfl_xor_sync(0xffffffffu, note, 2));
    if ((lane & 3) == 0) s_group[tid >> 2] = note;
    if (tid == 0) s_count = s_n_again = s_n_kept = 0;
    __syncthreads();
    // the n-th largest, four threads a note; they differ from one another, but for those that are 0
    const int i = tid >> 2;
    const Key own = s_group[i];
    int r = 0;
#pragma unroll
    for (int j = 0; j < kGroups / 4; ++j) {
      const int at = 4 * j + (tid & 3);
      const Key o = s_group[at];
      r += o > own || (o == own && at < i);
    }
    r += __shfl_xor_sync(0xffffffffu, r, 1);
    r += __shfl_xor_sync(0xffffffffu, r, 2);
    if ((tid & 3) == 0 && r == a.n_top - 1) s_bound = own;
    __syncthreads();
    bound = s_bound;
    least = bound == 0 ? -CUDART_INF_F : unordered((uint32_t)(bound >> 32));
    // a thread's best possible key: its value and the first token of the piece
    if (top_k >= 0 && key_of(top, front + top_k * P::kN) >= bound) s_again[atomicAdd(&s_n_again, 1)] = tid;
    __syncthreads();
    // the pieces of such threads, by equally many threads each, kBatch of them on their way at once
    const int each = s_n_again ? kThreads / s_n_again : 1, who = tid / each, step = each * kThreads;
    if (who < s_n_again) {
      for (int k = k0 + s_again[who] + (tid - who * each) * kThreads; k < end; k += kBatch * step) {
        P p[kBatch];
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (k + u * step < end) p[u].raw = __ldg(body + k + u * step);
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (k + u * step < end && p[u].largest() >= least) keep(p[u], k + u * step);
      }
    }
  };
  constexpr int kStep = kBatch * kThreads;
  const int whole = (k1 - k0) / kStep;
  // A thread's pieces come by asynchronous copies into places of its own, kStages - 1 batches
  // ahead; behind the last whole batch is a part of one.
  uint4* stage = s_stage + tid;
  auto fetch = [&](int b) {
    const int k = k0 + tid + b * kStep;
    uint4* dst = stage + b % kStages * kStep;
    if (b < whole) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u) copy_async16(dst + u * kThreads, body + k + u * kThreads);
    } else if (b == whole) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
        if (k + u * kThreads < k1) copy_async16(dst + u * kThreads, body + k + u * kThreads);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  auto arrived = [] { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory"); };
  // batches b0 .. b1 - 1, whole ones
  auto stream = [&](int b0, int b1, auto notes) {
    for (int b = b0; b < b1; ++b) {
      fetch(b + kStages - 1);
      arrived();
      P cur[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) cur[u].raw = stage[b % kStages * kStep + u * kThreads];
      const int k = k0 + tid + b * kStep;
      float m[kBatch], largest = -CUDART_INF_F;
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        m[u] = cur[u].largest();
        largest = fmaxf(largest, m[u]);
      }
      sums.follow(largest);
#pragma unroll
      for (int u = 0; u < kBatch; ++u) take(cur[u], k + u * kThreads, m[u], notes);
      sums.flush();
      if (TOP && !decltype(notes)::value) {
#pragma unroll
        for (int u = 0; u < kBatch; ++u)
          if (m[u] >= least) keep(cur[u], k + u * kThreads);
        __syncwarp();
      }
    }
  };
  auto rest = [&](auto notes) {
    fetch(whole + kStages - 1);
    arrived();
    const int k = k0 + tid + whole * kStep;
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
      if (k + u * kThreads < k1) {
        P p;
        p.raw = stage[whole % kStages * kStep + u * kThreads];
        const float m = p.largest();
        sums.follow(m);
        take(p, k + u * kThreads, m, notes);
        sums.flush();
        if (TOP && !decltype(notes)::value && m >= least) keep(p, k + u * kThreads);
      }
    __syncwarp();
  };
#pragma unroll
  for (int b = 0; b < kStages - 1; ++b) fetch(b);
  if (!TOP) {
    stream(0, whole, No());
    rest(No());
  } else {
    const int first = whole >= 8 ? whole / 4 : whole;
    stream(0, first, Yes());
    if (first == whole) rest(Yes());
    set_bound(first == whole ? k1 : k0 + first * kStep);
    if (first < whole) {
      stream(first, whole, No());
      rest(No());
    }
  }

  // ---- the CTA's maximum and sums
  float cta_top = fmaxf(top, loose_x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) cta_top = fmaxf(cta_top, __shfl_xor_sync(0xffffffffu, cta_top, o));
  if (lane == 0) s_part[warp][0] = cta_top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) cta_top = fmaxf(cta_top, s_part[w][0]);
  float s = sums.s, t = sums.t;
  // cta_top is below the reference only where nothing was added
  Sums::move(sums.ref, fmaxf(cta_top, sums.ref), s, t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    s += __shfl_xor_sync(0xffffffffu, s, o);
    t += __shfl_xor_sync(0xffffffffu, t, o);
  }
  __shared__ float s_sums[kWarps][2];
  if (lane == 0) {
    s_sums[warp][0] = s;
    s_sums[warp][1] = t;
  }
  __syncthreads();
  if (tid == 0) {
    s = t = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      s += s_sums[w][0];
      t += s_sums[w][1];
    }
    s_found.top = cta_top;
    s_found.s = s;
    s_found.t = t;
  }

  if (TOP) {
    // ---- the tokens that reach the bound
    static_assert(!TOP || S::kBytes >= kFound * (int)sizeof(Key), "s_keys");
    const int kept = s_n_kept;
    auto look_at_all = [&] {
      for (int k = k0 + tid; k < k1; k += kThreads) {
        P p;
        p.raw = __ldg(body + k);
        if (p.largest() >= least) look_at(p, k);
      }
    };
    if (loose_at >= 0) look(loose_x, loose_at);
    if (kept <= kKept) {
      for (int i = tid; i < kept; i += kThreads) {
        P p;
        p.raw = s_kept[i];
        look_at(p, s_kept_k[i]);
      }
    } else {
      look_at_all();
    }
    __syncthreads();
    int n = s_count;
    // Too many (values that rise, or stand close together): a bound between the last one, which
    // more than kFound tokens reach, and one that fewer than n_top reach, by halving.  Keys differ,
    // so that one with a count in between is found in at most 64 steps, whatever the row.
    // (lo is not 0: that needs a part of fewer tokens.)
    Key lo = bound, hi = ~0ull;
    if (n > kFound) hi = key_of(cta_top, 0) + 1;
    while (n > kFound || (n < a.n_top && lo != bound)) {
      if (n > kFound) lo = bound; else hi = bound;
      bound = lo + (hi - lo) / 2;
      least = unordered((uint32_t)(bound >> 32));
      __syncthreads();
      if (tid == 0) s_count = 0;
      __syncthreads();
      if (loose_at >= 0) look(loose_x, loose_at);
      look_at_all();
      __syncthreads();
      n = s_count;
    }
    // ranks; a CTA's part may hold fewer than n_top tokens
    if (tid < kMaxTop) s_found.best[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      const Key own = s_keys[i];
      int r = 0;
      for (int j = 0; j < n; ++j) r += s_keys[j] > own;
      if (r < a.n_top) s_found.best[r] = own;
    }
  }

  // ---- the row
  if (C > 1) cluster.sync(); else __syncthreads();
  if (rank == 0) {
    float row_top = -CUDART_INF_F;
    for (int c = 0; c < C; ++c) row_top = fmaxf(row_top, cluster.map_shared_rank(&s_found, c)->top);
    s = t = 0.0f;
    for (int c = 0; c < C; ++c) {
      const Found* f = cluster.map_shared_rank(&s_found, c);
      float cs = f->s, ct = f->t;
      const float from = f->top;
      if (from != row_top) Sums::move(from, row_top, cs, ct);
      s += cs;
      t += ct;
    }
    const float log_s = log2f(s);
    auto logprob = [&](float v) { return v == -CUDART_INF_F ? v : fmaf(-kLn2, log_s, v - row_top); };
    if (tid == 0) {
      const bool real = token >= 0 && token < a.V;
      a.logprob[row] = real ? logprob(token_x) : -CUDART_INF_F;
      const float h = s == 0.0f ? 0.0f : kLn2 * (log_s - t / s);   // nothing but -inf: 0
      a.entropy[row] = h < 0.0f ? 0.0f : h;                         // roundings, where one token has it all
    }
    if (TOP) {
      if (C > 1) {
        // the CTAs' best, ranked again
        for (int i = tid; i < C * a.n_top; i += kThreads)
          s_keys[i] = cluster.map_shared_rank(&s_found, i / a.n_top)->best[i % a.n_top];
        __syncthreads();
      }
      const int n = C > 1 ? C * a.n_top : a.n_top;
      const Key* keys = C > 1 ? s_keys : s_found.best;
      for (int i = tid; i < n; i += kThreads) {
        const Key own = keys[i];
        int r = 0;
        for (int j = 0; j < n; ++j) r += keys[j] > own;
        if (own == 0)
          for (int j = 0; j < i; ++j) r += keys[j] == 0;
        if (r < a.n_top) {
          // none are left only where NaN is not among them: any id, NaN
          a.top_ids[row * a.n_top + r] = own == 0 ? r : (int32_t)(0xFFFFFFFFu - (uint32_t)own);
          a.top_logprobs[row * a.n_top + r] = own == 0 ? CUDART_NAN_F : logprob(unordered((uint32_t)(own >> 32)));
        }
      }
    }
  }
  allow_dependent_launch();
  if (C > 1) cluster.sync();   // the first CTA has read the others' memory
}

template <typename T, bool TOP>
cudaError_t launch_t(const LogprobsArgs& a, cudaStream_t s) {
  // CTAs a row: as many as run at once, at most a portable cluster, with at least 1,024 pieces each
  int C = kMaxCluster;
  while (C > 1 && (a.n_rows * C > 4 * device_sm_count() || (int64_t)a.V * (int)sizeof(T) < (int64_t)C * 16384)) C >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.n_rows * C));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Stream<TOP>::kBytes;
  static bool configured[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(token_logprobs_kernel<T, TOP>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               Stream<TOP>::kBytes);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = C;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T, TOP>, a);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobsArgs& a, bool bf16, cudaStream_t s) {
  if (bf16) return a.n_top > 0 ? launch_t<__nv_bfloat16, true>(a, s) : launch_t<__nv_bfloat16, false>(a, s);
  return a.n_top > 0 ? launch_t<float, true>(a, s) : launch_t<float, false>(a, s);
}

}  // namespace lynx
