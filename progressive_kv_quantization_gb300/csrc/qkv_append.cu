// New tokens' queries, keys and values on their way to attention
// (lynx_qkv_append): the RMS norm of each query and key head, the rotation by
// the token's position, and the keys and values written into the channel-major
// pages at their slots.
//
//   y = x rsqrt(mean_c x_c^2 + eps) w            (no norm without a weight)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin) for the pairs (a, b) of
//   the first rot channels: (i, i + rot / 2), or (2i, 2i + 1) interleaved
// computed as rsqrt(..) (x_a (w_a cos) - x_b (w_b sin)), the brackets once for a
// row and all its heads; float32, rounded once to BF16.
//
// A half-warp holds one head of one row, 8 channels (16 bytes) a lane: 8 neighbours, or
// for half-split pairs four of the first half and the four that belong to them, so
// that a pair is in one lane (16 + 4 heads, 4,096 rows: 10.1 us; with 8 neighbours and an
// exchange between lanes 12.5).  A CTA takes 32 rows and either a group of query heads or
// one KV head (or a part of its channels).  Cosines and sines stay in registers over
// the heads of a row.  Keys and values pass through shared memory, token-major in, and
// leave with one token per lane: where slots follow one another (a chunk of one request)
// a warp's store is 64 contiguous bytes of a channel row.
//
// What bounds it on a GB300.  Many rows: memory; 40,000 rows of 32 + 8 heads take 166 us,
// 6.1 TB/s read and written (90% of a copy; the slots' 2-byte stores meet in L2, DRAM
// moves the algorithmic bytes), 27,292 rows with norms and a half of each head rotated
// interleaved 124 us (81%).  Some thousand rows, all in L2: latency at 32 warps an SM (64
// registers; 5.2 TB/s for 4,096 rows of 16 + 4 heads).  A decode step of 64 rows (2.8 us):
// the launch, the position and then the cosines at it.
//
// Pages in 8 bits (lynx_qkv_append_e4m3).  A block of 32 tokens has one scale, so that its
// new rows (a run: rows that follow one another in one block, whether or not all of them are
// written) are quantised together, and what stands in front of them is rounded again where the
// scale grows.  A CTA takes the
// runs that begin in its 32 rows, from the first one's first row on: 32 rows in registers, and where
// there are several runs up to 31 more in shared memory, wait as float32 for the runs' maxima.  A page's
// token is then one 128-byte store.
// Powers of two as scales make the rounding that of E4M3 alone, and rounding a code
// again under a larger one changes it only where it becomes subnormal.  27,292 rows of 32 + 8
// heads, half rotated: 121 us, 5.2 TB/s (76% of a copy), bound by instructions (issue slots 74%
// busy): 145 us with the rows put through shared memory between the two barriers.
// 3,689 rows of 16 + 4: 11.0 to 13.7 us, 64 rows of 32 + 8: 4.4 us, and where every block's scale grows
// 10 and 15 us with 15 and 31 tokens in front of each row.

#include "e4m3.cuh"
#include "f32x2.cuh"
#include "lynx_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>

namespace lynx {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kTile = 32;                  // rows per CTA
constexpr int kBatch = 4;                  // query heads of a row read at once
constexpr int kPitch = kH / 2 + 1;         // words per staged token: the reading lanes (one token each) hit all banks
constexpr int kRows8 = kTile - 1;          // pages in 8 bits: rows behind the first 32 that a tile's runs reach
constexpr int kSmem8 = kRows8 * kH * 6;    // their keys (float32) and values (BF16)

__device__ __forceinline__ void load4(const float* p, float* v) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
}

// A row's rotation with the norm weight in it, for the lane's 8 channels: with x'
// the pairs' other halves, y = rsqrt(..) (x c + x' s)
struct Turn {
  float c[8], s[8];
};

// `row`: the position's cosines and sines; ca, cb: the lane's channels, four from
// each (INTERLEAVED or behind the rotated ones: cb = ca + 4)
template <bool INTERLEAVED>
__device__ __forceinline__ Turn load_turn(const float* row, int rot, const float* weight, int ca, int cb) {
  Turn t;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.0f;
    t.s[i] = 0.0f;
  }
  if (ca < rot) {
    float c[4], s[4];
    load4(row + (INTERLEAVED ? ca / 2 : ca), c);
    load4(row + rot / 2 + (INTERLEAVED ? ca / 2 : ca), s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lo = INTERLEAVED ? 2 * i : i, hi = INTERLEAVED ? 2 * i + 1 : i + 4;
      t.c[lo] = t.c[hi] = c[i];
      t.s[lo] = -s[i];
      t.s[hi] = s[i];
    }
  }
  if (weight) {
    float w[8];
    load4(weight + ca, w);
    load4(weight + cb, w + 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t.c[i] *= w[i];
      t.s[i] *= w[INTERLEAVED ? i ^ 1 : i ^ 4];
    }
  }
  return t;
}

// One head; all lanes of a warp together.  Two channels an instruction.  turned: the
// lane's channels are rotated (WHOLE: every lane's).  Others take nothing from their
// partners, not even 0 times them, which is NaN where the partner is not finite; without
// a norm they are copied.  (That costs 27,292 rows with half of each head rotated 3 us;
// heads rotated as a whole have a kernel of their own, without it.)
template <bool INTERLEAVED, bool WHOLE>
__device__ __forceinline__ void norm_rotate(const uint4& x, const Turn& t, bool turned, bool norm, float eps, float* out) {
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
  float a[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    a[2 * i] = __uint_as_float(xw[i] << 16);
    a[2 * i + 1] = __uint_as_float(xw[i] & 0xFFFF0000u);
  }
  float r = 1.0f;
  if (norm) {
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], ss);
#pragma unroll
    for (int k = 8; k > 0; k >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, k);
    r = rsqrtf(ss * (1.0f / kH) + eps);
  }
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int o0 = INTERLEAVED ? i + 1 : i ^ 4, o1 = INTERLEAVED ? i : o0 + 1;
    const uint64_t own = pair(a[i], a[i + 1]), other = pair(a[o0], a[o1]);
    const uint64_t c = pair(t.c[i], t.c[i + 1]), s = pair(t.s[i], t.s[i + 1]);
    uint64_t y;
    if (WHOLE) {
      y = fma2(own, c, mul2(other, s));
    } else {
      y = mul2(own, c);
      if (turned) y = fma2(other, s, y);
    }
    unpair(mul2(y, pair(r, r)), out[i], out[i + 1]);
  }
}
// the same, rounded
template <bool INTERLEAVED, bool WHOLE>
__device__ __forceinline__ uint4 norm_rotate(const uint4& x, const Turn& t, bool turned, bool norm, float eps) {
  float y[8];
  norm_rotate<INTERLEAVED, WHOLE>(x, t, turned, norm, eps, y);
  const uint32_t xw[4] = {x.x, x.y, x.z, x.w};
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(y[i], y[i + 1]);
    w[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
  }
  if (!WHOLE && !norm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = turned ? w[i] : xw[i];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// four float32 values as codes
__device__ __forceinline__ uint32_t e4m3x4(float x0, float x1, float x2, float x3) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1), "f"(x0));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3), "f"(x2));
  return (uint32_t)lo | (uint32_t)hi << 16;
}
// four codes times f, rounded once
__device__ __forceinline__ uint32_t rescaled(uint32_t codes, float f) {
  const uint32_t lo = f16x2_of(codes), hi = f16x2_of_high(codes);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&lo)), y = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return e4m3x4(x.x * f, x.y * f, y.x * f, y.y * f);
}

// E: pages in 8 bits
template <bool INTERLEAVED, bool WHOLE, bool E>
__global__ void __launch_bounds__(kThreads, 4)
qkv_append_kernel(const AppendArgs a) {
  __shared__ uint32_t s_kv[2][E ? 1 : kTile * kPitch];
  const int tid = threadIdx.x, lane = tid & 31, lane16 = tid & 15, hw = tid >> 4;
  const unsigned n_jobs = a.q_jobs + a.Hkv * a.kv_parts, n_tiles = (unsigned)((a.n_rows + kTile - 1) / kTile);
  const int job = (int)(a.whole_rows ? blockIdx.x % n_jobs : blockIdx.x / n_tiles);
  const int64_t row0 = (int64_t)(a.whole_rows ? blockIdx.x / n_jobs : blockIdx.x % n_tiles) * kTile;
  const bool is_kv = job >= a.q_jobs;
  const int kv_head = is_kv ? (job - a.q_jobs) / a.kv_parts : 0;
  // the lane's channels: four at ca and four at cb, so that a pair's halves are in
  // one lane
  const bool apart = !INTERLEAVED && 8 * lane16 < a.rot;
  const int ca = (apart ? 4 : 8) * lane16, cb = apart ? ca + a.rot / 2 : ca + 4;
  allow_dependent_launch();
  wait_prerequisite_grids();
  const float* weight = is_kv ? a.k_weight : a.q_weight;
  auto finish = [&](const uint4& x, const Turn& turn) {
    return norm_rotate<INTERLEAVED, WHOLE>(x, turn, 8 * lane16 < a.rot, weight != nullptr, a.norm_eps);
  };
  // position of a row that takes part, or -1
  auto checked = [&](int pos) {
    if (a.rot > 0 && pos >= a.max_pos) {
      if (lane16 == 0) atomicExch(a.status, 4);
      return -1;
    }
    return pos;
  };
  auto turn_at = [&](int pos) {
    return load_turn<INTERLEAVED>(a.cos_sin + (int64_t)(pos < 0 ? 0 : pos) * a.rot, a.rot, weight, ca, cb);
  };
  // heads are read before their row's position is known (what is skipped is not written)
  auto head_at = [&](int64_t row, int h) {
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    if (row < a.n_rows) {
      const uint16_t* src = a.qkv + row * a.row_stride + (int64_t)h * kH;
      if (INTERLEAVED) {
        x = *reinterpret_cast<const uint4*>(src + ca);
      } else {
        const uint2 lo = *reinterpret_cast<const uint2*>(src + ca), hi = *reinterpret_cast<const uint2*>(src + cb);
        x = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
    return x;
  };
  constexpr int kSteps = kTile / kHalfWarps;   // rows of a half-warp
  const int64_t row_hw = row0 + hw;
  int pos[kSteps];
#pragma unroll
  for (int k = 0; k < kSteps; ++k) {
    const int64_t row = row_hw + k * kHalfWarps;
    pos[k] = row < a.n_rows ? a.positions[row] : -1;
  }

  if (!is_kv) {
    // ---- queries, kBatch heads at a time, the next ones on their way
    const int h0 = job * a.heads_per_job, h1 = min(h0 + a.heads_per_job, a.Hq);
    uint4 x[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h0 + i < h1) x[i] = head_at(row_hw, h0 + i);
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int64_t row = row_hw + k * kHalfWarps;
      const int p = checked(pos[k]);
      const Turn turn = turn_at(p);
      for (int h = h0; h < h1; h += kBatch) {
        uint4 next[kBatch];
        const bool last = h + kBatch >= h1;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int hn = last ? h0 + i : h + kBatch + i;
          if (hn < h1 && (!last || k + 1 < kSteps)) next[i] = head_at(last ? row + kHalfWarps : row, hn);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (h + i >= h1) break;
          const uint4 r = finish(x[i], turn);
          if (p < 0) continue;
          uint16_t* dst = a.q_out + (row * a.Hq + h + i) * kH;
          if (INTERLEAVED) {
            *reinterpret_cast<uint4*>(dst + ca) = r;
          } else {
            *reinterpret_cast<uint2*>(dst + ca) = make_uint2(r.x, r.y);
            *reinterpret_cast<uint2*>(dst + cb) = make_uint2(r.z, r.w);
          }
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) x[i] = next[i];
      }
    }
    return;
  }

  if constexpr (E) {
    // ---- a KV head into blocks of 32 tokens
    extern __shared__ __align__(16) float s_dyn[];
    float4* s_k = reinterpret_cast<float4*>(s_dyn);                        // [row][the lane's two fours][lane]
    uint4* s_v = reinterpret_cast<uint4*>(s_dyn + kRows8 * kH);            // [row][lane]
    __shared__ int64_t s_slots[3 * kTile - 1];
    int64_t* const s_slot = s_slots + kTile - 1;   // [i]: of row row0 - 1 + i, from i = -31 on; -1: not written
    __shared__ uint32_t s_top[2][2 * kTile]; // at a run's first row: largest magnitude of keys and values, as bits
    __shared__ int s_pos[2 * kTile], s_old[2 * kTile];
    if (tid < 3 * kTile - 1) {
      const int i = tid - (kTile - 1);
      const int64_t row = row0 - 1 + i;
      int64_t slot = row < 0 ? INT64_MAX : -1;   // (nothing goes on from in front of the first row)
      int p = -1;
      if (row >= 0 && row < a.n_rows) {
        p = a.positions[row];
        slot = a.slots[row * a.Hkv + kv_head];
        if (a.rot > 0 && p >= a.max_pos) {
          if (i > 0 && i <= kTile) atomicExch(a.status, 4);
          p = -1;
        }
        if (p < 0) slot = -1;
        if (slot >= a.n_pool * kP) {
          atomicExch(a.status, 5);
          slot = -1;
        }
      }
      s_slot[i] = slot < 0 ? -1 : slot;
      if (i >= 0) {
        s_pos[i] = p;
        s_top[0][i] = s_top[1][i] = 0u;
      }
    }
    __syncthreads();
    // Rows that begin a run, as every warp sees them.  One that is not written does not end it: with
    // two runs in one block, each would take the scale that the block had before the call, and both
    // would set it.
    unsigned long long starts = 0;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int i = 32 * x + lane;
      const int64_t slot = s_slot[i], before = s_slot[i - 1];
      bool first = i > 0 && slot >= 0 && (slot % kC == 0 || before != slot - 1);
      if (__any_sync(0xffffffffu, first && before < 0)) {   // is there one of the block in front of such rows?
#pragma unroll 1
        for (int d = 2; first && d <= (int)(slot % kC) && s_slot[i - d + 1] < 0; ++d) first = s_slot[i - d] != slot - d;
        __syncwarp();
      }
      starts |= (unsigned long long)__ballot_sync(0xffffffffu, first) << (32 * x);
    }
    // first row of row i's run, or 0 if that is none of the tile's
    auto run_of = [&](int i) {
      const int st = i < 2 * kTile && s_slot[i] >= 0 ? 63 - __clzll((long long)(starts & ((2ull << i) - 1))) : 0;
      return st > 0 && st <= kTile ? st : 0;
    };
    // The tile's runs, from the first one's first row on; 32 rows unless there are several
    const unsigned own = (unsigned)(starts >> 1);
    if (own == 0) return;
    const int i0 = __ffs(own);
    // and up to 31 rows behind the last one's first, or the next tile's first run
    const unsigned next = (unsigned)(starts >> 33);
    const int i1 = min(32 - __clz(own) + kTile - 1, next ? 32 + __ffs(next) - 1 : 2 * kTile - 1);
    // a key's channels from the lane, and the largest magnitudes of both to the row's run
    auto prepare = [&](int i, int run, const uint4& xk_i, const uint4& xv_i, float* y) {
      norm_rotate<INTERLEAVED, WHOLE>(xk_i, turn_at(run ? s_pos[i] : -1), 8 * lane16 < a.rot, weight != nullptr, a.norm_eps, y);
      float mk = fmaxf(fabsf(y[0]), fabsf(y[1]));
#pragma unroll
      for (int e = 2; e < 8; ++e) mk = fmaxf(mk, fabsf(y[e]));
      const __nv_bfloat162* v2 = reinterpret_cast<const __nv_bfloat162*>(&xv_i);
      const __nv_bfloat162 v4 = __hmax2(__hmax2(__habs2(v2[0]), __habs2(v2[1])), __hmax2(__habs2(v2[2]), __habs2(v2[3])));
      // (a maximum of nothing but NaN counts as 0: the block's other tokens keep their scale)
      uint32_t top_k = __float_as_uint(fmaxf(mk, 0.0f)), top_v = __float_as_uint(fmaxf(fmaxf(__low2float(v4), __high2float(v4)), 0.0f));
      // a maximum does not depend on the order
      if (__all_sync(0xffffffffu, run == __shfl_sync(0xffffffffu, run, 0))) {   // both rows of one run, as in a prompt
        top_k = __reduce_max_sync(0xffffffffu, top_k);
        top_v = __reduce_max_sync(0xffffffffu, top_v);
        if (lane == 0 && run > 0) {
          atomicMax(&s_top[0][run], top_k);
          atomicMax(&s_top[1][run], top_v);
        }
      } else {
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) {
          top_k = max(top_k, __shfl_xor_sync(0xffffffffu, top_k, o));
          top_v = max(top_v, __shfl_xor_sync(0xffffffffu, top_v, o));
        }
        if (lane16 == 0 && run > 0) {
          atomicMax(&s_top[0][run], top_k);
          atomicMax(&s_top[1][run], top_v);
        }
      }
    };
    // the scales that a run's block had, 0 if the run begins the block: the keys' in the lower half
    if (tid > 0 && tid <= kTile && run_of(tid) == tid) {
      const int64_t first = s_slot[tid];
      const uint8_t* s = a.scales + first / kP * kScaleBytes + first % kP / kC;
      s_old[tid] = first % kC == 0 ? 0 : min(max((int)s[0], kScaleLo), kScaleHi) | min(max((int)s[kChunks], kScaleLo), kScaleHi) << 16;
    }
    float y[kSteps][8];
    uint4 xv[kSteps];
    int run[kSteps];
    {
      uint4 xk[kSteps];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int i = i0 + k * kHalfWarps + hw;
        run[k] = run_of(i);
        const int64_t row = run[k] ? row0 + i - 1 : a.n_rows;   // (none is read there)
        xk[k] = head_at(row, a.Hq + kv_head);
        xv[k] = head_at(row, a.Hq + a.Hkv + kv_head);
      }
#pragma unroll
      for (int k = 0; k < kSteps; ++k)
        if (__any_sync(0xffffffffu, run[k] > 0)) prepare(i0 + k * kHalfWarps + hw, run[k], xk[k], xv[k], y[k]);
    }
    // rows behind the first 32, of several runs: their keys and values wait in shared memory
    constexpr int kBehind = kTile;
#pragma unroll 1
    for (int i = i0 + kBehind + hw; i - hw <= i1; i += kHalfWarps) {
      const int run = run_of(i), place = i - i0 - kBehind;
      if (!__any_sync(0xffffffffu, run > 0)) continue;
      const int64_t row = run ? row0 + i - 1 : a.n_rows;
      const uint4 v = head_at(row, a.Hq + a.Hkv + kv_head);
      float z[8];
      prepare(i, run, head_at(row, a.Hq + kv_head), v, z);
      if (run > 0) {
        s_k[place * 32 + lane16] = make_float4(z[0], z[1], z[2], z[3]);
        s_k[place * 32 + 16 + lane16] = make_float4(z[4], z[5], z[6], z[7]);
        s_v[place * 16 + lane16] = v;
      }
    }
    __syncthreads();
    auto write = [&](int i, int run, const float* y, const uint4& v) {
      if (run == 0) return;
      const int64_t slot = s_slot[i];
      const int old_k = s_old[run] & 0xFFFF, old_v = s_old[run] >> 16;
      const int sk = max(scale_byte(__uint_as_float(s_top[0][run])), old_k);
      const int sv = max(scale_byte(__uint_as_float(s_top[1][run])), old_v);
      const float fk = __uint_as_float((uint32_t)(254 - sk) << 23), fv = __uint_as_float((uint32_t)(254 - sv) << 23);
      auto low = [&](uint32_t w) { return __uint_as_float(w << 16) * fv; };
      auto high = [&](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u) * fv; };
      uint8_t* kd = a.k_codes + slot * kH;
      uint8_t* vd = a.v_codes + slot * kH;
      const uint2 kc = make_uint2(e4m3x4(y[0] * fk, y[1] * fk, y[2] * fk, y[3] * fk), e4m3x4(y[4] * fk, y[5] * fk, y[6] * fk, y[7] * fk));
      const uint2 vc = make_uint2(e4m3x4(low(v.x), high(v.x), low(v.y), high(v.y)), e4m3x4(low(v.z), high(v.z), low(v.w), high(v.w)));
      if (INTERLEAVED) {
        *reinterpret_cast<uint2*>(kd + ca) = kc;
        *reinterpret_cast<uint2*>(vd + ca) = vc;
      } else {
        *reinterpret_cast<uint32_t*>(kd + ca) = kc.x;
        *reinterpret_cast<uint32_t*>(kd + cb) = kc.y;
        *reinterpret_cast<uint32_t*>(vd + ca) = vc.x;
        *reinterpret_cast<uint32_t*>(vd + cb) = vc.y;
      }
      if (i != run) return;
      // the block's scales, and what stands in front of the run under grown ones
      if (lane16 == 0) {
        uint8_t* s = a.scales + slot / kP * kScaleBytes + slot % kP / kC;
        s[0] = (uint8_t)sk;
        s[kChunks] = (uint8_t)sv;
      }
      const int64_t first = slot / kC * kC;
#pragma unroll 1
      for (int which = 0; which < 2; ++which) {
        const int was = which ? old_v : old_k, now = which ? sv : sk;
        if (was == 0 || now <= was) continue;
        const float f = now - was > 126 ? 0.0f : __uint_as_float((uint32_t)(127 - (now - was)) << 23);
        for (int64_t t = first; t < slot; ++t) {
          uint2* d = reinterpret_cast<uint2*>((which ? a.v_codes : a.k_codes) + t * kH) + lane16;
          const uint2 x = *d;
          *d = make_uint2(rescaled(x.x, f), rescaled(x.y, f));
        }
      }
    };
#pragma unroll
    for (int k = 0; k < kSteps; ++k) write(i0 + k * kHalfWarps + hw, run[k], y[k], xv[k]);
#pragma unroll 1
    for (int i = i0 + kBehind + hw; i <= i1; i += kHalfWarps) {
      const int run = run_of(i), place = i - i0 - kBehind;
      if (run == 0) continue;
      const float4 k0 = s_k[place * 32 + lane16], k1 = s_k[place * 32 + 16 + lane16];
      const float z[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
      write(i, run, z, s_v[place * 16 + lane16]);
    }
  } else {
    // ---- a KV head: keys and values to shared memory, then out by channel
    uint4 xk[kSteps], xv[kSteps];
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      xk[k] = head_at(row_hw + k * kHalfWarps, a.Hq + kv_head);
      xv[k] = head_at(row_hw + k * kHalfWarps, a.Hq + a.Hkv + kv_head);
    }
    const int64_t slot_row = row0 + lane;
    const int slot_pos = slot_row < a.n_rows ? a.positions[slot_row] : -1;
    int64_t slot = slot_row < a.n_rows ? a.slots[slot_row * a.Hkv + kv_head] : -1;
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const int t = k * kHalfWarps + hw;
      const uint4 r = finish(xk[k], turn_at(checked(pos[k])));
      const uint4 v = xv[k];
      uint32_t* dk = s_kv[0] + t * kPitch;
      uint32_t* dv = s_kv[1] + t * kPitch;
      dk[ca / 2] = r.x; dk[ca / 2 + 1] = r.y; dk[cb / 2] = r.z; dk[cb / 2 + 1] = r.w;
      dv[ca / 2] = v.x; dv[ca / 2 + 1] = v.y; dv[cb / 2] = v.z; dv[cb / 2 + 1] = v.w;
    }
    __syncthreads();
    // one token per lane, a pair of channels at a time
    if (slot_pos < 0 || (a.rot > 0 && slot_pos >= a.max_pos)) slot = -1;
    if (slot >= a.n_pool * kP) {
      if (tid < 32) atomicExch(a.status, 5);
      slot = -1;
    }
    if (slot >= 0) {
      const int64_t at = (slot / kP) * kPageElems + slot % kP;
      uint16_t* kd = a.k_pages + at;
      uint16_t* vd = a.v_pages + at;
      // the part's channel pairs
      const int n_c2 = kH / 2 / a.kv_parts, c20 = (job - a.q_jobs) % a.kv_parts * n_c2;
#pragma unroll 4
      for (int c2 = c20 + (tid >> 5); c2 < c20 + n_c2; c2 += kThreads / 32) {
        const uint32_t kw = s_kv[0][lane * kPitch + c2], vw = s_kv[1][lane * kPitch + c2];
        kd[(2 * c2) * kP] = (uint16_t)kw;
        kd[(2 * c2 + 1) * kP] = (uint16_t)(kw >> 16);
        vd[(2 * c2) * kP] = (uint16_t)vw;
        vd[(2 * c2 + 1) * kP] = (uint16_t)(vw >> 16);
      }
    }
  }
}

template <bool E>
cudaError_t launch_kernel(const AppendArgs& a, unsigned grid, cudaStream_t s) {
  const bool whole = a.rot == kH;
  auto* const kernel = a.interleaved ? whole ? qkv_append_kernel<true, true, E> : qkv_append_kernel<true, false, E>
                                     : whole ? qkv_append_kernel<false, true, E> : qkv_append_kernel<false, false, E>;
  if (E) {
    static bool configured[64][4] = {{false}};
    int dev = 0;
    cudaGetDevice(&dev);
    bool* done = dev >= 0 && dev < 64 ? &configured[dev][2 * (a.interleaved != 0) + whole] : nullptr;
    if (!done || !*done) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem8);
      if (e != cudaSuccess) return e;
      if (done) *done = true;
    }
  }
  return launch_programmatic(kernel, dim3(grid), dim3(kThreads), E ? kSmem8 : 0, s, a);
}

}  // namespace

cudaError_t launch_qkv_append(AppendArgs a, cudaStream_t s) {
  const int64_t tiles = (a.n_rows + kTile - 1) / kTile;
  // query heads per CTA: eight, or fewer while the grid would leave SMs idle
  a.heads_per_job = 8;
  while (a.heads_per_job > 1 && tiles * (a.Hkv + (a.Hq + a.heads_per_job - 1) / a.heads_per_job) < 2 * device_sm_count())
    a.heads_per_job >>= 1;
  a.q_jobs = (a.Hq + a.heads_per_job - 1) / a.heads_per_job;
  // few rows: the channels of a KV head's keys and values are written by up to
  // eight CTAs (each norms and rotates the whole head), since every token of a
  // decode step writes 2 bytes of a sector of its own in each channel
  a.kv_parts = 1;
  while (!a.k_codes && a.kv_parts < 8 && tiles * (a.q_jobs + a.Hkv * a.kv_parts) < 2 * device_sm_count()) a.kv_parts <<= 1;
  // Order of the CTAs: one job's tiles side by side (neighbours write
  // neighbouring slots while the lines are in L2), or, where rows and pages exceed
  // L2, one tile's jobs (what runs at a time reads whole rows of DRAM).  us for
  // 4,096 rows of 16 + 4 heads: 10.1 against 13.1; 40,000 rows of 32 + 8: 180
  // against 166.
  a.whole_rows = a.n_rows * (a.Hq + 2 * a.Hkv) * (4 * kH) > ((int64_t)100 << 20);
  const unsigned grid = (unsigned)(tiles * (a.q_jobs + a.Hkv * a.kv_parts));
  return a.k_codes ? launch_kernel<true>(a, grid, s) : launch_kernel<false>(a, grid, s);
}

}  // namespace lynx
