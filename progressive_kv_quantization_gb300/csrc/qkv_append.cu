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

#include "f32x2.cuh"
#include "lynx_internal.cuh"

#include <cuda_bf16.h>

namespace lynx {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kTile = 32;                  // rows per CTA
constexpr int kBatch = 4;                  // query heads of a row read at once
constexpr int kPitch = kH / 2 + 1;         // words per staged token: the reading lanes (one token each) hit all banks

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
__device__ __forceinline__ uint4 norm_rotate(const uint4& x, const Turn& t, bool turned, bool norm, float eps) {
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
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const int o0 = INTERLEAVED ? i + 1 : i ^ 4, o1 = INTERLEAVED ? i : o0 + 1;
    float y0, y1;
    const uint64_t own = pair(a[i], a[i + 1]), other = pair(a[o0], a[o1]);
    const uint64_t c = pair(t.c[i], t.c[i + 1]), s = pair(t.s[i], t.s[i + 1]);
    uint64_t y;
    if (WHOLE) {
      y = fma2(own, c, mul2(other, s));
    } else {
      y = mul2(own, c);
      if (turned) y = fma2(other, s, y);
    }
    unpair(mul2(y, pair(r, r)), y0, y1);
    const __nv_bfloat162 p = __floats2bfloat162_rn(y0, y1);
    w[i / 2] = *reinterpret_cast<const uint32_t*>(&p);
  }
  if (!WHOLE && !norm) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = turned ? w[i] : xw[i];
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool INTERLEAVED, bool WHOLE>
__global__ void __launch_bounds__(kThreads, 4)
qkv_append_kernel(const AppendArgs a) {
  __shared__ uint32_t s_kv[2][kTile * kPitch];
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
  while (a.kv_parts < 8 && tiles * (a.q_jobs + a.Hkv * a.kv_parts) < 2 * device_sm_count()) a.kv_parts <<= 1;
  // Order of the CTAs: one job's tiles side by side (neighbours write
  // neighbouring slots while the lines are in L2), or, where rows and pages exceed
  // L2, one tile's jobs (what runs at a time reads whole rows of DRAM).  us for
  // 4,096 rows of 16 + 4 heads: 10.1 against 13.1; 40,000 rows of 32 + 8: 180
  // against 166.
  a.whole_rows = a.n_rows * (a.Hq + 2 * a.Hkv) * (4 * kH) > ((int64_t)100 << 20);
  const unsigned grid = (unsigned)(tiles * (a.q_jobs + a.Hkv * a.kv_parts));
  const bool whole = a.rot == kH;
  auto* const kernel = a.interleaved ? whole ? qkv_append_kernel<true, true> : qkv_append_kernel<true, false>
                                     : whole ? qkv_append_kernel<false, true> : qkv_append_kernel<false, false>;
  return launch_programmatic(kernel, dim3(grid), dim3(kThreads), 0, s, a);
}

}  // namespace lynx
