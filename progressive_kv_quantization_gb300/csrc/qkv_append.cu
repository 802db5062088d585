// New tokens' queries, keys and values on their way to attention
// (lynx_qkv_append): the RMS norm of each query and key head, the rotation by
// the token's position, and the keys and values written into the channel-major
// pages at their slots.
//
//   y = x rsqrt(mean_c x_c^2 + eps) w            (no norm without a weight)
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin) for the pairs (a, b) of
//   the first rot channels: (i, i + rot / 2), or (2i, 2i + 1) interleaved
// All in float32, rounded once to BF16.
//
// A half-warp holds one head of one row, 8 channels (16 bytes) a lane; a pair's
// other half is rot / 16 lanes away (a shuffle) or in the same lane.  A CTA
// takes 32 rows and either a group of query heads or one KV head (or a part of its
// channels).  Cosines and
// sines stay in registers over the heads of a row.  Keys and values pass
// through shared memory, token-major in, and leave with one token per lane:
// where slots follow one another (a chunk of one request) a warp's store is 64
// contiguous bytes of a channel row.

#include "lynx_internal.cuh"

#include <cuda_bf16.h>

namespace lynx {
namespace {

constexpr int kThreads = 256;
constexpr int kHalfWarps = kThreads / 16;
constexpr int kTile = 32;                  // rows per CTA
constexpr int kBatch = 4;                  // query heads of a row read at once
constexpr int kPitch = kH / 2 + 1;         // words per staged token: the reading lanes (one token each) hit all banks

struct Head {
  float v[8];
};

__device__ __forceinline__ Head unpack(const uint4& x) {
  Head h;
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    h.v[2 * i] = __uint_as_float(w[i] << 16);
    h.v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  return h;
}
__device__ __forceinline__ uint4 pack(const Head& h) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 p = __floats2bfloat162_rn(h.v[2 * i], h.v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// the lane's 8 factors of a norm weight; all lanes of a warp call the norm together
__device__ __forceinline__ void rms_norm(Head& h, const float (&w)[8], float eps) {
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(h.v[i], h.v[i], ss);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float r = rsqrtf(ss * (1.0f / kH) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) h.v[i] = h.v[i] * r * w[i];
}

// cosines and sines of the lane's 8 channels, sines signed: y = y cos + other sin
struct Turn {
  float c[8], s[8];
};

template <bool INTERLEAVED>
__device__ __forceinline__ Turn load_turn(const float* row, int rot, int lane16) {
  Turn t;
  const int half = rot >> 1, c0 = 8 * lane16;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    t.c[i] = 1.0f;
    t.s[i] = 0.0f;
  }
  if (c0 < rot) {
    if (INTERLEAVED) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + c0 / 2));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + c0 / 2));
      const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        t.c[2 * i] = t.c[2 * i + 1] = cc[i];
        t.s[2 * i] = -sc[i];
        t.s[2 * i + 1] = sc[i];
      }
    } else {
      const bool low = c0 < half;
      const int i0 = low ? c0 : c0 - half;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const float4 c = __ldg(reinterpret_cast<const float4*>(row + i0 + 4 * q));
        const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i0 + 4 * q));
        const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          t.c[4 * q + i] = cc[i];
          t.s[4 * q + i] = low ? -sc[i] : sc[i];
        }
      }
    }
  }
  return t;
}

template <bool INTERLEAVED>
__device__ __forceinline__ void rotate(Head& h, const Turn& t, int partner) {
  Head o;
#pragma unroll
  for (int i = 0; i < 8; ++i) o.v[i] = INTERLEAVED ? h.v[i ^ 1] : __shfl_sync(0xffffffffu, h.v[i], partner);
#pragma unroll
  for (int i = 0; i < 8; ++i) h.v[i] = fmaf(h.v[i], t.c[i], o.v[i] * t.s[i]);
}

template <bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 4)
qkv_append_kernel(const AppendArgs a) {
  __shared__ uint32_t s_kv[2][kTile * kPitch];
  const int tid = threadIdx.x, lane = tid & 31, lane16 = tid & 15, hw = tid >> 4;
  const unsigned n_jobs = a.q_jobs + a.Hkv * a.kv_parts, n_tiles = (unsigned)((a.n_rows + kTile - 1) / kTile);
  const int job = (int)(a.whole_rows ? blockIdx.x % n_jobs : blockIdx.x / n_tiles);
  const int64_t row0 = (int64_t)(a.whole_rows ? blockIdx.x / n_jobs : blockIdx.x % n_tiles) * kTile;
  const bool is_kv = job >= a.q_jobs;
  const int kv_head = is_kv ? (job - a.q_jobs) / a.kv_parts : 0;
  const int half = a.rot >> 1;
  // the lane that holds the other halves of this lane's pairs
  int partner = lane;
  if (!INTERLEAVED && 8 * lane16 < a.rot) partner = 8 * lane16 < half ? lane + half / 8 : lane - half / 8;

  const float* weight = is_kv ? a.k_weight : a.q_weight;
  float w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = weight ? weight[8 * lane16 + i] : 1.0f;

  const int h0 = is_kv ? a.Hq + kv_head : job * a.heads_per_job;
  const int h1 = is_kv ? h0 + 1 : min(h0 + a.heads_per_job, a.Hq);

  int positions[kTile / kHalfWarps];
#pragma unroll
  for (int k = 0; k < kTile / kHalfWarps; ++k) {
    const int64_t row = row0 + k * kHalfWarps + hw;
    positions[k] = row < a.n_rows ? __ldg(a.positions + row) : -1;
  }
#pragma unroll
  for (int k = 0; k < kTile / kHalfWarps; ++k) {
    const int t = k * kHalfWarps + hw;
    const int64_t row = row0 + t;
    const int pos = positions[k];
    const bool far = pos >= a.max_pos && a.rot > 0;
    if (far && lane16 == 0) atomicExch(a.status, 4);
    const bool on = pos >= 0 && !far;
    const Turn turn = load_turn<INTERLEAVED>(a.cos_sin + (int64_t)(on ? pos : 0) * a.rot, a.rot, lane16);
    const uint4* src = reinterpret_cast<const uint4*>(a.qkv + (on ? row : 0) * a.row_stride) + lane16;
    if (!is_kv) {
      for (int h = h0; h < h1; h += kBatch) {
        uint4 x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          x[i] = make_uint4(0u, 0u, 0u, 0u);
          if (on && h + i < h1) x[i] = __ldg(src + (h + i) * (kH / 8));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          if (h + i >= h1) break;
          Head y = unpack(x[i]);
          if (weight) rms_norm(y, w, a.norm_eps);
          if (a.rot > 0) rotate<INTERLEAVED>(y, turn, partner);
          if (on) *(reinterpret_cast<uint4*>(a.q_out + (row * a.Hq + h + i) * kH) + lane16) = pack(y);
        }
      }
    } else {
      uint4 x = make_uint4(0u, 0u, 0u, 0u), v = x;
      if (on) {
        x = __ldg(src + h0 * (kH / 8));
        v = __ldg(src + (h0 + a.Hkv) * (kH / 8));
      }
      Head y = unpack(x);
      if (weight) rms_norm(y, w, a.norm_eps);
      if (a.rot > 0) rotate<INTERLEAVED>(y, turn, partner);
      const uint4 r = pack(y);
      uint32_t* dk = s_kv[0] + t * kPitch + 4 * lane16;
      uint32_t* dv = s_kv[1] + t * kPitch + 4 * lane16;
      dk[0] = r.x; dk[1] = r.y; dk[2] = r.z; dk[3] = r.w;
      dv[0] = v.x; dv[1] = v.y; dv[2] = v.z; dv[3] = v.w;
    }
  }
  if (!is_kv) return;
  __syncthreads();
  // one token per lane, a pair of channels at a time
  const int64_t row = row0 + lane;
  int64_t slot = -1;
  if (row < a.n_rows) {
    const int pos = __ldg(a.positions + row);
    if (pos >= 0 && (pos < a.max_pos || a.rot == 0)) slot = a.slots[row * a.Hkv + kv_head];
    if (slot >= a.n_pool * kP) {
      if (tid < 32) atomicExch(a.status, 5);
      slot = -1;
    }
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
  // 4,096 rows of 16 + 4 heads: 11.1 against 13.4; 40,000 rows of 32 + 8: 206
  // against 190.
  a.whole_rows = a.n_rows * (a.Hq + 2 * a.Hkv) * (4 * kH) > ((int64_t)100 << 20);
  const unsigned grid = (unsigned)(tiles * (a.q_jobs + a.Hkv * a.kv_parts));
  if (a.interleaved)
    qkv_append_kernel<true><<<grid, kThreads, 0, s>>>(a);
  else
    qkv_append_kernel<false><<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lynx
