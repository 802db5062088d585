// Decode and verification attention over pages in 8 bits
// (lynx_decode_attn_e4m3): a few query rows a KV head, dequantised on the way to
// the tensor cores.
//
//   x = code 2^(s - 127) with one s for 32 tokens of a head's keys, one for its values
//   S = Q K^T,  p = 2^(c S - m),  O = (sum p V) / (sum p),  lse = (m + log2 sum p) ln 2
//
// A CTA takes 8, 16 or 24 query rows (NT tiles of 8) of a request and KV head and goes
// through the keys in units of half a page (128 tokens; a page for 24 rows), K and V tile one
// behind the other through a ring that one lane fills by TMA.  Each of four (eight) warps owns a
// block of 32 tokens of every unit, with a softmax of its own, and they are joined at the end.  Two
// CTAs an SM (one): what one waits for (a join, an item's first copy) the other covers.
//
//   K side  f16 m16n8k16.  A lane reads 16 codes of a token at once; a k-step takes 4 of them, so
//           that channels come in the order (64 j + 16 t + 4 w ..) and the query fragments with
//           them.  The token of place n of 8 is (n >> 1) + 4 (n & 1): lanes that read together
//           then hit rows that differ in bit 2, whose 16-byte pieces the 128-byte swizzle of the
//           copy keeps in other banks.  Up to 8 rows: S = Q K^T, query rows as M (half of it
//           empty), and P stands as the V side wants it.  More rows: S^T = K Q^T, half the products a
//           row, and P is transposed 8 x 8 at a time (one tile of 8 rows that way: 159 us for the
//           48 requests below against 155).
//   V side  U[16 channels x 8 rows] = V P^T, channels as M.  A lane reads 16 channels of
//           four tokens, 8 at a time, and interleaves two tokens' bytes (prmt); a code pair
//           becomes an FP16 pair in one instruction.  Lane group g holds channels 16 c(g) .. + 15,
//           c(g) = (g >> 1) + 4 (g & 1), for the banks' sake again.
//
// Numbers.  Codes are exact in FP16.  A query row is scaled by a power of two to a
// largest value of 2^14..2^15, which leaves BF16's 8 bits exact down to 2^-30 of it.  p is
// split into two FP16 numbers (2^10 p, so that what is below 2^-35 is lost), 22 bits;
// products sum in float32.  A block's scales are factors of its scores' (warp-wide) and of
// its U, which is added to O in float32: the tensor core's accumulators, which cut off and
// do not round, only ever sum 32 tokens.  Of p a unit's are summed before they go to the row's
// sum: roundings that all go one way make 1.4e-5 of it over 1,024 units, one by one 1.2e-4.
//
// Work split: the units of all requests and heads (and kItemCost for the start and end of
// each) stand on one line that is cut into equal parts, one a CTA.  A CTA whose part
// begins or ends inside an item leaves O, m and l in the workspace, and
// decode_e4m3_join adds up what belongs together; ragged batches and one long
// context fill the machine alike, and nothing depends on timing.
//
// What bounds it (GB300, 128 channels).  Up to 8 rows: memory.  48 requests of up to 16,383 keys, 32 / 8
// heads: 155 us, 6.5 TB/s of codes and scales (95% of a copy); 4 of 131,071, 64 / 8: 83 us (90%, of
// which some 8 us are the start, the last units and the join).  One request of 983 keys: 8.0 us, the two
// launches and one unit's chain.  More rows: latency, at two warps a scheduler that the registers of
// O leave; 5 tokens of 8 requests up to 32,000 keys, 16 / 4 heads (20 rows): 60 us against 26 of
// memory, tensor pipe 41% busy, an instruction every 6.3 clocks of a warp.
//
// A warp that has given up a wait goes on through the items without waiting or
// reading, because the others meet it at the joins.

#include "e4m3.cuh"
#include "lynx_internal.cuh"
#include "tma_ptx.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

namespace lynx {
namespace {

constexpr int kSlots = 5;
constexpr int kItemCost = 1;                  // units
constexpr int kMinCost = 2;                   // units of a CTA's part, at least
constexpr int kMaxCtas = 512;
constexpr int kQPitch = 2 * kH + 16;          // bytes of a query row
constexpr int kOPitch = kH + 4;               // floats of a row at the join of the warps
constexpr float kLazyLog2 = 5.0f;             // lead of a score over the running maximum that moves it
constexpr float kUpLog2 = 10.0f;              // p is held times 2^10
constexpr float kLn2 = 0.6931471805599453f;

// NT: tiles of 8 query rows, W: consuming warps
template <int NT, int W>
struct Layout {
  // The producer is one warp.  Tiles of more rows than 8 do not fit the 168 registers that are left to
  // a thread then: three idle warps complete its warpgroup, which gives registers up; of 128 or 168
  // each at launch, 128 x 216 + 128 x 40 = 256 x 128, 256 x 232 + 128 x 40 = 384 x 168.
  static constexpr bool kSplit = NT > 1;
  static constexpr int kThreads = 32 * (W + (kSplit ? 4 : 1));
  static constexpr int kRegs = W == 4 ? 216 : 232, kRegsProducer = 40;
  static constexpr int kCtas = 8 / W;                       // an SM
  static constexpr int kRows = 8 * NT;
  static constexpr int kUnit = 32 * W;                      // keys
  static constexpr int kTile = kUnit * kH;                  // bytes of a K or V tile
  static constexpr int kOffRing = 0;
  static constexpr int kOffScale = kOffRing + kSlots * kTile;
  static constexpr int kOffRaw = kOffScale + kSlots * kScaleBytes;     // two items' query rows as they are
  static constexpr int kOffQ = kOffRaw + 2 * kRows * kQPitch;          // as operands [NT][k-step pair][lane] 16 bytes
  static constexpr int kOffRow = kOffQ + NT * 4 * 32 * 16;             // a row's factor and visible keys
  static constexpr int kOffO = kOffRow + 2 * kRows * 4;                // [warp][8 rows][kOPitch]
  static constexpr int kOffM = kOffO + W * 8 * kOPitch * 4;            // m [warp][row], l [warp][row]
  static constexpr int kOffBar = kOffM + 2 * W * kRows * 4;
  static constexpr int kSmem = kOffBar + 8 * (2 * kSlots + 4) + 16;
  static constexpr int kSmemAlloc = kSmem + 1024;
  static_assert(kCtas * (kSmemAlloc + 1024) <= 233472, "shared memory");
};

// what a CTA tells the join: its part of an item that an earlier CTA began (a_*), and
// the item that it began and did not end (b_*)
struct Header {
  int a_state;    // 0: nothing, 1: a part in slot 2 c, 2: the whole item, already written out
  int a_ends;     // the item ends in this CTA
  int b_open;     // 0: no such item
  int b_state;    // as a_state, slot 2 c + 1
  int b, h, row0, rows;
};
enum Kind { kDirect = 0, kPartA = 1, kPartB = 2, kNothing = 3 };
struct Part {
  int b, h, row0, rows, ctx, k0, k1, kind;
  bool starts, ends;
  int units;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) { return __byte_perm(a, b, sel); }
__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t half2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// two BF16 values times f as FP16
__device__ __forceinline__ uint32_t scaled_half2(uint32_t w, float f) {
  return half2_bits(__floats2half2_rn(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f));
}
// an 8 x 8 matrix of 16-bit values, a row's pair a lane, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t v) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// This CTA's part of the line, item by item; every warp goes through it by itself
// and all of them see the same.
template <int Unit>
struct Walk {
  const DecodeE4m3Args& a;
  long long x, x1;
  int b, j, off, units, ctx;

  __device__ void load(int i) {
    const int c = i < a.B ? a.ctx_len[i] : 0;
    ctx = min(max(c, 0), a.max_pages * kP);
    units = (ctx + Unit - 1) / Unit;
  }
  __device__ explicit Walk(const DecodeE4m3Args& args) : a(args) {
    const int lane = threadIdx.x & 31;
    const long long M = (long long)a.Hkv * a.n_tiles;
    load(lane);   // of the first 32 requests, a lane each
    const int first_ctx = ctx, first_units = units;
    long long sum = lane < a.B ? units + kItemCost : 0;
    for (int i = lane + 32; i < a.B; i += 32) {
      load(i);
      sum += units + kItemCost;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const long long W = sum * M;
    const int grid = (int)gridDim.x;
    const int n = W >= (long long)grid * kMinCost ? grid : max(1, (int)W / kMinCost);
    const int i = min((int)blockIdx.x + (lane & 1), n);
    // W i / n; short lines without a 64-bit division
    const long long at = W < 0x7fffffff / kMaxCtas ? (int)W * i / n : W * i / n;
    x = __shfl_sync(0xffffffffu, at, 0);
    x1 = __shfl_sync(0xffffffffu, at, 1);
    b = a.B;
    j = off = 0;
    if (x >= x1) return;
    long long before = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
      if (b0 == 0) {
        ctx = first_ctx;
        units = first_units;
      } else {
        load(b0 + lane);
      }
      const long long len = b0 + lane < a.B ? (units + kItemCost) * M : 0;
      long long end = len;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, end, o);
        if (lane >= o) end += u;
      }
      end += before;
      const unsigned in = __ballot_sync(0xffffffffu, x < end);
      if (in) {
        const int l = __ffs(in) - 1;
        b = b0 + l;
        before = __shfl_sync(0xffffffffu, end - len, l);
        ctx = __shfl_sync(0xffffffffu, ctx, l);
        units = __shfl_sync(0xffffffffu, units, l);
        break;
      }
      before = __shfl_sync(0xffffffffu, end, 31);
    }
    const long long rem = x - before;
    const int L = units + kItemCost;
    j = rem <= 0x7fffffff ? (int)rem / L : (int)(rem / L);
    off = (int)(rem - (long long)j * L);
  }
  __device__ bool next(Part& p) {
    if (x >= x1) return false;
    const int L = units + kItemCost;
    const int hi = (int)min((long long)L, off + (x1 - x));
    const int tile = a.n_tiles == 1 ? 0 : j % a.n_tiles;
    p.b = b;
    p.h = a.n_tiles == 1 ? j : j / a.n_tiles;
    p.row0 = tile * a.tile_rows;
    p.rows = min(a.tile_rows, a.T * a.G - p.row0);
    p.ctx = ctx;
    p.units = units;
    p.starts = off == 0;
    p.ends = hi == L;
    p.k0 = max(off - kItemCost, 0);
    p.k1 = p.ends ? units : max(hi - kItemCost, 0);
    const bool whole = p.k0 == 0 && p.k1 == units && (units > 0 || p.starts);
    p.kind = whole ? kDirect : p.k0 >= p.k1 ? kNothing : p.starts ? kPartB : kPartA;
    x += hi - off;
    off = 0;
    if (p.ends && ++j == a.Hkv * a.n_tiles) {
      j = 0;
      load(++b);
    }
    return true;
  }
};

template <int NT, int W>
__global__ void __launch_bounds__(Layout<NT, W>::kThreads, Layout<NT, W>::kCtas)
decode_e4m3_kernel(const DecodeE4m3Args a, const __grid_constant__ CUtensorMap tm_k,
                   const __grid_constant__ CUtensorMap tm_v) {
  using S = Layout<NT, W>;
  constexpr int R = S::kRows, kUnit = S::kUnit, kTile = S::kTile, kPerPage = kP / kUnit;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;
  const int c = blockIdx.x;

  const uint32_t bars = base + S::kOffBar;
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kSlots + s); };
  auto q_full = [&](int s) { return bars + 8 * (2 * kSlots + s); };
  auto q_empty = [&](int s) { return bars + 8 * (2 * kSlots + 2 + s); };
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + S::kOffBar + 8 * (2 * kSlots + 4));
  auto sync_consumers = [] { asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory"); };

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), W);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(q_full(s), 1);
      mbar_init(q_empty(s), W);
    }
    *s_abort = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (tid == 32 * W) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  __syncthreads();
  // every access to global memory follows this wait
  wait_prerequisite_grids();
  allow_dependent_launch();   // the join's CTAs come as these leave

  Walk<kUnit> walk(a);
  Part p;
  uint32_t n_tiles = 0, n_q = 0;   // tiles through the ring, and query tiles
  bool failed = false;

  if (warp >= W) {
    if (S::kSplit) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsProducer));
    if (warp > W) return;
    // ================= producer
    uint32_t issued_q = 0;
    while (!failed && walk.next(p)) {
      if (p.starts && lane == 0) {
        const int len = a.ctx_len[p.b];
        if (len < 0 || len > a.max_pages * kP) atomicExch(a.status, 3);
      }
      if (p.k0 >= p.k1) continue;
      // the rows' queries, a row a lane
      const int qs = n_q & 1;
      if (n_q >= 2) failed = __any_sync(0xffffffffu, !mbar_wait(q_empty(qs), ((n_q >> 1) - 1) & 1, a.wait_ns));
      if (failed) break;
      if (lane == 0) mbar_expect_tx(q_full(qs), p.rows * 2 * kH);
      __syncwarp();
      if (lane < p.rows) {
        const int row = p.row0 + lane, token = row / a.G;
        bulk_g2s(base + S::kOffRaw + qs * R * kQPitch + lane * kQPitch,
                 a.q + (((int64_t)p.b * a.T + token) * a.Hq + p.h * a.G + row - token * a.G) * kH, 2 * kH, q_full(qs));
      }
      __syncwarp();
      ++n_q;
      ++issued_q;
      if (lane == 0) {
        const int32_t* ids = a.page_table + ((int64_t)p.b * a.Hkv + p.h) * a.max_pages;
        int next_id = ids[p.k0 / kPerPage];
        int64_t id = 0;
        for (int k = p.k0; k < p.k1 && !failed; ++k) {
          if (k == p.k0 || k % kPerPage == 0) {
            id = next_id;
            if ((k / kPerPage + 1) * kPerPage < p.k1) next_id = ids[k / kPerPage + 1];
            if (id < 0 || id >= a.n_pool) {
              atomicExch(a.status, 2);
              id = 0;
            }
          }
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            const int s = n_tiles % kSlots;
            if (n_tiles >= kSlots && !mbar_wait(empty(s), (n_tiles / kSlots - 1) & 1, a.wait_ns)) {
              failed = true;
              break;
            }
            ++n_tiles;
            if (a.inject && n_tiles == 2) continue;   // test hook: the first V tile never arrives
            mbar_expect_tx(full(s), kTile + kScaleBytes);
#pragma unroll
            for (int x = 0; x < kUnit; x += 128)      // boxes of 128 tokens
              tma_tile_g2s(base + S::kOffRing + s * kTile + x * kH, kv ? &tm_v : &tm_k, 0,
                           (int)(id * kP) + k % kPerPage * kUnit + x, full(s));
            bulk_g2s(base + S::kOffScale + s * kScaleBytes, a.scales + id * kScaleBytes, kScaleBytes, full(s));
          }
        }
      }
      failed = __any_sync(0xffffffffu, failed);
    }
    if (lane == 0 && failed) {
      atomicExch(a.status, 1);
      *s_abort = 1;
      // the copies in flight end before the memory they go to is given up
      for (uint32_t u = n_tiles > kSlots ? n_tiles - kSlots : 0; u < n_tiles; ++u)
        if (!(a.inject && u == 1)) mbar_wait(full(u % kSlots), (u / kSlots) & 1, a.wait_ns);
      for (uint32_t u = issued_q > 2 ? issued_q - 2 : 0; u < issued_q; ++u) mbar_wait(q_full(u & 1), (u >> 1) & 1, a.wait_ns);
    }
    __syncwarp();
  } else {
    // ================= consumers: warp w has tokens 32 w .. 32 w + 31 of each unit
    if (S::kSplit) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegs));
    Header hdr{0, 0, 0, 0, 0, 0, 0, 0};
    float* s_o = reinterpret_cast<float*>(smem + S::kOffO);
    float* s_m = reinterpret_cast<float*>(smem + S::kOffM);
    float* s_l = s_m + W * R;
    uint4* s_q = reinterpret_cast<uint4*>(smem + S::kOffQ);
    float* s_factor = reinterpret_cast<float*>(smem + S::kOffRow);
    int* s_seen = reinterpret_cast<int*>(s_factor + R);
    const uint8_t* s_scale = smem + S::kOffScale;
    const int n_of = (g >> 1) | ((g & 1) << 2);   // the token of row g of a K fragment, and the lane's 16 channels of V
    // byte offsets in a tile: K row n_of and pieces t, 4 + t; V rows t and t + 4, piece n_of, whose
    // second half comes first in every other pair of lane groups
    const uint32_t v_half = 4 * (g & 2);
    const uint32_t k_at = (uint32_t)(32 * warp + n_of) * kH, k_piece0 = (uint32_t)(t ^ n_of) << 4,
                   k_piece1 = (uint32_t)((4 + t) ^ n_of) << 4;
    const uint32_t v_at0 = (uint32_t)(32 * warp + t) * kH + ((uint32_t)(n_of ^ t) << 4) + v_half,
                   v_at1 = (uint32_t)(32 * warp + t + 4) * kH + ((uint32_t)(n_of ^ (t + 4)) << 4) + v_half;

    while (walk.next(p)) {
      if (tid == 0) {
        const int state = p.units > 0 && p.kind == kDirect ? 2 : p.k1 > p.k0 ? 1 : 0;
        if (!p.starts) {
          hdr.a_state = state;
          hdr.a_ends = p.ends;
        } else if (!p.ends && p.units > 0) {
          hdr.b_open = 1;
          hdr.b_state = state;
          hdr.b = p.b;
          hdr.h = p.h;
          hdr.row0 = p.row0;
          hdr.rows = p.rows;
        }
      }
      if (p.kind == kNothing) continue;
      // the lane's query rows are 8 nr + 2 t + e (NT = 1: g, in [0][0])
      float m_run[NT][2], l_run[NT][2], sc[NT][2];
      float O[8][NT][4];
      uint4 own_q[4];   // NT = 1: the operands that s_q holds otherwise
      const int own_seen = g >= p.rows ? 0 : a.causal ? p.ctx - a.T + (p.row0 + g) / a.G + 1 : p.ctx;
#pragma unroll
      for (int nr = 0; nr < NT; ++nr) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          m_run[nr][e] = -CUDART_INF_F;
          l_run[nr][e] = sc[nr][e] = 0.0f;
        }
#pragma unroll
        for (int mt = 0; mt < 8; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) O[mt][nr][e] = 0.0f;
      }
      if (p.k0 < p.k1) {
        if (!failed) failed = __any_sync(0xffffffffu, !mbar_wait(q_full(n_q & 1), (n_q >> 1) & 1, a.wait_ns));
        const uint32_t q_rows = base + S::kOffRaw + (n_q & 1) * R * kQPitch;
        // the operands of a tile of 8 rows, a warp a tile (a single one: every warp its own): row g, of k-step 4 j + w the channels
        // 64 j + 16 t + 4 w + 0, 1 then + 2, 3
        for (int nr = NT == 1 ? 0 : warp; nr < NT; nr += W) {
          const int r = 8 * nr + g;
          const bool real = r < p.rows && !failed;   // rows past the item's last are zeros
          uint4 x[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x[i] = real ? lds16(q_rows + r * kQPitch + 128 * (i >> 1) + 32 * t + 16 * (i & 1)) : make_uint4(0u, 0u, 0u, 0u);
          uint32_t top = 0;   // largest magnitude, as BF16 bits
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // 2^(14 - exponent of the largest); the scale and its inverse stay normal numbers.  A row with
          // an infinity is NaN (it would be nothing but weights of 0 where all its scores are -inf).
          const int up = top == 0 ? 0 : min(max(14 + 127 - (int)(top >> 7), -113), 126);
          const float f = top >= 0x7F80u ? CUDART_NAN_F : __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {   // 8 channels: two k-steps
            const uint4 h = make_uint4(scaled_half2(x[i].x, f), scaled_half2(x[i].y, f), scaled_half2(x[i].z, f), scaled_half2(x[i].w, f));
            if (NT == 1) own_q[i] = h; else s_q[(nr * 4 + i) * 32 + lane] = h;
          }
          const float factor = a.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
          if (NT == 1) {
            sc[0][0] = factor;
          } else if (t == 0) {
            s_factor[r] = factor;
            s_seen[r] = r >= p.rows ? 0 : a.causal ? p.ctx - a.T + (p.row0 + r) / a.G + 1 : p.ctx;
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(q_empty(n_q & 1));
        ++n_q;
        if (NT > 1) {
          sync_consumers();
#pragma unroll
          for (int nr = 0; nr < NT; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) sc[nr][e] = s_factor[8 * nr + 2 * t + e];
        }
      }

      // the key that the last row sees last, and those that all rows see
      const int last = a.causal ? p.ctx - a.T + (p.row0 + p.rows - 1) / a.G + 1 : p.ctx;
      const int common = a.causal ? p.ctx - a.T + p.row0 / a.G + 1 : p.ctx;
      for (int k = p.k0; k < p.k1; ++k, n_tiles += 2) {
        if (failed) continue;
        const int s_k = n_tiles % kSlots, s_v = (n_tiles + 1) % kSlots;
        const int pos = k * kUnit + 32 * warp;   // of the block's first token
        const bool any = pos < last;             // the warp's block holds a key that is seen
        const int block = k % kPerPage * (kUnit / kC) + warp;
        if (!mbar_wait(full(s_k), (n_tiles / kSlots) & 1, a.wait_ns)) failed = true;
        failed = __any_sync(0xffffffffu, failed);
        if (failed) continue;
        // [16 tokens]: rows 2 t, 2 t + 1 of token n_of, then of n_of + 8 (NT = 1: row g of tokens t, t + 4, t + 8, t + 12)
        float s[2][NT][4];
        float corr[NT][2];
        bool grow = false;
        if (any) {
          const uint32_t tile = base + S::kOffRing + s_k * kTile + k_at;
          if constexpr (NT == 1) {
            // query rows as M: four products side by side, and P as the next products want it
            float d[4][4];   // [8 tokens]: row g of tokens t and t + 4
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
              for (int e = 0; e < 4; ++e) d[nt][e] = 0.0f;
#pragma unroll
              for (int jj = 0; jj < 2; ++jj) {
                const uint4 x = lds16(tile + nt * 8 * kH + (jj ? k_piece1 : k_piece0));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const uint4& q = own_q[2 * jj + (e >> 1)];
                  mma_f16(d[nt], e & 1 ? q.z : q.x, 0u, e & 1 ? q.w : q.y, 0u, f16x2_of(w[e]), f16x2_of_high(w[e]));
                }
              }
            }
            const float ks = scale_of(s_scale[s_k * kScaleBytes + block]);
            __syncwarp();
            if (lane == 0) mbar_arrive(empty(s_k));
            __syncwarp();
            const float f = clamped(sc[0][0] * ks);
            const bool whole = pos + 32 <= common;
            float top = -CUDART_INF_F;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (!whole && pos + 8 * nt + t + 4 * e >= own_seen) d[nt][e] = -CUDART_INF_F;
                top = fmaxf(top, d[nt][e]);
              }
            top *= f;
            float m = m_run[0][0];
            grow = __any_sync(0xffffffffu, top > m + kLazyLog2);
            if (grow) {
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
              top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
              m = fmaxf(m, top);
              const float own = m == -CUDART_INF_F ? 1.0f : ex2(m_run[0][0] - m);
              l_run[0][0] *= own;
              m_run[0][0] = m;
              corr[0][0] = __shfl_sync(0xffffffffu, own, 8 * t);
              corr[0][1] = __shfl_sync(0xffffffffu, own, 8 * t + 4);
            }
            const float ref = m == -CUDART_INF_F ? 0.0f : kUpLog2 - m;   // a masked score gives 0 in any case
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float& v = s[nt >> 1][0][2 * (nt & 1) + e];
                v = ex2(fmaf(d[nt][e], f, ref));
                sum[e] += v;
              }
            l_run[0][0] += sum[0] + sum[1];
          } else {
            // The scales belong to the slot as the codes do: they are read before it is given back, since
            // the next tile's may land there from then on.
            const float ks = scale_of(s_scale[s_k * kScaleBytes + block]);
#pragma unroll
            for (int mt = 0; mt < 2; ++mt)
#pragma unroll
              for (int nr = 0; nr < NT; ++nr)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][nr][e] = 0.0f;
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              uint4 x[2][2];
#pragma unroll
              for (int i = 0; i < 4; ++i) x[i >> 1][i & 1] = lds16(tile + i * 8 * kH + (jj ? k_piece1 : k_piece0));
              if (jj == 1) {   // the last reads of the slot are behind
                __syncwarp();
                if (lane == 0) mbar_arrive(empty(s_k));
                __syncwarp();
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {   // two k-steps
                uint4 q[NT];
#pragma unroll
                for (int nr = 0; nr < NT; ++nr) q[nr] = s_q[(nr * 4 + 2 * jj + h) * 32 + lane];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                  for (int mt = 0; mt < 2; ++mt) {
                    auto word = [&](const uint4& v) { return h == 0 ? e == 0 ? v.x : v.y : e == 0 ? v.z : v.w; };
                    const uint32_t w0 = word(x[mt][0]), w1 = word(x[mt][1]);
                    const uint32_t a0 = f16x2_of(w0), a1 = f16x2_of(w1), a2 = f16x2_of_high(w0), a3 = f16x2_of_high(w1);
#pragma unroll
                    for (int nr = 0; nr < NT; ++nr)
                      mma_f16(s[mt][nr], a0, a1, a2, a3, e == 0 ? q[nr].x : q[nr].z, e == 0 ? q[nr].y : q[nr].w);
                  }
              }
            }
            const bool whole = pos + 32 <= common;
            float f[NT][2], top[NT][2];
#pragma unroll
            for (int nr = 0; nr < NT; ++nr)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                f[nr][e] = clamped(sc[nr][e] * ks);
                if (!whole) {
                  const int seen = s_seen[8 * nr + 2 * t + e] - pos - n_of;
#pragma unroll
                  for (int i = 0; i < 4; ++i)
                    if (8 * i >= seen) s[i >> 1][nr][2 * (i & 1) + e] = -CUDART_INF_F;
                }
                top[nr][e] = fmaxf(fmaxf(s[0][nr][e], s[0][nr][2 + e]), fmaxf(s[1][nr][e], s[1][nr][2 + e])) * f[nr][e];
                grow |= top[nr][e] > m_run[nr][e] + kLazyLog2;
              }
            grow = __any_sync(0xffffffffu, grow);
#pragma unroll
            for (int nr = 0; nr < NT; ++nr)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float m = m_run[nr][e];
                if (grow) {
                  float x = top[nr][e];
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                  m = fmaxf(m, x);
                  corr[nr][e] = m == -CUDART_INF_F ? 1.0f : ex2(m_run[nr][e] - m);
                  l_run[nr][e] *= corr[nr][e];
                  m_run[nr][e] = m;
                }
                const float ref = m == -CUDART_INF_F ? 0.0f : kUpLog2 - m;   // a masked score gives 0 in any case
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  float& v = s[i >> 1][nr][2 * (i & 1) + e];
                  v = ex2(fmaf(v, f[nr][e], ref));
                  sum += v;
                }
                l_run[nr][e] += sum;
              }
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(s_k));
          __syncwarp();
        }

        if (!mbar_wait(full(s_v), ((n_tiles + 1) / kSlots) & 1, a.wait_ns)) failed = true;
        failed = __any_sync(0xffffffffu, failed);
        if (failed) continue;
        if (any) {
          // p as two FP16 numbers, in pairs of tokens (transposed to them): (b0, b1) of k-step kv
          uint32_t hi[2][NT][2], lo[2][NT][2];
#pragma unroll
          for (int kv = 0; kv < 2; ++kv)
#pragma unroll
            for (int nr = 0; nr < NT; ++nr)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float p0 = s[kv][nr][2 * i], p1 = s[kv][nr][2 * i + 1];
                const __half2 h = __floats2half2_rn(p0, p1);
                const float2 r = __half22float2(h);
                const uint32_t rest = half2_bits(__floats2half2_rn(p0 - r.x, p1 - r.y));
                hi[kv][nr][i] = NT == 1 ? half2_bits(h) : transposed(half2_bits(h));
                lo[kv][nr][i] = NT == 1 ? rest : transposed(rest);
              }
          if (grow) {
#pragma unroll
            for (int nr = 0; nr < NT; ++nr)
#pragma unroll
              for (int mt = 0; mt < 8; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) O[mt][nr][e] *= corr[nr][e & 1];
          }
          const uint32_t tile = base + S::kOffRing + s_v * kTile;
          const float vs = scale_of(s_scale[s_v * kScaleBytes + kChunks + block]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // 8 of the lane's 16 channels
            uint2 x[2][4];   // [kv][tokens t, t + 4, t + 8, t + 12]
#pragma unroll
            for (int kv = 0; kv < 2; ++kv)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                x[kv][i] = lds8(tile + ((i & 1 ? v_at1 : v_at0) ^ (8 * h)) + (16 * kv + 8 * (i >> 1)) * kH);
            if (pos + 32 > p.ctx) {   // what is behind the context may be anything, and 0 * NaN is NaN
#pragma unroll
              for (int kv = 0; kv < 2; ++kv)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (pos + 16 * kv + 4 * i + t >= p.ctx) x[kv][i] = make_uint2(0u, 0u);
            }
            if (h == 1) {
              __syncwarp();
              if (lane == 0) mbar_arrive(empty(s_v));
              __syncwarp();
            }
#pragma unroll
            for (int w = 0; w < 2; ++w) {
              float U[2][NT][4];
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nr = 0; nr < NT; ++nr)
#pragma unroll
                  for (int e = 0; e < 4; ++e) U[i][nr][e] = 0.0f;
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                auto word = [&](int i) { return w == 0 ? x[kv][i].x : x[kv][i].y; };
                uint32_t v[2][4];
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // channels 4 w + 2 i, + 1 of the 8
                  const uint32_t ab = prmt(word(0), word(1), i ? 0x7362u : 0x5140u), cd = prmt(word(2), word(3), i ? 0x7362u : 0x5140u);
                  v[i][0] = f16x2_of(ab);
                  v[i][1] = f16x2_of_high(ab);
                  v[i][2] = f16x2_of(cd);
                  v[i][3] = f16x2_of_high(cd);
                }
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int nr = 0; nr < NT; ++nr)
                    mma_f16(U[i][nr], v[i][0], v[i][1], v[i][2], v[i][3], hi[kv][nr][0], hi[kv][nr][1]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                  for (int nr = 0; nr < NT; ++nr)
                    mma_f16(U[i][nr], v[i][0], v[i][1], v[i][2], v[i][3], lo[kv][nr][0], lo[kv][nr][1]);
              }
#pragma unroll
              for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int nr = 0; nr < NT; ++nr)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    float& o = O[4 * h + 2 * w + i][nr][e];
                    o = fmaf(U[i][nr][e], vs, o);
                  }
            }
          }
        } else {
          __syncwarp();
          if (lane == 0) mbar_arrive(empty(s_v));
          __syncwarp();
        }
      }

      // ---- the warps' sums, joined and written (8 rows at a time)
      if constexpr (NT == 1) {
        float l = l_run[0][0];
        l += __shfl_xor_sync(0xffffffffu, l, 1);
        l += __shfl_xor_sync(0xffffffffu, l, 2);
        if (t == 0) {
          s_m[warp * R + g] = m_run[0][0];
          s_l[warp * R + g] = l;
        }
      } else {
#pragma unroll
        for (int nr = 0; nr < NT; ++nr)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float l = l_run[nr][e];
            l += __shfl_xor_sync(0xffffffffu, l, 4);
            l += __shfl_xor_sync(0xffffffffu, l, 8);
            l += __shfl_xor_sync(0xffffffffu, l, 16);
            if (g == 0) {
              s_m[warp * R + 8 * nr + 2 * t + e] = m_run[nr][e];
              s_l[warp * R + 8 * nr + 2 * t + e] = l;
            }
          }
      }
      float* slot = a.ws_o + (int64_t)(2 * c + (p.kind == kPartB)) * a.tile_rows * (kH + 2);
#pragma unroll
      for (int nr = 0; nr < NT; ++nr) {
        if (8 * nr >= p.rows) break;
        // channels 16 n_of + 4 i' .. + 3 of rows 2 t and 2 t + 1 (i' = i, or its halves the other way round)
        float* o = s_o + (warp * 8 + 2 * t) * kOPitch + 16 * n_of;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float(&u)[4] = O[2 * i][nr];
          const float(&v)[4] = O[2 * i + 1][nr];
          *reinterpret_cast<float4*>(o + ((4 * i) ^ v_half)) = make_float4(u[0], u[2], v[0], v[2]);
          *reinterpret_cast<float4*>(o + kOPitch + ((4 * i) ^ v_half)) = make_float4(u[1], u[3], v[1], v[3]);
        }
        sync_consumers();
        // a row of 8 by 4 W lanes, four channels each at a time
        constexpr int kLanes = 4 * W;
        const int rr = tid / kLanes, r = 8 * nr + rr, ch = 4 * (tid % kLanes);
        float mw[W], m = -CUDART_INF_F, l = 0.0f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
          mw[w] = s_m[w * R + r];
          m = fmaxf(m, mw[w]);
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          mw[w] = mw[w] == -CUDART_INF_F ? 0.0f : ex2(mw[w] - m);   // the warp's factor
          l = fmaf(s_l[w * R + r], mw[w], l);
        }
        float4 u[kH / (4 * kLanes)];
#pragma unroll
        for (int x = 0; x < kH / (4 * kLanes); ++x) {
          u[x] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < W; ++w) {
            const float4 v = *reinterpret_cast<const float4*>(s_o + (w * 8 + rr) * kOPitch + 4 * kLanes * x + ch);
            u[x].x = fmaf(v.x, mw[w], u[x].x);
            u[x].y = fmaf(v.y, mw[w], u[x].y);
            u[x].z = fmaf(v.z, mw[w], u[x].z);
            u[x].w = fmaf(v.w, mw[w], u[x].w);
          }
        }
        if (r < p.rows && !failed) {
          if (p.kind == kDirect) {
            const int row = p.row0 + r, token = row / a.G;
            const int64_t at = ((int64_t)p.b * a.T + token) * a.Hq + p.h * a.G + row - token * a.G;
            const float f = l > 0.0f ? 1.0f / l : l;   // 0 for a row without keys, NaN stays
#pragma unroll
            for (int x = 0; x < kH / (4 * kLanes); ++x)
              *reinterpret_cast<float4*>(a.out + at * kH + 4 * kLanes * x + ch) =
                  make_float4(u[x].x * f, u[x].y * f, u[x].z * f, u[x].w * f);
            if (ch == 0 && a.lse) a.lse[at] = l == 0.0f ? -CUDART_INF_F : (m - kUpLog2 + log2f(l)) * kLn2;
          } else {
#pragma unroll
            for (int x = 0; x < kH / (4 * kLanes); ++x)
              *reinterpret_cast<float4*>(slot + r * kH + 4 * kLanes * x + ch) = u[x];
            if (ch == 0) *reinterpret_cast<float2*>(slot + a.tile_rows * kH + 2 * r) = make_float2(m, l);
          }
        }
        sync_consumers();   // the area is free again
      }
    }
    if (failed && lane == 0) {
      atomicExch(a.status, 1);
      *s_abort = 1;
    }
    sync_consumers();
    if (tid == 0) a.ws_hdr_as<Header>()[c] = *s_abort ? Header{0, 0, 0, 0, 0, 0, 0, 0} : hdr;
  }
}

// ------------------------------------------------------------------ join of the parts

constexpr int kJoinWarps = 8;

// CTA (c, r) joins row r of the item that CTA c of the kernel above began and did
// not end; a warp takes every eighth part, a lane four channels.
__global__ void __launch_bounds__(32 * kJoinWarps)
decode_e4m3_join(const DecodeE4m3Args a) {
  __shared__ float s_o[kJoinWarps][kH];
  __shared__ float2 s_ml[kJoinWarps];
  const int c = blockIdx.x, r = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  allow_dependent_launch();
  wait_prerequisite_grids();
  const Header* hdr = a.ws_hdr_as<Header>();
  const Header hd = hdr[c];
  if (!hd.b_open || hd.b_state == 2 || r >= hd.rows) return;
  const int R = a.tile_rows;
  float m = -CUDART_INF_F, l = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  auto add = [&](int slot) {
    const float* o = a.ws_o + (int64_t)slot * R * (kH + 2);
    const float2 ml = *reinterpret_cast<const float2*>(o + R * kH + 2 * r);
    const float4 v = *reinterpret_cast<const float4*>(o + r * kH + 4 * lane);
    const float m_new = fmaxf(m, ml.x);
    const float f = m == -CUDART_INF_F ? 0.0f : ex2(m - m_new);
    // a part without keys weighs nothing, one whose sum is NaN stays NaN
    const float g = ml.x == -CUDART_INF_F ? (ml.y == ml.y ? 0.0f : 1.0f) : ex2(ml.x - m_new);
    l = fmaf(l, f, ml.y * g);
    acc.x = fmaf(acc.x, f, v.x * g);
    acc.y = fmaf(acc.y, f, v.y * g);
    acc.z = fmaf(acc.z, f, v.z * g);
    acc.w = fmaf(acc.w, f, v.w * g);
    m = m_new;
  };
  if (warp == 0 && hd.b_state == 1) add(2 * c + 1);
  // the CTAs behind, up to the one where the item ends, 32 at a time
  for (int d0 = c + 1; d0 < (int)gridDim.x; d0 += 32) {
    const int d = d0 + lane;
    const int state = d < (int)gridDim.x ? hdr[d].a_state : 0;
    const int ends = d < (int)gridDim.x ? hdr[d].a_ends : 1;
    const unsigned e = __ballot_sync(0xffffffffu, ends != 0);
    const unsigned within = e ? (e & -e) | ((e & -e) - 1) : 0xffffffffu;
    if (__ballot_sync(0xffffffffu, state == 2) & within) return;   // one CTA had it all (and all warps see so)
    unsigned valid = __ballot_sync(0xffffffffu, state == 1) & within;
    valid &= 0x01010101u << warp;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (valid >> (8 * i + warp) & 1) add(2 * (d0 + 8 * i + warp));
    if (e) break;
  }
  *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = acc;
  if (lane == 0) s_ml[warp] = make_float2(m, l);
  __syncthreads();
  if (warp != 0) return;
  float top = -CUDART_INF_F, sum = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, s_ml[w].x);
  acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    const float2 ml = s_ml[w];
    const float g = ml.x == -CUDART_INF_F ? (ml.y == ml.y ? 0.0f : 1.0f) : ex2(ml.x - top);
    const float4 v = *reinterpret_cast<const float4*>(&s_o[w][4 * lane]);
    sum = fmaf(ml.y, g, sum);
    acc.x = fmaf(v.x, g, acc.x);
    acc.y = fmaf(v.y, g, acc.y);
    acc.z = fmaf(v.z, g, acc.z);
    acc.w = fmaf(v.w, g, acc.w);
  }
  const float f = sum > 0.0f ? 1.0f / sum : sum;
  const int row = hd.row0 + r, token = row / a.G;
  const int64_t at = ((int64_t)hd.b * a.T + token) * a.Hq + hd.h * a.G + row - token * a.G;
  *reinterpret_cast<float4*>(a.out + at * kH + 4 * lane) = make_float4(acc.x * f, acc.y * f, acc.z * f, acc.w * f);
  if (lane == 0 && a.lse) a.lse[at] = sum == 0.0f ? -CUDART_INF_F : (top - kUpLog2 + log2f(sum)) * kLn2;
}

template <int NT, int W>
cudaError_t launch(DecodeE4m3Args a, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  using S = Layout<NT, W>;
  static bool configured[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(decode_e4m3_kernel<NT, W>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemAlloc);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  const int n_cta = device_sm_count() * S::kCtas;
  cudaError_t e = launch_programmatic(decode_e4m3_kernel<NT, W>, dim3(n_cta < kMaxCtas ? n_cta : kMaxCtas),
                                      dim3(S::kThreads), S::kSmemAlloc, s, a, tk, tv);
  if (e != cudaSuccess) return e;
  const int rows = a.T * a.G;
  return launch_programmatic(decode_e4m3_join, dim3(n_cta < kMaxCtas ? n_cta : kMaxCtas, rows < a.tile_rows ? rows : a.tile_rows),
                             dim3(32 * kJoinWarps), 0, s, a);
}

// Rows of a tile.  One pass over the keys takes about 26, 37 and 49 us with 8, 16 and 24 rows (8
// requests of up to 32,000 keys, 4 KV heads); tiles of 32 rows spill, 92 us.
int tile_rows(int rows) {
  if (rows <= 8) return 8;
  return 4 * ((rows + 23) / 24) < 3 * ((rows + 15) / 16) ? 24 : 16;
}

}  // namespace

size_t decode_e4m3_ws_bytes(int rows) {
  const int n = 2 * device_sm_count();
  return (size_t)kMaxCtas * sizeof(Header) + (size_t)2 * (n < kMaxCtas ? n : kMaxCtas) * tile_rows(rows) * (kH + 2) * 4;
}

cudaError_t launch_decode_e4m3(DecodeE4m3Args a, void* workspace, cudaStream_t s) {
  const int rows = a.T * a.G;
  a.tile_rows = tile_rows(rows);
  a.n_tiles = (rows + a.tile_rows - 1) / a.tile_rows;
  a.ws_hdr = workspace;
  a.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kMaxCtas * sizeof(Header));
  CUtensorMap tk, tv;
  // a page is two tiles of 128 rows of 128 bytes
  if (!plane_map(&tk, a.k_pages, 2 * a.n_pool) || !plane_map(&tv, a.v_pages, 2 * a.n_pool)) return cudaErrorInvalidValue;
  switch (a.tile_rows) {
    case 8: return launch<1, 4>(a, tk, tv, s);
    case 16: return launch<2, 4>(a, tk, tv, s);
    default: return launch<3, 8>(a, tk, tv, s);
  }
}

}  // namespace lynx
