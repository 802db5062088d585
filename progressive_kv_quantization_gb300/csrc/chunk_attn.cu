// Attention of ragged chunks of new tokens over BF16 pages on the 5th-generation
// tensor cores (lynx_chunk_attn_bf16): chunked prefill, mixed batches, and single
// tokens.
//
//   S = Q K^T,  P = 2^(S c - m),  O = (sum P V) / (sum P),  c = sm_scale log2(e)
//   lse = (m + log2 sum P) ln 2
//
// Tile.  The query rows of a request that share a KV head are its tokens times
// the G = Hq / Hkv heads of the group (row = token G + head): a tile is 256 of
// them, two groups of 128, against 128 keys at a time.  A page is stored
// channel-major, so a K half page [128 channels][128 tokens] is the MN-major B
// operand of S = Q K^T and a V half page the K-major B operand of O = P V as they
// lie: nothing is transposed.
//
// Warps.  0-3 and 4-7: softmax of the two groups, one row a thread; 8 and 11:
// issue the groups' tcgen05.mma; 9: TMA of K and V tiles through a ring; 10: the
// lists of tiles.  S and O of both groups live in tensor memory (4 x 128 columns).
// P overwrites S as BF16 and is the A operand of O += P V from there.  While one
// group does its softmax the tensor core works for the other, one block of products
// (P V, the next Q K^T) at a time.
//
// Softmax in one pass over the keys.  The running maximum moves only where a
// score leads it by more than 8 in log2 units, so that O is rescaled (a round
// trip through registers) on few tiles; P is at most 2^8.  P is taken against the
// maximum as it stands, beside the search for the tile's, and again if that moves
// it.  Row sums are taken of the float32 probabilities.  P is rounded to BF16 for
// the matrix product (kind::f16 wants V's type): half a step, 2^-8 of a term at
// most, either way, so that over many keys it falls below the BF16 output's own
// rounding.
//
// Sums of long contexts.  What the tensor core's float32 accumulator does not hold is
// cut off and not rounded, so that the errors of O's additions add up: -5e-5 of the value
// over 16,384 keys, -4.8e-4 over 131,072, -4e-3 over a million (values of one sign).  So O
// is taken out every 16,384 keys and added up, rounded, in the workspace: some 6,000
// clocks for both groups, most of them L2's for 128 KB a CTA, 3% of 131,072 keys' time.
//
// What bounds it (GB300, 16 or 32 query heads over 4 or 8 KV heads).  Many rows: the
// tensor core, 4 x 128 x 128 x 128 products in 2,048 clocks for two groups; a tile of
// keys takes 1.4 us against 1.08 at the clock seen.  2,048 tokens at the end of 131,072
// keys run at some 1,620 TFLOP/s call after call (power-capped; the library's BF16
// matrix product does 1,849 in a burst, 1,663 sustained).  The rest is a group's chain:
// softmax ~1,350 clocks, its products 1,024, hand-overs ~400.  A tile's start and end cost
// ~4.5 us (first scores, last products, output), so that 3,000 tokens of six requests
// over 8,000 keys run at 1,330.  One token a request over long contexts: memory, 6.27 TB/s
// of keys and values (93% of a copy).  A short prompt: 12.8 us, of which the two launches,
// the lists (~2.5 us) and one tile's chain of waits are all but one.
//
// Work split.  The tiles of all requests and heads stand on one line, each as
// long as its estimated cost; the line is cut into equal parts, one a CTA, one
// CTA an SM.  A tile that a cut goes through is computed in parts that leave
// their unnormalised O, m and sum in the workspace, and chunk_combine_kernel
// joins them; so a long chunk, a ragged batch and a single token over a long
// context all fill the machine, and the result does not depend on timing.
//
// A list is gone through from its end.  Where a CTA's part is the end of one tile
// and the beginning of the next, the CTAs of a head then all begin at key 0 and,
// behind their second tile's part, all go on at the same distance from it: the
// keys and values of a context that L2 does not hold are read from memory twice,
// not once a tile (128 tiles over 131,072 keys: 6.4 GB in the other order).
//
// Keys past ctx_len in the last page take no part: their scores are replaced, and
// their V rows are zeroed in shared memory (0 x NaN would be NaN).

#include "lynx_internal.cuh"
#include "f32x2.cuh"
#include "tma_ptx.cuh"

#include <cuda_bf16.h>
#include <math_constants.h>

namespace lynx {
namespace {

constexpr int kGroupRows = 128;
constexpr int kTileRows = 2 * kGroupRows;
constexpr int kTileKeys = 128;
constexpr int kBox = 16384;                    // TMA box: 64 tokens x 128 channels
constexpr int kSlot = 2 * kBox;                // one K or V tile
constexpr int kSlots = 5;
constexpr int kQBytes = 2 * kBox;              // a group's queries: two halves [128 rows][64 channels]
constexpr int kMmaWarp = 8, kTmaWarp = 9, kListWarp = 10, kMmaWarp1 = 11;
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 208, kRegsOther = 80;   // of 168 each at launch: 256 x 208 + 128 x 80 <= 384 x 168
constexpr int kMaxItems = 24;
// Tiles of keys of a part, at least: a smaller one goes to the CTA with the rest, whose
// tile then needs no join.  us with 1 / 2 / 3 / 4 / 6: one prompt of 2,048 tokens (32 / 8
// heads) 50.6 / 45.5 / 50.0 / 49.4 / 51.8, eight of 1,024 59.2 / 57.1 / 57.1 / 57.3 / 59.8, 12
// chunks of 300 before 5,000 keys 52.7 / 53.6 / 52.0 / 52.1 / 57.4.  Not where a CTA gets
// fewer than 1,024 keys: 17 tokens over 1,000 keys 13.1 / 13.6.
constexpr int kLeastPart = 2, kLeastPartKeysLog2 = 10;
constexpr int kMaxCtas = 256;                  // of the grid; the GB300's 152 SMs get one each
constexpr float kLazyLog2 = 8.0f;
// Tiles of keys that are summed up in tensor memory.  Error (131,072 keys, values with an
// offset) and us with 64 / 128 / 256: 3.1e-5, 1,371 / 6.7e-5, 1,345 / 1.3e-4, 1,332; never
// taken out: 4.9e-4, 1,307.
constexpr int kSumTiles = 128;
static_assert(kSumTiles > 0 && (kSumTiles & (kSumTiles - 1)) == 0, "kSumTiles");
constexpr int kBusyPolls = 4096;               // some 100 us
constexpr int kMinKeysLog2 = 7;                // least cost of a CTA's part of the work, in keys; us for 17 tokens
                                               // over 1,000 keys: 12.8 (7), 13.2 (8), 16.1 (9)

constexpr int kOffQ = 0;
constexpr int kOffRing = kOffQ + 2 * kQBytes;
constexpr int kOffBar = kOffRing + kSlots * kSlot;
constexpr int kNumBars = 2 * kSlots + 10;
constexpr int kOffItems = kOffBar + 8 * kNumBars;
constexpr int kItemInts = 10;
constexpr int kOffMisc = kOffItems + ((kMaxItems * kItemInts * 4 + 15) / 16) * 16;
constexpr int kSmem = kOffMisc + 80;   // items, header (at 16), tensor memory (at 64), abort and busy flags
constexpr int kSmemAlloc = kSmem + 1024;
static_assert(kSmemAlloc <= 232448, "shared memory (chunk attention)");

// one tile, or the part of one, of a CTA
struct Item {
  int b, h, q_base, row0, rows, T, ctx, k0, k1, kind;
};
enum Kind { kDirect = 0, kPartA = 1, kPartB = 2, kNothing = 3 };
static_assert(sizeof(Item) == kItemInts * 4, "Item");

// what a CTA tells the combine: its part of a tile that an earlier CTA began
// (a_*), and the tile that it began and did not end (b_*)
struct Header {
  int a_state;    // 0: nothing, 1: a part in slot 2 c, 2: the whole tile, already written out
  int a_ends;     // the tile ends in this CTA
  int b_open;     // 0: no such tile
  int b_state;    // as a_state, slot 2 c + 1
  int h, q_base, row0, rows;
};

// ------------------------------------------------------------------ PTX

__device__ __forceinline__ void fence_proxy_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// 16 bytes, or zeros where `bytes` is 0
__device__ __forceinline__ void copy_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_done() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// one lane of a whole warp, the same one every time
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// mask of the first n of two packed 16-bit values
__device__ __forceinline__ uint32_t keep2(int n) { return n >= 2 ? 0xFFFFFFFFu : n == 1 ? 0x0000FFFFu : 0u; }
// a value that all lanes of the warp share
template <typename V>
__device__ __forceinline__ V uni(V v) {
  return __shfl_sync(0xffffffffu, v, 0);
}
// shared-memory operand, 128-byte swizzle.  K-major: rows of 128 bytes along K,
// 8-row groups 1024 bytes apart.  MN-major: rows of 64 values along MN, 8-row
// (K) groups 1024 bytes apart, the next 64 along MN one TMA box on.
__device__ __forceinline__ uint64_t desc_k(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | (1ull << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(kBox >> 4) << 16) | (64ull << 32) | (1ull << 46) | (2ull << 61);
}
// float32 accumulators, BF16 operands, 128 x 128; the B operand K-major or MN-major
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10) | (16u << 17) | (8u << 24);
constexpr uint32_t kIdescMn = kIdesc | (1u << 16);

#define LYNX_R8(v, o) "=r"(v[o]), "=r"(v[o + 1]), "=r"(v[o + 2]), "=r"(v[o + 3]), "=r"(v[o + 4]), "=r"(v[o + 5]), "=r"(v[o + 6]), "=r"(v[o + 7])
#define LYNX_I8(v, o) "r"(v[o]), "r"(v[o + 1]), "r"(v[o + 2]), "r"(v[o + 3]), "r"(v[o + 4]), "r"(v[o + 5]), "r"(v[o + 6]), "r"(v[o + 7])
// 32 columns of the thread's tensor-memory row
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : LYNX_R8(v, 0), LYNX_R8(v, 8), LYNX_R8(v, 16), LYNX_R8(v, 24)
      : "r"(addr));
}
// 16 columns, waited for
__device__ __forceinline__ void tmem_ld16(uint32_t addr, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
      "[%16];\n\ttcgen05.wait::ld.sync.aligned;"
      : LYNX_R8(v, 0), LYNX_R8(v, 8)
      : "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15};" ::LYNX_I8(v, 0),
      LYNX_I8(v, 8), "r"(addr)
      : "memory");
}
// the loaded registers hold their values only behind the wait: pass them through it
#define LYNX_P8(v, o) "+r"(v[o]), "+r"(v[o + 1]), "+r"(v[o + 2]), "+r"(v[o + 3]), "+r"(v[o + 4]), "+r"(v[o + 5]), "+r"(v[o + 6]), "+r"(v[o + 7])
__device__ __forceinline__ void tmem_wait_ld32(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : LYNX_P8(v, 0), LYNX_P8(v, 8), LYNX_P8(v, 16), LYNX_P8(v, 24)
               :
               : "memory");
}
__device__ __forceinline__ void tmem_hold32(uint32_t* v) {
  asm volatile("" : LYNX_P8(v, 0), LYNX_P8(v, 8), LYNX_P8(v, 16), LYNX_P8(v, 24) : : "memory");
}
__device__ __forceinline__ void tmem_wait_st_() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// 32 bytes: a whole sector at once, if the address is a multiple of 32
__device__ __forceinline__ void store32(void* p, const uint32_t* v, int wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), LYNX_I8(v, 0) : "memory");
  } else {
    uint4* d = static_cast<uint4*>(p);
    d[0] = make_uint4(v[0], v[1], v[2], v[3]);
    d[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

// x / d for 32-bit x, with magic = ceil(2^64 / d) (0 for d = 1): exact
__device__ __forceinline__ int div_by(int x, unsigned long long magic) {
  return magic ? (int)__umul64hi((unsigned long long)(unsigned)x, magic) : x;
}

// ------------------------------------------------------------------ work split

// A request's tiles on the cost line of one head, in 1/256 keys: tile m costs
// its keys (those before the chunk plus 256 / G more with every tile under a
// causal mask) and, for its start and end, 512 keys, or 256 if one group does
// (512 and 256 are the best of 384, 448, 512, 640 and 192, 256, 384).
struct Request {
  int q_base, T, ctx, tiles;
  long long base, step;
  __device__ long long at(int m) const { return m * base + step * ((long long)m * (m + 1) / 2); }
  __device__ int tile_of(long long x) const {   // the tile that holds x, at(0) <= x < at(tiles)
    int lo = 0, hi = tiles;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (at(mid) <= x) lo = mid; else hi = mid;
    }
    return lo;
  }
};

__device__ __forceinline__ Request load_request(const ChunkArgs& a, int b) {
  Request r{0, 0, 0, 0, 0, 0};
  if (b >= a.B) return r;
  const int lo = a.cu_q[b], hi = a.cu_q[b + 1];
  const int ctx = a.ctx_len[b];
  const int max_keys = a.max_pages * kP;
  if (ctx < 0 || ctx > max_keys) atomicExch(a.status, 3);
  if (lo < 0 || hi < lo || hi > a.n_rows) {
    atomicExch(a.status, 6);
    return r;
  }
  r.q_base = lo;
  r.T = hi - lo;
  r.ctx = min(max(ctx, 0), max_keys);
  r.tiles = (r.T * a.G + kTileRows - 1) / kTileRows;
  r.base = (long long)((a.causal ? max(r.ctx - r.T, 0) : r.ctx) + (r.T * a.G > kGroupRows ? 512 : 256)) << 8;
  r.step = a.causal ? div_by(65536, a.by_G) : 0;
  return r;
}

// keys that the rows of a token see
__device__ __forceinline__ int visible(const ChunkArgs& a, int ctx, int T, int token) {
  return a.causal ? max(ctx - T + token + 1, 0) : ctx;
}

// All warps meet here from their own loops, some of which one lane alone goes through.
// (bar.sync and the .aligned instructions below, tcgen05.ld and .st among them, want the
// warp's lanes together; behind code that may part them a __syncwarp brings them so.)
__device__ __forceinline__ void sync_all() {
  __syncwarp();
  asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory");
}

template <typename V>
__device__ __forceinline__ V warp_scan(V v) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V u = __shfl_up_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) >= o) v += u;
  }
  return v;
}

// The list warp: measures the line, finds this CTA's part of it and hands out
// the part's items, the tiles of one head at a time and at most kMaxItems.
// Requests are taken 32 at a time, one a lane; each list starts again from the
// first.  (One warp and one place in the code: the list's instructions are fetched
// once, which is most of the time that a short list takes.)
__device__ __forceinline__ void make_lists(const ChunkArgs& a, Item* items, volatile int* s_n_items, Header* s_hdr,
                                           const volatile int* s_abort) {
  const int lane = threadIdx.x & 31;
  const Request first = load_request(a, lane);
  long long Wh = 0;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const Request r = b0 == 0 ? first : load_request(a, b0 + lane);
    Wh += __shfl_sync(0xffffffffu, warp_scan(r.at(r.tiles)), 31);
  }
  const long long W = Wh * a.Hkv;
  // CTAs that get a part (divisions would take as long as the rest of this)
  int n_cta = (int)max(1ll, min((long long)gridDim.x, W >> (kMinKeysLog2 + 8)));
  // A multiple of the heads, where that leaves no more than 1/32 of the CTAs idle
  // or they are not all used anyway: then each head has its own CTAs.
  const int grid = (int)gridDim.x, each = div_by(n_cta, a.by_heads), over = n_cta - each * a.Hkv;
  const bool by_head = n_cta >= a.Hkv && (n_cta < grid || over * 32 <= grid);
  if (by_head) n_cta -= over;
  const int least_part = W >> (kLeastPartKeysLog2 + 8) >= n_cta ? kLeastPart : 1;
  const int per = by_head ? each : n_cta;
  // about 2^32 / per: the same for all CTAs, and (per - 1) shares stay below 2^32
  const unsigned share = __float2uint_rz(__fdividef(4294967040.0f, (float)per));
  auto cut = [&](int i) {   // where CTA i begins
    if (i >= n_cta) return W;
    // i / per: i + 1/2 is 1 / (2 per) away from its multiples, and both are 256 at most
    const unsigned whole = by_head ? (unsigned)__fdividef((float)i + 0.5f, (float)per) : 0u;
    const unsigned long long len = by_head ? Wh : W;
    return (long long)(whole * len + __umul64hi(len, (unsigned long long)((i - whole * per) * share) << 32));
  };
  long long x0 = cut((int)blockIdx.x);
  const long long x1 = cut((int)blockIdx.x + 1);
  while (x0 < x1) {
    long long h = (long long)__fdividef(__ll2float_rn(x0), __ll2float_rn(Wh));   // off by one at most
    h -= h * Wh > x0;
    h += (h + 1) * Wh <= x0;
    const long long seg0 = x0 - h * Wh, seg1 = min(x1 - h * Wh, Wh);
    long long before = 0, next = h * Wh + seg1;
    int n_items = 0;
    for (int b0 = 0; b0 < a.B && before < seg1; b0 += 32) {
      const Request r = b0 == 0 ? first : load_request(a, b0 + lane);
      const long long len = r.at(r.tiles);
      const long long end = before + warp_scan(len), p = end - len;
      before = __shfl_sync(0xffffffffu, end, 31);
      if (before <= seg0) continue;
      const long long lo = max(seg0 - p, 0ll), hi = min(seg1 - p, len);
      int m0 = 0, m1 = -1;
      if (lo < hi) {
        m0 = r.tile_of(lo);
        m1 = r.tile_of(hi - 1);
      }
      int at = n_items + warp_scan(m1 - m0 + 1);
      n_items = __shfl_sync(0xffffffffu, at, 31);
      at -= m1 - m0 + 1;
      long long stop = next;
      for (int m = m0; m <= m1; ++m, ++at) {
        if (at >= kMaxItems) {
          if (at == kMaxItems) stop = h * Wh + p + r.at(m);
          break;
        }
        const int last = min(r.T - 1, div_by(kTileRows * (m + 1) - 1, a.by_G));
        const int n_kv = (visible(a, r.ctx, r.T, last) + kTileKeys - 1) / kTileKeys;
        const long long from = r.at(m), cost = r.at(m + 1) - from;
        const bool starts = lo <= from, ends = hi >= from + cost;
        Item it;
        it.b = b0 + lane;
        it.h = (int)h;
        it.q_base = r.q_base;
        it.row0 = m * kTileRows;
        it.rows = min(kTileRows, r.T * a.G - it.row0);
        it.T = r.T;
        it.ctx = r.ctx;
        // where a cut falls among the tile's keys: the same function on both of its sides, not decreasing
        auto key_tile = [&](long long x) {
          const int k = (int)(__ll2float_rn(x - from) * (float)n_kv / __ll2float_rn(cost));
          return k < least_part ? 0 : k > n_kv - least_part ? n_kv : k;
        };
        it.k0 = starts ? 0 : key_tile(lo);
        it.k1 = ends ? n_kv : key_tile(hi);
        const bool whole = it.k0 == 0 && it.k1 == n_kv && (n_kv > 0 || starts);
        it.kind = whole ? kDirect : it.k0 == it.k1 ? kNothing : starts ? kPartB : kPartA;
        items[at] = it;
        const int state = n_kv > 0 && whole ? 2 : it.k1 > it.k0 ? 1 : 0;
        if (!starts) {
          s_hdr->a_state = state;
          s_hdr->a_ends = ends;
        } else if (!ends && n_kv > 0) {
          s_hdr->b_open = 1;
          s_hdr->b_state = state;
          s_hdr->h = it.h;
          s_hdr->q_base = it.q_base;
          s_hdr->row0 = it.row0;
          s_hdr->rows = it.rows;
        }
      }
      __syncwarp();   // the lanes' loops end at different times
      // the lane that ran out of room knows where the next list begins
      const unsigned cutter = __ballot_sync(0xffffffffu, stop != next);
      if (cutter) next = __shfl_sync(0xffffffffu, stop, __ffs(cutter) - 1);
      if (n_items > kMaxItems) break;
    }
    x0 = next;
    if (lane == 0) *s_n_items = min(n_items, kMaxItems);
    __syncwarp();
    sync_all();   // the list is there
    sync_all();   // and done with
    if (*s_abort) return;
  }
  if (lane == 0) *s_n_items = 0;
  __syncwarp();
  sync_all();
}

// ------------------------------------------------------------------ kernel

__global__ void __launch_bounds__(kThreads, 1)
chunk_attn_kernel(const ChunkArgs a, const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int c = blockIdx.x;

  Item* items = reinterpret_cast<Item*>(smem + kOffItems);
  volatile int* s_n_items = reinterpret_cast<volatile int*>(smem + kOffMisc);
  Header* s_hdr = reinterpret_cast<Header*>(smem + kOffMisc + 16);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + kOffMisc + 64);
  volatile int* s_busy = reinterpret_cast<volatile int*>(smem + kOffMisc + 72);   // a group's products are being issued
  volatile int* s_abort = reinterpret_cast<volatile int*>(smem + kOffMisc + 68);

  const uint32_t bar0 = base + kOffBar;
  auto kv_full = [&](int s) { return bar0 + 8 * s; };
  auto kv_empty = [&](int s) { return bar0 + 8 * (kSlots + s); };
  const uint32_t bars = bar0 + 8 * 2 * kSlots;
  auto q_full = [&](int g) { return bars + 8 * g; };
  auto s_full = [&](int g) { return bars + 8 * (2 + g); };
  auto p_full = [&](int g) { return bars + 8 * (4 + g); };
  auto o_done = [&](int g) { return bars + 8 * (6 + g); };
  const uint32_t drained = bars + 8 * 8;   // used once, by a CTA that gives up
  const uint32_t met = bars + 8 * 9;       // both groups, behind a sum that was taken out

  if (tid == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(kv_full(s), 1);
      mbar_init(kv_empty(s), 2);   // both groups
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(q_full(g), kGroupRows);
      mbar_init(s_full(g), 1);
      mbar_init(p_full(g), kGroupRows);
      mbar_init(o_done(g), 1);
    }
    mbar_init(drained, 2);
    mbar_init(met, 2 * kGroupRows);
    *s_hdr = Header{0, 0, 0, 0, 0, 0, 0, 0};
    *s_abort = 0;
    s_busy[0] = s_busy[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(s_tmem)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    tc_fence_before();
  }
  if (warp == kTmaWarp && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_k)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tm_v)) : "memory");
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *s_tmem;
  // every access to global memory follows this wait
  wait_prerequisite_grids();

  const unsigned long long wait_ns = a.wait_ns;
  auto give_up = [&]() {
    atomicExch(a.status, 1);
    *s_abort = 1;
  };
  // counters of each role, running over all items
  uint32_t n_kv_ring = 0;     // K and V tiles through the ring (producer; MMA warp)
  uint32_t n_tile_g = 0;      // S tiles of this thread's group (softmax)
  uint32_t n_met = 0;         // phases of `met`
  uint32_t mma_items = 0, mma_tiles = 0;   // of the tensor-core warp's group
  bool failed = false;

  // Every role goes through the lists of items that the list warp makes, and
  // meets the others in front of and behind each.
  auto next_list = [&]() {
    sync_all();
    return *s_n_items;
  };
  auto list_done = [&]() {   // false: a wait has run out somewhere
    sync_all();
    return *s_abort == 0;
  };

  if (warp >= kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp == kListWarp) {
      make_lists(a, items, s_n_items, s_hdr, s_abort);
    } else {
    while (const int n_items = next_list()) {
      if (warp == kTmaWarp) {
        // ================= producer: K and V tiles in the order of use
        if (lane == 0) {
          for (int i = n_items - 1; i >= 0 && !failed; --i) {
            const Item it = items[i];
            if (it.kind == kNothing || it.k0 == it.k1) continue;
            const int32_t* row = a.page_table + ((int64_t)it.b * a.Hkv + it.h) * a.max_pages;
            int next_id = row[it.k0 >> 1];
            int64_t id = 0;
            for (int k = it.k0; k < it.k1 && !failed; ++k) {
              if (k == it.k0 || !(k & 1)) {
                id = next_id;
                if (((k >> 1) + 1) * 2 < it.k1) next_id = row[(k >> 1) + 1];
                if (id < 0 || id >= a.n_pool) {
                  atomicExch(a.status, 2);
                  id = 0;
                }
              }
#pragma unroll
              for (int kv = 0; kv < 2; ++kv) {
                const int s = n_kv_ring % kSlots;
                if (n_kv_ring >= kSlots && !mbar_wait(kv_empty(s), (n_kv_ring / kSlots - 1) & 1, wait_ns)) {
                  give_up();
                  failed = true;
                  break;
                }
                if (a.inject && n_kv_ring == 1) {   // test hook: the first V tile never arrives
                  ++n_kv_ring;
                  continue;
                }
                const uint32_t dst = base + kOffRing + s * kSlot;
                mbar_expect_tx(kv_full(s), kSlot);
                tma_tile_g2s(dst, kv ? &tm_v : &tm_k, (k & 1) * kTileKeys, (int)(id * kH), kv_full(s));
                tma_tile_g2s(dst + kBox, kv ? &tm_v : &tm_k, (k & 1) * kTileKeys + 64, (int)(id * kH), kv_full(s));
                ++n_kv_ring;
              }
            }
          }
        }
      } else {
        // ================= tensor-core warp of group g: while it waits, the other
        // group's products run.  Everything that the products' operands are made of
        // is the same in all lanes and known to be (uni), and one elected lane
        // issues: the compiler keeps descriptors in uniform registers then.  66
        // clocks a product of 128 x 128 x 16 against 79 under lane == 0; the tensor
        // core takes 64.
        const int g = warp == kMmaWarp ? 0 : 1;
        const uint32_t t_s = uni(tmem) + g * 128, t_o = uni(tmem) + 256 + g * 128;
        const uint64_t q_desc = desc_k(uni(base) + kOffQ + g * kQBytes);
        const uint64_t k_desc = desc_mn(uni(base) + kOffRing), v_desc = desc_k(uni(base) + kOffRing);
        for (int i = n_items - 1; i >= 0 && !failed; --i) {
          const int n = uni(items[i].k1 - items[i].k0);
          const bool both = uni(items[i].rows) > kGroupRows;
          const int keys = uni(items[i].ctx - items[i].k0 * kTileKeys);   // from the first tile on
          if (uni(items[i].kind) == kNothing || n == 0) continue;
          const uint32_t u0 = n_kv_ring;
          n_kv_ring += 2 * n;
          auto wait = [&](uint32_t bar, uint32_t parity) {
            if (!mbar_wait(bar, parity, wait_ns)) failed = true;
            failed = __any_sync(0xffffffffu, failed);
            return !failed;
          };
          if (g == 1 && !both) {
            // The first group is alone.  The slots are taken and given back all the
            // same: a warp that ran ahead of the ring could not tell a phase of a
            // slot's barrier from the one before the last.
            for (uint32_t u = u0; u != n_kv_ring; ++u) {
              if (!wait(kv_full(u % kSlots), (u / kSlots) & 1)) break;
              if (lane == 0) mbar_arrive(kv_empty(u % kSlots));
            }
            continue;
          }
          // S of the K tile in slot s; by the elected lane
          auto qk = [&](uint32_t s) {
            const uint64_t k = k_desc + (uint64_t)(s * (kSlot >> 4));
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              mma_ss(t_s, q_desc + (ks >> 2) * (kBox >> 4) + (ks & 3) * 2, k + ks * 128, kIdescMn, ks > 0);
            tc_commit(s_full(g));
          };
          if (!wait(kv_full(u0 % kSlots), (u0 / kSlots) & 1) || !wait(q_full(g), mma_items & 1)) break;
          ++mma_items;
          tc_fence_after();
          const uint32_t s0 = uni(u0 % kSlots);
          if (elected()) {
            qk(s0);
            tc_commit(kv_empty(s0));
          }
          __syncwarp();
          for (int j = 0; j < n; ++j) {
            const uint32_t uv = u0 + 2 * j + 1, uk = uv + 1;
            const uint32_t sv = uni(uv % kSlots), sk = uni(uk % kSlots);
            if (!wait(kv_full(sv), (uv / kSlots) & 1)) break;
            const int tail = keys - j * kTileKeys;   // valid keys of the tile
            const int steps = uni(min(8, (tail + 15) >> 4));   // products of 16 keys that hold valid ones
            if (tail < steps * 16) {
              // Zero the V rows of the last product's tokens past the context: 16-byte
              // pieces of 8 tokens, the one that the context ends in value by value.
              // (Both groups' warps do so; they write the same.)
#pragma unroll
              for (int x = 0; x < kH / 32; ++x) {
                const int ch = 32 * x + lane;
                uint8_t* v = smem + kOffRing + sv * kSlot + ch * 128;
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const int piece = 2 * steps - 2 + y, left = tail - piece * 8;
                  uint4* at = reinterpret_cast<uint4*>(v + (piece >> 3) * kBox + (((piece & 7) ^ (ch & 7)) << 4));
                  if (left <= 0) {
                    *at = make_uint4(0u, 0u, 0u, 0u);
                  } else if (left < 8) {
                    uint4 w = *at;
                    w.x &= keep2(left);
                    w.y &= keep2(left - 2);
                    w.z &= keep2(left - 4);
                    w.w &= keep2(left - 6);
                    *at = w;
                  }
                }
              }
              fence_proxy_async();
              __syncwarp();
            }
            if (j + 1 < n && !wait(kv_full(sk), (uk / kSlots) & 1)) break;
            if (!wait(p_full(g), mma_tiles & 1)) break;
            ++mma_tiles;
            // One group's block of products (this P V, the next Q K) at a time: mixed, both
            // blocks end late, the groups' softmaxes fall together and stay so, 2.0 us a tile
            // of keys against 1.4.  A group says that it wants to before it looks at the
            // other, and the second one steps back, so that no two begin at once.  (A matter
            // of speed alone: nobody waits for long.)
            if (both) {
              s_busy[g] = 1;
              for (int x = 0; x < kBusyPolls && s_busy[1 - g] != 0; ++x) {
                if (g == 1) {
                  s_busy[1] = 0;
                  for (; x < kBusyPolls && s_busy[0] != 0; ++x) {}
                  s_busy[1] = 1;
                }
              }
            }
            tc_fence_after();
            const bool more = (j & (kSumTiles - 1)) != 0;   // to the sum in O, or O begins again
            if (elected()) {
              const uint64_t v = v_desc + (uint64_t)(sv * (kSlot >> 4));
              if (steps == 8) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks)
                  mma_ts(t_o, t_s + ks * 8, v + (ks >> 2) * (kBox >> 4) + (ks & 3) * 2, kIdesc, more || ks > 0);
              } else {
                for (int ks = 0; ks < steps; ++ks)
                  mma_ts(t_o, t_s + ks * 8, v + (ks >> 2) * (kBox >> 4) + (ks & 3) * 2, kIdesc, more || ks > 0);
              }
              tc_commit(o_done(g));
              tc_commit(kv_empty(sv));
              if (j + 1 < n) {
                qk(sk);
                tc_commit(kv_empty(sk));
              }
            }
            __syncwarp();
            if (both && lane == 0) s_busy[g] = 0;
          }
        }
        if (failed && lane == 0) give_up();
      }
      if (!list_done()) break;
    }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int two_tokens = 2 / a.G, two_rows = 2 - two_tokens * a.G;
    while (const int n_items = next_list()) {
      // ================= softmax: group g, one row a thread
      const int g = warp >> 2;
      const int r = (warp & 3) * 32 + lane;               // row of the group, tensor-memory lane
      const uint32_t t_lane = tmem + ((uint32_t)((warp & 3) * 32) << 16);
      const uint32_t t_s = t_lane + g * 128, t_o = t_lane + 256 + g * 128;
      auto next_active = [&](int i) {   // the next item that this group has rows of, -1 behind the last
        while (i >= 0 && (items[i].kind == kNothing || items[i].rows <= g * kGroupRows)) --i;
        return i;
      };
      // An item's queries on their way to shared memory, swizzled, 16 lanes a row; the
      // products that read the item's before have all been seen to be done.
      auto load_queries = [&](const Item& it) {
        if (it.k0 == it.k1) return;
        const int rows = it.rows - g * kGroupRows;
        const int r0 = (warp & 3) * 32 + (lane >> 4), row = it.row0 + g * kGroupRows + r0;
        int token = row / a.G, head = row - token * a.G;
        const uint16_t* src = a.q + (int64_t)it.q_base * a.q_stride + it.h * a.G * kH + 8 * (lane & 15);
        const uint32_t q = base + kOffQ + g * kQBytes + ((lane & 15) >> 3) * kBox;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const int rx = r0 + 2 * x;
          const bool real = rx < rows;   // rows past the item's last are zeros
          copy_async16(q + rx * 128 + (((lane & 7) ^ (rx & 7)) << 4),
                       real ? src + (int64_t)token * a.q_stride + head * kH : a.q, real ? 16 : 0);
          head += two_rows;
          token += two_tokens;
          if (head >= a.G) {
            head -= a.G;
            ++token;
          }
        }
        __syncwarp();
      };
      auto queries_there = [&](const Item& it) {
        if (it.k0 == it.k1) return;
        copies_done();
        fence_proxy_async();
        mbar_arrive(q_full(g));
      };
      int i = next_active(n_items - 1);
      if (i >= 0) {
        load_queries(items[i]);
        queries_there(items[i]);
      }
      while (i >= 0 && !failed) {
        const Item& it = items[i];
        i = next_active(i - 1);
        const int row = it.row0 + g * kGroupRows + r;
        const bool real = g * kGroupRows + r < it.rows;
        const int token = row / a.G, hq = it.h * a.G + row - token * a.G;
        const int64_t out_row = ((int64_t)(it.q_base + token)) * a.Hq + hq;
        float m = -CUDART_INF_F, l = 0.0f;
        const int n = it.k1 - it.k0;
        if (n > 0) {
          // rows past the tile's last hold zero queries: whatever they sum up is not written
          const int seen = real ? visible(a, it.ctx, it.T, token) : 0x7fffffff;
          const float sc = a.scale_log2;
          for (int j = 0;;) {
            const int j0 = j, j1 = min(n, j0 + kSumTiles);
            for (; j < j1; ++j) {
              if (!mbar_wait(s_full(g), n_tile_g & 1, wait_ns)) failed = true;
              failed = __any_sync(0xffffffffu, failed);
              if (failed) break;
              tc_fence_after();
              if (j == n - 1 && i >= 0) load_queries(items[i]);   // the last product with this item's is done
              uint32_t s[128];
#pragma unroll
              for (int x = 0; x < 4; ++x) tmem_ld32(t_s + 32 * x, s + 32 * x);
              tmem_wait_ld32(s);
              tmem_hold32(s + 32);
              tmem_hold32(s + 64);
              tmem_hold32(s + 96);
              const int left = seen - (it.k0 + j) * kTileKeys;
              if (__any_sync(0xffffffffu, left < kTileKeys)) {
#pragma unroll
                for (int x = 0; x < 128; ++x)
                  if (x >= left) s[x] = 0xFF800000u;   // -inf
                __syncwarp();
              }
              // P against the running maximum as it stands, and the tile's maximum beside
              // it: the two do not wait for one another (1.36 us a tile of keys against 1.5 one
              // after the other).  Where the maximum has to move P is computed again.
              const uint64_t sc2 = pair(sc, sc);
              uint64_t sum[4];
              auto exps = [&](float ref) {
                const uint64_t ref2 = pair(ref, ref);
#pragma unroll
                for (int x = 0; x < 4; ++x) sum[x] = 0ull;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                  uint32_t p[16];
#pragma unroll
                  for (int e = 0; e < 16; ++e) {
                    float p0, p1;
                    unpair(fma2(pair(s[32 * x + 2 * e], s[32 * x + 2 * e + 1]), sc2, ref2), p0, p1);
                    p0 = ex2(p0);
                    p1 = ex2(p1);
                    sum[e & 3] = add2(sum[e & 3], pair(p0, p1));
                    p[e] = bf16x2(p0, p1);
                  }
                  tmem_st16(t_s + 16 * x, p);
                }
              };
              exps(m == -CUDART_INF_F ? 0.0f : -m);
              float mx[8];
#pragma unroll
              for (int x = 0; x < 8; ++x) mx[x] = fmaxf(__uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]));
#pragma unroll
              for (int x = 8; x < 64; ++x)
                mx[x & 7] = max3(mx[x & 7], __uint_as_float(s[2 * x]), __uint_as_float(s[2 * x + 1]));
              const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7])) * sc;
              if (__any_sync(0xffffffffu, top > m + kLazyLog2)) {
                const float m_new = fmaxf(m, top);
                const float f = m == -CUDART_INF_F ? 0.0f : ex2(m - m_new);
                __syncwarp();
                if (j > j0) {   // rescale O, to which the product before has been added (its commit came first)
                  const float fo = m == -CUDART_INF_F ? 1.0f : f;   // O is 0 there
#pragma unroll
                  for (int x = 0; x < 8; ++x) {
                    uint32_t o[16];
                    tmem_ld16(t_o + 16 * x, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fo);
                    tmem_st16(t_o + 16 * x, o);
                  }
                }
                l *= f;
                m = m_new;
                exps(m == -CUDART_INF_F ? 0.0f : -m);
              }
              float l0, l1;
              unpair(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), l0, l1);
              l += l0 + l1;
              tmem_wait_st_();
              tc_fence_before();
              mbar_arrive(p_full(g));
              ++n_tile_g;
            }
            if (failed || n <= kSumTiles) break;
            // O, once the last product of a segment of keys from j0 on is done, goes to the
            // row's sum in the CTA's third slot, which is laid out as a part with the maximum
            // that it is against; behind the last segment the sum goes to O.
            const bool last = j == n;
            if (!mbar_wait(last ? o_done(g) : s_full(g), (last ? n_tile_g - 1 : n_tile_g) & 1, wait_ns)) failed = true;
            failed = __any_sync(0xffffffffu, failed);
            if (failed) break;
            tc_fence_after();
            float* sum = a.ws_o + (int64_t)(2 * a.n_cta + c) * a.slot_rows * (kH + 2);
            float* sum_max = sum + a.slot_rows * kH + g * kGroupRows + r;
            float4* sum_o = reinterpret_cast<float4*>(sum) + g * kGroupRows + r;
            const bool add = j0 > 0 && real;
            const float m_sum = add ? *sum_max : -CUDART_INF_F;
            const float f = m_sum == -CUDART_INF_F ? 1.0f : ex2(m_sum - m);   // no keys yet: the sum is 0, or NaN and stays so
#pragma unroll 1
            for (int x = 0; x < 2; ++x) {
              uint32_t o[64];
              float4 u[16];
#pragma unroll
              for (int e = 0; e < 16; ++e)
                u[e] = add ? sum_o[(16 * x + e) * a.slot_rows] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
              __syncwarp();
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                tmem_ld32(t_o + 64 * x + 32 * y, o + 32 * y);
                tmem_wait_ld32(o + 32 * y);
              }
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                o[4 * e] = __float_as_uint(fmaf(u[e].x, f, __uint_as_float(o[4 * e])));
                o[4 * e + 1] = __float_as_uint(fmaf(u[e].y, f, __uint_as_float(o[4 * e + 1])));
                o[4 * e + 2] = __float_as_uint(fmaf(u[e].z, f, __uint_as_float(o[4 * e + 2])));
                o[4 * e + 3] = __float_as_uint(fmaf(u[e].w, f, __uint_as_float(o[4 * e + 3])));
                if (real && !last)
                  reinterpret_cast<uint4*>(sum_o)[(16 * x + e) * a.slot_rows] =
                      make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              }
              __syncwarp();
              if (last) {
#pragma unroll
                for (int y = 0; y < 4; ++y) tmem_st16(t_o + 64 * x + 16 * y, o + 16 * y);
              }
            }
            if (last) {
              tmem_wait_st_();
              break;
            }
            if (real) *sum_max = m;
            // Begun one behind the other by more than a tile of keys, the groups stay so
            // and leave the ring no room to load ahead: 3,300 clocks a tile of keys against
            // 2,740.
            if (it.rows > kGroupRows) {
              mbar_arrive(met);
              if (!mbar_wait(met, n_met & 1, wait_ns)) failed = true;
              ++n_met;
              failed = __any_sync(0xffffffffu, failed);
              if (failed) break;
            }
          }
          if (failed) break;
          // the next item's first product runs while this one's output is written
          if (i >= 0) queries_there(items[i]);
          if (!mbar_wait(o_done(g), (n_tile_g - 1) & 1, wait_ns)) failed = true;
          failed = __any_sync(0xffffffffu, failed);
          if (failed) break;
          tc_fence_after();
        } else if (i >= 0) {
          load_queries(items[i]);
          queries_there(items[i]);
        }
        // ---- the row's output, or its part
        const bool part = it.kind != kDirect;
        const float scale = part ? 1.0f : l > 0.0f ? 1.0f / l : l;   // 0 for a row without keys, NaN stays
        const int rr = g * kGroupRows + r;
        float* slot = a.ws_o + (int64_t)(2 * c + (it.kind == kPartB)) * a.slot_rows * (kH + 2);
        if (part) {
          if (real) *reinterpret_cast<float2*>(slot + a.slot_rows * kH + 2 * rr) = make_float2(m, l);
        } else if (real && a.lse) {
          a.lse[out_row] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          uint32_t o[32];
          __syncwarp();
          if (n > 0) {
            tmem_ld32(t_o + 32 * x, o);
            tmem_wait_ld32(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * scale);
          if (part) {   // [four channels][row]: a warp's stores are contiguous
            if (real) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                *reinterpret_cast<uint4*>(slot + ((8 * x + e) * a.slot_rows + rr) * 4) =
                    make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
            }
          } else if (real && a.out_f32) {
            float* dst = static_cast<float*>(a.out) + out_row * kH + 32 * x;
#pragma unroll
            for (int e = 0; e < 4; ++e) store32(dst + 8 * e, o + 8 * e, a.out_wide);
          } else if (real) {
            uint16_t* dst = static_cast<uint16_t*>(a.out) + out_row * kH + 32 * x;
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            store32(dst, o, a.out_wide);
            store32(dst + 16, o + 8, a.out_wide);
          }
        }
        tc_fence_before();   // O has been read before the next item's first product
      }
      if (failed && lane == 0) give_up();
      if (!list_done()) break;
    }
  }

  allow_dependent_launch();
  if (*s_abort) {
    copies_done();
    // the copies and products in flight end before the memory they use is given up
    if (warp == kTmaWarp && lane == 0) {
      for (uint32_t u = n_kv_ring > kSlots ? n_kv_ring - kSlots : 0; u < n_kv_ring; ++u)
        if (!(a.inject && u == 1)) mbar_wait(kv_full(u % kSlots), (u / kSlots) & 1, wait_ns);
    }
    if (warp == kMmaWarp || warp == kMmaWarp1) {
      if (elected()) tc_commit(drained);
      __syncwarp();
      mbar_wait(drained, 0, wait_ns);
      __syncwarp();
    }
  }
  if (tid == 0) reinterpret_cast<Header*>(a.ws_hdr)[c] = *s_abort ? Header{0, 0, 0, 0, 0, 0, 0, 0} : *s_hdr;
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

// ------------------------------------------------------------------ join of the parts

constexpr int kJoinThreads = 256;

// CTA (c, y) joins rows 32 y .. of the tile that CTA c of the kernel above began
// and did not end; a row a lane, 16 channels a warp, two parts at a time:
// with m the running maximum, O = sum 2^(m_i - m) O_i, l = sum 2^(m_i - m) l_i.
__global__ void __launch_bounds__(kJoinThreads)
chunk_combine_kernel(const ChunkArgs a) {
  const int c = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  wait_prerequisite_grids();
  const Header* hdr = reinterpret_cast<const Header*>(a.ws_hdr);
  const Header hd = hdr[c];
  // the CTAs behind, up to the one where the tile ends, 32 at a time
  int state = 0, ends = 0;
  auto read_window = [&](int d0) {
    const int d = d0 + lane;
    state = d < a.n_cta ? hdr[d].a_state : 0;
    ends = d < a.n_cta ? hdr[d].a_ends : 1;
  };
  read_window(c + 1);
  if (!hd.b_open || hd.b_state == 2 || (int)blockIdx.y * 32 >= hd.rows) return;
  const int r = blockIdx.y * 32 + lane;
  const bool on = r < hd.rows;
  const int64_t stride = (int64_t)a.slot_rows * (kH + 2);
  const float* ml = a.ws_o + (int64_t)a.slot_rows * kH + 2 * (on ? r : 0);
  const float* po = a.ws_o + (int64_t)(4 * warp * a.slot_rows + (on ? r : 0)) * 4;
  float acc[16], l = 0.0f, m = -CUDART_INF_F;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.0f;
  bool any = false;
  auto join = [&](int s0, int s1) {   // s1 < 0: one part
    const int64_t at0 = s0 * stride, at1 = (s1 < 0 ? s0 : s1) * stride;
    const float2 t0 = *reinterpret_cast<const float2*>(ml + at0), t1 = *reinterpret_cast<const float2*>(ml + at1);
    float4 o0[4], o1[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      o0[x] = *reinterpret_cast<const float4*>(po + at0 + (int64_t)x * a.slot_rows * 4);
      o1[x] = *reinterpret_cast<const float4*>(po + at1 + (int64_t)x * a.slot_rows * 4);
    }
    const float m_new = max3(m, t0.x, t1.x);
    // a part without keys weighs nothing, one whose sum is NaN stays NaN
    auto factor = [&](float mi, float li) { return mi == -CUDART_INF_F ? (li == li ? 0.0f : 1.0f) : ex2(mi - m_new); };
    const float f = any ? factor(m, l) : 0.0f, f0 = factor(t0.x, t0.y), f1 = s1 < 0 ? 0.0f : factor(t1.x, t1.y);
    l = fmaf(l, f, fmaf(t0.y, f0, s1 < 0 ? 0.0f : t1.y * f1));
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float u0[4] = {o0[x].x, o0[x].y, o0[x].z, o0[x].w}, u1[4] = {o1[x].x, o1[x].y, o1[x].z, o1[x].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[4 * x + e] = fmaf(acc[4 * x + e], f, fmaf(u0[e], f0, s1 < 0 ? 0.0f : u1[e] * f1));
    }
    m = m_new;
    any = true;
  };
  int waiting = hd.b_state == 1 ? 2 * c + 1 : -1;   // a part without a second one yet
  for (int d0 = c + 1; d0 < a.n_cta; d0 += 32) {
    if (d0 > c + 1) read_window(d0);
    const unsigned e = __ballot_sync(0xffffffffu, ends != 0);
    const unsigned within = e ? (e & -e) | ((e & -e) - 1) : 0xffffffffu;
    if (__ballot_sync(0xffffffffu, state == 2) & within) return;   // one CTA had it all and wrote it out
    unsigned valid = __ballot_sync(0xffffffffu, state == 1) & within;
    while (valid) {
      const int s = 2 * (d0 + __ffs(valid) - 1);
      valid &= valid - 1;
      if (waiting < 0) {
        waiting = s;
      } else {
        join(waiting, s);
        waiting = -1;
      }
    }
    if (e) break;
  }
  if (waiting >= 0) join(waiting, -1);
  if (!any || !on) return;
  const float scale = l > 0.0f ? 1.0f / l : l;
  const int row = hd.row0 + r;
  const int token = row / a.G;
  const int64_t out_row = (int64_t)(hd.q_base + token) * a.Hq + hd.h * a.G + row - token * a.G;
  uint32_t w[16];
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(acc[e] * scale);
  if (a.out_f32) {
    float* dst = static_cast<float*>(a.out) + out_row * kH + 16 * warp;
    store32(dst, w, a.out_wide);
    store32(dst + 8, w + 8, a.out_wide);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = bf16x2(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
    store32(static_cast<uint16_t*>(a.out) + out_row * kH + 16 * warp, w, a.out_wide);
  }
  if (warp == 0 && a.lse) a.lse[out_row] = l == 0.0f ? -CUDART_INF_F : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

int chunk_ctas() {
  const int n = device_sm_count();
  return n < kMaxCtas ? n : kMaxCtas;
}

// partial rows per slot: those of a tile, or all that the batch has
int chunk_slot_rows(int64_t n_rows, int G) {
  const int64_t rows = (n_rows * G + 1) & ~(int64_t)1;
  return rows < kTileRows ? (int)rows : kTileRows;
}

size_t chunk_ws_bytes(int64_t n_rows, int G) {
  return (size_t)kMaxCtas * sizeof(Header) + (size_t)3 * chunk_ctas() * chunk_slot_rows(n_rows, G) * (kH + 2) * 4;
}

cudaError_t launch_chunk_attn(ChunkArgs a, void* workspace, cudaStream_t s) {
  static bool configured[64] = {false};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev < 0 || dev >= 64 || !configured[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(chunk_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemAlloc);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) configured[dev] = true;
  }
  if (n_pool_too_large(a.n_pool)) return cudaErrorInvalidValue;
  CUtensorMap tk, tv;
  if (!bf16_page_map(&tk, a.k_pages, a.n_pool) || !bf16_page_map(&tv, a.v_pages, a.n_pool))
    return cudaErrorInvalidValue;
  a.n_cta = chunk_ctas();
  a.by_G = a.G > 1 ? ~0ull / a.G + 1 : 0;
  a.by_heads = a.Hkv > 1 ? ~0ull / a.Hkv + 1 : 0;
  a.out_wide = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
  a.slot_rows = chunk_slot_rows(a.n_rows, a.G);
  a.ws_hdr = workspace;
  a.ws_o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kMaxCtas * sizeof(Header));
  cudaError_t e = launch_programmatic(chunk_attn_kernel, dim3(a.n_cta), dim3(kThreads), kSmemAlloc, s, a, tk, tv);
  if (e != cudaSuccess) return e;
  return launch_programmatic(chunk_combine_kernel, dim3(a.n_cta, (a.slot_rows + 31) / 32), dim3(kJoinThreads), 0, s, a);
}

}  // namespace lynx
