// Pages, positions and slots of a step's new tokens, from the requests' lengths
// (lynx_assign_pages).
//
//   held_b  = ceil(ctx_b / 256)                 pages the request has
//   need_b  = ceil((ctx_b + new_b) / 256) - held_b
//   end_b   = sum of Hkv need_b up to and with b; cu_b = sum of new_b before b
//   fresh page held_b + i of KV head h takes free[end_b - Hkv need_b + i Hkv + h]
//   row r of request b:  pos = ctx_b + r - cu_b,
//                        slot of head h = 256 table[b][h][pos / 256] + pos % 256
//
// One launch.  Every CTA takes a tile of rows and forms the two running sums over
// the requests itself (kThreads requests at a time, 8 bytes each, from L2)
// until its rows are covered, so that no CTA waits on another; the first CTA
// goes through all requests and writes the per-request outputs.  A row finds
// its request by bisection in the sums of the current kThreads requests.  The
// row that stands at the start of a page writes that page's table entries: the
// fresh pages' first positions are all new rows, and no other row reads those
// entries (it takes the id from the free list itself), so nothing races.
//
// Bound by the launch and the chain lengths -> sums -> row -> table -> slot: 3.1 us for a
// decode step of 64 requests (the host's call; 2.6 us on the GPU), 5.5 us for 100,000
// rows of 8 heads, whose slots (8 bytes a row and head) would take 1 us at the memory's
// rate.

#include "lynx_internal.cuh"

namespace lynx {
namespace {

constexpr int kThreads = 256;
// Sums stop here: past every number of rows and of free ids (2^30 at most), and
// two such numbers still add up within 32 bits.  Addition cut off at a bound is
// associative, so the sums are the same in any order.
constexpr int kMost = (1 << 30) + 1;
static_assert(kThreads == 256, "eight steps of bisection; a row of a CTA's tile a thread");

__device__ __forceinline__ int add(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)kMost); }

// A row of the tile: where its page's id stands for head 0 and how far on for the
// next head (the page table, or the free list for a fresh page), and its place in
// the page; kBegins: the first row of a fresh page; -1: a row without a slot
struct Row {
  const int32_t* ids;
  int stride;
  int at;
};
constexpr int kBegins = kP;

template <int kTile>   // rows per CTA
__global__ void __launch_bounds__(kThreads, 1)   // 48 registers: all ids of a thread in flight (34: 11% slower)
assign_pages_kernel(const AssignArgs a) {
  __shared__ int s_rows[kThreads];   // rows before request i of the group
  __shared__ int s_free[kThreads];   // first free-list index of request i
  __shared__ int s_ctx[kThreads];
  __shared__ int s_held[kThreads];   // pages held; -1: refused
  __shared__ int2 s_warp[kThreads / 32];
  __shared__ int s_taken;
  __shared__ Row s_row[kTile];
  __shared__ int64_t s_entry[kTile];   // of rows at kBegins: the table entry of their page, head 0

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row0 = blockIdx.x * kTile;
  const int row1 = min(row0 + kTile, a.n_rows);
  const bool first = blockIdx.x == 0;
  const int max_keys = a.max_pages * kP;

  int pos = -1;   // of row row0 + tid
  if (tid < kTile) s_row[tid].at = -1;
  if (tid == 0) s_taken = 0;
  allow_dependent_launch();
  wait_prerequisite_grids();

  auto lengths = [&](int b) { return b < a.B ? make_int2(a.ctx_len[b], a.new_len[b]) : make_int2(0, 0); };
  int2 next = lengths(tid);   // of the next group, on their way
  int rows_before = 0, free_before = 0;   // over the groups behind us
  for (int b0 = 0; b0 < a.B && (first || rows_before < row1); b0 += kThreads) {
    const int b = b0 + tid;
    const bool in = b < a.B;
    const int ctx = next.x, asked = next.y;
    next = lengths(b + kThreads);
    bool valid = in && ctx >= 0 && asked >= 0 && (long long)ctx + asked <= max_keys;
    if (in && !valid && first) atomicExch(a.status, 3);
    const int rows = min(max(asked, 0), kMost);
    const int held = (ctx + kP - 1) / kP;
    const int need = valid ? (ctx + rows + kP - 1) / kP - held : 0;
    const int ids = (int)min((long long)need * a.Hkv, (long long)kMost);
    // Inclusive sums of rows and ids, side by side.  The ids of a request whose
    // rows do not fit count too: behind it no request with rows fits, so no sum
    // that matters has them.
    int row_end = rows, free_end = ids;
    auto scan = [&](int steps) {
#pragma unroll
      for (int o = 1; o < steps; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, row_end, o), v = __shfl_up_sync(0xffffffffu, free_end, o);
        if (lane >= o) {
          row_end = add(row_end, u);
          free_end = add(free_end, v);
        }
      }
    };
    scan(32);
    if (lane == 31) s_warp[warp] = make_int2(row_end, free_end);
    __syncthreads();
    // the sums of the warps in front of this one, and of all
    const int row_mine = row_end, free_mine = free_end;
    const int2 u = lane < kThreads / 32 ? s_warp[lane] : make_int2(0, 0);
    row_end = u.x;
    free_end = u.y;
    scan(kThreads / 32);
    const int before = max(warp - 1, 0);
    int rows_warp = __shfl_sync(0xffffffffu, row_end, before), free_warp = __shfl_sync(0xffffffffu, free_end, before);
    rows_warp = add(rows_before, warp > 0 ? rows_warp : 0);
    free_warp = add(free_before, warp > 0 ? free_warp : 0);
    rows_before = add(rows_before, __shfl_sync(0xffffffffu, row_end, kThreads / 32 - 1));
    free_before = add(free_before, __shfl_sync(0xffffffffu, free_end, kThreads / 32 - 1));
    row_end = row_mine;
    free_end = free_mine;
    row_end = add(row_end, rows_warp);
    free_end = add(free_end, free_warp);
    valid = valid && row_end <= a.n_rows;
    const bool granted = valid && (need == 0 || free_end <= a.n_free);
    // The first row is the sum of the requests in front, not row_end - rows: that is too
    // small where the sum has been cut off, and the bisection needs s_rows in order.
    const int rows_lanes = __shfl_up_sync(0xffffffffu, row_mine, 1);
    s_rows[tid] = add(rows_warp, lane > 0 ? rows_lanes : 0);
    s_free[tid] = free_end - ids;   // read of granted requests, whose sums are whole
    s_ctx[tid] = ctx;
    s_held[tid] = granted ? held : -1;
    if (first && in) {
      if (b == 0) a.cu_new[0] = 0;
      a.cu_new[b + 1] = min(row_end, a.n_rows);
      a.ctx_out[b] = granted ? ctx + rows : ctx;
      // the running sum of the granted requests does not decrease
      if (granted && need > 0) atomicMax(&s_taken, free_end);
    }
    __syncthreads();
    // the tile's rows that lie in this group
    const int lo = s_rows[0], r = row0 + tid;
    if (tid < kTile && r < row1 && r >= lo && r < rows_before) {
      int i = 0, j = kThreads;   // last request whose rows begin at or before r: those in front of it end there
#pragma unroll
      for (int step = 0; step < 8; ++step) {   // log2 kThreads
        const int mid = (i + j) >> 1;
        if (s_rows[mid] <= r) i = mid; else j = mid;
      }
      if (s_held[i] >= 0) {
        pos = s_ctx[i] + r - s_rows[i];
        const int page = pos / kP;
        const int64_t entry = (int64_t)(b0 + i) * a.Hkv * a.max_pages + page;
        Row row;
        row.at = pos % kP;
        if (page < s_held[i]) {
          row.ids = a.page_table + entry;
          row.stride = a.max_pages;
        } else {
          row.ids = a.free_pages + s_free[i] + (page - s_held[i]) * a.Hkv;
          row.stride = 1;
          if (row.at == 0) {
            row.at = kBegins;
            s_entry[tid] = entry;
          }
        }
        s_row[tid] = row;
      }
    }
    __syncthreads();
  }
  if (first && tid == 0) a.n_taken[0] = s_taken;

  if (tid < row1 - row0) a.positions[row0 + tid] = pos;
  // slots, kBatch a thread at a time, so that their ids are read together
  constexpr int kBatch = 1024 / kTile;
  const int n_out = (row1 - row0) * a.Hkv;
  const int dr = kThreads / a.Hkv, dh = kThreads - dr * a.Hkv;
  int r = tid / a.Hkv, h = tid - r * a.Hkv;
  int64_t* slots = a.slots + (int64_t)row0 * a.Hkv;
  for (int i0 = tid; i0 < n_out; i0 += kBatch * kThreads) {
    int id[kBatch], at[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      at[k] = -1;
      id[k] = 0;
      if (i0 + k * kThreads < n_out) {
        const Row row = s_row[r];
        at[k] = row.at;
        if (row.at >= 0) id[k] = row.ids[(int64_t)h * row.stride];
      }
      r += dr;
      h += dh;
      if (h >= a.Hkv) {
        h -= a.Hkv;
        ++r;
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * kThreads;
      if (i >= n_out) break;
      if (at[k] == kBegins) {
        const int row = i / a.Hkv;
        a.page_table[s_entry[row] + (int64_t)(i - row * a.Hkv) * a.max_pages] = id[k];
      }
      slots[i] = at[k] >= 0 ? (int64_t)id[k] * kP + at[k] % kP : -1;
    }
  }
}

}  // namespace

cudaError_t launch_assign_pages(const AssignArgs& a, cudaStream_t s) {
  // 128 rows a CTA, or 256 where the sums would be formed by too many CTAs: by more than
  // eight an SM, or four where a CTA has few slots to write.  us with 128 against 256, by
  // rows and heads: 70,000 x 4 4.4 / 4.7, 90,000 x 4 4.4 / 4.0, 120,000 x 1 4.8 / 4.4, 250,000 x 1
  // 7.7 / 5.3, 60,000 x 8 4.7 / 6.0, 100,000 x 8 5.5 / 6.0, 120,000 x 8 6.0 / 6.1, of 1,000 requests
  // 60,000 x 8 6.8 / 6.0.
  const int64_t groups = (a.B + kThreads - 1) / kThreads;
  const bool wide = a.n_rows * groups > (int64_t)128 * (a.Hkv > 4 ? 8 : 4) * device_sm_count();
  const int tile = wide ? 256 : 128;
  const int grid = a.n_rows > tile ? (a.n_rows + tile - 1) / tile : 1;
  return launch_programmatic(wide ? assign_pages_kernel<256> : assign_pages_kernel<128>, dim3(grid), dim3(kThreads), 0, s,
                             a);
}

}  // namespace lynx
