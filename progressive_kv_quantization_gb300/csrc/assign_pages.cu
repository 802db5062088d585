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
// One launch.  Every CTA takes kTile rows and forms the two running sums over
// the requests itself (kThreads requests at a time, 8 bytes each, from L2)
// until its rows are covered, so that no CTA waits on another; the first CTA
// goes through all requests and writes the per-request outputs.  A row finds
// its request by bisection in the sums of the current kThreads requests.  The
// row that stands at the start of a page writes that page's table entries: the
// fresh pages' first positions are all new rows, and no other row reads those
// entries (it takes the id from the free list itself), so nothing races.
//
// Bound by the launch for a decode step and by the slots written (8 bytes a row
// and head) for prompts.

#include "lynx_internal.cuh"

namespace lynx {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 128;    // rows per CTA

__global__ void __launch_bounds__(kThreads)
assign_pages_kernel(const AssignArgs a) {
  __shared__ long long s_rows[kThreads + 1];   // rows before request i of the group; [n]: behind the last
  __shared__ long long s_free[kThreads];       // first free-list index of request i
  __shared__ int s_ctx[kThreads];
  __shared__ int s_held[kThreads];             // pages held; -1: refused
  __shared__ long long s_warp[2][kThreads / 32];
  __shared__ long long s_taken;
  __shared__ int r_pos[kTile];                 // position of the tile's row; -1: none
  __shared__ int r_req[kTile];
  __shared__ long long r_free[kTile];          // free-list index of the row's page, head 0; -1: in the table

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int row0 = blockIdx.x * kTile;
  const int row1 = min(row0 + kTile, a.n_rows);
  const bool first = blockIdx.x == 0;
  const int max_keys = a.max_pages * kP;

  if (tid < kTile) r_pos[tid] = -1;
  if (tid == 0) s_taken = 0;
  __syncthreads();

  long long rows_before = 0, free_before = 0;   // over the groups behind us
  for (int b0 = 0; b0 < a.B && (first || rows_before < row1); b0 += kThreads) {
    const int n = min(kThreads, a.B - b0);
    const int b = b0 + tid;
    int ctx = 0, rows = 0;
    bool valid = false;
    if (tid < n) {
      ctx = a.ctx_len[b];
      rows = a.new_len[b];
      valid = ctx >= 0 && rows >= 0 && (long long)ctx + rows <= max_keys;
      if (!valid && first) atomicExch(a.status, 3);
      rows = max(rows, 0);
    }
    // inclusive sums of the rows, then of the pages of the requests that can be granted
    auto block_scan = [&](long long v, int which) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
      }
      if (lane == 31) s_warp[which][warp] = v;
      __syncthreads();
      long long before = 0;
      for (int w = 0; w < warp; ++w) before += s_warp[which][w];
      return v + before;
    };
    const long long row_end = rows_before + block_scan(rows, 0);
    valid = valid && row_end <= a.n_rows;
    const int held = (ctx + kP - 1) / kP;
    const int need = valid ? (ctx + rows + kP - 1) / kP - held : 0;
    const long long free_end = free_before + block_scan((long long)need * a.Hkv, 1);
    const bool granted = valid && (need == 0 || free_end <= a.n_free);
    s_rows[tid] = row_end - rows;
    if (tid == kThreads - 1) s_rows[kThreads] = row_end;
    s_free[tid] = free_end - (long long)need * a.Hkv;
    s_ctx[tid] = ctx;
    s_held[tid] = granted ? held : -1;
    if (first) {
      if (tid < n) {
        if (b == 0) a.cu_new[0] = 0;
        a.cu_new[b + 1] = (int)min(row_end, (long long)a.n_rows);
        a.ctx_out[b] = granted ? ctx + rows : ctx;
        // the running sum of the granted requests does not decrease
        if (granted && need > 0) atomicMax(&s_taken, free_end);
      }
    }
    __syncthreads();
    rows_before = s_rows[kThreads];
    if (lane == 31) s_warp[0][warp] = free_end;
    const long long lo = s_rows[0];
    // the tile's rows that lie in this group
    if (tid < kTile && row0 + tid < row1 && row0 + tid >= lo && row0 + tid < rows_before) {
      const int r = row0 + tid;
      int i = 0, j = kThreads;   // last request whose rows begin at or before r: those in front of it end there
      while (j - i > 1) {
        const int mid = (i + j) >> 1;
        if (s_rows[mid] <= r) i = mid; else j = mid;
      }
      if (s_held[i] >= 0) {
        const int pos = s_ctx[i] + (int)(r - s_rows[i]);
        const int page = pos / kP;
        r_pos[tid] = pos;
        r_req[tid] = b0 + i;
        r_free[tid] = page < s_held[i] ? -1 : s_free[i] + (long long)(page - s_held[i]) * a.Hkv;
      }
    }
    __syncthreads();
    free_before = s_warp[0][kThreads / 32 - 1];
    __syncthreads();
  }
  if (first && tid == 0) a.n_taken[0] = (int)s_taken;

  if (tid < row1 - row0) a.positions[row0 + tid] = r_pos[tid];
  const int n_out = (row1 - row0) * a.Hkv;
  for (int i = tid; i < n_out; i += kThreads) {
    const int r = i / a.Hkv, h = i - r * a.Hkv;
    const int pos = r_pos[r];
    int64_t slot = -1;
    if (pos >= 0) {
      const int page = pos / kP;
      int32_t* entry = a.page_table + ((int64_t)r_req[r] * a.Hkv + h) * a.max_pages + page;
      const long long f = r_free[r];
      const int id = f < 0 ? *entry : a.free_pages[f + h];
      if (f >= 0 && pos % kP == 0) *entry = id;
      slot = (int64_t)id * kP + pos % kP;
    }
    a.slots[(int64_t)row0 * a.Hkv + i] = slot;
  }
}

}  // namespace

cudaError_t launch_assign_pages(const AssignArgs& a, cudaStream_t s) {
  const int grid = a.n_rows > kTile ? (a.n_rows + kTile - 1) / kTile : 1;
  assign_pages_kernel<<<grid, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace lynx
