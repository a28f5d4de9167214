// step_tables.hip -- the page tables, slot maps, positions and offsets of a
// serving step, built on the GPU from the requests' lengths.
//
//   have_r = ceil(held_r / page), need_r = ceil((held_r + new_r) / page)
//   request r takes need_r - have_r pages, in request order, from
//   free_pages[used + sum_{s<r} (need_s - have_s)] on.
#include <hip/hip_runtime.h>

#include "fast_div.h"
#include "layer_launch.h"

namespace flare {
namespace {

constexpr int kThreads = 512;

// Pages that n tokens take.
__device__ __forceinline__ int32_t pages_of(uint32_t n, const FastDiv &d) { return n ? fast_div(n - 1, d) + 1 : 0; }

// Every workgroup scans all lengths (8 bytes a request, from the L2) and keeps
// the two offsets of each request in LDS; then it fills its own share of the
// rows.  One launch instead of a scan and a fill.  Latency bounds it: the lengths'
// loads, the scan's two barriers, a search of log2 R steps and a page's load follow on
// each other.  256 requests x 4 tokens 5.1 us; 700 requests with 700 K tokens, 16 a
// page, in 1.4 M rows 13.3 us for 17 MB (rows behind the last token are written too).
__global__ __launch_bounds__(kThreads) void step_tables_kernel(StepTablesArgs a, FastDiv pd, int rows_per_block) {
  extern __shared__ int32_t lds[];
  // of each request: tokens and new pages before it, and the tokens it holds
  int32_t *cu = lds, *first = lds + a.num_req, *have = lds + 2 * a.num_req;
  __shared__ int64_t wave_tok[kThreads / 64], wave_pg[kThreads / 64];
  __shared__ int bad;
  const int R = a.num_req, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int32_t used = *a.pages_used;
  if (tid == 0) bad = 0;
  for (int r = tid; r < R; r += kThreads) {
    have[r] = a.seq_lens[r];
    cu[r] = a.new_lens[r];
  }
  __syncthreads();
  // a thread sums a run of requests, the workgroup scans the threads' sums once
  const int64_t limit = (int64_t)a.max_pages * a.page;
  const int run = (R + kThreads - 1) / kThreads, r0 = tid * run, r1 = r0 + run < R ? r0 + run : R;
  int64_t tokens = 0, pages = 0;
  int why = 0;  // the largest of the thread's reasons
  for (int r = r0; r < r1; ++r) {
    const int64_t held = have[r], add = cu[r];
    if (held < 0 || add < 0) {
      why = FLARE_TABLES_BAD_LENGTH;
    } else {
      if ((held + add > limit || held + add + a.position_offset > INT32_MAX) && why < FLARE_TABLES_TOO_LONG)
        why = FLARE_TABLES_TOO_LONG;
      tokens += add;
      if (held + add <= INT32_MAX) pages += pages_of((uint32_t)(held + add), pd) - pages_of((uint32_t)held, pd);
    }
  }
  int64_t st = tokens, sp = pages;
  for (int o = 1; o < 64; o <<= 1) {
    const int64_t ut = __shfl_up(st, o), up = __shfl_up(sp, o);
    if (lane >= o) {
      st += ut;
      sp += up;
    }
  }
  if (lane == 63) {
    wave_tok[wave] = st;
    wave_pg[wave] = sp;
  }
  if (why) atomicMax(&bad, why);
  __syncthreads();
  int64_t tok0 = 0, pg0 = 0;  // totals
  st -= tokens;
  sp -= pages;
  for (int w = 0; w < kThreads / 64; ++w) {
    if (w < wave) {
      st += wave_tok[w];
      sp += wave_pg[w];
    }
    tok0 += wave_tok[w];
    pg0 += wave_pg[w];
  }
  // beyond 32 bits only where the call is refused below
  for (int r = r0; r < r1; ++r) {
    const uint32_t held = (uint32_t)have[r], add = (uint32_t)cu[r];
    cu[r] = (int32_t)st;
    first[r] = (int32_t)sp;
    st += add;
    sp += pages_of(held + add, pd) - pages_of(held, pd);
  }
  __syncthreads();
  int status = used < 0 ? FLARE_TABLES_BAD_LENGTH : bad;
  if (status == 0 && tok0 > a.max_tokens) status = FLARE_TABLES_TOO_MANY_TOKENS;
  if (status == 0 && used + pg0 > a.num_free) status = FLARE_TABLES_NO_PAGES;
  const int64_t total = status ? 0 : tok0;

  // the per-request outputs, spread over the workgroups
  for (int r = blockIdx.x * kThreads + tid; r < R; r += gridDim.x * kThreads) {
    a.cu_new[r] = status ? 0 : cu[r];
    a.seq_lens_out[r] = have[r] + (status ? 0 : a.new_lens[r]);
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_new[R] = (int32_t)total;
    *a.pages_used_out = used + (status ? 0 : (int32_t)pg0);
    *a.status = status;
  }
  // four rows of a thread side by side: their searches and page loads overlap
  const int64_t row0 = (int64_t)blockIdx.x * rows_per_block;
  int top = 1;
  while (2 * top < R) top *= 2;
  for (int i = tid; i < rows_per_block; i += 4 * kThreads) {
    int req[4];
    int32_t id[4], pos[4];
    bool live[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      req[k] = 0;
      live[k] = i + k * kThreads < rows_per_block && row0 + i + k * kThreads < total;
    }
    // the request of a row: the last one that starts at or before it (no branches:
    // the four rows' LDS reads and page loads are then in flight together)
    for (int step = top; step > 0; step >>= 1) {
      int32_t at[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) at[k] = cu[req[k] + step < R ? req[k] + step : req[k]];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        req[k] += req[k] + step < R && at[k] <= (int32_t)(row0 + i + k * kThreads) ? step : 0;
    }
    const int32_t *from[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int r = req[k];
      const int32_t held = have[r];
      pos[k] = held + ((int32_t)(row0 + i + k * kThreads) - cu[r]);
      const int32_t pg = fast_div(pos[k], pd), old = pages_of(held, pd);
      from[k] = pg >= old ? a.free_pages + (used + first[r] + pg - old) : a.block_table + ((int64_t)r * a.max_pages + pg);
      if (!live[k]) from[k] = a.pages_used;  // padding: any readable place
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) id[k] = *from[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int64_t row = row0 + i + k * kThreads;
      if (i + k * kThreads >= rows_per_block || row >= a.max_tokens) continue;
      const int32_t pg = fast_div(pos[k], pd), off = pos[k] - pg * a.page;
      // the row that opens a page enters it into the table
      if (live[k] && off == 0 && pg >= pages_of(have[req[k]], pd))
        a.block_table[(int64_t)req[k] * a.max_pages + pg] = id[k];
      a.positions[row] = live[k] ? pos[k] + a.position_offset : 0;
      a.slots[row] = live[k] ? (int64_t)id[k] * a.page + off : -1;
    }
  }
}

}  // namespace

hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t st) {
  // few workgroups where there are many rows: each of them scans all lengths
  int64_t rows = (a.max_tokens + 511) / 512;
  rows = rows < 1024 ? 1024 : (rows + kThreads - 1) / kThreads * kThreads;
  int64_t grid = (a.max_tokens + rows - 1) / rows;
  if (grid < 1) grid = 1;
  const FastDiv pd = make_fast_div(a.page);
  TimedLaunch tl(K_STEP_TABLES, st);
  step_tables_kernel<<<(int)grid, kThreads, (size_t)3 * (a.num_req > 0 ? a.num_req : 1) * sizeof(int32_t), st>>>(a, pd, (int)rows);
  return hipGetLastError();
}

}  // namespace flare
