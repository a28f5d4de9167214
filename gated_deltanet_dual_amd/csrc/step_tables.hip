// step_tables.hip -- the page tables, slot maps, positions and offsets of a
// serving step, built on the GPU from the requests' lengths.
//
//   have_r = ceil(held_r / page), need_r = ceil((held_r + new_r) / page)
//   request r takes need_r - have_r pages, in request order, from
//   free_pages[used + sum_{s<r} (need_s - have_s)] on.
#include <hip/hip_runtime.h>

#include "layer_launch.h"

namespace flare {
namespace {

constexpr int kThreads = 512;

// Every workgroup scans all lengths (8 bytes a request, from the L2) and keeps
// the two offsets of each request in LDS; then it fills its own share of the
// rows.  One launch instead of a scan and a fill.
__global__ __launch_bounds__(kThreads) void step_tables_kernel(StepTablesArgs a, int rows_per_block) {
  extern __shared__ int32_t lds[];
  int32_t *cu = lds, *first = lds + a.num_req;  // tokens and new pages before each request
  __shared__ int64_t wave_tok[kThreads / 64], wave_pg[kThreads / 64];
  __shared__ int bad;
  const int R = a.num_req, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid == 0) bad = 0;
  __syncthreads();
  const int64_t limit = (int64_t)a.max_pages * a.page;
  int64_t tok0 = 0, pg0 = 0;
  int why = 0;  // the largest of the thread's reasons
  for (int base = 0; base < R; base += kThreads) {
    const int r = base + tid;
    int64_t held = 0, fresh = 0;
    int64_t tokens = 0;
    if (r < R) {
      held = a.seq_lens[r];
      tokens = a.new_lens[r];
      if (held < 0 || tokens < 0) {
        why = FLARE_TABLES_BAD_LENGTH;
        held = tokens = 0;
      }
      if (held + tokens > limit || held + tokens + a.position_offset > INT32_MAX) {
        why = why > FLARE_TABLES_TOO_LONG ? why : FLARE_TABLES_TOO_LONG;
      }
      fresh = (held + tokens + a.page - 1) / a.page - (held + a.page - 1) / a.page;
    }
    int64_t st = tokens, sp = fresh;
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
    __syncthreads();
    int64_t bt = tok0, bp = pg0;
    for (int w = 0; w < kThreads / 64; ++w) {
      if (w < wave) {
        bt += wave_tok[w];
        bp += wave_pg[w];
      }
      tok0 += wave_tok[w];
      pg0 += wave_pg[w];
    }
    if (r < R) {
      // beyond 32 bits only where the call is refused below
      cu[r] = (int32_t)(bt + st - tokens);
      first[r] = (int32_t)(bp + sp - fresh);
    }
    __syncthreads();
  }
  const int32_t used = *a.pages_used;
  if (used < 0) why = FLARE_TABLES_BAD_LENGTH;
  if (why) atomicMax(&bad, why);
  __syncthreads();
  int status = bad;
  if (status == 0 && tok0 > a.max_tokens) status = FLARE_TABLES_TOO_MANY_TOKENS;
  if (status == 0 && used + pg0 > a.num_free) status = FLARE_TABLES_NO_PAGES;
  const int64_t total = status ? 0 : tok0;

  // the per-request outputs, spread over the workgroups
  for (int r = blockIdx.x * kThreads + tid; r < R; r += gridDim.x * kThreads) {
    a.cu_new[r] = status ? 0 : cu[r];
    a.seq_lens_out[r] = a.seq_lens[r] + (status ? 0 : a.new_lens[r]);
  }
  if (blockIdx.x == 0 && tid == 0) {
    a.cu_new[R] = (int32_t)total;
    *a.pages_used_out = used + (status ? 0 : (int32_t)pg0);
    *a.status = status;
  }
  const int64_t row0 = (int64_t)blockIdx.x * rows_per_block;
  for (int i = tid; i < rows_per_block; i += kThreads) {
    const int64_t row = row0 + i;
    if (row >= a.max_tokens) break;
    if (row >= total) {
      a.positions[row] = 0;
      a.slots[row] = -1;
      continue;
    }
    // the request of this row: the last one that starts at or before it
    int lo = 0, hi = R - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= (int32_t)row) lo = mid;
      else hi = mid - 1;
    }
    const int32_t held = a.seq_lens[lo];
    const int32_t pos = held + ((int32_t)row - cu[lo]);
    const int32_t pg = pos / a.page, have = (held + a.page - 1) / a.page;
    int32_t *entry = a.block_table + (int64_t)lo * a.max_pages + pg;
    int32_t id;
    if (pg >= have) {
      id = a.free_pages[used + first[lo] + pg - have];
      // the row that opens a page enters it into the table
      if (pos == pg * a.page) *entry = id;
    } else {
      id = *entry;
    }
    a.positions[row] = pos + a.position_offset;
    a.slots[row] = (int64_t)id * a.page + (pos - pg * a.page);
  }
}

}  // namespace

hipError_t launch_step_tables(const StepTablesArgs &a, hipStream_t st) {
  int rows = 1024;
  int64_t grid = (a.max_tokens + rows - 1) / rows;
  if (grid < 1) grid = 1;
  TimedLaunch tl(K_STEP_TABLES, st);
  step_tables_kernel<<<(int)grid, kThreads, (size_t)2 * (a.num_req > 0 ? a.num_req : 1) * sizeof(int32_t), st>>>(a, rows);
  return hipGetLastError();
}

}  // namespace flare
