/* The HIP functions that a kernel launch calls, for tests without a GPU: launches
 * are recorded and nothing runs.  Loaded with RTLD_GLOBAL before the library, whose
 * calls then arrive here.  stub_fail_at(n): launch n (from 0) is refused, as are all
 * grids that HIP refuses (a dimension of 2^32 work items or more). */
#include <stddef.h>
#include <stdint.h>

typedef struct { uint32_t x, y, z; } dim3;
typedef int hipError_t;

enum { kInvalidConfiguration = 9, kMost = 64 };
static dim3 pushed_grid, pushed_block;
static size_t pushed_shared;
static void *pushed_stream;
static uint64_t items[kMost];
static const void *functions[kMost];
static int launches, fail_at = -1;
static hipError_t last;

void stub_reset(void) { launches = 0, fail_at = -1, last = 0; }
void stub_fail_at(int n) { fail_at = n; }
int stub_launches(void) { return launches; }
uint64_t stub_items(int n) { return items[n]; }
const void *stub_function(int n) { return functions[n]; }

hipError_t __hipPushCallConfiguration(dim3 grid, dim3 block, size_t shared, void *stream) {
  pushed_grid = grid, pushed_block = block, pushed_shared = shared, pushed_stream = stream;
  return 0;
}
hipError_t __hipPopCallConfiguration(dim3 *grid, dim3 *block, size_t *shared, void **stream) {
  *grid = pushed_grid, *block = pushed_block, *shared = pushed_shared, *stream = pushed_stream;
  return 0;
}
hipError_t hipLaunchKernel(const void *f, dim3 grid, dim3 block, void **args, size_t shared, void *stream) {
  (void)args, (void)shared, (void)stream;
  const uint64_t x = (uint64_t)grid.x * block.x;
  const int refused = launches == fail_at || x >> 32 || grid.x == 0 || grid.y == 0;
  if (launches < kMost) items[launches] = x, functions[launches] = f;
  ++launches;
  if (refused) last = kInvalidConfiguration;
  return refused ? kInvalidConfiguration : 0;
}
hipError_t hipGetLastError(void) {
  const hipError_t e = last;
  last = 0;
  return e;
}
