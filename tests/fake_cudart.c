/* A stand-in for the CUDA runtime calls that hs_append and hs_mla_prefix make, preloaded before the real library so that
 * their checks of arguments run to the end on a machine without a GPU: there is one device, every call succeeds, and a
 * launch only writes down its grid. */
#include <stddef.h>
#include <stdint.h>

static int launches;
static unsigned grid[64][3]; /* of each launch */

int fake_launches(void) { return launches; }
const unsigned *fake_grid(int i) { return grid[i % 64]; }

int cudaGetDevice(int *device) {
  *device = 0;
  return 0;
}
static int last_error, fail_at; /* fail_at: launches from this one on fail (1: the next); 0: none does */
void fake_fail(int at) { fail_at = at; }
int fake_last_error(void) { return last_error; }
int cudaGetLastError(void) {
  const int e = last_error;
  last_error = 0;
  return e;
}
int cudaFuncSetAttribute(const void *f, int attr, int value) {
  (void)f, (void)attr, (void)value;
  return 0;
}
int cudaOccupancyMaxActiveClusters(int *clusters, const void *f, const void *config) {
  (void)f, (void)config;
  *clusters = 76;
  return 0;
}
static int held = 8; /* blocks of any kernel that an SM holds */
void fake_hold(int blocks) { held = blocks; }
int cudaOccupancyMaxActiveBlocksPerMultiprocessor(int *blocks, const void *f, int threads, size_t smem) {
  (void)f, (void)threads, (void)smem;
  *blocks = held;
  return held ? 0 : 2;
}
static int encode_tensor_map(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char *symbol, void **f, unsigned version, unsigned long long flags, int *found) {
  (void)symbol, (void)version, (void)flags;
  *f = (void *)encode_tensor_map;
  if (found) *found = 0;
  return 0;
}
/* cudaLaunchConfig_t begins with the grid's three numbers */
int cudaLaunchKernelExC(const void *config, const void *f, void **args) {
  (void)f, (void)args;
  if (fail_at == 1) return last_error = 1;
  if (fail_at > 1) --fail_at;
  for (int i = 0; i < 3; ++i) grid[launches % 64][i] = ((const unsigned *)config)[i];
  ++launches;
  return 0;
}
