/* Preloaded before fake_cudart.so: the two queries of the device that can fail, failing when they are told to. */
static int queries, fail_query, error; /* queries made; the one that fails next (1: the next), 0: none; and with what */
static int largest = 16, held = 76;    /* CTAs of the largest cluster that the device takes, and clusters that it holds */

static int last;                       /* error of a query, until it is taken */

int cudaGetLastError(void) {
  const int e = last;
  last = 0;
  return e;
}
int fake_query_error(void) { return last; }
int fake_queries(void) { return queries; }
void fake_fail_query(int at, int with) { fail_query = at, error = with; }
void fake_clusters(int ctas, int count) { largest = ctas, held = count; }
static int fails(void) {
  ++queries;
  return fail_query && --fail_query == 0;
}
static const void *set[64]; /* kernels that have been given their shared memory: the others do not fit on the device */
static int nset, ask_first;
void fake_ask_first(int on) { ask_first = on; }
int cudaFuncSetAttribute(const void *f, int attr, int value) {
  (void)value;
  if (fails()) return last = error;
  if (attr == 8 && nset < 64) set[nset++] = f; /* cudaFuncAttributeMaxDynamicSharedMemorySize */
  return 0;
}
/* cudaLaunchConfig_t begins with the grid's three numbers */
int cudaOccupancyMaxActiveClusters(int *clusters, const void *f, const void *config) {
  int known = !ask_first;
  for (int i = 0; i < nset; ++i) known |= set[i] == f;
  if (fails()) return last = error;
  if (*(const unsigned *)config > (unsigned)largest) return last = 912; /* cudaErrorInvalidClusterSize */
  *clusters = known ? held : 0;
  return 0;
}
