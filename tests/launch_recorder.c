/* Stands in for the HIP runtime's launch calls on a machine without a GPU
 * (LD_PRELOAD): a launch computes nothing, its grid and block are appended to
 * the file that LAUNCH_LOG names, and a launch of 2^32 threads or more fails as
 * the runtime's does. */
#include <stddef.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

typedef struct { uint32_t x, y, z; } dim3_t;
static dim3_t s_grid, s_block;
static int s_error;

int hipGetDevice(int* d) { *d = 0; return 0; }
int hipGetDeviceCount(int* n) { *n = 1; return 0; }
int hipDeviceGetAttribute(int* v, int what, int dev) { (void)what; (void)dev; *v = 256; return 0; }
int hipExtStreamGetCUMask(void* st, uint32_t n, uint32_t* m) { (void)st; (void)n; (void)m; return 1; }
int hipGetLastError(void) { const int e = s_error; s_error = 0; return e; }
int hipPeekAtLastError(void) { return s_error; }
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t lds, void* st) {
  (void)lds; (void)st;
  s_grid = g;
  s_block = b;
  return 0;
}
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* lds, void** st) {
  *g = s_grid;
  *b = s_block;
  *lds = 0;
  *st = NULL;
  return 0;
}
int hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** args, size_t lds, void* st) {
  (void)f; (void)args; (void)lds; (void)st;
  const int ok = (uint64_t)g.x * b.x < (1ull << 32);
  FILE* log = fopen(getenv("LAUNCH_LOG"), "a");
  if (!log) abort();
  fprintf(log, "%u %u %d\n", g.x, b.x, ok);
  fclose(log);
  if (!ok) s_error = 9;
  return ok ? 0 : 9;
}
