/* HIP calls that succeed without a GPU: device work is left out, host work runs.  Preloaded by the tests of the host side. */
#include <stdlib.h>

typedef int hipError_t;

hipError_t hipGetDevice(int* d) { *d = 0; return 0; }
hipError_t hipSetDevice(int d) { (void)d; return 0; }
hipError_t hipEventCreateWithFlags(void** e, unsigned f) { (void)f; *e = malloc(1); return *e ? 0 : 2; }
hipError_t hipEventDestroy(void* e) { free(e); return 0; }
hipError_t hipEventSynchronize(void* e) { (void)e; return 0; }
hipError_t hipEventRecord(void* e, void* s) { (void)e; (void)s; return 0; }
hipError_t hipHostMalloc(void** p, size_t n, unsigned f) { (void)f; *p = malloc(n); return *p ? 0 : 2; }
hipError_t hipHostFree(void* p) { free(p); return 0; }
hipError_t hipMemcpyAsync(void* d, const void* s, size_t n, int k, void* st) {
  (void)d; (void)s; (void)n; (void)k; (void)st;
  return 0;
}
typedef struct { unsigned x, y, z; } dim3_t;
static int fails_at = -1, last;
/* The launch after n more ones fails (n < 0: none does). */
void kv_stub_fail_launch(int n) { fails_at = n; last = 0; }
/* An error that some earlier call of the program's left. */
void kv_stub_leave_error(void) { last = 2; }
hipError_t hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** a, size_t l, void* s) {
  (void)f; (void)b; (void)a; (void)l; (void)s;
  const int e = (fails_at >= 0 && fails_at-- == 0) || !g.x;
  if (e) last = e;
  return e;
}
/* What kernel<<<...>>> passes through. */
static struct { dim3_t g, b; size_t l; void* s; } call;
hipError_t __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t l, void* s) {
  call.g = g, call.b = b, call.l = l, call.s = s;
  return 0;
}
hipError_t __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* l, void** s) {
  *g = call.g, *b = call.b, *l = call.l, *s = call.s;
  return 0;
}
hipError_t hipStreamIsCapturing(void* s, int* c) { *c = s == (void*)0xC0; return 0; }
hipError_t hipStreamSynchronize(void* s) { (void)s; return 0; }
hipError_t hipGetLastError(void) { int e = last; last = 0; return e; }
const char* hipGetErrorString(hipError_t e) { (void)e; return "a stub's error"; }
