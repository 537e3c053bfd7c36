/* A stand-in for the HIP runtime that runs nothing: it keeps the current
 * device and writes one line per call that reaches a device, so that a test
 * without a GPU can see which device each call of the library is made on. */
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

typedef struct {
    uint32_t x, y, z;
} dim3_t;

static int device;
static char text[1 << 16];
static size_t used;
static dim3_t grid_, block_;
static size_t shared_;
static void* stream_;

static void note(const char* what, const void* p)
{
    used += (size_t)snprintf(text + used, sizeof(text) - used, "%s %d %p\n", what, device, p);
}

const char* fake_log(void) { return text; }
void fake_clear(void) { used = 0, text[0] = 0; }

int hipGetDevice(int* d) { *d = device; return 0; }
int hipSetDevice(int d) { device = d; return 0; }
int hipDeviceGetAttribute(int* v, int what, int d) { (void)what, (void)d; *v = 256; return 0; }
int hipGetLastError(void) { return 0; }
int hipMalloc(void** p, size_t n) { note("malloc", NULL); *p = aligned_alloc(256, (n + 255) / 256 * 256); return *p ? 0 : 2; }
int hipFree(void* p) { note("free", p); free(p); return 0; }
int hipMemsetAsync(void* p, int v, size_t n, void* s) { (void)p, (void)v, (void)n; note("memset", s); return 0; }
int hipMemcpyAsync(void* d, const void* s, size_t n, int k, void* st) { (void)d, (void)s, (void)n, (void)k; note("memcpy", st); return 0; }
int hipGetSymbolAddress(void** p, const void* s) { static char a[256]; (void)s; *p = a; return 0; }
int hipStreamSynchronize(void* s) { note("synchronize", s); return 0; }
int hipEventCreate(void** e) { note("event", NULL); *e = malloc(1); return 0; }
int hipEventDestroy(void* e) { note("destroy", NULL); free(e); return 0; }
int hipEventRecord(void* e, void* s) { (void)e; note("record", s); return 0; }
int hipEventSynchronize(void* e) { (void)e; return 0; }
int hipEventElapsedTime(float* ms, void* a, void* b) { (void)a, (void)b; *ms = 0; return 0; }
int hipLaunchKernel(const void* f, dim3_t g, dim3_t b, void** a, size_t n, void* s)
{
    (void)f, (void)g, (void)b, (void)a, (void)n;
    note("launch", s);
    return 0;
}
int __hipPushCallConfiguration(dim3_t g, dim3_t b, size_t n, void* s)
{
    grid_ = g, block_ = b, shared_ = n, stream_ = s;
    return 0;
}
int __hipPopCallConfiguration(dim3_t* g, dim3_t* b, size_t* n, void** s)
{
    *g = grid_, *b = block_, *n = shared_, *s = stream_;
    return 0;
}
void** __hipRegisterFatBinary(const void* p) { static void* h; (void)p; return &h; }
void __hipUnregisterFatBinary(void** h) { (void)h; }
void __hipRegisterFunction(void** h, const void* f, char* d, const char* n, unsigned t, void* a, void* b, void* c, void* e, int* w)
{
    (void)h, (void)f, (void)d, (void)n, (void)t, (void)a, (void)b, (void)c, (void)e, (void)w;
}
void __hipRegisterVar(void** h, void* v, char* d, const char* n, int e, size_t s, int c, int g)
{
    (void)h, (void)v, (void)d, (void)n, (void)e, (void)s, (void)c, (void)g;
}
