/* Stand-ins for the CUDA runtime functions that the operators' host code calls, so that its answers
 * to failing launches can be tested without a GPU: nothing is launched, and the call numbered
 * `fake_fail_at` (launches and memsets, counted from 0) fails the way the runtime's calls do. */
#include <stddef.h>

typedef struct { unsigned x, y, z; } Dim3;
enum { kInvalidConfiguration = 9, kLaunchFailure = 719 };

int fake_fail_at = -1, fake_calls;
static int last_error;

static int call(void) {
    if (fake_calls++ != fake_fail_at) return 0;
    last_error = kInvalidConfiguration;
    return last_error;
}
void fake_reset(int fail_at) {
    fake_fail_at = fail_at;
    fake_calls = 0;
    last_error = 0;
}

int cudaLaunchKernel(const void *f, Dim3 g, Dim3 b, void **a, size_t s, void *st) { return call(); }
int cudaLaunchKernelExC(const void *cfg, const void *f, void **a) { return call(); }
int cudaMemsetAsync(void *p, int v, size_t n, void *st) { return call(); }
int cudaGetLastError(void) {
    const int e = last_error;
    last_error = 0;
    return e;
}
int cudaGetDevice(int *d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int *v, int attr, int dev) { *v = 148; return 0; }
int cudaFuncSetAttribute(const void *f, int attr, int v) { return 0; }
int cudaOccupancyMaxActiveClusters(int *n, const void *f, const void *cfg) { *n = 16; return 0; }
int cudaMemcpyFromSymbol(void *d, const void *s, size_t n, size_t o, int k) { return 0; }
int cudaMemcpyToSymbol(const void *s, const void *d, size_t n, size_t o, int k) { return 0; }
static int encode_tiled(void) { return 0; }
int cudaGetDriverEntryPoint(const char *name, void **fn, unsigned long long flags, int *q) {
    *fn = (void *)encode_tiled;
    if (q) *q = 0;
    return 0;
}
unsigned __cudaPushCallConfiguration(Dim3 g, Dim3 b, size_t s, void *st) { return 0; }
int __cudaPopCallConfiguration(Dim3 *g, Dim3 *b, size_t *s, void *st) { return 0; }
void **__cudaRegisterFatBinary(void *bin) { static void *handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void **h) {}
void __cudaUnregisterFatBinary(void **h) {}
void __cudaRegisterFunction(void **h, const char *f, char *n, const char *d, int l, void *t, void *b, void *bd, void *gd,
                            int *w) {}
void __cudaRegisterVar(void **h, char *v, char *a, const char *n, int e, size_t s, int c, int g) {}
