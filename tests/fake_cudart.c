/* Stand-ins for the CUDA runtime calls of creating a problem, preloaded into a
 * process without a GPU: device memory is host memory, and work queued on a
 * stream stays pending until somebody waits for that stream. */
#include <stdlib.h>
#include <string.h>

#define STREAMS 8

static int pending[STREAMS + 1];      /* [0]: the legacy default stream */
static int made;
static size_t allocated;

static int slot(void *stream) { return stream ? (int)(size_t)stream : 0; }

int fake_pending(void) {
    int n = 0;
    for (int i = 0; i <= STREAMS; ++i) n += pending[i];
    return n;
}
size_t fake_allocated(void) { return allocated; }

int cudaGetDevice(int *d) { *d = 0; return 0; }
int cudaDeviceGetAttribute(int *v, int attr, int dev) { (void)attr; (void)dev; *v = 152; return 0; }
int cudaMalloc(void **p, size_t n) {
    allocated += n;
    /* Address space only; nothing of a workspace is touched. */
    *p = n <= (size_t)1 << 20 ? malloc(n) : malloc(64);
    if (*p) memset(*p, 0xa5, n <= (size_t)1 << 20 ? n : 64);
    return *p ? 0 : 2;
}
int cudaFree(void *p) { free(p); return 0; }
int cudaMemset(void *p, int v, size_t n) { (void)p; (void)v; (void)n; ++pending[0]; return 0; }
int cudaMemsetAsync(void *p, int v, size_t n, void *st) {
    (void)p; (void)v; (void)n;
    ++pending[slot(st)];
    return 0;
}
int cudaStreamCreateWithFlags(void **st, unsigned flags) {
    (void)flags;
    if (made == STREAMS) return 2;
    *st = (void *)(size_t)++made;
    return 0;
}
int cudaStreamDestroy(void *st) { (void)st; return 0; }
int cudaStreamSynchronize(void *st) { pending[slot(st)] = 0; return 0; }
int cudaDeviceSynchronize(void) { memset(pending, 0, sizeof pending); return 0; }
