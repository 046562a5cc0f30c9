/* A stand-in for the CUDA runtime calls that liblattice's host code makes, for tests of that code without a GPU.
 * Nothing runs: every call is noted in a list, launches and stream waits can be told to fail, and
 * every pointer is as good as any other. */
#include <stdint.h>
#include <string.h>

enum { LAUNCH = 1, ATTRIBUTE, RECORD, WAIT };
struct note {
    int64_t what;    /* one of the above */
    int64_t a, b, c; /* LAUNCH: function, stream, dynamic shared memory; ATTRIBUTE: function, which, value;
                        RECORD: event, stream; WAIT: stream, event */
    int64_t status;
};
#define NOTES 4096
static struct note notes[NOTES];
static int count, fail_at;
static int64_t handles = 0x1000;

/* Forgets the notes; the call that becomes note number `fail` (from 0; negative: none) returns an error. */
void fake_reset(int fail) {
    count = 0;
    fail_at = fail;
}
int fake_notes(struct note **out) {
    *out = notes;
    return count;
}
static int note(int64_t what, int64_t a, int64_t b, int64_t c) {
    const int status = count == fail_at ? 719 : 0; /* any error */
    if (count < NOTES) notes[count] = (struct note){what, a, b, c, status};
    ++count;
    return status;
}

/* cudaLaunchConfig_t as far as the stream (two dim3, a size_t, a cudaStream_t) */
struct config {
    uint32_t grid[3], block[3];
    size_t smem;
    void *stream;
};
int cudaLaunchKernelExC(const struct config *c, const void *f, void **args) {
    (void)args;
    return note(LAUNCH, (int64_t)f, (int64_t)c->stream, (int64_t)c->smem);
}
int cudaFuncSetAttribute(const void *f, int which, int value) { return note(ATTRIBUTE, (int64_t)f, which, value); }
int cudaEventRecord(void *e, void *s) { return note(RECORD, (int64_t)e, (int64_t)s, 0); }
int cudaStreamWaitEvent(void *s, void *e, unsigned flags) {
    (void)flags;
    return note(WAIT, (int64_t)s, (int64_t)e, 0);
}

int cudaGetDevice(int *d) { return *d = 0; }
int cudaDeviceGetAttribute(int *v, int which, int d) {
    (void)which, (void)d;
    *v = 148;
    return 0;
}
int cudaStreamCreateWithFlags(void **s, unsigned flags) {
    (void)flags;
    *s = (void *)(handles += 16);
    return 0;
}
int cudaEventCreateWithFlags(void **e, unsigned flags) {
    (void)flags;
    *e = (void *)(handles += 16);
    return 0;
}
int cudaStreamGetCaptureInfo_v2(void *s, int *status, unsigned long long *id, void **graph, void **deps, size_t *n) {
    (void)s, (void)graph, (void)deps, (void)n;
    *status = 0;
    if (id) *id = 0;
    return 0;
}
int cudaLaunchKernel(const void *f, uint64_t g0, uint32_t g1, uint64_t b0, uint32_t b1, void **args, size_t smem, void *s) {
    (void)g0, (void)g1, (void)b0, (void)b1, (void)args;
    return note(LAUNCH, (int64_t)f, (int64_t)s, (int64_t)smem);
}

/* what the compiler's registration of kernels calls */
void **__cudaRegisterFatBinary(void *p) {
    (void)p;
    return (void **)&handles;
}
void __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void __cudaUnregisterFatBinary(void **h) { (void)h; }
void __cudaRegisterFunction(void **h, const char *f, char *df, const char *n, int l, void *t, void *b, void *bd, void *gd, int *w) {
    (void)h, (void)f, (void)df, (void)n, (void)l, (void)t, (void)b, (void)bd, (void)gd, (void)w;
}
int __cudaPopCallConfiguration(void *g, void *b, size_t *s, void *st) {
    (void)g, (void)b, (void)s, (void)st;
    return 0;
}
