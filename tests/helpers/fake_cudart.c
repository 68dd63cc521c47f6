/* A stand-in for the CUDA runtime, for the library's host code alone: devices
 * are numbers, opt-ins to more than 48 KB of dynamic shared memory are kept per
 * (kernel, device) as the runtime keeps them, and a launch without the one it
 * needs is refused.  Nothing is ever launched. */
#include <stddef.h>
#include <stdint.h>

typedef struct { unsigned x, y, z; } Dim3;
typedef struct { Dim3 grid, block; size_t smem; void *stream; void *attrs; unsigned num_attrs; } Config;

enum { kOk = 0, kInvalidValue = 1, kMaxDynamicShared = 8, kKernels = 4096 };

static int g_device, g_launches, g_queries;
static struct { const void *func; int device, bytes; } g_optin[kKernels];
static int g_optins;

void fake_set_device(int d) { g_device = d; }
int fake_launches(void) { return g_launches; }
int fake_queries(void) { return g_queries; }

static int allowed(const void *func)
{
    int best = 48 * 1024;
    for (int i = 0; i < g_optins; ++i)
        if (g_optin[i].func == func && g_optin[i].device == g_device) best = g_optin[i].bytes;
    return best;
}

int cudaGetDevice(int *d) { *d = g_device; return kOk; }
int cudaDeviceGetAttribute(int *v, int attr, int d) { (void)attr; (void)d; *v = 152; return kOk; }
int cudaGetLastError(void) { return kOk; }
int cudaDeviceSynchronize(void) { return kOk; }
int cudaGetSymbolAddress(void **p, const void *s) { (void)s; *p = (void *)(uintptr_t)0x1000; return kOk; }
int cudaMemcpyToSymbol(const void *s, const void *p, size_t n, size_t o, int k) { (void)s; (void)p; (void)n; (void)o; (void)k; return kOk; }
int cudaMemcpyFromSymbol(void *p, const void *s, size_t n, size_t o, int k) { (void)s; (void)p; (void)n; (void)o; (void)k; return kOk; }

int cudaFuncSetAttribute(const void *func, int attr, int value)
{
    if (attr != kMaxDynamicShared || value > 227 * 1024 || g_optins == kKernels) return kInvalidValue;
    g_optin[g_optins].func = func;
    g_optin[g_optins].device = g_device;
    g_optin[g_optins++].bytes = value;
    return kOk;
}

int cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int *n, const void *func, int threads, size_t smem, unsigned flags)
{
    (void)threads; (void)flags;
    ++g_queries;
    *n = smem <= (size_t)allowed(func) ? 2 : 0;
    return kOk;
}

int cudaLaunchKernelExC(const Config *c, const void *func, void **args)
{
    (void)args;
    if (c->smem > (size_t)allowed(func)) return kInvalidValue;
    ++g_launches;
    return kOk;
}

static int encode_map() { return 0; }
int cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned version, unsigned long long flags, int *status)
{
    (void)name; (void)version; (void)flags;
    *fn = (void *)encode_map;
    *status = 0;
    return kOk;
}

/* what a translation unit calls when it is loaded, and its launch stubs */
void **__cudaRegisterFatBinary(void *p) { static void *h; (void)p; return &h; }
void __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void __cudaUnregisterFatBinary(void **h) { (void)h; }
void __cudaRegisterFunction() {}
void __cudaRegisterVar() {}
int __cudaPushCallConfiguration() { return kOk; }
int __cudaPopCallConfiguration() { return kOk; }
int __cudaGetKernel() { return kOk; }
int __cudaLaunchKernel() { return kOk; }
