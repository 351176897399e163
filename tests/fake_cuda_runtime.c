/* A CUDA runtime with two made-up devices, for tests of the host code without
 * a GPU: launches are checked and recorded, nothing runs.  A launch with more
 * than 48 KB of dynamic shared memory fails unless its kernel has been allowed
 * that much on the current device, as a real one does. */
#include <cuda_runtime_api.h>
#include <stddef.h>

static int g_dev;
static const int g_sms[2] = {152, 100};
static struct { const void *fn; int dev, bytes; } g_allowed[512];
static int g_n_allowed;
static unsigned g_grid[64];
static int g_launches;

void fake_set_device(int dev) { g_dev = dev; }
int fake_launches(void) { return g_launches; }
unsigned fake_grid(int i) { return g_grid[i % 64]; } /* x of launch i */

static cudaError_t launch(const void *fn, unsigned grid, size_t smem) {
  size_t allowed = 48 << 10;
  for (int i = 0; i < g_n_allowed; ++i)
    if (g_allowed[i].fn == fn && g_allowed[i].dev == g_dev) allowed = (size_t)g_allowed[i].bytes;
  if (smem > allowed) return cudaErrorInvalidValue;
  g_grid[g_launches++ % 64] = grid;
  return cudaSuccess;
}

cudaError_t cudaFuncSetAttribute(const void *fn, enum cudaFuncAttribute attr, int value) {
  if (attr != cudaFuncAttributeMaxDynamicSharedMemorySize || g_n_allowed == 512)
    return cudaErrorInvalidValue;
  g_allowed[g_n_allowed].fn = fn;
  g_allowed[g_n_allowed].dev = g_dev;
  g_allowed[g_n_allowed++].bytes = value;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *fn, void **args) {
  (void)args;
  return launch(fn, cfg->gridDim.x, cfg->dynamicSmemBytes);
}
static dim3 g_pushed;
static size_t g_pushed_smem;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, void *stream) {
  (void)block, (void)stream;
  g_pushed = grid;
  g_pushed_smem = smem;
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3 *grid, dim3 *block, size_t *smem, void *stream) {
  (void)block;
  *grid = g_pushed;
  *smem = g_pushed_smem;
  *(void **)stream = NULL;
  return cudaSuccess;
}
cudaError_t __cudaGetKernel(void **kernel, const void *fn) {
  *kernel = (void *)fn;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(void *kernel, dim3 grid, dim3 block, void **args, size_t smem,
                               void *stream) {
  (void)block, (void)args, (void)stream;
  return launch(kernel, grid.x, smem);
}

static void *g_fat;
void **__cudaRegisterFatBinary(void *p) {
  (void)p;
  return &g_fat;
}
void __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void __cudaUnregisterFatBinary(void **h) { (void)h; }
void __cudaRegisterFunction(void) {}
void __cudaRegisterVar(void) {}

cudaError_t cudaGetDevice(int *dev) {
  *dev = g_dev;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int *value, enum cudaDeviceAttr attr, int dev) {
  if (attr != cudaDevAttrMultiProcessorCount) return cudaErrorInvalidValue;
  *value = g_sms[dev];
  return cudaSuccess;
}
cudaError_t cudaPointerGetAttributes(struct cudaPointerAttributes *at, const void *p) {
  at->type = cudaMemoryTypeDevice;
  at->device = g_dev;
  at->devicePointer = (void *)p;
  at->hostPointer = NULL;
  return cudaSuccess;
}
static int encode_nothing(void) { return 0; }
cudaError_t cudaGetDriverEntryPointByVersion(const char *name, void **fn, unsigned version,
                                             unsigned long long flags,
                                             enum cudaDriverEntryPointQueryResult *found) {
  (void)name, (void)version, (void)flags;
  *fn = (void *)encode_nothing;
  *found = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void **p, const void *symbol) {
  (void)symbol;
  *p = (void *)(size_t)(1 << 20);
  return cudaSuccess;
}
const char *cudaGetErrorString(cudaError_t e) { return e == cudaSuccess ? "no error" : "an error"; }
cudaError_t cudaGetLastError(void) { return cudaSuccess; }
cudaError_t cudaMemsetAsync(void *p, int v, size_t n, cudaStream_t s) {
  (void)p, (void)v, (void)n, (void)s;
  return cudaSuccess;
}
/* no side stream: calls stay on one */
cudaError_t cudaStreamIsCapturing(cudaStream_t s, enum cudaStreamCaptureStatus *st) {
  (void)s;
  *st = cudaStreamCaptureStatusActive;
  return cudaSuccess;
}
