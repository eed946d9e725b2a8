// A stand-in for the CUDA runtime, linked to the library's own objects in place of it, so that the host side of
// the entry points runs without a GPU and with as many devices as a test likes.  It launches nothing: a launch is
// counted, and refused when its dynamic shared memory was not asked for on the current device.  A kernel's own arrays,
// which the stand-in does not know, count among the 48 KB that go without asking: 2 KB stand for them.
#include <cuda_runtime_api.h>

#include <map>
#include <utility>

namespace {
int device = 0;
long launches = 0;
std::map<std::pair<int, const void*>, int> granted;   // dynamic shared memory by (device, kernel)

cudaError_t launch(const void* kernel, size_t smem) {
  ++launches;
  const auto at = granted.find({device, kernel});
  return smem > size_t(at == granted.end() ? 46 * 1024 : at->second) ? cudaErrorInvalidValue : cudaSuccess;
}
int encode_tensor_map() { return 0; }
}  // namespace

extern "C" {

void fake_device(int d) { device = d; }
long fake_launches() { return launches; }

cudaError_t cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) { return *v = 152, cudaSuccess; }
cudaError_t cudaGetLastError() { return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) granted[{device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) { return *n = 76, cudaSuccess; }
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) { return launch(f, c->dynamicSmemBytes); }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** f, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *f = reinterpret_cast<void*>(encode_tensor_map);
  return *q = cudaDriverEntryPointSuccess, cudaSuccess;
}

// what the compiler's host stubs call
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* f) {
  return *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(f)), cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void**, size_t smem, cudaStream_t) { return launch(k, smem); }
struct Call {
  dim3 grid, block;
  size_t smem;
  cudaStream_t stream;
};
static Call call;
unsigned __cudaPushCallConfiguration(dim3 grid, dim3 block, size_t smem, cudaStream_t stream) {
  return call = {grid, block, smem, stream}, 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* grid, dim3* block, size_t* smem, void* stream) {
  *grid = call.grid, *block = call.block, *smem = call.smem, *static_cast<cudaStream_t*>(stream) = call.stream;
  return cudaSuccess;
}
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}

}  // extern "C"
