// fake_cuda.cpp — the CUDA runtime calls that libw4 makes, without a GPU: a
// launch is written down (thread, kernel, stream) and nothing runs.  Linked
// with libw4's own objects it shows, on any machine, what a call enqueues and
// in which order.
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <unistd.h>

#include <atomic>
#include <cstdint>
#include <functional>
#include <map>
#include <mutex>
#include <string>
#include <thread>
#include <vector>

namespace {
struct Launch {
  uint64_t thread;
  std::string kernel;
  void* stream;
};
std::mutex mu;
std::vector<Launch> launches;
std::atomic<int> pause_us{0};

std::map<const void*, std::string>& kernels() {  // host function -> mangled name
  static std::map<const void*, std::string> m;
  return m;
}

void record(const void* fn, void* stream) {
  {
    std::lock_guard<std::mutex> lock(mu);
    const auto it = kernels().find(fn);
    launches.push_back({std::hash<std::thread::id>()(std::this_thread::get_id()),
                        it == kernels().end() ? "?" : it->second, stream});
  }
  if (pause_us > 0) usleep(pause_us);  // another thread's turn
}

CUresult encode_tiled(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                      const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                      CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                      CUtensorMapFloatOOBfill) {
  return CUDA_SUCCESS;
}
thread_local struct {
  dim3 grid, block;
  size_t smem;
  void* stream;
} pushed;
}  // namespace

extern "C" {
// ------------------------------------------------------------- for the tests
void fake_reset(int pause) {
  std::lock_guard<std::mutex> lock(mu);
  launches.clear();
  pause_us = pause;
}
int fake_count() {
  std::lock_guard<std::mutex> lock(mu);
  return static_cast<int>(launches.size());
}
uint64_t fake_thread(int i) { return launches[i].thread; }
const char* fake_kernel(int i) { return launches[i].kernel.c_str(); }

// ------------------------------------------------- what compiled code registers
void** __cudaRegisterFatBinary(void*) {
  static void* handle;
  return &handle;
}
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, void*, void*,
                            void*, void*, int*) {
  kernels()[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* fn) {
  *k = reinterpret_cast<cudaKernel_t>(const_cast<void*>(fn));
  return cudaSuccess;
}
unsigned __cudaPushCallConfiguration(dim3 g, dim3 b, size_t smem, void* stream) {
  pushed = {g, b, smem, stream};
  return 0;
}
cudaError_t __cudaPopCallConfiguration(dim3* g, dim3* b, size_t* smem, void* stream) {
  *g = pushed.grid;
  *b = pushed.block;
  *smem = pushed.smem;
  *static_cast<void**>(stream) = pushed.stream;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t k, dim3, dim3, void**, size_t, cudaStream_t s) {
  record(reinterpret_cast<const void*>(k), s);
  return cudaSuccess;
}

// ------------------------------------------------------------- the runtime's
cudaError_t cudaLaunchKernel(const void* fn, dim3, dim3, void**, size_t, cudaStream_t s) {
  record(fn, s);
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* fn, void**) {
  record(fn, c->stream);
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = 0;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int) {
  *v = a == cudaDevAttrMultiProcessorCount ? 152 : 0;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { return cudaSuccess; }
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t* c) {
  int size = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) size = c->attrs[i].val.clusterDim.x;
  *n = 152 / size;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t,
                                                                   unsigned) {
  *n = 1;
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }
const char* cudaGetErrorString(cudaError_t) { return "fake"; }
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t s) {
  record(nullptr, s);
  return cudaSuccess;
}
cudaError_t cudaMemset(void*, int, size_t) { return cudaSuccess; }
cudaError_t cudaMemcpy(void*, const void*, size_t, cudaMemcpyKind) { return cudaErrorNotSupported; }
cudaError_t cudaStreamSynchronize(cudaStream_t) { return cudaSuccess; }
cudaError_t cudaStreamIsCapturing(cudaStream_t, cudaStreamCaptureStatus* st) {
  *st = cudaStreamCaptureStatusNone;
  return cudaSuccess;
}
cudaError_t cudaGetSymbolAddress(void**, const void*) { return cudaErrorInvalidSymbol; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  *p = reinterpret_cast<void*>(&encode_tiled);
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
}
