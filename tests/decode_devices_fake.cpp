// A stand-in for the CUDA runtime with two devices, linked with the launcher of the layer for a few tokens: every launch
// with more than 48 KB of shared memory must have been allowed on the device that is current (kernel attributes hold for
// one device).  Prints the launches that were not; exits with their number.
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdio>
#include <map>
#include <utility>

#include "decode.h"

namespace {
int g_device = 0, g_refused = 0, g_launches = 0;
std::map<std::pair<int, const void*>, int> g_allowed;
CUresult encode(...) { return CUDA_SUCCESS; }
}  // namespace

extern "C" {
void** __cudaRegisterFatBinary(void*) { static void* handle; return &handle; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char*, char*, const char*, int, uint3*, uint3*, dim3*, dim3*, int*) {}
int __cudaGetKernel(void*, const void*) { return 0; }
int __cudaLaunchKernel(...) { return 0; }
int __cudaPopCallConfiguration(...) { return 0; }
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void*, int, size_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaGetDriverEntryPointByVersion(const char*, void** fn, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* r) {
  *fn = reinterpret_cast<void*>(&encode);
  *r = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) g_allowed[{g_device, f}] = v;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void**) {
  ++g_launches;
  if (static_cast<int>(c->dynamicSmemBytes) <= g_allowed[{g_device, f}]) return cudaSuccess;
  std::printf("device %d: %zu bytes of shared memory not allowed\n", g_device, c->dynamicSmemBytes);
  ++g_refused;
  return cudaErrorInvalidValue;
}
}

namespace moe {
void trace_begin(int, cudaStream_t) {}
void trace_end(int, cudaStream_t) {}
int num_sms() { return 152; }
}  // namespace moe

int main() {
  alignas(256) static unsigned char p[256];
  uint16_t* a = reinterpret_cast<uint16_t*>(p);
  for (g_device = 0; g_device < 2; ++g_device)
    for (int y_type : {0, 1})
      for (int group : {0, 32, 64, 128}) {
        const moe::DecodeWeight w{p, group ? a : nullptr};
        moe::launch_linear(moe::LinearArgs{1, 64, 128, group, a, w, p, y_type, p, 0}, nullptr);
        const moe_cfg c{1, 128, 128, 4, 2, 0, 0};
        const float* z = reinterpret_cast<const float*>(p);
        moe::launch_decode(moe::DecodeArgs{c, group, z, a, w, w, w, p, y_type, reinterpret_cast<int32_t*>(p),
                                           reinterpret_cast<float*>(p), p, 0}, nullptr);
      }
  std::printf("%d launches, %d refused\n", g_launches, g_refused);
  return g_launches == 32 ? g_refused : 99;
}
