// A stand-in for the CUDA runtime, linked under the library's own objects so that its host code runs without a GPU:
// devices that differ in nothing, of which one is current. Function attributes belong to the device that is current when
// they are set, and a launch that needs one which that device does not have fails, as the runtime's does. No kernel runs.
#include <cuda_runtime_api.h>

#include <map>
#include <tuple>

namespace {
int g_device = 0, g_failures = 0, g_launches = 0;
std::map<std::tuple<int, const void *, int>, int> g_attr;

int attribute(const void *func, cudaFuncAttribute attr) {
  const auto it = g_attr.find({g_device, func, static_cast<int>(attr)});
  return it == g_attr.end() ? 0 : it->second;
}
}  // namespace

extern "C" {

void fake_use_device(int device) { g_device = device; }
void fake_fail_attributes(int count) { g_failures = count; }   // the next calls that set one fail
int fake_launches(void) { return g_launches; }

cudaError_t CUDARTAPI cudaGetDevice(int *device) {
  *device = g_device;
  return cudaSuccess;
}

cudaError_t CUDARTAPI cudaDeviceGetAttribute(int *value, cudaDeviceAttr attr, int) {
  *value = attr == cudaDevAttrComputeCapabilityMajor   ? 10
           : attr == cudaDevAttrComputeCapabilityMinor ? 3
           : attr == cudaDevAttrMultiProcessorCount    ? 152
                                                       : 0;
  return cudaSuccess;
}

cudaError_t CUDARTAPI cudaFuncSetAttribute(const void *func, cudaFuncAttribute attr, int value) {
  if (g_failures > 0) {
    --g_failures;
    return cudaErrorMemoryAllocation;
  }
  g_attr[{g_device, func, static_cast<int>(attr)}] = value;
  return cudaSuccess;
}

cudaError_t CUDARTAPI cudaLaunchKernelExC(const cudaLaunchConfig_t *cfg, const void *func, void **) {
  if (cfg->dynamicSmemBytes > 48 * 1024 &&
      cfg->dynamicSmemBytes > static_cast<size_t>(attribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize)))
    return cudaErrorInvalidValue;
  for (unsigned i = 0; i < cfg->numAttrs; ++i)
    if (cfg->attrs[i].id == cudaLaunchAttributeClusterDimension && cfg->attrs[i].val.clusterDim.x > 8 &&
        attribute(func, cudaFuncAttributeNonPortableClusterSizeAllowed) == 0)
      return cudaErrorInvalidClusterSize;
  ++g_launches;
  return cudaSuccess;
}

// What the other objects name, and nothing here calls.
#define ABSENT(name) \
  int name(void) { return static_cast<int>(cudaErrorNotSupported); }
ABSENT(__cudaGetKernel)
ABSENT(__cudaLaunchKernel)
ABSENT(__cudaPopCallConfiguration)
void *__cudaRegisterFatBinary(void *) { return &g_attr; }
void __cudaRegisterFatBinaryEnd(void **) {}
void __cudaUnregisterFatBinary(void **) {}
void __cudaRegisterFunction(void) {}
void __cudaRegisterVar(void) {}

}  // extern "C"

// Declared by the header with arguments that do not matter here: defined under their linker names.
#define ABSENT_API(name)           \
  extern "C" int absent_##name(void) __asm__(#name); \
  extern "C" int absent_##name(void) { return static_cast<int>(cudaErrorNotSupported); }
ABSENT_API(cudaEventCreate)
ABSENT_API(cudaEventDestroy)
ABSENT_API(cudaEventElapsedTime)
ABSENT_API(cudaEventRecord)
ABSENT_API(cudaEventSynchronize)
ABSENT_API(cudaGetDriverEntryPointByVersion)
ABSENT_API(cudaGetSymbolAddress)
ABSENT_API(cudaMemcpy)
ABSENT_API(cudaMemset)
ABSENT_API(cudaMemsetAsync)
ABSENT_API(cudaOccupancyMaxActiveClusters)
ABSENT_API(cudaStreamSynchronize)
