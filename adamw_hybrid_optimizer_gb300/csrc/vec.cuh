// Small device and launch helpers shared by the bandwidth-bound kernels: groups of eight values as 16-byte
// accesses, single values, a warp's sum, and the dependent launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <utility>

namespace muon {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T>
__device__ __forceinline__ void load8(const T *p, float *f);
template <>
__device__ __forceinline__ void load8<float>(const float *p, float *f) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0];
  const float4 b = reinterpret_cast<const float4 *>(p)[1];
  f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float *f) {
  const uint4 w = reinterpret_cast<const uint4 *>(p)[0];
  const __nv_bfloat162 *h = reinterpret_cast<const __nv_bfloat162 *>(&w);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 x = __bfloat1622float2(h[e]);
    f[2 * e] = x.x;
    f[2 * e + 1] = x.y;
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float *f);
template <>
__device__ __forceinline__ void store8<float>(float *p, const float *f) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
template <>
__device__ __forceinline__ void store8<__nv_bfloat16>(__nv_bfloat16 *p, const float *f) {
  uint4 w;
  __nv_bfloat162 *h = reinterpret_cast<__nv_bfloat162 *>(&w);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2bfloat162_rn(f[2 * e], f[2 * e + 1]);
  reinterpret_cast<uint4 *>(p)[0] = w;
}

template <typename T>
__device__ __forceinline__ float load1(const T *p, long long i);
template <>
__device__ __forceinline__ float load1<float>(const float *p, long long i) { return p[i]; }
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16 *p, long long i) {
  return __bfloat162float(p[i]);
}
__device__ __forceinline__ void store1(float *p, long long i, float v) { p[i] = v; }
__device__ __forceinline__ void store1(__nv_bfloat16 *p, long long i, float v) { p[i] = __float2bfloat16_rn(v); }

// Launch with programmatic stream serialization (the kernel waits for its predecessor itself).
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                       Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

}  // namespace muon
