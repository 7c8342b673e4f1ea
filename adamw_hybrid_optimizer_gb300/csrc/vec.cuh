// Small device and launch helpers shared by the bandwidth-bound kernels: groups of eight values as 16-byte
// accesses, single values, a warp's sum, and the dependent launch.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <utility>

#include "ptx.cuh"

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

// Eight values as four pairs: pairs go through the two-wide fp32 instructions.
struct Oct {
  float2 p[4];
};

// Eight values as they lie in memory.
template <typename XT>
struct Raw8 {
  static constexpr int PIECES = sizeof(XT) / 2;   // 16-byte pieces
  uint4 w[PIECES];
  __device__ __forceinline__ Oct get() const {
    Oct o;
    if constexpr (sizeof(XT) == 4) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o.p[2 * i] = make_float2(__uint_as_float(w[i].x), __uint_as_float(w[i].y));
        o.p[2 * i + 1] = make_float2(__uint_as_float(w[i].z), __uint_as_float(w[i].w));
      }
    } else {
      const unsigned u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o.p[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    }
    return o;
  }
  __device__ __forceinline__ void load(const XT *p) {
#pragma unroll
    for (int i = 0; i < PIECES; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
  }
  __device__ __forceinline__ void set(const XT *f) {
    if constexpr (sizeof(XT) == 4) {
      const unsigned *u = reinterpret_cast<const unsigned *>(f);
      w[0] = make_uint4(u[0], u[1], u[2], u[3]);
      w[PIECES - 1] = make_uint4(u[4], u[5], u[6], u[7]);
    } else {
      const unsigned short *h = reinterpret_cast<const unsigned short *>(f);
      w[0] = make_uint4(h[0] | (static_cast<unsigned>(h[1]) << 16), h[2] | (static_cast<unsigned>(h[3]) << 16),
                        h[4] | (static_cast<unsigned>(h[5]) << 16), h[6] | (static_cast<unsigned>(h[7]) << 16));
    }
  }
};

template <typename T>
__device__ __forceinline__ void store_oct(T *p, const Oct &o) {
  const float f[8] = {o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y, o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y};
  store8(p, f);
}

// Asynchronous copies to shared memory, 16 bytes each.
__device__ __forceinline__ void copy_async16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

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
