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

// N values as pairs: pairs go through the two-wide fp32 instructions.
template <int N>
struct Vals {
  float2 p[N / 2];
};

template <typename T>
__device__ __forceinline__ T bits_to(unsigned u);
template <>
__device__ __forceinline__ float bits_to<float>(unsigned u) { return __uint_as_float(u); }
template <>
__device__ __forceinline__ __nv_bfloat16 bits_to<__nv_bfloat16>(unsigned u) {
  return __ushort_as_bfloat16(static_cast<unsigned short>(u));
}

// N values as they lie in memory, read and written as one access of 8 or 16 bytes (or two of 16).
template <typename T, int N>
struct Raw {
  static constexpr int BYTES = N * sizeof(T), WORDS = BYTES / 4;
  unsigned w[WORDS];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (BYTES == 8) {
      const uint2 u = *reinterpret_cast<const uint2 *>(p);
      w[0] = u.x, w[1] = u.y;
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i) {
        const uint4 u = reinterpret_cast<const uint4 *>(p)[i];
        w[4 * i] = u.x, w[4 * i + 1] = u.y, w[4 * i + 2] = u.z, w[4 * i + 3] = u.w;
      }
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (BYTES == 8) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int i = 0; i < BYTES / 16; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
  }
  // value e from its bits (the low 16 of a bf16), e ascending from an all-zero start
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < WORDS; ++i) w[i] = 0u;
  }
  __device__ __forceinline__ void put(int e, T x) {
    if constexpr (sizeof(T) == 4) {
      w[e] = __float_as_uint(x);
    } else {
      const unsigned u = __bfloat16_as_ushort(x);
      w[e / 2] = e % 2 ? (w[e / 2] & 0xffffu) | (u << 16) : (w[e / 2] & 0xffff0000u) | u;
    }
  }
  __device__ __forceinline__ Vals<N> get() const {
    Vals<N> o;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (sizeof(T) == 4) o.p[i] = make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
      else o.p[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    return o;
  }
  __device__ __forceinline__ void from(const Vals<N> &o) {   // rounds to nearest
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      if constexpr (sizeof(T) == 4) {
        w[2 * i] = __float_as_uint(o.p[i].x);
        w[2 * i + 1] = __float_as_uint(o.p[i].y);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(o.p[i].x, o.p[i].y);
        w[i] = *reinterpret_cast<const unsigned *>(&h);
      }
    }
  }
};

template <typename T, int N>
__device__ __forceinline__ void store_vals(T *p, const Vals<N> &o) {
  Raw<T, N> r;
  r.from(o);
  r.store(p);
}

// Asynchronous copies to shared memory, of 8 or 16 bytes.
template <int BYTES>
__device__ __forceinline__ void copy_async(void *dst, const void *src) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
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
