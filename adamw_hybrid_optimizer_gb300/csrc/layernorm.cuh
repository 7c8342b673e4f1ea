// What the forward and the backward kernels of layer norm share: how threads hold a row's columns, the rows on their
// way, the weights, and the sums between the warps of a row.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int LONG_THREADS = 1024;     // block of the kernels for rows beyond MAX_ROW
constexpr int MAX_ROW = 16384;

// weight / bias value c; a null weight is 1 and a null bias 0
__device__ __forceinline__ float param_at(const void *p, int dt, int c, float absent) {
  if (p == nullptr) return absent;
  return dt == MUON_F32 ? static_cast<const float *>(p)[c]
                        : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
}

// The columns of thread t of the T that hold a row: chunk k's eight are contiguous on the vector path (which needs a
// width of whole eights), and one per sweep of the group otherwise, so that a warp's accesses stay contiguous whatever
// the alignment. Both number a thread's columns 8 k + e in increasing order, so one count says which of them the row
// has.
struct Cols {
  int t, T, count;
};
template <bool VEC>
__device__ __forceinline__ Cols cols_of(int t, int T, int D) {
  if (VEC) return {t, T, (D / 8 - t + T - 1) / T * 8};
  return {t, T, (D - t + T - 1) / T};
}
template <bool VEC>
__device__ __forceinline__ int col(const Cols &c, int k, int e) {
  return VEC ? (k * c.T + c.t) * 8 + e : (k * 8 + e) * c.T + c.t;
}
template <bool VEC>
__device__ __forceinline__ bool has(const Cols &c, int k, int e) {
  return (VEC ? 8 * k : 8 * k + e) < c.count;
}

template <typename XT>
__device__ __forceinline__ XT zero_of() { return XT(0.f); }
template <>
__device__ __forceinline__ __nv_bfloat16 zero_of<__nv_bfloat16>() { return __ushort_as_bfloat16(0); }

// Columns that the row does not have read as 0.
template <typename XT, bool VEC>
__device__ __forceinline__ void load_chunk(const XT *p, const Cols &c, int k, Raw8<XT> &r) {
  XT f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = zero_of<XT>();
  if constexpr (VEC) {
    if (has<true>(c, k, 0)) r.load(p + col<true>(c, k, 0));
    else r.set(f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (has<false>(c, k, e)) f[e] = p[col<false>(c, k, e)];
    r.set(f);
  }
}

template <typename XT, bool VEC>
__device__ __forceinline__ void store_chunk(XT *p, const Cols &c, int k, const Oct &o) {
  const float f[8] = {o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y, o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y};
  if constexpr (VEC) {
    if (has<true>(c, k, 0)) store8(p + col<true>(c, k, 0), f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (has<false>(c, k, e)) store1(p, col<false>(c, k, e), f[e]);
  }
}

// The thread's weights (or biases): `absent` where there are none.
template <bool VEC>
__device__ __forceinline__ Oct param_chunk(const void *p, int dt, const Cols &c, int k, float absent) {
  Oct o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = make_float2(absent, absent);
  if (p == nullptr) return o;
  if constexpr (VEC) {
    if (!has<true>(c, k, 0)) return o;
    if (dt == MUON_F32) {
      Raw8<float> r;
      r.load(static_cast<const float *>(p) + col<true>(c, k, 0));
      return r.get();
    }
    Raw8<__nv_bfloat16> r;
    r.load(static_cast<const __nv_bfloat16 *>(p) + col<true>(c, k, 0));
    return r.get();
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (has<false>(c, k, e)) (e % 2 ? o.p[e / 2].y : o.p[e / 2].x) = param_at(p, dt, col<false>(c, k, e), absent);
    return o;
  }
}

// Zero where the row has no column (without the vector path; on it a chunk is there or not).
template <bool VEC>
__device__ __forceinline__ float2 only(const Cols &c, int k, int i, float2 v) {
  if (!VEC) {
    if (!has<false>(c, k, 2 * i)) v.x = 0.f;
    if (!has<false>(c, k, 2 * i + 1)) v.y = 0.f;
  }
  return v;
}

// The rows to come. On the vector path they are copied into a ring of STAGES places in shared memory, of which every
// thread writes and reads its own columns only: its own wait orders them, and no registers hold them meanwhile.
// Without it the next row's loads wait in registers. Layout: [stage][chunk][piece][thread].
template <typename XT, int C, int THREADS>
struct Ring {
  static constexpr int PIECES = Raw8<XT>::PIECES;
  uint4 *base;   // of this thread
  __device__ __forceinline__ void fetch(const XT *row, const Cols &c, int stage) const {
    uint4 *to = base + stage * (C * PIECES * THREADS);
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (has<true>(c, k, 0)) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
          copy_async16(to + (k * PIECES + p) * THREADS, reinterpret_cast<const uint4 *>(row + col<true>(c, k, 0)) + p);
      }
  }
  __device__ __forceinline__ Oct get(int k, int stage) const {
    const uint4 *from = base + stage * (C * PIECES * THREADS);
    Raw8<XT> r;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) r.w[p] = from[(k * PIECES + p) * THREADS];
    return r.get();
  }
};

// A vector of weights (or biases), as each thread wants its own columns of it row after row: in registers where there
// is one chunk, as fp32 in shared memory up to 8192 columns of several chunks, and read where it is beyond that (and
// without the vector path, for several chunks).
template <int C, int THREADS, bool VEC, bool SHARED>
struct Params {
  const void *p;
  int dt;
  float absent;
  float4 *base;   // SHARED: of this thread, [2 chunk + half][thread]
  Oct one;
  __device__ __forceinline__ void init(const Cols &c) {
    if constexpr (C == 1) one = param_chunk<VEC>(p, dt, c, 0, absent);
    if constexpr (SHARED) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const Oct o = param_chunk<VEC>(p, dt, c, k, absent);
        base[(2 * k) * THREADS] = make_float4(o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y);
        base[(2 * k + 1) * THREADS] = make_float4(o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y);
      }
    }
  }
  __device__ __forceinline__ Oct get(const Cols &c, int k) const {
    if constexpr (C == 1) return one;
    if constexpr (SHARED) {
      const float4 u = base[(2 * k) * THREADS], v = base[(2 * k + 1) * THREADS];
      return {{make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(v.x, v.y), make_float2(v.z, v.w)}};
    }
    return param_chunk<VEC>(p, dt, c, k, absent);
  }
};

// Sums over all 32 lanes, or over groups of LANES that hold copies of the same values.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
template <int LANES>
__device__ __forceinline__ float2 lanes_sum2(float2 v) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    v = __fadd2_rn(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  return v;
}

// The exchange between the W warps that hold a row, one of R in the block: every warp puts a pair, and after the
// block's barrier lane i of every warp reads the pair of warp i mod LANES, the next power of two (0 beyond W), so that
// sums over LANES lanes reach all. Calls alternate between two buffers: a thread can write one again only after the
// barrier of the call in between, which every reader of that buffer has reached.
template <int W, int R>
struct Exchange {
  static constexpr int LANES = W <= 1 ? 1 : W <= 2 ? 2 : W <= 4 ? 4 : W <= 8 ? 8 : W <= 16 ? 16 : 32;
  float2 (*buf)[R][W];   // two
  int slot, w, turn;
  __device__ __forceinline__ float2 put_get(float a, float b) {
    float2 *r = buf[turn][slot];
    const int lane = threadIdx.x % 32, from = lane & (LANES - 1);
    if (lane == 0) r[w] = make_float2(a, b);
    __syncthreads();
    turn ^= 1;
    return from < W ? r[from] : make_float2(0.f, 0.f);
  }
};

// Sums over a block of 32 warps, for the kernels that give a block to a row.
__device__ __forceinline__ float block_sum(float v, float (*red)[32], int &turn) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) red[turn][threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < 32; ++w) v += red[turn][w];
  turn ^= 1;
  return v;
}

// ------------------------------------------------------------------------------------------ host

constexpr int SM_SHARED = 227 * 1024;
constexpr int STATIC_SHARED = 12 * 1024;   // more than any kernel's static share

// Once for each kernel: it may take more than 48 KB, and the multiprocessor is to hold as many blocks of it as fit.
template <typename K>
cudaError_t allow_shared(K kernel) {
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_SHARED - STATIC_SHARED);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(kernel, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool natural(const void *p, int dt) {
  return (reinterpret_cast<uintptr_t>(p) & (dt == MUON_F32 ? 3 : 1)) == 0;
}
inline bool dtype_ok(int dt) { return dt == MUON_F32 || dt == MUON_BF16; }
inline muon_status status_of(cudaError_t e) { return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA; }

inline muon_status check_dims(int64_t N, int64_t D) {
  if (N < 0 || D < 1) return MUON_ERR_INVALID_ARG;
  return N > (1ll << 30) || D > (1ll << 20) ? MUON_ERR_SHAPE : MUON_OK;
}

// Warps for a row of D columns held in C chunks per thread: what it takes, rounded up to a width that is compiled.
inline int warps_of(long long D, int C) {
  const int need = static_cast<int>((D + 256 * C - 1) / (256 * C));
  for (int w : {1, 2, 3, 4, 6, 8, 12, 16}) if (need <= w) return w;
  return 32;
}

}  // namespace
}  // namespace muon
