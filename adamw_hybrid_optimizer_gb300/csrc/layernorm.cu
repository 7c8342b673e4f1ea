// Layer norm over the rows of an N x D matrix, forward and backward.
//
//   mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps), xh = (x - mu) r, y = xh w + b
//   g = dy w,  dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Both passes are bound by bandwidth: a row is read once into registers (as fp32), its sums are exchanged inside
// the group of warps that holds it, and the result is stored. The variance is taken around the mean in a second
// sweep over the registers, so no E[x^2] - mu^2 cancels. The backward pass keeps each thread's columns of dw and db
// in registers over all rows of its block, stores one partial row per block, and a second kernel adds the partial
// rows in block order: no atomics, so the same inputs give the same bits.
//
//   layernorm_forward_kernel, layernorm_backward_kernel  rows of up to 16384 columns, W warps per row
//   layernorm_forward_long_kernel, layernorm_dx_long_kernel, layernorm_columns_kernel  longer rows: a block per row,
//                             re-reading it (from L2) for each sweep; dw and db by columns
//   layernorm_reduce_kernel   the partial rows' sum
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int SHORT_THREADS = 128;     // block of the one-warp-per-row kernels: four rows at a time
constexpr int LONG_THREADS = 1024;     // block of the kernels for rows beyond MAX_ROW
constexpr int MAX_ROW = 16384;
constexpr int REDUCE_COLS = 32;
constexpr int REDUCE_WARPS = 16;

// weight / bias value c; a null weight is 1 and a null bias 0
__device__ __forceinline__ float param_at(const void *p, int dt, int c, float absent) {
  if (p == nullptr) return absent;
  return dt == MUON_F32 ? static_cast<const float *>(p)[c]
                        : __bfloat162float(static_cast<const __nv_bfloat16 *>(p)[c]);
}

__device__ __forceinline__ void param8(const void *p, int dt, int c, float absent, float *f) {
  if (p == nullptr) {
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = absent;
  } else if (dt == MUON_F32) {
    load8(static_cast<const float *>(p) + c, f);
  } else {
    load8(static_cast<const __nv_bfloat16 *>(p) + c, f);
  }
}

// The columns of a thread: chunk k's eight are contiguous on the vector path, and one per group-wide sweep otherwise
// (so that a warp's accesses stay contiguous whatever the alignment).
template <int T, bool VEC>
__device__ __forceinline__ int col_of(int k, int e, int t) {
  return VEC ? (k * T + t) * 8 + e : (k * 8 + e) * T + t;
}

template <typename XT, int T, bool VEC>
__device__ __forceinline__ void load_chunk(const XT *p, int k, int t, int D, float *f) {
  if constexpr (VEC) {
    if (col_of<T, true>(k, 7, t) < D) {
      load8(p + col_of<T, true>(k, 0, t), f);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = col_of<T, VEC>(k, e, t);
    f[e] = c < D ? load1(p, c) : 0.f;
  }
}

template <typename XT, int T, bool VEC>
__device__ __forceinline__ void store_chunk(XT *p, int k, int t, int D, const float *f) {
  if constexpr (VEC) {
    if (col_of<T, true>(k, 7, t) < D) {
      store8(p + col_of<T, true>(k, 0, t), f);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = col_of<T, VEC>(k, e, t);
    if (c < D) store1(p, c, f[e]);
  }
}

template <int T, bool VEC>
__device__ __forceinline__ void param_chunk(const void *p, int dt, int k, int t, int D, float absent, float *f) {
  if constexpr (VEC) {
    if (col_of<T, true>(k, 7, t) < D) {
      param8(p, dt, col_of<T, true>(k, 0, t), absent, f);
      return;
    }
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const int c = col_of<T, VEC>(k, e, t);
    f[e] = c < D ? param_at(p, dt, c, absent) : 0.f;
  }
}

// Sums over the W warps of a row. Successive calls alternate between the two halves of `red`: a thread can write a
// half again only after the barrier of the call in between, which every reader of that half has passed.
template <int W>
__device__ __forceinline__ float group_sum(float v, float (*red)[W], int &turn) {
  v = warp_sum(v);
  if constexpr (W > 1) {
    if (threadIdx.x % 32 == 0) red[turn][threadIdx.x / 32] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) v += red[turn][w];
    turn ^= 1;
  }
  return v;
}

struct ForwardArgs {
  const void *x, *w, *b;
  void *y;
  long long ldx, ldy, N;
  float *mean, *rstd;
  float eps;
  int wdt, D;
};

template <typename XT, typename YT, int W, int C, bool VEC>
__global__ void __launch_bounds__(W == 1 ? SHORT_THREADS : W * 32) layernorm_forward_kernel(const ForwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int T = W * 32, ROWS = W == 1 ? SHORT_THREADS / 32 : 1;
  __shared__ float red[2][W];
  int turn = 0;
  const int t = threadIdx.x % T, D = a.D;
  const float inv = 1.f / static_cast<float>(D);
  const long long step = static_cast<long long>(gridDim.x) * ROWS;
  for (long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / T; row < a.N; row += step) {
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    float v[C][8];
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) load_chunk<XT, T, VEC>(x, k, t, D, v[k]);
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[k][e];
    const float mean = group_sum<W>(s, red, turn) * inv;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[k][e] -= mean;
        if (col_of<T, VEC>(k, e, t) < D) q = fmaf(v[k][e], v[k][e], q);
      }
    const float rstd = 1.f / sqrtf(group_sum<W>(q, red, turn) * inv + a.eps);
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    YT *y = static_cast<YT *>(a.y) + row * a.ldy;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float w[8], b[8];
      param_chunk<T, VEC>(a.w, a.wdt, k, t, D, 1.f, w);
      param_chunk<T, VEC>(a.b, a.wdt, k, t, D, 0.f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = fmaf(v[k][e] * rstd, w[e], b[e]);
      store_chunk<YT, T, VEC>(y, k, t, D, v[k]);
    }
  }
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_THREADS) layernorm_forward_long_kernel(const ForwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int W = LONG_THREADS / 32;
  __shared__ float red[2][W];
  int turn = 0;
  const float inv = 1.f / static_cast<float>(a.D);
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    YT *y = static_cast<YT *>(a.y) + row * a.ldy;
    float s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) s += load1(x, c);
    const float mean = group_sum<W>(s, red, turn) * inv;
    float q = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) {
      const float d = load1(x, c) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = 1.f / sqrtf(group_sum<W>(q, red, turn) * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS)
      store1(y, c, fmaf((load1(x, c) - mean) * rstd, param_at(a.w, a.wdt, c, 1.f), param_at(a.b, a.wdt, c, 0.f)));
  }
}

struct BackwardArgs {
  const void *dy, *x, *w;
  void *dx;
  long long lddy, ldx, lddx, N;
  const float *mean, *rstd;
  float *part;      // [2][parts][ldp]: dw's partial rows, then db's; null: neither is wanted
  long long parts, ldp;
  int wdt, D;
};

template <typename XT, typename YT, int W, int C, bool VEC>
__global__ void __launch_bounds__(W == 1 ? SHORT_THREADS : W * 32) layernorm_backward_kernel(const BackwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int T = W * 32, ROWS = W == 1 ? SHORT_THREADS / 32 : 1;
  __shared__ float red[2][W];
  __shared__ float join[W == 1 ? ROWS : 1][W == 1 ? C * 256 : 1];
  int turn = 0;
  const int t = threadIdx.x % T, D = a.D;
  const float inv = 1.f / static_cast<float>(D);
  float aw[C][8], ab[C][8];
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[k][e] = ab[k][e] = 0.f;
  const long long step = static_cast<long long>(gridDim.x) * ROWS;
  for (long long row = static_cast<long long>(blockIdx.x) * ROWS + threadIdx.x / T; row < a.N; row += step) {
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    const YT *dy = static_cast<const YT *>(a.dy) + row * a.lddy;
    float xh[C][8], g[C][8];
#pragma unroll
    for (int k = 0; k < C; ++k) {
      load_chunk<XT, T, VEC>(x, k, t, D, xh[k]);
      load_chunk<YT, T, VEC>(dy, k, t, D, g[k]);
    }
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float w[8];
      param_chunk<T, VEC>(a.w, a.wdt, k, t, D, 1.f, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // columns past the row's end hold dy = 0 (and w = 0), so they add nothing to any sum
        xh[k][e] = (xh[k][e] - mean) * rstd;
        if (col_of<T, VEC>(k, e, t) < D) {
          aw[k][e] = fmaf(g[k][e], xh[k][e], aw[k][e]);
          ab[k][e] += g[k][e];
          g[k][e] *= w[e];
          s1 += g[k][e];
          s2 = fmaf(g[k][e], xh[k][e], s2);
        }
      }
    }
    s1 = group_sum<W>(s1, red, turn) * inv;
    s2 = group_sum<W>(s2, red, turn) * inv;
    if (a.dx != nullptr) {
      XT *dx = static_cast<XT *>(a.dx) + row * a.lddx;
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[k][e] = rstd * (g[k][e] - s1 - xh[k][e] * s2);
        store_chunk<XT, T, VEC>(dx, k, t, D, g[k]);
      }
    }
  }
  if (a.part == nullptr) return;
  float *pw = a.part + static_cast<long long>(blockIdx.x) * a.ldp;
  float *pb = a.part + (a.parts + blockIdx.x) * a.ldp;
  if constexpr (W == 1) {
    // the block's four warps hold the same columns: add them in warp order
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < C; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) join[threadIdx.x / 32][col_of<T, VEC>(k, e, t)] = z == 0 ? aw[k][e] : ab[k][e];
      __syncthreads();
      for (int c = threadIdx.x; c < D; c += SHORT_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) s += join[r][c];
        (z == 0 ? pw : pb)[c] = s;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      store_chunk<float, T, VEC>(pw, k, t, D, aw[k]);
      store_chunk<float, T, VEC>(pb, k, t, D, ab[k]);
    }
  }
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_THREADS) layernorm_dx_long_kernel(const BackwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int W = LONG_THREADS / 32;
  __shared__ float red[2][W];
  int turn = 0;
  const float inv = 1.f / static_cast<float>(a.D);
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    const YT *dy = static_cast<const YT *>(a.dy) + row * a.lddy;
    XT *dx = static_cast<XT *>(a.dx) + row * a.lddx;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) {
      const float g = load1(dy, c) * param_at(a.w, a.wdt, c, 1.f);
      s1 += g;
      s2 = fmaf(g, (load1(x, c) - mean) * rstd, s2);
    }
    s1 = group_sum<W>(s1, red, turn) * inv;
    s2 = group_sum<W>(s2, red, turn) * inv;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) {
      const float g = load1(dy, c) * param_at(a.w, a.wdt, c, 1.f);
      store1(dx, c, rstd * (g - s1 - (load1(x, c) - mean) * rstd * s2));
    }
  }
}

// dw and db of long rows: block (b, z) sums 256 columns over row slice z, one column per thread.
template <typename XT, typename YT>
__global__ void __launch_bounds__(256) layernorm_columns_kernel(const BackwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= a.D) return;
  const long long r0 = a.N * blockIdx.y / a.parts, r1 = a.N * (blockIdx.y + 1) / a.parts;
  float sw = 0.f, sb = 0.f;
#pragma unroll 4
  for (long long r = r0; r < r1; ++r) {
    const float g = load1(static_cast<const YT *>(a.dy) + r * a.lddy, c);
    sw = fmaf(g, (load1(static_cast<const XT *>(a.x) + r * a.ldx, c) - a.mean[r]) * a.rstd[r], sw);
    sb += g;
  }
  a.part[static_cast<long long>(blockIdx.y) * a.ldp + c] = sw;
  a.part[(a.parts + blockIdx.y) * a.ldp + c] = sb;
}

// dw (blockIdx.y = 0) and db (1): 32 columns per block, warp w adds partial rows w, w + 16, ...
__global__ void __launch_bounds__(REDUCE_WARPS * 32) layernorm_reduce_kernel(const float *part, long long parts,
                                                                             long long ldp, int D, void *dw, void *db,
                                                                             int gdt, int accumulate) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  void *out = blockIdx.y == 0 ? dw : db;
  if (out == nullptr) return;
  __shared__ float red[REDUCE_WARPS][REDUCE_COLS];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const int c = blockIdx.x * REDUCE_COLS + lane;
  const float *p = part + blockIdx.y * parts * ldp;
  float s = 0.f;
  if (c < D) {
#pragma unroll 8
    for (long long r = w; r < parts; r += REDUCE_WARPS) s += p[r * ldp + c];
  }
  red[w][lane] = s;
  __syncthreads();
  if (w != 0 || c >= D) return;
  s = 0.f;
#pragma unroll
  for (int k = 0; k < REDUCE_WARPS; ++k) s += red[k][lane];
  if (gdt == MUON_F32) {
    float *o = static_cast<float *>(out);
    store1(o, c, accumulate ? s + load1(o, c) : s);
  } else {
    __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(out);
    store1(o, c, accumulate ? s + load1(o, c) : s);
  }
}

// ------------------------------------------------------------------------------------------ host

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool natural(const void *p, int dt) { return (reinterpret_cast<uintptr_t>(p) & (dt == MUON_F32 ? 3 : 1)) == 0; }
bool dtype_ok(int dt) { return dt == MUON_F32 || dt == MUON_BF16; }
muon_status status_of(cudaError_t e) { return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA; }

// Partial rows of the backward pass: one per block, and blocks enough to fill the GPU.
constexpr long long PARTS = 152 * 8;
long long parts_for(long long N, long long D) {
  if (D > MAX_ROW) return std::max(1LL, std::min(N, 64LL));
  const long long rows = D <= 1024 ? SHORT_THREADS / 32 : 1;
  return std::max(1LL, std::min((N + rows - 1) / rows, PARTS));
}
long long part_pitch(long long D) { return (D + 7) / 8 * 8; }

template <typename XT, typename YT, int W, int C>
cudaError_t forward_launch(const ForwardArgs &a, bool vec, cudaStream_t s) {
  constexpr int THREADS = W == 1 ? SHORT_THREADS : W * 32;
  constexpr long long ROWS = THREADS / (W * 32);
  const long long sms = device_sm_count();
  const dim3 grid(static_cast<unsigned>(std::min((a.N + ROWS - 1) / ROWS, sms * (2048 / THREADS)))), block(THREADS);
  return vec ? launch_pdl(layernorm_forward_kernel<XT, YT, W, C, true>, grid, block, 0, s, a)
             : launch_pdl(layernorm_forward_kernel<XT, YT, W, C, false>, grid, block, 0, s, a);
}

template <typename XT, typename YT>
cudaError_t forward_route(const ForwardArgs &a, bool vec, cudaStream_t s) {
  if (a.D <= 256) return forward_launch<XT, YT, 1, 1>(a, vec, s);
  if (a.D <= 512) return forward_launch<XT, YT, 1, 2>(a, vec, s);
  if (a.D <= 768) return forward_launch<XT, YT, 1, 3>(a, vec, s);
  if (a.D <= 1024) return forward_launch<XT, YT, 1, 4>(a, vec, s);
  if (a.D <= 2048) return forward_launch<XT, YT, 4, 2>(a, vec, s);
  if (a.D <= 4096) return forward_launch<XT, YT, 8, 2>(a, vec, s);
  if (a.D <= 8192) return forward_launch<XT, YT, 16, 2>(a, vec, s);
  if (a.D <= MAX_ROW) return forward_launch<XT, YT, 32, 2>(a, vec, s);
  const dim3 grid(static_cast<unsigned>(std::min<long long>(a.N, device_sm_count() * 2))), block(LONG_THREADS);
  return launch_pdl(layernorm_forward_long_kernel<XT, YT>, grid, block, 0, s, a);
}

template <typename XT, typename YT, int W, int C>
cudaError_t backward_launch(const BackwardArgs &a, bool vec, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.parts)), block(W == 1 ? SHORT_THREADS : W * 32);
  return vec ? launch_pdl(layernorm_backward_kernel<XT, YT, W, C, true>, grid, block, 0, s, a)
             : launch_pdl(layernorm_backward_kernel<XT, YT, W, C, false>, grid, block, 0, s, a);
}

template <typename XT, typename YT>
cudaError_t backward_route(const BackwardArgs &a, bool vec, cudaStream_t s) {
  if (a.D <= 256) return backward_launch<XT, YT, 1, 1>(a, vec, s);
  if (a.D <= 512) return backward_launch<XT, YT, 1, 2>(a, vec, s);
  if (a.D <= 768) return backward_launch<XT, YT, 1, 3>(a, vec, s);
  if (a.D <= 1024) return backward_launch<XT, YT, 1, 4>(a, vec, s);
  if (a.D <= 2048) return backward_launch<XT, YT, 4, 2>(a, vec, s);
  if (a.D <= 4096) return backward_launch<XT, YT, 8, 2>(a, vec, s);
  if (a.D <= 8192) return backward_launch<XT, YT, 16, 2>(a, vec, s);
  if (a.D <= MAX_ROW) return backward_launch<XT, YT, 32, 2>(a, vec, s);
  // the columns first: dx may take the place of dy or x
  if (a.part != nullptr) {
    const dim3 cgrid(static_cast<unsigned>((a.D + 255) / 256), static_cast<unsigned>(a.parts));
    const cudaError_t e = launch_pdl(layernorm_columns_kernel<XT, YT>, cgrid, dim3(256), 0, s, a);
    if (e != cudaSuccess || a.dx == nullptr) return e;
    launch_end(s);
    launch_begin(KK_LN_BWD, s);
  }
  const dim3 grid(static_cast<unsigned>(std::min<long long>(a.N, device_sm_count() * 2))), block(LONG_THREADS);
  return launch_pdl(layernorm_dx_long_kernel<XT, YT>, grid, block, 0, s, a);
}

muon_status check_dims(int64_t N, int64_t D) {
  if (N < 0 || D < 1) return MUON_ERR_INVALID_ARG;
  return N > (1ll << 30) || D > (1ll << 20) ? MUON_ERR_SHAPE : MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status layernorm_forward(const void *x, muon_dtype xdt, int64_t ldx, const void *weight, const void *bias,
                              muon_dtype wdt, void *y, muon_dtype ydt, int64_t ldy, float *mean, float *rstd, int64_t N,
                              int64_t D, float eps, muon_stream_t stream) {
  if (N > 0 && (x == nullptr || y == nullptr)) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(N, D);
  if (st != MUON_OK) return st;
  if (ldx < D || ldy < D || !std::isfinite(eps) || eps < 0.f) return MUON_ERR_INVALID_ARG;
  if (!dtype_ok(xdt) || !dtype_ok(ydt) || !dtype_ok(wdt)) return MUON_ERR_DTYPE;
  if (!natural(x, xdt) || !natural(y, ydt) || !natural(weight, wdt) || !natural(bias, wdt) ||
      !natural(mean, MUON_F32) || !natural(rstd, MUON_F32))
    return MUON_ERR_ALIGNMENT;
  if ((st = device_check()) != MUON_OK) return st;
  if (N == 0) return MUON_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const ForwardArgs a{x, weight, bias, y, ldx, ldy, N, mean, rstd, eps, wdt, static_cast<int>(D)};
  const bool vec = aligned16(x) && aligned16(y) && aligned16(weight) && aligned16(bias) && ldx % 8 == 0 && ldy % 8 == 0;
  launch_begin(KK_LN_FWD, s);
  cudaError_t e;
  if (xdt == MUON_F32)
    e = ydt == MUON_F32 ? forward_route<float, float>(a, vec, s) : forward_route<float, __nv_bfloat16>(a, vec, s);
  else
    e = ydt == MUON_F32 ? forward_route<__nv_bfloat16, float>(a, vec, s)
                        : forward_route<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
  launch_end(s);
  return status_of(e);
}

size_t layernorm_workspace_bytes(int64_t N, int64_t D) {
  if (N < 0 || D < 1) return 0;
  return align_up(static_cast<size_t>(8) * parts_for(N, D) * part_pitch(D), 256);
}

muon_status layernorm_backward(const void *dy, muon_dtype ydt, int64_t lddy, const void *x, muon_dtype xdt, int64_t ldx,
                               const void *weight, muon_dtype wdt, const float *mean, const float *rstd, void *dx,
                               int64_t lddx, void *dweight, void *dbias, muon_dtype gdt, int accumulate, int64_t N,
                               int64_t D, void *ws, size_t ws_bytes, muon_stream_t stream) {
  if (N > 0 && (dy == nullptr || x == nullptr || mean == nullptr || rstd == nullptr)) return MUON_ERR_INVALID_ARG;
  if ((N > 0 && dx == nullptr) && dweight == nullptr && dbias == nullptr) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(N, D);
  if (st != MUON_OK) return st;
  if (lddy < D || ldx < D || (dx != nullptr && lddx < D)) return MUON_ERR_INVALID_ARG;
  if (!dtype_ok(xdt) || !dtype_ok(ydt) || !dtype_ok(wdt) || !dtype_ok(gdt)) return MUON_ERR_DTYPE;
  if (!natural(dy, ydt) || !natural(x, xdt) || !natural(weight, wdt) || !natural(mean, MUON_F32) ||
      !natural(rstd, MUON_F32) || !natural(dx, xdt) || !natural(dweight, gdt) || !natural(dbias, gdt))
    return MUON_ERR_ALIGNMENT;
  const bool sums = dweight != nullptr || dbias != nullptr;
  if (sums) {
    if (ws == nullptr) return MUON_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return MUON_ERR_ALIGNMENT;
    if (ws_bytes < layernorm_workspace_bytes(N, D)) return MUON_ERR_WORKSPACE;
  }
  if ((st = device_check()) != MUON_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  BackwardArgs a{dy, x, weight, dx, lddy, ldx, lddx, N, mean, rstd, sums ? static_cast<float *>(ws) : nullptr,
                 parts_for(N, D), part_pitch(D), wdt, static_cast<int>(D)};
  const bool vec = aligned16(dy) && aligned16(x) && aligned16(weight) && aligned16(dx) && lddy % 8 == 0 &&
                   ldx % 8 == 0 && (dx == nullptr || lddx % 8 == 0);
  if (N == 0) a.parts = 0;
  if (N > 0) {
    launch_begin(KK_LN_BWD, s);
    cudaError_t e;
    if (xdt == MUON_F32)
      e = ydt == MUON_F32 ? backward_route<float, float>(a, vec, s) : backward_route<float, __nv_bfloat16>(a, vec, s);
    else
      e = ydt == MUON_F32 ? backward_route<__nv_bfloat16, float>(a, vec, s)
                          : backward_route<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
    launch_end(s);
    if (e != cudaSuccess) return MUON_ERR_CUDA;
  }
  if (!sums) return MUON_OK;
  const dim3 grid(static_cast<unsigned>((D + REDUCE_COLS - 1) / REDUCE_COLS), 2);
  launch_begin(KK_LN_REDUCE, s);
  const cudaError_t e = launch_pdl(layernorm_reduce_kernel, grid, dim3(REDUCE_WARPS * 32), 0, s,
                                   static_cast<const float *>(a.part), a.parts, a.ldp, a.D, dweight, dbias,
                                   static_cast<int>(gdt), accumulate != 0 ? 1 : 0);
  launch_end(s);
  return status_of(e);
}

}  // extern "C"
