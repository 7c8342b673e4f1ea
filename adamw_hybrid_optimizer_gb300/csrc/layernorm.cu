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

constexpr int LONG_THREADS = 1024;     // block of the kernels for rows beyond MAX_ROW
constexpr int MAX_ROW = 16384;
constexpr int BLOCK_WARPS = 8;         // warps of a block that holds several short rows
constexpr int REDUCE_COLS = 32;
constexpr int REDUCE_WARPS = 16;

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

// Eight values as loaded, converted only when they are used: the next row waits in half the registers.
template <typename XT>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void get(float *f) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void set(const float *f) {
    a = make_float4(f[0], f[1], f[2], f[3]);
    b = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 w;
  __device__ __forceinline__ void get(float *f) const {
    const unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[2 * e] = __uint_as_float(u[e] << 16);
      f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { w = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void set(const __nv_bfloat16 *f) {
    const unsigned short *h = reinterpret_cast<const unsigned short *>(f);
    w = make_uint4(h[0] | (static_cast<unsigned>(h[1]) << 16), h[2] | (static_cast<unsigned>(h[3]) << 16),
                   h[4] | (static_cast<unsigned>(h[5]) << 16), h[6] | (static_cast<unsigned>(h[7]) << 16));
  }
};

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
__device__ __forceinline__ void store_chunk(XT *p, const Cols &c, int k, const float *f) {
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
__device__ __forceinline__ void param_chunk(const void *p, int dt, const Cols &c, int k, float absent, float *f) {
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = absent;
  if (p == nullptr) return;
  if constexpr (VEC) {
    if (!has<true>(c, k, 0)) return;
    if (dt == MUON_F32) load8(static_cast<const float *>(p) + col<true>(c, k, 0), f);
    else load8(static_cast<const __nv_bfloat16 *>(p) + col<true>(c, k, 0), f);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (has<false>(c, k, e)) f[e] = param_at(p, dt, col<false>(c, k, e), absent);
  }
}

__device__ __forceinline__ float2 warp_sum2(float a, float b) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    a += __shfl_xor_sync(0xffffffffu, a, o);
    b += __shfl_xor_sync(0xffffffffu, b, o);
  }
  return make_float2(a, b);
}

// The exchange between the W warps that hold a row: every warp puts a pair, and after one barrier of the row's own (a
// named one, since a block may hold several rows) lane i of every warp reads the pair of warp i. Calls alternate
// between two buffers: a thread can write one again only after the barrier of the call in between, which every
// reader of that buffer has reached.
struct Group {
  float2 (*buf)[32];
  int W, w, id, turn;
  __device__ __forceinline__ float2 exchange(float a, float b) {
    float2 *r = buf[turn];
    const int lane = threadIdx.x % 32;
    if (lane == 0) r[w] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(W * 32) : "memory");
    turn ^= 1;
    return lane < W ? r[lane] : make_float2(0.f, 0.f);
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

// The most warps of a block, by the chunks C per thread and the row's width, and the blocks that the compiler is to
// leave registers for on a multiprocessor.
constexpr int fwd_blocks(int C, int MAXW) { return C == 1 ? 4 : MAXW == 16 ? 2 : 1; }
constexpr int bwd_blocks(int C, int MAXW) { return C == 1 ? 3 : 1; }

struct ForwardArgs {
  const void *x, *w, *b;
  void *y;
  long long ldx, ldy, N;
  float *mean, *rstd;
  float eps;
  int wdt, D;
};

// blockDim.x / (32 W) rows at a time, W warps each. The next row's loads are issued before the current row's sums are
// exchanged, so that the barrier and the stores run under them. Mean and variance take one exchange: each warp sums
// its own columns and their squared distances from the warp's own mean, and
//   sum (x - mean)^2 = sum over warps of (own squares + n_w (mean_w - mean)^2).
template <typename XT, typename YT, int C, int MAXW, int FIXED>
__global__ void __launch_bounds__(MAXW * 32, fwd_blocks(C, MAXW)) layernorm_forward_kernel(const ForwardArgs a,
                                                                                           int warps) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ float2 red[BLOCK_WARPS][2][32];
  constexpr bool VEC = FIXED == 0;
  const int W = VEC ? warps : FIXED;
  const int T = W * 32, rows = blockDim.x / T, slot = threadIdx.x / T, t = threadIdx.x - slot * T, D = a.D;
  Group grp{red[slot], W, t / 32, slot + 1, 0};
  const float inv = 1.f / static_cast<float>(D);
  const Cols c = cols_of<VEC>(t, T, D);
  // columns of this warp, and of the warp whose pair this lane reads in the exchange
  const float n_w = warp_sum(static_cast<float>(max(c.count, 0))), inv_n = n_w > 0.f ? 1.f / n_w : 0.f;
  float n_lane = n_w;
  if (W > 1) n_lane = grp.exchange(n_w, 0.f).x;
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long row = static_cast<long long>(blockIdx.x) * rows + slot;
  Raw8<XT> raw[C];
  if (row < a.N) {
#pragma unroll
    for (int k = 0; k < C; ++k)
      load_chunk<XT, VEC>(static_cast<const XT *>(a.x) + row * a.ldx, c, k, raw[k]);
  }
  for (; row < a.N; row += step) {
    float v[C][8];
#pragma unroll
    for (int k = 0; k < C; ++k) raw[k].get(v[k]);
    if (row + step < a.N) {
#pragma unroll
      for (int k = 0; k < C; ++k)
        load_chunk<XT, VEC>(static_cast<const XT *>(a.x) + (row + step) * a.ldx, c, k, raw[k]);
    }
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += v[k][e];
    s = warp_sum(s);
    const float own = s * inv_n;
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = v[k][e] - own;
        if (has<VEC>(c, k, e)) q = fmaf(d, d, q);
      }
    q = warp_sum(q);
    float mean = own;
    if (W > 1) {
      const float2 r = grp.exchange(own, q);
      mean = warp_sum(n_lane * r.x) * inv;
      const float d = r.x - mean;
      q = warp_sum(fmaf(n_lane * d, d, r.y));
    }
    const float rstd = 1.f / sqrtf(q * inv + a.eps);
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    YT *y = static_cast<YT *>(a.y) + row * a.ldy;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float w[8], b[8];
      param_chunk<VEC>(a.w, a.wdt, c, k, 1.f, w);
      param_chunk<VEC>(a.b, a.wdt, c, k, 0.f, b);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[k][e] = fmaf((v[k][e] - mean) * rstd, w[e], b[e]);
      store_chunk<YT, VEC>(y, c, k, v[k]);
    }
  }
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_THREADS) layernorm_forward_long_kernel(const ForwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ float red[2][32];
  int turn = 0;
  const float inv = 1.f / static_cast<float>(a.D);
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    YT *y = static_cast<YT *>(a.y) + row * a.ldy;
    float s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) s += load1(x, c);
    const float mean = block_sum(s, red, turn) * inv;
    float q = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) {
      const float d = load1(x, c) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = 1.f / sqrtf(block_sum(q, red, turn) * inv + a.eps);
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

// Rows and prefetch as in the forward kernel. Each thread keeps its columns of dw and db over all rows of its slot, in
// registers, or in shared memory for rows of more than 8192 columns (MAXW = 32: 1024 threads have 64 registers each,
// and the next row is fetched ahead only where it fits them); the block's slots are added in order at the end.
template <typename XT, typename YT, int C, int MAXW, int FIXED>
__global__ void __launch_bounds__(MAXW * 32, bwd_blocks(C, MAXW)) layernorm_backward_kernel(const BackwardArgs a,
                                                                                            int warps) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr bool IN_SHARED = MAXW == 32, AHEAD = !IN_SHARED || sizeof(XT) + sizeof(YT) == 4;
  extern __shared__ float4 sums[];   // IN_SHARED: [4 C][threads]: two of dw, two of db for each chunk
  __shared__ float2 red[BLOCK_WARPS][2][32];
  __shared__ float join[C == 1 ? BLOCK_WARPS * 256 : 1];
  constexpr bool VEC = FIXED == 0;
  const int W = VEC ? warps : FIXED;
  const int T = W * 32, rows = blockDim.x / T, slot = threadIdx.x / T, t = threadIdx.x - slot * T, D = a.D;
  Group grp{red[slot], W, t / 32, slot + 1, 0};
  const float inv = 1.f / static_cast<float>(D);
  const Cols c = cols_of<VEC>(t, T, D);
  float aw[C][8], ab[C][8];
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) aw[k][e] = ab[k][e] = 0.f;
  if constexpr (IN_SHARED) {
#pragma unroll
    for (int i = 0; i < 4 * C; ++i) sums[i * T + t] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long row = static_cast<long long>(blockIdx.x) * rows + slot;
  Raw8<XT> rx[C];
  Raw8<YT> rdy[C];
  float mean = 0.f, rstd = 0.f;
  auto fetch = [&](long long r) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      load_chunk<XT, VEC>(static_cast<const XT *>(a.x) + r * a.ldx, c, k, rx[k]);
      load_chunk<YT, VEC>(static_cast<const YT *>(a.dy) + r * a.lddy, c, k, rdy[k]);
    }
    mean = a.mean[r];
    rstd = a.rstd[r];
  };
  if (AHEAD && row < a.N) fetch(row);
  for (; row < a.N; row += step) {
    if constexpr (!AHEAD) fetch(row);
    float xh[C][8], g[C][8];
    const float mu = mean, rs = rstd;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      rx[k].get(xh[k]);
      rdy[k].get(g[k]);
    }
    if (AHEAD && row + step < a.N) fetch(row + step);
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int k = 0; k < C; ++k) {
      float w[8];
      param_chunk<VEC>(a.w, a.wdt, c, k, 1.f, w);
      if constexpr (IN_SHARED) {
        Raw8<float> r;
        r.a = sums[(4 * k) * T + t];
        r.b = sums[(4 * k + 1) * T + t];
        r.get(aw[k]);
        r.a = sums[(4 * k + 2) * T + t];
        r.b = sums[(4 * k + 3) * T + t];
        r.get(ab[k]);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        xh[k][e] = (xh[k][e] - mu) * rs;
        // where the row has no column dy is 0, but xh need not be finite
        if (has<VEC>(c, k, e)) {
          aw[k][e] = fmaf(g[k][e], xh[k][e], aw[k][e]);
          ab[k][e] += g[k][e];
          g[k][e] *= w[e];
          s1 += g[k][e];
          s2 = fmaf(g[k][e], xh[k][e], s2);
        }
      }
      if constexpr (IN_SHARED) {
        Raw8<float> r;
        r.set(aw[k]);
        sums[(4 * k) * T + t] = r.a;
        sums[(4 * k + 1) * T + t] = r.b;
        r.set(ab[k]);
        sums[(4 * k + 2) * T + t] = r.a;
        sums[(4 * k + 3) * T + t] = r.b;
      }
    }
    float2 sum = warp_sum2(s1, s2);
    if (W > 1) {
      sum = grp.exchange(sum.x, sum.y);
      sum = warp_sum2(sum.x, sum.y);
    }
    s1 = sum.x * inv;
    s2 = sum.y * inv;
    if (a.dx != nullptr) {
      XT *dx = static_cast<XT *>(a.dx) + row * a.lddx;
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[k][e] = rs * (g[k][e] - s1 - xh[k][e] * s2);
        store_chunk<XT, VEC>(dx, c, k, g[k]);
      }
    }
  }
  if (a.part == nullptr) return;
  float *pw = a.part + static_cast<long long>(blockIdx.x) * a.ldp;
  float *pb = a.part + (a.parts + blockIdx.x) * a.ldp;
  if (C > 1 || rows == 1) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      if constexpr (IN_SHARED) {
        Raw8<float> r;
        r.a = sums[(4 * k) * T + t];
        r.b = sums[(4 * k + 1) * T + t];
        r.get(aw[k]);
        r.a = sums[(4 * k + 2) * T + t];
        r.b = sums[(4 * k + 3) * T + t];
        r.get(ab[k]);
      }
      store_chunk<float, VEC>(pw, c, k, aw[k]);
      store_chunk<float, VEC>(pb, c, k, ab[k]);
    }
    return;
  }
  // several slots only where C = 1: rows * D <= BLOCK_WARPS * 256 columns
  for (int z = 0; z < 2; ++z) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (has<VEC>(c, 0, e)) join[slot * D + col<VEC>(c, 0, e)] = z == 0 ? aw[0][e] : ab[0][e];
    }
    __syncthreads();
    for (int j = threadIdx.x; j < D; j += blockDim.x) {
      float s = 0.f;
      for (int r = 0; r < rows; ++r) s += join[r * D + j];
      (z == 0 ? pw : pb)[j] = s;
    }
  }
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_THREADS) layernorm_dx_long_kernel(const BackwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ float red[2][32];
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
    s1 = block_sum(s1, red, turn) * inv;
    s2 = block_sum(s2, red, turn) * inv;
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

// How a row of D columns is held: C chunks of eight columns per thread, W warps, and several rows in a block of up to
// BLOCK_WARPS warps where C is 1. Without the vector path W is a power of two, which the kernels know when they are
// compiled: each column is an access of its own there, and its offset has to be a constant to take no register.
struct Shape {
  int C, W, rows;
};
Shape shape_for(long long D, bool vec) {
  const int C = D <= 1024 ? 1 : 2;
  int W = static_cast<int>((D + 256 * C - 1) / (256 * C));
  if (!vec) {
    int p = 1;
    while (p < W) p *= 2;
    W = p;
  }
  return {C, W, C == 1 ? std::max(1, BLOCK_WARPS / W) : 1};
}

// Blocks of the backward pass, each of which leaves one partial row of dw and db: as many as the GPU holds at once,
// so that there are few partial rows to add.
long long parts_for(long long N, long long D, bool vec) {
  if (D > MAX_ROW) return std::max(1LL, std::min(N, 64LL));
  const Shape h = shape_for(D, vec);
  const long long resident = h.C == 1 ? bwd_blocks(1, BLOCK_WARPS) : std::max(1, 16 / h.W);
  return std::max(1LL, std::min((N + h.rows - 1) / h.rows, 152 * resident));
}
long long part_pitch(long long D) { return (D + 7) / 8 * 8; }

template <typename XT, typename YT, int C, int MAXW, int FIXED>
cudaError_t forward_launch(const ForwardArgs &a, const Shape &h, cudaStream_t s) {
  const int threads = h.W * h.rows * 32;
  const long long sms = device_sm_count();
  const dim3 grid(static_cast<unsigned>(std::min((a.N + h.rows - 1) / h.rows, sms * (2048 / threads))));
  return launch_pdl(layernorm_forward_kernel<XT, YT, C, MAXW, FIXED>, grid, dim3(threads), 0, s, a, h.W);
}

template <typename XT, typename YT>
cudaError_t forward_route(const ForwardArgs &a, bool vec, cudaStream_t s) {
  if (a.D > MAX_ROW) {
    const dim3 grid(static_cast<unsigned>(std::min<long long>(a.N, device_sm_count() * 2))), block(LONG_THREADS);
    return launch_pdl(layernorm_forward_long_kernel<XT, YT>, grid, block, 0, s, a);
  }
  const Shape h = shape_for(a.D, vec);
  if (vec) {
    if (h.C == 1) return forward_launch<XT, YT, 1, BLOCK_WARPS, 0>(a, h, s);
    return h.W <= 16 ? forward_launch<XT, YT, 2, 16, 0>(a, h, s) : forward_launch<XT, YT, 2, 32, 0>(a, h, s);
  }
  if (h.C == 1)
    return h.W == 1   ? forward_launch<XT, YT, 1, BLOCK_WARPS, 1>(a, h, s)
           : h.W == 2 ? forward_launch<XT, YT, 1, BLOCK_WARPS, 2>(a, h, s)
                      : forward_launch<XT, YT, 1, BLOCK_WARPS, 4>(a, h, s);
  return h.W == 4    ? forward_launch<XT, YT, 2, 16, 4>(a, h, s)
         : h.W == 8  ? forward_launch<XT, YT, 2, 16, 8>(a, h, s)
         : h.W == 16 ? forward_launch<XT, YT, 2, 16, 16>(a, h, s)
                     : forward_launch<XT, YT, 2, 32, 32>(a, h, s);
}

template <typename XT, typename YT, int C, int MAXW, int FIXED>
cudaError_t backward_launch(const BackwardArgs &a, const Shape &h, cudaStream_t s) {
  auto kernel = layernorm_backward_kernel<XT, YT, C, MAXW, FIXED>;
  const int threads = h.W * h.rows * 32;
  const size_t smem = MAXW == 32 ? static_cast<size_t>(threads) * 4 * C * sizeof(float4) : 0;
  if (MAXW == 32) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(MAXW * 32 * 4 * C * sizeof(float4)));
    if (e != cudaSuccess) return e;
  }
  return launch_pdl(kernel, dim3(static_cast<unsigned>(a.parts)), dim3(threads), smem, s, a, h.W);
}

template <typename XT, typename YT>
cudaError_t backward_route(const BackwardArgs &a, bool vec, cudaStream_t s) {
  if (a.D > MAX_ROW) {
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
  const Shape h = shape_for(a.D, vec);
  if (vec) {
    if (h.C == 1) return backward_launch<XT, YT, 1, BLOCK_WARPS, 0>(a, h, s);
    return h.W <= 16 ? backward_launch<XT, YT, 2, 16, 0>(a, h, s) : backward_launch<XT, YT, 2, 32, 0>(a, h, s);
  }
  if (h.C == 1)
    return h.W == 1   ? backward_launch<XT, YT, 1, BLOCK_WARPS, 1>(a, h, s)
           : h.W == 2 ? backward_launch<XT, YT, 1, BLOCK_WARPS, 2>(a, h, s)
                      : backward_launch<XT, YT, 1, BLOCK_WARPS, 4>(a, h, s);
  return h.W == 4    ? backward_launch<XT, YT, 2, 16, 4>(a, h, s)
         : h.W == 8  ? backward_launch<XT, YT, 2, 16, 8>(a, h, s)
         : h.W == 16 ? backward_launch<XT, YT, 2, 16, 16>(a, h, s)
                     : backward_launch<XT, YT, 2, 32, 32>(a, h, s);
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
  const bool vec = aligned16(x) && aligned16(y) && aligned16(weight) && aligned16(bias) && ldx % 8 == 0 && ldy % 8 == 0 &&
                   D % 8 == 0;
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
  return align_up(static_cast<size_t>(8) * std::max(parts_for(N, D, true), parts_for(N, D, false)) * part_pitch(D), 256);
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
  const bool vec = aligned16(dy) && aligned16(x) && aligned16(weight) && aligned16(dx) && lddy % 8 == 0 &&
                   ldx % 8 == 0 && (dx == nullptr || lddx % 8 == 0) && D % 8 == 0;
  BackwardArgs a{dy, x, weight, dx, lddy, ldx, lddx, N, mean, rstd, sums ? static_cast<float *>(ws) : nullptr,
                 parts_for(N, D, vec), part_pitch(D), wdt, static_cast<int>(D)};
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
