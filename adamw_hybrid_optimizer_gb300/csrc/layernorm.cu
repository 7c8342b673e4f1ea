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
// Without it the next row's loads wait in registers.
// One matrix's part of the ring: [stage][chunk][piece][thread].
template <typename XT, int C>
struct Ring {
  static constexpr int PIECES = Raw8<XT>::PIECES;
  uint4 *base;
  __device__ __forceinline__ uint4 *at(int stage, int k, int p) const {
    return base + ((stage * C + k) * PIECES + p) * blockDim.x + threadIdx.x;
  }
  __device__ __forceinline__ void fetch(const XT *row, const Cols &c, int stage) const {
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (has<true>(c, k, 0)) {
#pragma unroll
        for (int p = 0; p < PIECES; ++p)
          copy_async16(at(stage, k, p), reinterpret_cast<const uint4 *>(row + col<true>(c, k, 0)) + p);
      }
  }
  __device__ __forceinline__ Oct get(const Cols &c, int k, int stage) const {
    Raw8<XT> r;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) r.w[p] = has<true>(c, k, 0) ? *at(stage, k, p) : make_uint4(0, 0, 0, 0);
    return r.get();
  }
};

__device__ __forceinline__ float2 warp_sum2(float2 v, int lanes = 32) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= lanes) continue;
    v = __fadd2_rn(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  }
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    if (o < lanes) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The exchange between the W warps that hold a row: every warp puts a pair, and after one barrier of the row's own (a
// named one, since a block may hold several rows) lane i of every warp reads the pair of warp i, for i below the next
// power of two `lanes` (and again for every further `lanes` lanes, so that sums over `lanes` lanes reach all). Calls
// alternate between two buffers: a thread can write one again only after the barrier of the call in between, which
// every reader of that buffer has reached.
struct Group {
  float2 (*buf)[32];
  int W, w, id, lanes, turn;
  __device__ __forceinline__ float2 exchange(float a, float b) {
    float2 *r = buf[turn];
    const int lane = threadIdx.x % 32, from = lane & (lanes - 1);
    if (lane == 0) r[w] = make_float2(a, b);
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(W * 32) : "memory");
    turn ^= 1;
    return from < W ? r[from] : make_float2(0.f, 0.f);
  }
};

__device__ __forceinline__ Group group_of(float2 (*buf)[32], int W, int t, int slot) {
  int lanes = 1;
  while (lanes < W) lanes *= 2;
  return {buf, W, t / 32, slot + 1, lanes, 0};
}

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
constexpr int fwd_blocks(int C, int MAXW) { return C == 1 ? 4 : C == 2 ? 32 / MAXW : MAXW == 4 ? 6 : 1; }
constexpr int bwd_blocks(int C, int MAXW) { return C == 1 ? 3 : MAXW == 8 ? 2 : 1; }
constexpr int STAGES = 3;

struct ForwardArgs {
  const void *x, *w, *b;
  void *y;
  long long ldx, ldy, N;
  float *mean, *rstd;
  float eps;
  int wdt, D;
};

// blockDim.x / (32 W) rows at a time, W warps each, with the next rows on their way. Mean and variance take one
// exchange: each warp sums its own columns and their squared distances from the warp's own mean, and
//   sum (x - mean)^2 = sum over warps of (own squares + n_w (mean_w - mean)^2).
template <typename XT, typename YT, int C, int MAXW, int FIXED>
__global__ void __launch_bounds__(MAXW * 32, fwd_blocks(C, MAXW)) layernorm_forward_kernel(const ForwardArgs a,
                                                                                           int warps) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr bool VEC = FIXED == 0;
  extern __shared__ uint4 ahead[];
  __shared__ float2 red[BLOCK_WARPS][2][32];
  const int W = VEC ? warps : FIXED;
  const int T = W * 32, rows = blockDim.x / T, slot = threadIdx.x / T, t = threadIdx.x - slot * T, D = a.D;
  Group grp = group_of(red[slot], W, t, slot);
  const float inv = 1.f / static_cast<float>(D);
  const Cols c = cols_of<VEC>(t, T, D);
  const Ring<XT, C> ring{ahead};
  // columns of this warp, and of the warp whose pair this lane reads in the exchange
  const float n_w = warp_sum(static_cast<float>(max(c.count, 0))), inv_n = n_w > 0.f ? 1.f / n_w : 0.f;
  float n_lane = n_w;
  if (W > 1) n_lane = grp.exchange(n_w, 0.f).x;
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long row = static_cast<long long>(blockIdx.x) * rows + slot;
  auto x_of = [&](long long r) { return static_cast<const XT *>(a.x) + r * a.ldx; };
  Raw8<XT> raw[VEC ? 1 : C];
  int stage = 0;
  if constexpr (VEC) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      if (row + i * step < a.N) ring.fetch(x_of(row + i * step), c, i);
      copy_async_commit();
    }
  } else if (row < a.N) {
#pragma unroll
    for (int k = 0; k < C; ++k) load_chunk<XT, false>(x_of(row), c, k, raw[k]);
  }
  for (; row < a.N; row += step) {
    Oct v[C];
    if constexpr (VEC) {
      copy_async_wait<STAGES - 2>();
#pragma unroll
      for (int k = 0; k < C; ++k) v[k] = ring.get(c, k, stage);
      // the place of the row before this one, whose values are long used, takes the row STAGES - 1 ahead
      const int free = stage == 0 ? STAGES - 1 : stage - 1;
      const long long r = row + (STAGES - 1) * step;
      if (r < a.N) ring.fetch(x_of(r), c, free);
      copy_async_commit();
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) v[k] = raw[k].get();
      if (row + step < a.N) {
#pragma unroll
        for (int k = 0; k < C; ++k) load_chunk<XT, false>(x_of(row + step), c, k, raw[k]);
      }
    }
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, v[k].p[i]);
    const float own = warp_sum(s.x + s.y) * inv_n;
    float2 q = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k)
      if (!VEC || has<true>(c, k, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 d = only<VEC>(c, k, i, __fadd2_rn(v[k].p[i], make_float2(-own, -own)));
          q = __ffma2_rn(d, d, q);
        }
      }
    float sq = warp_sum(q.x + q.y), mean = own;
    if (W > 1) {
      const float2 r = grp.exchange(own, sq);
      mean = lanes_sum(n_lane * r.x, grp.lanes) * inv;
      const float d = r.x - mean;
      sq = lanes_sum(fmaf(n_lane * d, d, r.y), grp.lanes);
    }
    const float rstd = rsqrtf(sq * inv + a.eps);
    if (t == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
    YT *y = static_cast<YT *>(a.y) + row * a.ldy;
    const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const Oct w = param_chunk<VEC>(a.w, a.wdt, c, k, 1.f), b = param_chunk<VEC>(a.b, a.wdt, c, k, 0.f);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[k].p[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[k].p[i], m2), r2), w.p[i], b.p[i]);
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
// and the rest of shared memory has no room for a ring, so the next row waits in registers where it fits them); the
// block's slots are added in order at the end.
template <typename XT, typename YT, int C, int MAXW, int FIXED>
__global__ void __launch_bounds__(MAXW * 32, bwd_blocks(C, MAXW)) layernorm_backward_kernel(const BackwardArgs a,
                                                                                            int warps) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr bool VEC = FIXED == 0, IN_SHARED = MAXW == 32, RING = VEC && !IN_SHARED;
  constexpr bool AHEAD = !RING && (!IN_SHARED || sizeof(XT) + sizeof(YT) == 4);
  extern __shared__ uint4 ahead[];   // the rings, or IN_SHARED: [4 C][threads]: two of dw, two of db for each chunk
  __shared__ float2 red[BLOCK_WARPS][2][32];
  __shared__ __align__(16) float join[C == 1 ? BLOCK_WARPS * 256 : 1];
  const int W = VEC ? warps : FIXED;
  const int T = W * 32, rows = blockDim.x / T, slot = threadIdx.x / T, t = threadIdx.x - slot * T, D = a.D;
  Group grp = group_of(red[slot], W, t, slot);
  const float inv = 1.f / static_cast<float>(D);
  const Cols c = cols_of<VEC>(t, T, D);
  float4 *sums = reinterpret_cast<float4 *>(ahead);
  const Ring<XT, C> ring_x{ahead};
  const Ring<YT, C> ring_dy{ahead + STAGES * C * Raw8<XT>::PIECES * blockDim.x};
  Oct aw[C], ab[C];
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) aw[k].p[i] = ab[k].p[i] = make_float2(0.f, 0.f);
  auto sums_get = [&](int k) {
    if constexpr (IN_SHARED) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 u = sums[(4 * k + h) * T + t], v = sums[(4 * k + 2 + h) * T + t];
        aw[k].p[2 * h] = make_float2(u.x, u.y);
        aw[k].p[2 * h + 1] = make_float2(u.z, u.w);
        ab[k].p[2 * h] = make_float2(v.x, v.y);
        ab[k].p[2 * h + 1] = make_float2(v.z, v.w);
      }
    }
  };
  auto sums_put = [&](int k) {
    if constexpr (IN_SHARED) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 u = aw[k].p[2 * h], u1 = aw[k].p[2 * h + 1], v = ab[k].p[2 * h], v1 = ab[k].p[2 * h + 1];
        sums[(4 * k + h) * T + t] = make_float4(u.x, u.y, u1.x, u1.y);
        sums[(4 * k + 2 + h) * T + t] = make_float4(v.x, v.y, v1.x, v1.y);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < C; ++k) sums_put(k);
  const long long step = static_cast<long long>(gridDim.x) * rows;
  long long row = static_cast<long long>(blockIdx.x) * rows + slot;
  auto x_of = [&](long long r) { return static_cast<const XT *>(a.x) + r * a.ldx; };
  auto dy_of = [&](long long r) { return static_cast<const YT *>(a.dy) + r * a.lddy; };
  Raw8<XT> rx[RING ? 1 : C];
  Raw8<YT> rdy[RING ? 1 : C];
  auto fetch = [&](long long r) {
    if constexpr (!RING) {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        load_chunk<XT, VEC>(x_of(r), c, k, rx[k]);
        load_chunk<YT, VEC>(dy_of(r), c, k, rdy[k]);
      }
    }
  };
  float mean = 0.f, rstd = 0.f;
  int stage = 0;
  if (row < a.N) {
    mean = a.mean[row];
    rstd = a.rstd[row];
    if constexpr (AHEAD) fetch(row);
  }
  if constexpr (RING) {
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i) {
      if (row + i * step < a.N) {
        ring_x.fetch(x_of(row + i * step), c, i);
        ring_dy.fetch(dy_of(row + i * step), c, i);
      }
      copy_async_commit();
    }
  }
  for (; row < a.N; row += step) {
    if constexpr (!RING && !AHEAD) fetch(row);
    const float rs = rstd;
    const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rs, rs);
    if (row + step < a.N) {
      mean = a.mean[row + step];
      rstd = a.rstd[row + step];
    }
    Oct xh[C], g[C];
    if constexpr (RING) {
      copy_async_wait<STAGES - 2>();
#pragma unroll
      for (int k = 0; k < C; ++k) {
        xh[k] = ring_x.get(c, k, stage);
        g[k] = ring_dy.get(c, k, stage);
      }
      // the place of the row before this one, whose values are long used, takes the row STAGES - 1 ahead
      const int free = stage == 0 ? STAGES - 1 : stage - 1;
      const long long r = row + (STAGES - 1) * step;
      if (r < a.N) {
        ring_x.fetch(x_of(r), c, free);
        ring_dy.fetch(dy_of(r), c, free);
      }
      copy_async_commit();
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        xh[k] = rx[k].get();
        g[k] = rdy[k].get();
      }
      if (AHEAD && row + step < a.N) fetch(row + step);
    }
    float2 s1 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k) {
      const Oct w = param_chunk<VEC>(a.w, a.wdt, c, k, 1.f);
      sums_get(k);
      // where the row has no column dy is 0, but xh need not be finite
      if (!VEC || has<true>(c, k, 0)) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 h = only<VEC>(c, k, i, __fmul2_rn(__fadd2_rn(xh[k].p[i], m2), r2));
          xh[k].p[i] = h;
          aw[k].p[i] = __ffma2_rn(g[k].p[i], h, aw[k].p[i]);
          ab[k].p[i] = __fadd2_rn(ab[k].p[i], g[k].p[i]);
          g[k].p[i] = __fmul2_rn(g[k].p[i], w.p[i]);
          s1 = __fadd2_rn(s1, g[k].p[i]);
          s2 = __ffma2_rn(g[k].p[i], h, s2);
        }
      }
      sums_put(k);
    }
    float2 sum = warp_sum2(make_float2(s1.x + s1.y, s2.x + s2.y));
    if (W > 1) {
      sum = grp.exchange(sum.x, sum.y);
      sum = warp_sum2(sum, grp.lanes);
    }
    if (a.dx != nullptr) {
      const float2 c1 = make_float2(-sum.x * inv, -sum.x * inv), c2 = make_float2(-sum.y * inv, -sum.y * inv);
      XT *dx = static_cast<XT *>(a.dx) + row * a.lddx;
#pragma unroll
      for (int k = 0; k < C; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          g[k].p[i] = __fmul2_rn(__ffma2_rn(xh[k].p[i], c2, __fadd2_rn(g[k].p[i], c1)), r2);
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
      sums_get(k);
      store_chunk<float, VEC>(pw, c, k, aw[k]);
      store_chunk<float, VEC>(pb, c, k, ab[k]);
    }
    return;
  }
  // several slots only where C = 1: rows * D <= BLOCK_WARPS * 256 columns
  for (int z = 0; z < 2; ++z) {
    __syncthreads();
    const Oct o = z == 0 ? aw[0] : ab[0];
    store_chunk<float, VEC>(join + slot * D, c, 0, o);
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
  int threads() const { return W * rows * 32; }
};
Shape shape_of(long long D, bool vec, int C) {
  int W = static_cast<int>((D + 256 * C - 1) / (256 * C));
  if (!vec) {
    int p = 1;
    while (p < W) p *= 2;
    W = p;
  }
  return {C, W, C == 1 ? std::max(1, BLOCK_WARPS / W) : 1};
}
// The forward pass takes four chunks where it can: the shuffles and the exchange of a row are shared by more columns.
Shape fwd_shape(long long D, bool vec) { return shape_of(D, vec, D <= 1024 ? 1 : vec ? 4 : 2); }
Shape bwd_shape(long long D, bool vec) { return shape_of(D, vec, D <= 1024 ? 1 : 2); }

// Blocks of the backward pass, each of which leaves one partial row of dw and db: as many as the GPU holds at once,
// so that there are few partial rows to add.
long long parts_for(long long N, long long D, bool vec) {
  if (D > MAX_ROW) return std::max(1LL, std::min(N, 64LL));
  const Shape h = bwd_shape(D, vec);
  const long long resident = std::max(1, (h.C == 1 ? 768 : 512) / h.threads());
  return std::max(1LL, std::min((N + h.rows - 1) / h.rows, 152 * resident));
}
long long part_pitch(long long D) { return (D + 7) / 8 * 8; }

constexpr int SM_SHARED = 227 * 1024;
constexpr int STATIC_SHARED = 16 * 1024;   // more than any kernel's static share

// Once for each kernel that may take more than 48 KB.
template <typename K>
cudaError_t allow_shared(K kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM_SHARED - STATIC_SHARED);
}

template <typename XT, typename YT, int C, int MAXW, int FIXED>
cudaError_t forward_launch(const ForwardArgs &a, const Shape &h, cudaStream_t s) {
  auto kernel = layernorm_forward_kernel<XT, YT, C, MAXW, FIXED>;
  static const cudaError_t allowed = allow_shared(kernel);
  if (allowed != cudaSuccess) return allowed;
  const size_t smem = FIXED == 0 ? static_cast<size_t>(STAGES) * C * 8 * sizeof(XT) * h.threads() : 0;
  const long long sms = device_sm_count();
  const size_t held = smem + 6 * 1024;   // with the kernel's static share and the system's
  const long long resident = std::min<long long>(fwd_blocks(C, MAXW) * MAXW * 32 / h.threads(), SM_SHARED / held);
  const dim3 grid(static_cast<unsigned>(std::min((a.N + h.rows - 1) / h.rows, sms * resident)));
  return launch_pdl(kernel, grid, dim3(h.threads()), smem, s, a, h.W);
}

template <typename XT, typename YT>
cudaError_t forward_route(const ForwardArgs &a, bool vec, cudaStream_t s) {
  if (a.D > MAX_ROW) {
    const dim3 grid(static_cast<unsigned>(std::min<long long>(a.N, device_sm_count() * 2))), block(LONG_THREADS);
    return launch_pdl(layernorm_forward_long_kernel<XT, YT>, grid, block, 0, s, a);
  }
  const Shape h = fwd_shape(a.D, vec);
  if (vec)
    return h.C == 1    ? forward_launch<XT, YT, 1, BLOCK_WARPS, 0>(a, h, s)
           : h.W <= 4  ? forward_launch<XT, YT, 4, 4, 0>(a, h, s)
                       : forward_launch<XT, YT, 4, 16, 0>(a, h, s);
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
  static const cudaError_t allowed = allow_shared(kernel);
  if (allowed != cudaSuccess) return allowed;
  const size_t per_thread = MAXW == 32 ? 4 * C * sizeof(float4)
                            : FIXED == 0 ? static_cast<size_t>(STAGES) * C * 8 * (sizeof(XT) + sizeof(YT)) : 0;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(a.parts)), dim3(h.threads()), per_thread * h.threads(), s, a,
                    h.W);
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
  const Shape h = bwd_shape(a.D, vec);
  if (vec)
    return h.C == 1    ? backward_launch<XT, YT, 1, BLOCK_WARPS, 0>(a, h, s)
           : h.W <= 8  ? backward_launch<XT, YT, 2, 8, 0>(a, h, s)
           : h.W <= 16 ? backward_launch<XT, YT, 2, 16, 0>(a, h, s)
                       : backward_launch<XT, YT, 2, 32, 0>(a, h, s);
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
