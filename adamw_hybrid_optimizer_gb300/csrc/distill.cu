// Distillation from a teacher's top logits: for each row, the Kullback-Leibler divergence of the student's softmax
// over V logits from the teacher's softmax over its K kept entries, at a temperature T.
//
//   q = softmax(t / T) over the row's valid entries (index in [0, V), value above -inf)
//   m = max_j z_j,  l = log sum_j exp((z_j - m) / T),  log p_j = (z_j - m) / T - l
//   loss = w T^2 sum_k q_k (log q_k - log p_{idx_k})
//   d loss / d z_j = w T (p_j - sum_{k : idx_k = j} q_k)
//
// A row of weight 0, or without a valid entry, has loss 0 and gradient 0, and its logits are not used. m and l are
// kept apart (stats), so that p = exp((z - m) / T - l) keeps its precision for logits of any size. All three forms
// are bound by bandwidth: forward reads the logits once, with a running maximum and sum; backward reads them once
// and writes the gradient; the joint form does both on one row in the same block, so that its second reading comes
// from L2.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_K = 1024;
constexpr float LOG2E = 1.4426950408889634f;

struct DistillArgs {
  const void *z;              // N x V student logits; dz may be the same buffer
  const void *t_idx, *t_val;  // N x K
  const float *weights, *grad;
  float *losses, *stats;      // stats: N x 2 (m, l), written by the forward forms, read by backward
  void *dz;
  long long ldz, ldd, N;
  int V, K, itype, tdt;
  float inv_t, temp, grad_scale;
};

// The row's teacher entries: index (-1: none), q, and the student's logit there (read before dz overwrites it).
struct Teacher {
  int idx[MAX_K];
  float q[MAX_K], z[MAX_K];
};

__device__ __forceinline__ float block_max(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < WARPS; ++w) v = fmaxf(v, red[w]);
  __syncthreads();
  return v;
}

__device__ __forceinline__ float block_sum(float v, float *red) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  v = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) v += red[w];
  __syncthreads();
  return v;
}

// exp(x * c), c = log2(e) / T; the difference x is taken in the logits' own unit, where it is exact or nearly so
__device__ __forceinline__ float exp_scaled(float x, float c) { return exp2f(x * c); }

// Loads the row's teacher entries and makes q. Returns whether the row has a valid one; lse_t: the log of the
// teacher's sum, tmax its largest value.
template <typename ZT>
__device__ __forceinline__ bool load_teacher(const DistillArgs &a, long long row, const ZT *z, Teacher &s, float *red,
                                             float &tmax, float &sum) {
  const long long at = row * a.K;
  float mx = -INFINITY;
  bool any = false;
  for (int k = threadIdx.x; k < a.K; k += THREADS) {
    const long long id = a.itype == MUON_I32 ? static_cast<long long>(static_cast<const int *>(a.t_idx)[at + k])
                                             : static_cast<const long long *>(a.t_idx)[at + k];
    const float t = a.tdt == MUON_F32 ? static_cast<const float *>(a.t_val)[at + k]
                                      : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.t_val)[at + k]);
    const bool ok = id >= 0 && id < a.V && !(t == -INFINITY);   // a NaN is kept, and shows in the loss
    s.idx[k] = ok ? static_cast<int>(id) : -1;
    s.q[k] = t;
    s.z[k] = ok ? load1(z, id) : 0.f;
    if (ok) {
      mx = fmaxf(mx, t);
      any = true;
    }
  }
  any = __syncthreads_or(any);
  tmax = block_max(mx, red);
  const float c = a.inv_t * LOG2E;
  float part = 0.f;
  for (int k = threadIdx.x; k < a.K; k += THREADS)
    if (s.idx[k] >= 0) part += exp_scaled(s.q[k] - tmax, c);
  sum = block_sum(part, red);
  return any;
}

// Eight logits to a running (max, sum); a chunk of -inf leaves both alone.
__device__ __forceinline__ void online8(const float *f, float c, float &m, float &s) {
  float mx = f[0];
#pragma unroll
  for (int e = 1; e < 8; ++e) mx = fmaxf(mx, f[e]);
  if (mx > m) {
    s *= exp_scaled(m - mx, c);
    m = mx;
  }
  const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
  for (int e = 0; e < 8; ++e) s += exp_scaled(f[e] - ref, c);
}

// m and the sum of exp((z - m) / T) over the row. A row of nothing but -inf has no softmax: its sum is NaN.
template <typename ZT, bool VEC>
__device__ __forceinline__ void row_stats(const ZT *z, int V, float c, float *red, float &m, float &sum) {
  float mt = -INFINITY, st = 0.f;
  constexpr int U = 4;
  int j0 = 0;
  if constexpr (VEC) {
    const int whole = V / (THREADS * 8 * U) * (THREADS * 8 * U);
    for (; j0 < whole; j0 += THREADS * 8 * U) {
      float f[U][8];
#pragma unroll
      for (int u = 0; u < U; ++u) load8(z + j0 + (u * THREADS + threadIdx.x) * 8, f[u]);
#pragma unroll
      for (int u = 0; u < U; ++u) online8(f[u], c, mt, st);
    }
    for (; j0 + THREADS * 8 <= V; j0 += THREADS * 8) {
      float f[8];
      load8(z + j0 + threadIdx.x * 8, f);
      online8(f, c, mt, st);
    }
  }
  for (; j0 < V; j0 += THREADS * 8) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + e * THREADS + threadIdx.x;
      f[e] = j < V ? load1(z, j) : -INFINITY;
    }
    online8(f, c, mt, st);
  }
  m = block_max(mt, red);
  const float ref = m == -INFINITY ? 0.f : m;
  sum = block_sum(st * exp_scaled(mt - ref, c), red);
  if (m == -INFINITY) sum = NAN;
}

// dz over columns [a0, a1): scale * (exp((z - m) / T) * inv - q), the q part by the entries themselves afterwards.
template <typename ZT, typename DT, bool VEC>
__device__ __forceinline__ void write_grad(const ZT *z, DT *dz, int V, float c, float m, float inv, float scale) {
  int j0 = 0;
  const float si = scale * inv;
  if constexpr (VEC) {
    for (; j0 + THREADS * 8 <= V; j0 += THREADS * 8) {
      const int j = j0 + threadIdx.x * 8;
      float f[8];
      load8(z + j, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = exp_scaled(f[e] - m, c) * si;
      store8(dz + j, f);
    }
  }
  for (; j0 < V; j0 += THREADS * 8) {
    float f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + e * THREADS + threadIdx.x;
      if (j < V) f[e] = load1(z, j);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = j0 + e * THREADS + threadIdx.x;
      if (j < V) store1(dz, j, exp_scaled(f[e] - m, c) * si);
    }
  }
}

template <typename DT>
__device__ __forceinline__ void zero_row(DT *dz, int V) {
  for (int j = threadIdx.x; j < V; j += THREADS) store1(dz, j, 0.f);
}

// The teacher's entries of a row whose p parts are written: the first entry of each index subtracts the q of all
// entries of that index.
template <typename DT>
__device__ __forceinline__ void subtract_teacher(const DistillArgs &a, const Teacher &s, DT *dz, float c, float m,
                                                 float inv, float scale, float tmax, float tinv) {
  for (int k = threadIdx.x; k < a.K; k += THREADS) {
    const int id = s.idx[k];
    if (id < 0) continue;
    bool first = true;
    float q = 0.f;
    for (int i = 0; i < a.K; ++i) {
      if (s.idx[i] != id) continue;
      if (i < k) {
        first = false;
        break;
      }
      q += exp_scaled(s.q[i] - tmax, c) * tinv;
    }
    if (first) store1(dz, id, scale * (exp_scaled(s.z[k] - m, c) * inv - q));
  }
}

// GRAD false: losses and stats. GRAD true: dz too.
template <typename ZT, typename DT, bool VEC, bool GRAD>
__global__ void __launch_bounds__(THREADS) distill_forward_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ Teacher s;
  __shared__ float red[WARPS];
  const float c = a.inv_t * LOG2E;
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
    DT *dz = GRAD ? static_cast<DT *>(a.dz) + row * a.ldd : nullptr;
    const float w = a.weights != nullptr ? a.weights[row] : 1.f;
    float tmax, tsum;
    if (w == 0.f || !load_teacher(a, row, z, s, red, tmax, tsum)) {   // the same for the whole block
      if (threadIdx.x == 0) {
        a.losses[row] = 0.f;
        a.stats[2 * row] = 0.f;
        a.stats[2 * row + 1] = 0.f;
      }
      if constexpr (GRAD) zero_row(dz, a.V);
      continue;
    }
    float m, sum;
    row_stats<ZT, VEC>(z, a.V, c, red, m, sum);
    const float l = logf(sum), tl = logf(tsum), tinv = 1.f / tsum;
    float part = 0.f;
    for (int k = threadIdx.x; k < a.K; k += THREADS) {
      if (s.idx[k] < 0) continue;
      const float d = s.q[k] - tmax;
      const float q = exp_scaled(d, c) * tinv;
      // an entry whose q is 0 adds nothing, whatever the student gives it
      if (!(q == 0.f)) part = fmaf(q, (d * a.inv_t - tl) - (s.z[k] - m) * a.inv_t, part);
    }
    const float kl = block_sum(part, red) + l;
    if (threadIdx.x == 0) {
      a.losses[row] = w * a.temp * a.temp * kl;
      a.stats[2 * row] = m;
      a.stats[2 * row + 1] = l;
    }
    if constexpr (GRAD) {
      const float scale = a.grad_scale * w * a.temp, inv = 1.f / sum;
      write_grad<ZT, DT, VEC>(z, dz, a.V, c, m, inv, scale);
      __syncthreads();
      subtract_teacher(a, s, dz, c, m, inv, scale, tmax, tinv);
    }
    __syncthreads();   // the next row reuses s
  }
}

template <typename ZT, typename DT, bool VEC>
__global__ void __launch_bounds__(THREADS) distill_backward_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ Teacher s;
  __shared__ float red[WARPS];
  const float c = a.inv_t * LOG2E;
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
    DT *dz = static_cast<DT *>(a.dz) + row * a.ldd;
    const float w = a.weights != nullptr ? a.weights[row] : 1.f;
    float tmax, tsum;
    if (w == 0.f || !load_teacher(a, row, z, s, red, tmax, tsum)) {
      zero_row(dz, a.V);
      continue;
    }
    const float m = a.stats[2 * row], inv = expf(-a.stats[2 * row + 1]);
    const float scale = (a.grad != nullptr ? a.grad[row] : 1.f) * w * a.temp;
    write_grad<ZT, DT, VEC>(z, dz, a.V, c, m, inv, scale);
    __syncthreads();
    subtract_teacher(a, s, dz, c, m, inv, scale, tmax, 1.f / tsum);
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------ host

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool natural(const void *p, int dt) { return (reinterpret_cast<uintptr_t>(p) & (dt == MUON_F32 ? 3 : 1)) == 0; }
bool dtype_ok(int dt) { return dt == MUON_F32 || dt == MUON_BF16; }
muon_status status_of(cudaError_t e) { return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA; }

muon_status check_distill(const void *logits, muon_dtype zdt, int64_t ldz, const void *t_idx, muon_itype itype,
                          const void *t_val, muon_dtype tdt, const float *weights, const float *stats, int64_t N,
                          int64_t V, int64_t K, float temperature) {
  if (N < 0 || V < 1 || K < 1 || ldz < V) return MUON_ERR_INVALID_ARG;
  if (N > 0 && (logits == nullptr || t_idx == nullptr || t_val == nullptr || stats == nullptr))
    return MUON_ERR_INVALID_ARG;
  if (!(temperature >= 1e-4f && temperature <= 1e4f)) return MUON_ERR_INVALID_ARG;
  if (N > (1ll << 30) || V > (1ll << 30) || K > MAX_K) return MUON_ERR_SHAPE;
  if (!dtype_ok(zdt) || !dtype_ok(tdt) || (itype != MUON_I32 && itype != MUON_I64)) return MUON_ERR_DTYPE;
  if (!natural(logits, zdt) || !natural(t_val, tdt) || !natural(weights, MUON_F32) || !natural(stats, MUON_F32) ||
      (reinterpret_cast<uintptr_t>(t_idx) & (itype == MUON_I32 ? 3 : 7)) != 0)
    return MUON_ERR_ALIGNMENT;
  return MUON_OK;
}

DistillArgs distill_args(const void *logits, int64_t ldz, const void *t_idx, muon_itype itype, const void *t_val,
                         muon_dtype tdt, const float *weights, int64_t N, int64_t V, int64_t K, float temperature) {
  DistillArgs a{};
  a.z = logits;
  a.t_idx = t_idx;
  a.t_val = t_val;
  a.weights = weights;
  a.ldz = ldz;
  a.N = N;
  a.V = static_cast<int>(V);
  a.K = static_cast<int>(K);
  a.itype = itype;
  a.tdt = tdt;
  a.inv_t = 1.f / temperature;
  a.temp = temperature;
  a.grad_scale = 1.f;
  return a;
}

dim3 row_grid(int64_t N) { return dim3(static_cast<unsigned>(std::min<long long>(N, device_sm_count() * 64))); }

template <typename ZT, typename DT, bool GRAD>
cudaError_t launch_fwd(const DistillArgs &a, bool vec, cudaStream_t s) {
  return vec ? launch_pdl(distill_forward_kernel<ZT, DT, true, GRAD>, row_grid(a.N), dim3(THREADS), 0, s, a)
             : launch_pdl(distill_forward_kernel<ZT, DT, false, GRAD>, row_grid(a.N), dim3(THREADS), 0, s, a);
}

template <typename ZT, typename DT>
cudaError_t launch_bwd(const DistillArgs &a, bool vec, cudaStream_t s) {
  return vec ? launch_pdl(distill_backward_kernel<ZT, DT, true>, row_grid(a.N), dim3(THREADS), 0, s, a)
             : launch_pdl(distill_backward_kernel<ZT, DT, false>, row_grid(a.N), dim3(THREADS), 0, s, a);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status distill_forward(const void *logits, muon_dtype zdt, int64_t ldz, const void *t_idx, muon_itype itype,
                            const void *t_val, muon_dtype tdt, const float *weights, float *losses, float *stats,
                            int64_t N, int64_t V, int64_t K, float temperature, muon_stream_t stream) {
  muon_status st = check_distill(logits, zdt, ldz, t_idx, itype, t_val, tdt, weights, stats, N, V, K, temperature);
  if (st != MUON_OK) return st;
  if (N > 0 && losses == nullptr) return MUON_ERR_INVALID_ARG;
  if (!natural(losses, MUON_F32)) return MUON_ERR_ALIGNMENT;
  if ((st = device_check()) != MUON_OK) return st;
  if (N == 0) return MUON_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DistillArgs a = distill_args(logits, ldz, t_idx, itype, t_val, tdt, weights, N, V, K, temperature);
  a.losses = losses;
  a.stats = stats;
  const bool vec = aligned16(logits) && ldz % 8 == 0;
  launch_begin(KK_DISTILL_FWD, s);
  const cudaError_t e = zdt == MUON_F32 ? launch_fwd<float, float, false>(a, vec, s)
                                        : launch_fwd<__nv_bfloat16, float, false>(a, vec, s);
  launch_end(s);
  return status_of(e);
}

muon_status distill_backward(const void *logits, muon_dtype zdt, int64_t ldz, const void *t_idx, muon_itype itype,
                             const void *t_val, muon_dtype tdt, const float *weights, const float *stats,
                             const float *grad, void *dlogits, muon_dtype ddt, int64_t ldd, int64_t N, int64_t V,
                             int64_t K, float temperature, muon_stream_t stream) {
  muon_status st = check_distill(logits, zdt, ldz, t_idx, itype, t_val, tdt, weights, stats, N, V, K, temperature);
  if (st != MUON_OK) return st;
  if ((N > 0 && dlogits == nullptr) || ldd < V) return MUON_ERR_INVALID_ARG;
  if (!dtype_ok(ddt)) return MUON_ERR_DTYPE;
  if (dlogits == logits && N > 0 && (ddt != zdt || ldd != ldz)) return MUON_ERR_INVALID_ARG;
  if (!natural(dlogits, ddt) || !natural(grad, MUON_F32)) return MUON_ERR_ALIGNMENT;
  if ((st = device_check()) != MUON_OK) return st;
  if (N == 0) return MUON_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DistillArgs a = distill_args(logits, ldz, t_idx, itype, t_val, tdt, weights, N, V, K, temperature);
  a.stats = const_cast<float *>(stats);   // read only in this form
  a.grad = grad;
  a.dz = dlogits;
  a.ldd = ldd;
  const bool vec = aligned16(logits) && ldz % 8 == 0 && aligned16(dlogits) && ldd % 8 == 0;
  launch_begin(KK_DISTILL_BWD, s);
  cudaError_t e;
  if (zdt == MUON_F32)
    e = ddt == MUON_F32 ? launch_bwd<float, float>(a, vec, s) : launch_bwd<float, __nv_bfloat16>(a, vec, s);
  else
    e = ddt == MUON_F32 ? launch_bwd<__nv_bfloat16, float>(a, vec, s)
                        : launch_bwd<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
  launch_end(s);
  return status_of(e);
}

muon_status distill_forward_backward(const void *logits, muon_dtype zdt, int64_t ldz, const void *t_idx,
                                     muon_itype itype, const void *t_val, muon_dtype tdt, const float *weights,
                                     float grad_scale, float *losses, float *stats, void *dlogits, muon_dtype ddt,
                                     int64_t ldd, int64_t N, int64_t V, int64_t K, float temperature,
                                     muon_stream_t stream) {
  muon_status st = check_distill(logits, zdt, ldz, t_idx, itype, t_val, tdt, weights, stats, N, V, K, temperature);
  if (st != MUON_OK) return st;
  if ((N > 0 && (dlogits == nullptr || losses == nullptr)) || ldd < V || !std::isfinite(grad_scale))
    return MUON_ERR_INVALID_ARG;
  if (!dtype_ok(ddt)) return MUON_ERR_DTYPE;
  if (dlogits == logits && N > 0 && (ddt != zdt || ldd != ldz)) return MUON_ERR_INVALID_ARG;
  if (!natural(dlogits, ddt) || !natural(losses, MUON_F32)) return MUON_ERR_ALIGNMENT;
  if ((st = device_check()) != MUON_OK) return st;
  if (N == 0) return MUON_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  DistillArgs a = distill_args(logits, ldz, t_idx, itype, t_val, tdt, weights, N, V, K, temperature);
  a.losses = losses;
  a.stats = stats;
  a.dz = dlogits;
  a.ldd = ldd;
  a.grad_scale = grad_scale;
  const bool vec = aligned16(logits) && ldz % 8 == 0 && aligned16(dlogits) && ldd % 8 == 0;
  launch_begin(KK_DISTILL_STEP, s);
  cudaError_t e;
  if (zdt == MUON_F32)
    e = ddt == MUON_F32 ? launch_fwd<float, float, true>(a, vec, s) : launch_fwd<float, __nv_bfloat16, true>(a, vec, s);
  else
    e = ddt == MUON_F32 ? launch_fwd<__nv_bfloat16, float, true>(a, vec, s)
                        : launch_fwd<__nv_bfloat16, __nv_bfloat16, true>(a, vec, s);
  launch_end(s);
  return status_of(e);
}

}  // extern "C"
