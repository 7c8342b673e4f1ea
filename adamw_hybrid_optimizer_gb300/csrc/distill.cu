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
// and writes the gradient; the joint form keeps a row in shared memory between its two passes.
//
// A row is cut into granules of eight logits on 16-byte boundaries of memory: a row whose start is not on one (an odd
// vocabulary) has a short granule at each end, and everything between is whole vectors.
//
//   distill_forward_kernel   a cluster of 1 to 8 blocks per row, each with a slice of it: few rows still fill the GPU
//   distill_backward_kernel  a block per row and slice
//   distill_joint_kernel     a cluster per row, the slices in shared memory; while a thread writes the gradient of a
//                            granule it starts the copy of the next row's granule into the same place
//   distill_reread_kernel    the joint form for rows that do not fit: a block per row, which reads it twice
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <mutex>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int MAX_K = 1024;
constexpr int MAX_CLUSTER = 8;
constexpr float LOG2E = 1.4426950408889634f;

struct DistillArgs {
  const void *z;              // N x V student logits; dz may be the same buffer
  const void *t_idx, *t_val;  // N x K
  const float *weights, *grad;
  float *losses, *stats;      // stats: N x 2 (m, l), written by the forward forms, read by backward
  void *dz;
  long long ldz, ldd, N;
  int V, K, itype, tdt, slices;
  float inv_t, temp, grad_scale;
};

// exp(x * c), c = log2(e) / T; the difference x is taken in the logits' own unit, where it is exact or nearly so
__device__ __forceinline__ float exp_scaled(float x, float c) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * c));
  return y;
}

// exp_scaled of both differences from m
__device__ __forceinline__ float2 exp2_scaled(float2 x, float m, float c) {
  const float2 v = __fmul2_rn(__fadd2_rn(x, make_float2(-m, -m)), make_float2(c, c));
  float2 y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.x) : "f"(v.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y.y) : "f"(v.y));
  return y;
}

// ------------------------------------------------------------------------------------------ running softmax

// A maximum and the sum of exp((x - m) c) below it.
struct Soft {
  float m, s;
};

__device__ __forceinline__ Soft merge(const Soft &a, const Soft &b, float c) {
  const float m = fmaxf(a.m, b.m), ref = m == -INFINITY ? 0.f : m;
  return {m, fmaf(a.s, exp_scaled(a.m - ref, c), b.s * exp_scaled(b.m - ref, c))};
}

__device__ __forceinline__ Soft warp_merge(Soft a, float c) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    a = merge(a, {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, c);
  return a;
}

// A thread's running sum, as a pair.
struct Run {
  float m = -INFINITY;
  float2 s = {0.f, 0.f};
  // Eight logits; a granule of -inf leaves the sum alone.
  __device__ __forceinline__ void add(const Vals<8> &o, float c) {
    const float mx = fmaxf(fmaxf(fmaxf(o.p[0].x, o.p[0].y), fmaxf(o.p[1].x, o.p[1].y)),
                           fmaxf(fmaxf(o.p[2].x, o.p[2].y), fmaxf(o.p[3].x, o.p[3].y)));
    if (mx > m) {
      const float f = exp_scaled(m - mx, c);
      s = __fmul2_rn(s, make_float2(f, f));
      m = mx;
    }
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < 4; ++i) s = __fadd2_rn(s, exp2_scaled(o.p[i], ref, c));
  }
  __device__ __forceinline__ Soft soft() const { return {m, s.x + s.y}; }
};

// si * exp((z - m) / T) of eight logits
__device__ __forceinline__ Vals<8> grad_of(Vals<8> o, float m, float c, float si) {
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = __fmul2_rn(exp2_scaled(o.p[i], m, c), make_float2(si, si));
  return o;
}

// ------------------------------------------------------------------------------------------ granules

// Granules of one row. VEC: granule g holds logits 8 g - shift + e, where shift is the row's start past a boundary
// (the same for z and dz, whose pitches differ by a multiple of eight); otherwise shift is 0 and every access is
// of one element. All granules but the first and the last (the edges) are whole.
struct Granules {
  int shift, count, V;
  __device__ __forceinline__ int first(int g) const { return 8 * g - shift; }
  __device__ __forceinline__ bool has(int g, int e) const {
    return first(g) + e >= 0 && first(g) + e < V;
  }
  __device__ __forceinline__ bool whole(int g) const { return first(g) >= 0 && first(g) + 8 <= V; }
};

template <bool VEC>
__device__ __forceinline__ Granules granules(long long row, long long ld, int V) {
  const int shift = VEC ? static_cast<int>((row * ld) & 7) : 0;
  return {shift, (V + shift + 7) / 8, V};
}

// The part of a row that block `rank` of `slices` has: granules [g0, g1), of which [inner, inner + n) are not edges.
// Inner granule inner + i belongs to thread i mod THREADS; the row's first edge to thread HEAD and its last to thread
// TAIL, of two warps.
struct Slice {
  int g0, g1, inner, n;
  bool head, tail;
};
constexpr int HEAD = 0, TAIL = 32;

__device__ __forceinline__ Slice slice_of(const Granules &G, int rank, int slices) {
  Slice s;
  s.g0 = static_cast<int>(static_cast<long long>(G.count) * rank / slices);
  s.g1 = static_cast<int>(static_cast<long long>(G.count) * (rank + 1) / slices);
  s.inner = max(s.g0, 1);
  s.n = max(min(s.g1, G.count - 1) - s.inner, 0);
  s.head = s.g0 == 0 && s.g1 > 0;
  s.tail = s.g1 == G.count && s.g1 > s.g0 && G.count > 1;
  return s;
}

template <typename T>
__device__ __forceinline__ T neg_inf();
template <>
__device__ __forceinline__ float neg_inf<float>() { return -INFINITY; }
template <>
__device__ __forceinline__ __nv_bfloat16 neg_inf<__nv_bfloat16>() { return __ushort_as_bfloat16(0xff80); }

// Places that the row does not have read as -inf.
template <typename T, bool VEC>
__device__ __forceinline__ void load_granule(const T *p, const Granules &G, int g, Raw<T, 8> &r) {
  if (VEC && G.whole(g)) {
    r.load(p + G.first(g));
    return;
  }
  r.clear();
#pragma unroll
  for (int e = 0; e < 8; ++e) r.put(e, G.has(g, e) ? p[G.first(g) + e] : neg_inf<T>());
}

template <typename T, bool VEC>
__device__ __forceinline__ void store_granule(T *p, const Granules &G, int g, const Vals<8> &o) {
  if (VEC && G.whole(g)) {
    store_vals(p + G.first(g), o);
    return;
  }
  const float f[8] = {o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y, o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (G.has(g, e)) store1(p, G.first(g) + e, f[e]);
}

template <typename DT, bool VEC>
__device__ __forceinline__ void zero_granules(DT *dz, const Granules &G, const Slice &S) {
  Vals<8> o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = make_float2(0.f, 0.f);
  for (int g = S.g0 + threadIdx.x; g < S.g1; g += THREADS) store_granule<DT, VEC>(dz, G, g, o);
}

// A thread's granules of a slice, in batches: while one is used the loads of the next are in flight. run calls
// inner(i, values) and edge(g, values).
template <typename ZT, bool VEC>
struct Stream {
  static constexpr int U = sizeof(ZT) == 2 ? 4 : 2;
  const ZT *z;
  const ZT *next;   // of the thread's next batch to fetch
  const Granules &G;
  const Slice &S;
  int fetched, used;
  Raw<ZT, 8> a[U], b[U], e;
  __device__ __forceinline__ void fetch(Raw<ZT, 8> *r) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (fetched + u * THREADS < S.n) {
        if constexpr (VEC) r[u].load(next + u * THREADS * 8);
        else load_granule<ZT, false>(z, G, S.inner + fetched + u * THREADS, r[u]);
      }
    fetched += U * THREADS;
    next += U * THREADS * 8;
  }
  __device__ __forceinline__ Stream(const ZT *z_, const Granules &G_, const Slice &S_)
      : z(z_), next(z_ + G_.first(S_.inner) + 8 * threadIdx.x), G(G_), S(S_), fetched(threadIdx.x), used(threadIdx.x) {
    if (S.head && threadIdx.x == HEAD) load_granule<ZT, false>(z, G, 0, e);
    if (S.tail && threadIdx.x == TAIL) load_granule<ZT, false>(z, G, G.count - 1, e);
    fetch(a);
  }
  template <typename F>
  __device__ __forceinline__ void use(const Raw<ZT, 8> *r, F &&inner) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (used + u * THREADS < S.n) inner(used + u * THREADS, r[u].get());
    used += U * THREADS;
  }
  template <typename F, typename E>
  __device__ __forceinline__ void run(F &&inner, E &&edge) {
    while (used < S.n) {
      fetch(b);
      use(a, inner);
      if (used >= S.n) break;
      fetch(a);
      use(b, inner);
    }
    if (S.head && threadIdx.x == HEAD) edge(0, e.get());
    if (S.tail && threadIdx.x == TAIL) edge(G.count - 1, e.get());
  }
};

// ------------------------------------------------------------------------------------------ the teacher's entries

// A row's entries in (dynamic) shared memory, K of each: index (-1: none), value, and the student's logit there, read
// before dz overwrites it (for indices in [lo, hi) only: those of the block's slice, where others may be writing).
struct Teacher {
  int *idx;
  float *t, *z;
};

__device__ __forceinline__ Teacher teacher_at(void *smem, int K) {
  int *idx = static_cast<int *>(smem);
  const int pad = (K + 3) & ~3;
  return {idx, reinterpret_cast<float *>(idx + pad), reinterpret_cast<float *>(idx + 2 * pad)};
}
constexpr size_t teacher_bytes(int K) { return static_cast<size_t>((K + 3) & ~3) * 12; }

// One entry as loaded. ok: it is valid.
struct Entry {
  long long id;
  float t, z;
  bool ok;
};

__device__ __forceinline__ Entry load_entry(const DistillArgs &a, long long row, int k) {
  const long long at = row * a.K + k;
  Entry e;
  e.id = a.itype == MUON_I32 ? static_cast<long long>(static_cast<const int *>(a.t_idx)[at])
                             : static_cast<const long long *>(a.t_idx)[at];
  e.t = a.tdt == MUON_F32 ? static_cast<const float *>(a.t_val)[at]
                          : __bfloat162float(static_cast<const __nv_bfloat16 *>(a.t_val)[at]);
  e.ok = e.id >= 0 && e.id < a.V && !(e.t == -INFINITY);   // a NaN is kept, and shows in the loss
  return e;
}

template <typename ZT, bool ALL>
__device__ __forceinline__ float entry_logit(const Entry &e, const ZT *z, int lo, int hi) {
  return e.ok && (ALL || (e.id >= lo && e.id < hi)) ? load1(z, e.id) : 0.f;
}

// Puts entry k in its place and adds it to the thread's part of the teacher's sum. A NaN value goes into the sum as
// it is.
__device__ __forceinline__ void put_entry(const Teacher &s, int k, const Entry &e, float c, Soft &sum) {
  s.idx[k] = e.ok ? static_cast<int>(e.id) : -1;
  s.t[k] = e.t;
  s.z[k] = e.z;
  if (e.ok) sum = merge(sum, {e.t, e.t == e.t ? 1.f : e.t}, c);
}

// A thread's first entry (k = threadIdx.x) is loaded ahead; the rest of a long list, and the padding that
// subtract_teacher's vectors read, when the first is put.
template <typename ZT, bool ALL>
__device__ __forceinline__ Soft put_teacher(const DistillArgs &a, long long row, const ZT *z, const Teacher &s, int lo,
                                            int hi, float c, const Entry &ahead) {
  Soft sum{-INFINITY, 0.f};
  if (static_cast<int>(threadIdx.x) < a.K) put_entry(s, threadIdx.x, ahead, c, sum);
  for (int k = THREADS + threadIdx.x; k < a.K; k += THREADS) {
    Entry e = load_entry(a, row, k);
    e.z = entry_logit<ZT, ALL>(e, z, lo, hi);
    put_entry(s, k, e, c, sum);
  }
  for (int k = a.K + threadIdx.x; k < ((a.K + 3) & ~3); k += THREADS) s.idx[k] = -1;
  return sum;
}

// One exchange for the student's and the teacher's sums: every warp puts its pair, and after one barrier every warp
// merges all of them. Calls alternate between two buffers.
struct BlockRed {
  float4 buf[2][WARPS];
  float loss[2][WARPS];
};

// A thread can write a buffer again only after the barrier of the call in between, which every reader of that buffer
// has reached.
__device__ __forceinline__ void merge_all(BlockRed &r, int turn, float c, Soft &student, Soft &teacher) {
  student = warp_merge(student, c);
  teacher = warp_merge(teacher, c);
  const int lane = threadIdx.x % 32;
  if (lane == 0) r.buf[turn][threadIdx.x / 32] = make_float4(student.m, student.s, teacher.m, teacher.s);
  __syncthreads();
  const float4 v = lane < WARPS ? r.buf[turn][lane] : make_float4(-INFINITY, 0.f, -INFINITY, 0.f);
  student = warp_merge({v.x, v.y}, c);
  teacher = warp_merge({v.z, v.w}, c);
}

// The thread's part of sum_k q_k (log q_k - (z_k - m) / T); an entry whose q is 0 adds nothing, whatever the student
// gives it.
__device__ __forceinline__ float loss_part(const DistillArgs &a, const Teacher &s, const Soft &teacher, float m,
                                           float c) {
  const float tl = logf(teacher.s), tinv = 1.f / teacher.s;
  float part = 0.f;
  for (int k = threadIdx.x; k < a.K; k += THREADS) {
    if (s.idx[k] < 0) continue;
    const float d = s.t[k] - teacher.m;
    const float q = exp_scaled(d, c) * tinv;
    if (!(q == 0.f)) part = fmaf(q, (d * a.inv_t - tl) - (s.z[k] - m) * a.inv_t, part);
  }
  return warp_sum(part);
}

__device__ __forceinline__ void store_loss(const DistillArgs &a, long long row, float w, const float *parts,
                                           const Soft &student) {
  float kl = 0.f;
  for (int i = 0; i < WARPS; ++i) kl += parts[i];
  const float l = logf(student.s);
  a.losses[row] = w * a.temp * a.temp * (kl + l);
  a.stats[2 * row] = student.m;
  a.stats[2 * row + 1] = l;
}

__device__ __forceinline__ void store_nothing(const DistillArgs &a, long long row) {
  a.losses[row] = 0.f;
  a.stats[2 * row] = 0.f;
  a.stats[2 * row + 1] = 0.f;
}

// Where the p parts of columns [lo, hi) are written: the first entry of each index there subtracts the q of all
// entries of that index.
template <typename DT>
__device__ __forceinline__ void subtract_teacher(const DistillArgs &a, const Teacher &s, DT *dz, int lo, int hi,
                                                 float c, float m, float inv, float scale, const Soft &teacher) {
  const float tinv = 1.f / teacher.s;
  for (int k = threadIdx.x; k < a.K; k += THREADS) {
    const int id = s.idx[k];
    if (id < lo || id >= hi) continue;   // absent entries are -1, below every lo
    bool first = true;
    float q = 0.f;
    for (int i = 0; i < a.K; i += 4) {
      const int4 v = *reinterpret_cast<const int4 *>(s.idx + i);
      if (v.x != id && v.y != id && v.z != id && v.w != id) continue;
      const int u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (u[e] != id) continue;
        if (i + e < k) first = false;
        q += exp_scaled(s.t[i + e] - teacher.m, c) * tinv;
      }
    }
    if (first) store1(dz, id, scale * (exp_scaled(s.z[k] - m, c) * inv - q));
  }
}

// A row of nothing but -inf has no softmax.
__device__ __forceinline__ void no_softmax(Soft &student) {
  if (student.m == -INFINITY) student.s = NAN;
}

// ------------------------------------------------------------------------------------------ clusters

__device__ __forceinline__ float2 load_remote(const float2 *p, unsigned rank) {
  const uint32_t at = mapa_shared(smem_u32(p), rank);
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}

// The student's sums of all slices of the row: every block puts its own and reads the others', in rank order, so that
// all blocks get the same bits. `put` alternates between two places like the block's own exchange.
__device__ __forceinline__ void merge_cluster(float2 *put, int blocks, float c, Soft &student) {
  if (threadIdx.x == 0) *put = make_float2(student.m, student.s);
  cluster_sync();
  Soft all{-INFINITY, 0.f};
  for (int r = 0; r < blocks; ++r) {
    const float2 v = load_remote(put, r);
    all = merge(all, {v.x, v.y}, c);
  }
  student = all;
}

// ------------------------------------------------------------------------------------------ kernels

__device__ __forceinline__ float weight_of(const DistillArgs &a, long long row) {
  return a.weights != nullptr ? a.weights[row] : 1.f;
}

// dz of a slice without the q part: si * exp((z - m) / T).
template <typename ZT, typename DT, bool VEC>
__device__ __forceinline__ void write_grad(Stream<ZT, VEC> &stream, DT *dz, const Granules &G, const Slice &S, float m,
                                           float c, float si) {
  DT *inner = dz + G.first(S.inner);
  stream.run(
      [&](int i, const Vals<8> &o) {
        if constexpr (VEC) store_vals(inner + 8 * i, grad_of(o, m, c, si));
        else store_granule<DT, false>(dz, G, S.inner + i, grad_of(o, m, c, si));
      },
      [&](int g, const Vals<8> &o) { store_granule<DT, false>(dz, G, g, grad_of(o, m, c, si)); });
}

template <typename ZT, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) distill_forward_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed red;
  __shared__ float2 put;
  const Teacher s = teacher_at(smem, a.K);
  const float c = a.inv_t * LOG2E;
  const int slices = a.slices, rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long long row = blockIdx.x / slices;
  const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
  const Granules G = granules<VEC>(row, a.ldz, a.V);
  const Slice S = slice_of(G, rank, slices);
  const bool entry = rank == 0 && static_cast<int>(threadIdx.x) < a.K;
  const float w = weight_of(a, row);
  Entry e{};
  if (entry) e = load_entry(a, row, threadIdx.x);
  if (w == 0.f) {   // the same for the whole cluster
    if (rank == 0 && threadIdx.x == 0) store_nothing(a, row);
    return;
  }
  Stream<ZT, VEC> stream(z, G, S);
  if (entry) e.z = entry_logit<ZT, true>(e, z, 0, 0);
  Run run;
  auto add = [&](int, const Vals<8> &o) { run.add(o, c); };
  stream.run(add, add);
  Soft student = run.soft(), teacher{-INFINITY, 0.f};
  if (rank == 0) teacher = put_teacher<ZT, true>(a, row, z, s, 0, 0, c, e);
  merge_all(red, 0, c, student, teacher);
  if (slices > 1) merge_cluster(&put, slices, c, student);
  if (rank == 0) {
    no_softmax(student);
    const float part = loss_part(a, s, teacher, student.m, c);
    if (threadIdx.x % 32 == 0) red.loss[0][threadIdx.x / 32] = part;
    __syncthreads();
    if (threadIdx.x == 0) {
      if (teacher.s == 0.f) store_nothing(a, row);
      else store_loss(a, row, w, red.loss[0], student);
    }
  }
  if (slices > 1) cluster_sync();   // no block leaves while another reads its shared memory
}

template <typename ZT, typename DT, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) distill_backward_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed red;
  const Teacher s = teacher_at(smem, a.K);
  const float c = a.inv_t * LOG2E;
  const long long row = blockIdx.x / a.slices;
  const int rank = static_cast<int>(blockIdx.x - row * a.slices);
  const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
  DT *dz = static_cast<DT *>(a.dz) + row * a.ldd;
  const Granules G = granules<VEC>(row, a.ldz, a.V);
  const Slice S = slice_of(G, rank, a.slices);
  const int lo = max(G.first(S.g0), 0), hi = min(G.first(S.g1), a.V);
  const float w = weight_of(a, row);
  Entry e{};
  if (static_cast<int>(threadIdx.x) < a.K) e = load_entry(a, row, threadIdx.x);
  if (w == 0.f) {
    zero_granules<DT, VEC>(dz, G, S);
    return;
  }
  Stream<ZT, VEC> stream(z, G, S);
  const float m = a.stats[2 * row], l = a.stats[2 * row + 1], up = a.grad != nullptr ? a.grad[row] : 1.f;
  if (static_cast<int>(threadIdx.x) < a.K) e.z = entry_logit<ZT, false>(e, z, lo, hi);
  Soft teacher = put_teacher<ZT, false>(a, row, z, s, lo, hi, c, e), student{-INFINITY, 0.f};
  merge_all(red, 0, c, student, teacher);   // its barrier also ends the reads of z that dz may overwrite
  if (teacher.s == 0.f) {
    zero_granules<DT, VEC>(dz, G, S);
    return;
  }
  const float inv = expf(-l), scale = up * w * a.temp;
  write_grad<ZT, DT, VEC>(stream, dz, G, S, m, c, scale * inv);
  __syncthreads();
  subtract_teacher(a, s, dz, lo, hi, c, m, inv, scale, teacher);
}

// The joint form without room for the row: a block per row, whose second reading is left to L2.
template <typename ZT, typename DT, bool VEC>
__global__ void __launch_bounds__(THREADS, 2) distill_reread_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed red;
  const Teacher s = teacher_at(smem, a.K);
  const float c = a.inv_t * LOG2E;
  const long long row = blockIdx.x;
  const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
  DT *dz = static_cast<DT *>(a.dz) + row * a.ldd;
  const Granules G = granules<VEC>(row, a.ldz, a.V);
  const Slice S = slice_of(G, 0, 1);
  const float w = weight_of(a, row);
  Entry e{};
  if (static_cast<int>(threadIdx.x) < a.K) e = load_entry(a, row, threadIdx.x);
  if (w == 0.f) {
    if (threadIdx.x == 0) store_nothing(a, row);
    zero_granules<DT, VEC>(dz, G, S);
    return;
  }
  if (static_cast<int>(threadIdx.x) < a.K) e.z = entry_logit<ZT, true>(e, z, 0, 0);
  Run run;
  {
    Stream<ZT, VEC> stream(z, G, S);
    auto add = [&](int, const Vals<8> &o) { run.add(o, c); };
    stream.run(add, add);
  }
  Soft student = run.soft(), teacher = put_teacher<ZT, true>(a, row, z, s, 0, 0, c, e);
  merge_all(red, 0, c, student, teacher);
  if (teacher.s == 0.f) {
    if (threadIdx.x == 0) store_nothing(a, row);
    zero_granules<DT, VEC>(dz, G, S);
    return;
  }
  no_softmax(student);
  const float part = loss_part(a, s, teacher, student.m, c);
  if (threadIdx.x % 32 == 0) red.loss[0][threadIdx.x / 32] = part;
  const float scale = a.grad_scale * w * a.temp, inv = 1.f / student.s;
  Stream<ZT, VEC> stream(z, G, S);
  write_grad<ZT, DT, VEC>(stream, dz, G, S, student.m, c, scale * inv);
  __syncthreads();
  if (threadIdx.x == 0) store_loss(a, row, w, red.loss[0], student);
  subtract_teacher(a, s, dz, 0, a.V, c, student.m, inv, scale, teacher);
}

// ------------------------------------------------------------------------------------------ joint form

// The slice in shared memory: inner granule i at place i, the row's first edge at place room - 2 and its last at
// room - 1, in 16-byte pieces `room` apart, so that a warp's accesses to one piece are contiguous. Every place is
// written and read by one thread only, so a thread's own wait is all the ordering it needs.
template <typename ZT>
struct Kept {
  static constexpr int PIECES = static_cast<int>(sizeof(ZT)) / 2;
  uint4 *base;
  int room;
  __device__ __forceinline__ void fetch(int at, const ZT *src) const {
#pragma unroll
    for (int p = 0; p < PIECES; ++p) copy_async<16>(base + p * room + at, reinterpret_cast<const uint4 *>(src) + p);
  }
  __device__ __forceinline__ Vals<8> get(int at) const {
    Raw<ZT, 8> r;
#pragma unroll
    for (int p = 0; p < PIECES; ++p) {
      const uint4 u = base[p * room + at];
      r.w[4 * p] = u.x, r.w[4 * p + 1] = u.y, r.w[4 * p + 2] = u.z, r.w[4 * p + 3] = u.w;
    }
    return r.get();
  }
  // An edge that the row has only part of is copied whole where the rest of it lies in the rows around (V >= 8), whose
  // values edge() leaves out; only the ends of the whole matrix are read element by element.
  __device__ __forceinline__ void fetch_edges(const ZT *z, const Granules &G, const Slice &S, bool first_row,
                                              bool last_row) const {
    const bool head = S.head && threadIdx.x == HEAD;
    if (!head && !(S.tail && threadIdx.x == TAIL)) return;
    const int g = head ? 0 : G.count - 1, at = room - (head ? 2 : 1);
    if ((G.first(g) >= 0 || !first_row) && (G.first(g) + 8 <= G.V || !last_row)) {
      fetch(at, z + G.first(g));
    } else {
      Raw<ZT, 8> r;
      load_granule<ZT, false>(z, G, g, r);
#pragma unroll
      for (int p = 0; p < PIECES; ++p)
        base[p * room + at] = make_uint4(r.w[4 * p], r.w[4 * p + 1], r.w[4 * p + 2], r.w[4 * p + 3]);
    }
  }
  // f(g, values) of the edges that are the thread's
  template <typename F>
  __device__ __forceinline__ void edges(const Granules &G, const Slice &S, F &&f) const {
    const bool head = S.head && threadIdx.x == HEAD;
    if (!head && !(S.tail && threadIdx.x == TAIL)) return;
    const int g = head ? 0 : G.count - 1;
    Vals<8> o = get(room - (head ? 2 : 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!G.has(g, 2 * i)) o.p[i].x = -INFINITY;
      if (!G.has(g, 2 * i + 1)) o.p[i].y = -INFINITY;
    }
    f(g, o);
  }
};

template <typename ZT, typename DT>
__global__ void __launch_bounds__(THREADS, 2) distill_joint_kernel(const DistillArgs a, int room) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed red;
  __shared__ float2 put[2];
  const Kept<ZT> kept{reinterpret_cast<uint4 *>(smem), room};
  unsigned char *entries = smem + static_cast<size_t>(room) * sizeof(ZT) * 8;
  const float c = a.inv_t * LOG2E;
  const int slices = a.slices, rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long long step = gridDim.x / slices;
  long long row = blockIdx.x / slices;
  int turn = 0;
  const bool entry = static_cast<int>(threadIdx.x) < a.K;
  const int t = threadIdx.x;
  auto z_of = [&](long long r) { return static_cast<const ZT *>(a.z) + r * a.ldz; };
  float w_next = weight_of(a, row);   // the grid has no more clusters than there are rows
  Entry e_next{};
  if (entry) e_next = load_entry(a, row, t);
  Granules G_next = granules<true>(row, a.ldz, a.V);
  Slice S_next = slice_of(G_next, rank, slices);
  if (w_next != 0.f) {
    const ZT *src = z_of(row) + G_next.first(S_next.inner) + 8 * t;
    for (int i = t; i < S_next.n; i += THREADS, src += 8 * THREADS) kept.fetch(i, src);
    kept.fetch_edges(z_of(row), G_next, S_next, row == 0, row + 1 == a.N);
  }
  copy_async_commit();
  if (entry) e_next.z = entry_logit<ZT, true>(e_next, z_of(row), 0, 0);
  for (; row < a.N; row += step) {
    DT *dz = static_cast<DT *>(a.dz) + row * a.ldd;
    const Granules G = G_next;
    const Slice S = S_next;
    const float w = w_next;
    const Entry e = e_next;
    // the next row: its weight and entries now, its logits and the entries' own as this one's gradient is written
    const long long next = row + step;
    const bool more = next < a.N;
    if (more) {
      w_next = weight_of(a, next);
      if (entry) e_next = load_entry(a, next, t);
    }
    G_next = granules<true>(next, a.ldz, a.V);
    S_next = slice_of(G_next, rank, slices);
    const ZT *zn = z_of(next);
    const bool used = w != 0.f;   // the same for the whole cluster
    const Teacher s = teacher_at(entries + turn * teacher_bytes(a.K), a.K);
    Soft teacher{-INFINITY, 0.f}, student{-INFINITY, 0.f};
    if (used) {
      Run run;
      copy_async_wait<0>();
#pragma unroll 2
      for (int i = t; i < S.n; i += THREADS) run.add(kept.get(i), c);
      kept.edges(G, S, [&](int, const Vals<8> &o) { run.add(o, c); });
      student = run.soft();
      teacher = put_teacher<ZT, true>(a, row, z_of(row), s, 0, 0, c, e);
      merge_all(red, turn, c, student, teacher);
      if (slices > 1) merge_cluster(&put[turn], slices, c, student);
    }
    const bool wanted = more && w_next != 0.f;
    const int nn = wanted ? S_next.n : 0;
    const ZT *src = zn + G_next.first(S_next.inner) + 8 * t;
    if (more && entry) e_next.z = entry_logit<ZT, true>(e_next, zn, 0, 0);
    if (!used || teacher.s == 0.f) {
      if (rank == 0 && t == 0) store_nothing(a, row);
      zero_granules<DT, true>(dz, G, S);
      for (int i = t; i < nn; i += THREADS, src += 8 * THREADS) kept.fetch(i, src);
      if (wanted) kept.fetch_edges(zn, G_next, S_next, false, next + 1 == a.N);
      copy_async_commit();
      if (used) turn ^= 1;
      continue;
    }
    no_softmax(student);
    if (rank == 0) {
      const float part = loss_part(a, s, teacher, student.m, c);
      if (t % 32 == 0) red.loss[turn][t / 32] = part;
    }
    const float m = student.m, scale = a.grad_scale * w * a.temp, inv = 1.f / student.s, si = scale * inv;
    // a granule's values have gone into the store when its place is given to the next row's
    kept.edges(G, S, [&](int g, const Vals<8> &o) { store_granule<DT, false>(dz, G, g, grad_of(o, m, c, si)); });
    if (wanted) kept.fetch_edges(zn, G_next, S_next, false, next + 1 == a.N);
    DT *dst = dz + G.first(S.inner) + 8 * t;
    int i = t;
#pragma unroll 2
    for (; i < min(S.n, nn); i += THREADS, src += 8 * THREADS, dst += 8 * THREADS) {
      store_vals(dst, grad_of(kept.get(i), m, c, si));
      kept.fetch(i, src);
    }
    for (int j = i; j < S.n; j += THREADS, dst += 8 * THREADS) store_vals(dst, grad_of(kept.get(j), m, c, si));
    for (; i < nn; i += THREADS, src += 8 * THREADS) kept.fetch(i, src);
    copy_async_commit();
    // what follows may run beside the next row, which has its own half of everything shared
    __syncthreads();
    if (rank == 0 && t == 0) store_loss(a, row, w, red.loss[turn], student);
    subtract_teacher(a, s, dz, max(G.first(S.g0), 0), min(G.first(S.g1), a.V), c, m, inv, scale, teacher);
    turn ^= 1;
  }
  if (slices > 1) cluster_sync();   // no block leaves while another reads its shared memory
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
  if (N > (1ll << 30) || V > (1ll << 30) || N * V > (1ll << 40) || K > MAX_K) return MUON_ERR_SHAPE;
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

// A dependent launch of clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), long long blocks, int cluster, size_t smem, cudaStream_t s,
                            Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

// Blocks per row: as many as it takes to give every multiprocessor `per_sm` blocks, each with at least `least` logits.
int row_slices(const DistillArgs &a, int per_sm, int least, int most) {
  const long long want = static_cast<long long>(device_sm_count()) * per_sm;
  int n = 1;
  while (n < most && a.N * n < want && a.V / (2 * n) >= least) n *= 2;
  return n;
}

template <typename ZT>
cudaError_t launch_fwd(DistillArgs a, bool vec, cudaStream_t s) {
  a.slices = row_slices(a, 2, 4096, MAX_CLUSTER);
  const size_t smem = teacher_bytes(a.K);
  return vec ? launch_clusters(distill_forward_kernel<ZT, true>, a.N * a.slices, a.slices, smem, s, a)
             : launch_clusters(distill_forward_kernel<ZT, false>, a.N * a.slices, a.slices, smem, s, a);
}

template <typename ZT, typename DT>
cudaError_t launch_bwd(DistillArgs a, bool vec, cudaStream_t s) {
  // a block's start (its teacher entries) is paid back by some 32 Ki logits
  a.slices = row_slices(a, 3, 4096, MAX_CLUSTER);
  while (a.V / a.slices > 65536) a.slices *= 2;
  const size_t smem = teacher_bytes(a.K);
  const dim3 grid(static_cast<unsigned>(a.N * a.slices)), block(THREADS);
  return vec ? launch_pdl(distill_backward_kernel<ZT, DT, true>, grid, block, smem, s, a)
             : launch_pdl(distill_backward_kernel<ZT, DT, false>, grid, block, smem, s, a);
}

constexpr int SM_SHARED = 227 * 1024;          // what blocks of one multiprocessor can have together
constexpr int BLOCK_SHARED = 2048;             // a block's static share and the system's, rounded up
std::mutex g_joint_mu;

// Clusters of this shape that the GPU holds at once (a persistent grid of more would leave the rest for last).
template <typename ZT, typename DT>
cudaError_t joint_clusters(int cluster, size_t smem, int *n) {
  static int cached[MAX_CLUSTER + 1][3];       // by cluster size and blocks per multiprocessor; 0: not asked yet
  auto kernel = distill_joint_kernel<ZT, DT>;
  std::lock_guard<std::mutex> lk(g_joint_mu);
  const int per_sm = static_cast<int>(std::min<size_t>(2, SM_SHARED / (smem + BLOCK_SHARED)));
  int &c = cached[cluster][per_sm];
  if (c == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         SM_SHARED - BLOCK_SHARED);
    if (e != cudaSuccess) return e;
    if (cluster == 1) {
      c = device_sm_count() * per_sm;
    } else {
      cudaLaunchConfig_t cfg = {};
      cfg.gridDim = dim3(static_cast<unsigned>(cluster));
      cfg.blockDim = dim3(THREADS);
      cfg.dynamicSmemBytes = smem;
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = static_cast<unsigned>(cluster);
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      e = cudaOccupancyMaxActiveClusters(&c, kernel, &cfg);
      if (e != cudaSuccess) {
        c = 0;
        return e;
      }
    }
  }
  *n = std::max(1, c);
  return cudaSuccess;
}

template <typename ZT, typename DT>
cudaError_t launch_step(DistillArgs a, bool vec, cudaStream_t s) {
  const size_t entries = teacher_bytes(a.K), both = 2 * entries;
  // slices of at most half a multiprocessor's shared memory, or of all of it where eight of those are too few
  const size_t granule = 8 * sizeof(ZT), granules = (static_cast<size_t>(a.V) + 7 + 7) / 8;
  const size_t half = (SM_SHARED / 2 - BLOCK_SHARED - both) / granule, all = (SM_SHARED - BLOCK_SHARED - both) / granule;
  int slices = row_slices(a, 2, 4096, MAX_CLUSTER);
  // a slice's granules and two places for edges
  while (slices < MAX_CLUSTER && (granules + slices - 1) / slices + 2 > half) ++slices;
  const size_t room = (granules + slices - 1) / slices + 2;
  if (!vec || room > all || a.V < 8) {
    const dim3 grid(static_cast<unsigned>(a.N)), block(THREADS);
    return vec ? launch_pdl(distill_reread_kernel<ZT, DT, true>, grid, block, entries, s, a)
               : launch_pdl(distill_reread_kernel<ZT, DT, false>, grid, block, entries, s, a);
  }
  a.slices = slices;
  const size_t smem = room * granule + both;
  int clusters = 0;
  const cudaError_t e = joint_clusters<ZT, DT>(slices, smem, &clusters);
  if (e != cudaSuccess) return e;
  return launch_clusters(distill_joint_kernel<ZT, DT>, std::min<long long>(a.N, clusters) * slices, slices, smem, s, a,
                         static_cast<int>(room));
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
  const bool vec = aligned16(logits);
  launch_begin(KK_DISTILL_FWD, s);
  const cudaError_t e = zdt == MUON_F32 ? launch_fwd<float>(a, vec, s)
                                        : launch_fwd<__nv_bfloat16>(a, vec, s);
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
  const bool vec = aligned16(logits) && aligned16(dlogits) && (ldz - ldd) % 8 == 0;
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
  const bool vec = aligned16(logits) && aligned16(dlogits) && (ldz - ldd) % 8 == 0;
  launch_begin(KK_DISTILL_STEP, s);
  cudaError_t e;
  if (zdt == MUON_F32)
    e = ddt == MUON_F32 ? launch_step<float, float>(a, vec, s) : launch_step<float, __nv_bfloat16>(a, vec, s);
  else
    e = ddt == MUON_F32 ? launch_step<__nv_bfloat16, float>(a, vec, s)
                        : launch_step<__nv_bfloat16, __nv_bfloat16>(a, vec, s);
  launch_end(s);
  return status_of(e);
}

}  // extern "C"
