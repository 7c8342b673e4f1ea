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
// and writes the gradient; the joint form reads a row twice, the second time from L2 as far as the rows on their way at
// once and their gradients fit it.
//
// A row is cut into granules of eight logits (four where a matrix is fp32) on boundaries of memory: a row whose start
// is not on one (an odd vocabulary) has a short granule at each end, and everything between is whole vectors.
//
//   distill_forward_kernel   losses and stats: a block per row, or a cluster of 2 to 8 where there are few rows
//   distill_backward_kernel  the gradient: a block per row and slice of a row
//   distill_joint_kernel     both: blocks and clusters as in the forward kernel
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

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
  int V, K, itype, tdt, slices, bits;   // bits: of the table of the teacher's indices
  float inv_t, temp, grad_scale;
};

// exp(x * c), c = log2(e) / T; the difference x is taken in the logits' own unit, where it is exact or nearly so. The
// product is rounded before the exponential, which is good to two units in the last place: a relative error of 2^-22, and
// of |x / T| 2^-23 beside it (3e-6 at a weight of exp(-25)). Results below 2^-126 are 0, as weights too small to be seen
// beside the largest, 1.
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

// Over all lanes, or over groups of LANES that hold copies of the same values.
template <int LANES>
__device__ __forceinline__ Soft warp_merge(Soft a, float c) {
#pragma unroll
  for (int o = LANES / 2; o > 0; o >>= 1)
    a = merge(a, {__shfl_xor_sync(0xffffffffu, a.m, o), __shfl_xor_sync(0xffffffffu, a.s, o)}, c);
  return a;
}

// A thread's running sum, as a pair.
struct Run {
  float m = -INFINITY;
  float2 s = {0.f, 0.f};
  // A granule of -inf leaves the sum alone.
  template <int N>
  __device__ __forceinline__ void add(const Vals<N> &o, float c) {
    float mx = fmaxf(o.p[0].x, o.p[0].y);
#pragma unroll
    for (int i = 1; i < N / 2; ++i) mx = fmaxf(mx, fmaxf(o.p[i].x, o.p[i].y));
    if (mx > m) {
      const float f = exp_scaled(m - mx, c);
      s = __fmul2_rn(s, make_float2(f, f));
      m = mx;
    }
    const float ref = m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) s = __fadd2_rn(s, exp2_scaled(o.p[i], ref, c));
  }
  __device__ __forceinline__ Soft soft() const { return {m, s.x + s.y}; }
};

// si * exp((z - m) / T)
template <int N>
__device__ __forceinline__ Vals<N> grad_of(Vals<N> o, float m, float c, float si) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) o.p[i] = __fmul2_rn(exp2_scaled(o.p[i], m, c), make_float2(si, si));
  return o;
}

// ------------------------------------------------------------------------------------------ granules

template <typename A, typename B>
constexpr int granule_of() { return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4; }

// Granules of GE logits of one row. VEC: granule g holds logits GE g - shift + e, where shift is the row's start past a
// boundary (the same for z and dz, whose pitches differ by a multiple of eight); otherwise shift is 0 and every access
// is of one element. All granules but the first and the last (the edges) are whole.
template <int GE>
struct Granules {
  int shift, count, V;
  __device__ __forceinline__ int first(int g) const { return GE * g - shift; }
  __device__ __forceinline__ bool has(int g, int e) const { return first(g) + e >= 0 && first(g) + e < V; }
};

template <int GE, bool VEC>
__device__ __forceinline__ Granules<GE> granules(long long row, long long ld, int V) {
  const int shift = VEC ? static_cast<int>((row * ld) & (GE - 1)) : 0;
  return {shift, (V + shift + GE - 1) / GE, V};
}

// The part of a row that block `rank` of `slices` has: granules [g0, g1), of which [inner, inner + n) are not edges.
// Inner granule inner + i belongs to thread i mod TH; the row's first edge to thread HEAD and its last to thread TAIL.
struct Slice {
  int g0, g1, inner, n;
  bool head, tail;
};
constexpr int HEAD = 0, TAIL = 16;

template <int GE>
__device__ __forceinline__ Slice slice_of(const Granules<GE> &G, int rank, int slices) {
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

// Element by element; places that the row does not have read as -inf.
template <typename T, int GE>
__device__ __forceinline__ void load_values(const T *p, const Granules<GE> &G, int g, Raw<T, GE> &r) {
  r.clear();
#pragma unroll
  for (int e = 0; e < GE; ++e) r.put(e, G.has(g, e) ? p[G.first(g) + e] : neg_inf<T>());
}

template <typename T, int GE>
__device__ __forceinline__ void store_values(T *p, const Granules<GE> &G, int g, const Vals<GE> &o) {
#pragma unroll
  for (int e = 0; e < GE; ++e)
    if (G.has(g, e)) store1(p, G.first(g) + e, e % 2 ? o.p[e / 2].y : o.p[e / 2].x);
}

template <typename DT, int GE, int TH, bool VEC>
__device__ __forceinline__ void zero_granules(DT *dz, const Granules<GE> &G, const Slice &S) {
  Vals<GE> o;
#pragma unroll
  for (int i = 0; i < GE / 2; ++i) o.p[i] = make_float2(0.f, 0.f);
  for (int i = threadIdx.x; i < S.n; i += TH) {
    if constexpr (VEC) store_vals(dz + G.first(S.inner + i), o);
    else store_values(dz, G, S.inner + i, o);
  }
  if (S.head && threadIdx.x == HEAD) store_values(dz, G, 0, o);
  if (S.tail && threadIdx.x == TAIL) store_values(dz, G, G.count - 1, o);
}

// A thread's granules of a slice, in batches: while one is used the loads of the next are in flight. run() calls
// inner(i, values) and edge(g, values).
template <typename ZT, int GE, int TH, bool VEC>
struct Stream {
  static constexpr int U = 64 / (GE * static_cast<int>(sizeof(ZT)));   // 64 bytes to a batch
  const ZT *z, *next;   // the row; the thread's next batch to fetch
  const Granules<GE> &G;
  const Slice &S;
  int fetched, used;
  Raw<ZT, GE> a[U], b[U], e;
  __device__ __forceinline__ void fetch(Raw<ZT, GE> *r) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (fetched + u * TH < S.n) {
        if constexpr (VEC) r[u].load(next + u * TH * GE);
        else load_values(z, G, S.inner + fetched + u * TH, r[u]);
      }
    fetched += U * TH;
    next += U * TH * GE;
  }
  __device__ __forceinline__ Stream(const ZT *z_, const Granules<GE> &G_, const Slice &S_)
      : z(z_), next(z_ + G_.first(S_.inner) + GE * static_cast<int>(threadIdx.x)), G(G_), S(S_),
        fetched(threadIdx.x), used(threadIdx.x) {
    if (S.head && threadIdx.x == HEAD) load_values(z, G, 0, e);
    if (S.tail && threadIdx.x == TAIL) load_values(z, G, G.count - 1, e);
    fetch(a);
  }
  template <typename F>
  __device__ __forceinline__ void use(const Raw<ZT, GE> *r, F &&inner) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (used + u * TH < S.n) inner(used + u * TH, r[u].get());
    used += U * TH;
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
  // si * exp((z - m) / T) to dz
  template <typename DT>
  __device__ __forceinline__ void write_grad(DT *dz, float m, float c, float si) {
    DT *first = dz + G.first(S.inner);
    run(
        [&](int i, const Vals<GE> &o) {
          if constexpr (VEC) store_vals(first + GE * i, grad_of(o, m, c, si));
          else store_values(dz, G, S.inner + i, grad_of(o, m, c, si));
        },
        [&](int g, const Vals<GE> &o) { store_values(dz, G, g, grad_of(o, m, c, si)); });
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

// After them the forms that write the gradient of short rows (TABLE) have a flag that an index occurs twice and a table of
// the indices, 2^bits >= 2 K places of which -1 are free.
__device__ __forceinline__ int *twice_at(const Teacher &s, int K) { return s.idx + 3 * ((K + 3) & ~3); }
int table_bits(int K) {
  int bits = 1;
  while ((1 << bits) < 2 * K) ++bits;
  return bits;
}
size_t table_bytes(int K) { return 4 + (size_t{4} << table_bits(K)); }

// With a warp to a row the search of all entries for each entry's index is most of the work (16384 x 2000 bf16, joint: 56
// and 80 us with 64 and 200 entries, and 63 and 155 us with the search); beside longer rows the table costs as much as it
// saves.
template <int TH>
constexpr bool TABLE = TH == 32;

template <int TH>
__device__ __forceinline__ void clear_table(const DistillArgs &a, const Teacher &s) {
  int *twice = twice_at(s, a.K);
  if (threadIdx.x == 0) *twice = 0;
  for (int i = threadIdx.x; i < 1 << a.bits; i += TH) twice[1 + i] = -1;
}

// Once the table is clear and the entries are there. An index's search starts at the top bits of its product with an odd
// constant near 2^32 / golden ratio, and ends since half of the places stay free.
template <int TH>
__device__ __forceinline__ void fill_table(const DistillArgs &a, const Teacher &s) {
  int *twice = twice_at(s, a.K), *table = twice + 1;
  for (int k = threadIdx.x; k < a.K; k += TH) {
    const int id = s.idx[k];
    if (id < 0) continue;
    unsigned at = static_cast<unsigned>(id) * 0x9e3779b1u >> (32 - a.bits);
    int found = atomicCAS(table + at, -1, id);
    while (found != -1 && found != id) {
      at = (at + 1) & ((1u << a.bits) - 1);
      found = atomicCAS(table + at, -1, id);
    }
    if (found == id) *twice = 1;
  }
}

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
template <typename ZT, int TH, bool ALL>
__device__ __forceinline__ Soft put_teacher(const DistillArgs &a, long long row, const ZT *z, const Teacher &s, int lo,
                                            int hi, float c, const Entry &ahead) {
  Soft sum{-INFINITY, 0.f};
  if (static_cast<int>(threadIdx.x) < a.K) put_entry(s, threadIdx.x, ahead, c, sum);
  constexpr int U = ALL && TH == 32 ? 4 : 1;   // entries on their way at once
  int k = TH + threadIdx.x;
  if constexpr (U > 1)
    for (; k + (U - 1) * TH < a.K; k += U * TH) {
      Entry e[U];
#pragma unroll
      for (int u = 0; u < U; ++u) e[u] = load_entry(a, row, k + u * TH);
#pragma unroll
      for (int u = 0; u < U; ++u) e[u].z = entry_logit<ZT, ALL>(e[u], z, lo, hi);
#pragma unroll
      for (int u = 0; u < U; ++u) put_entry(s, k + u * TH, e[u], c, sum);
    }
  for (; k < a.K; k += TH) {
    Entry e = load_entry(a, row, k);
    e.z = entry_logit<ZT, ALL>(e, z, lo, hi);
    put_entry(s, k, e, c, sum);
  }
  for (k = a.K + threadIdx.x; k < ((a.K + 3) & ~3); k += TH) s.idx[k] = -1;
  return sum;
}

// What a block's warps exchange.
template <int TH>
struct BlockRed {
  float4 sums[TH / 32];
  float loss[TH / 32];
};

// The student's and the teacher's sums in one exchange: every warp puts its pairs, and after one barrier every warp
// merges all of them.
template <int TH>
__device__ __forceinline__ void merge_all(BlockRed<TH> &r, float c, Soft &student, Soft &teacher) {
  student = warp_merge<32>(student, c);
  teacher = warp_merge<32>(teacher, c);
  const int lane = threadIdx.x % 32;
  if (lane == 0) r.sums[threadIdx.x / 32] = make_float4(student.m, student.s, teacher.m, teacher.s);
  __syncthreads();
  const float4 v = r.sums[lane % (TH / 32)];
  student = warp_merge<TH / 32>({v.x, v.y}, c);
  teacher = warp_merge<TH / 32>({v.z, v.w}, c);
}

// The thread's part of sum_k q_k (log q_k - (z_k - m) / T); an entry whose q is 0 adds nothing, whatever the student
// gives it.
template <int TH>
__device__ __forceinline__ float loss_part(const DistillArgs &a, const Teacher &s, const Soft &teacher, float m,
                                           float c) {
  if (static_cast<int>(threadIdx.x & ~31u) >= a.K) return 0.f;   // the whole warp
  const float tl = logf(teacher.s), tinv = 1.f / teacher.s;
  float part = 0.f;
  for (int k = threadIdx.x; k < a.K; k += TH) {
    if (s.idx[k] < 0) continue;
    const float d = s.t[k] - teacher.m;
    const float q = exp_scaled(d, c) * tinv;
    if (!(q == 0.f)) part = fmaf(q, (d * a.inv_t - tl) - (s.z[k] - m) * a.inv_t, part);
  }
  return warp_sum(part);
}

template <int TH>
__device__ __forceinline__ void store_loss(const DistillArgs &a, long long row, float w, const float *parts,
                                           const Soft &student) {
  float kl = 0.f;
#pragma unroll
  for (int i = 0; i < TH / 32; ++i) kl += parts[i];
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

// Where the p parts of columns [lo, hi) are written: each entry subtracts its q, or, unless it is known that no index
// occurs twice, the first entry of each index subtracts the q of all of its entries, in order.
template <int TH, typename DT>
__device__ __forceinline__ void subtract_teacher(const DistillArgs &a, const Teacher &s, DT *dz, int lo, int hi,
                                                 float c, float m, float inv, float scale, const Soft &teacher) {
  const float tinv = 1.f / teacher.s;
  bool twice = true;
  if constexpr (TABLE<TH>) twice = *twice_at(s, a.K) != 0;
  for (int k = threadIdx.x; k < a.K; k += TH) {
    const int id = s.idx[k];
    if (id < lo || id >= hi) continue;   // absent entries are -1, below every lo
    bool first = true;
    float q = twice ? 0.f : exp_scaled(s.t[k] - teacher.m, c) * tinv;
    for (int i = 0; twice && i < a.K; i += 4) {
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
// all blocks get the same bits. 
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

// Blocks of a multiprocessor for TH threads, at 64 registers each.
constexpr int blocks_of(int TH) { return std::min(32, 1024 / TH); }

// Loss and stats. One pass with a running maximum and sum per thread, and one exchange of both softmaxes' pairs between
// the block's warps. Bound by the rate at which a block's chains of loads start and end more than by memory's: 8192 x 50304
// bf16 in 150 us, 5.5 TB/s; 4096 x 128256 in 171 us, 6.1 TB/s, and of fp32 in 291 us, 7.2 TB/s.
template <typename ZT, int TH, bool VEC>
__global__ void __launch_bounds__(TH, blocks_of(TH)) distill_forward_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int GE = granule_of<ZT, ZT>();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed<TH> red;
  __shared__ float2 put;
  const Teacher s = teacher_at(smem, a.K);
  const float c = a.inv_t * LOG2E;
  const int t = threadIdx.x, slices = a.slices, rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long long row = blockIdx.x / slices;
  const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
  const Granules<GE> G = granules<GE, VEC>(row, a.ldz, a.V);
  const Slice S = slice_of(G, rank, slices);
  const bool entry = rank == 0 && t < a.K;
  const float w = weight_of(a, row);
  Entry e{};
  if (entry) e = load_entry(a, row, t);
  if (w == 0.f) {   // the same for the whole cluster
    if (rank == 0 && t == 0) store_nothing(a, row);
    return;
  }
  Stream<ZT, GE, TH, VEC> stream(z, G, S);
  if (entry) e.z = entry_logit<ZT, true>(e, z, 0, 0);
  Run run;
  auto add = [&](int, const Vals<GE> &o) { run.add(o, c); };
  stream.run(add, add);
  Soft student = run.soft(), teacher{-INFINITY, 0.f};
  if (rank == 0) teacher = put_teacher<ZT, TH, true>(a, row, z, s, 0, 0, c, e);
  merge_all<TH>(red, c, student, teacher);
  if (slices > 1) merge_cluster(&put, slices, c, student);
  if (rank == 0) {
    no_softmax(student);
    const float part = loss_part<TH>(a, s, teacher, student.m, c);
    if (t % 32 == 0) red.loss[t / 32] = part;
    __syncthreads();
    if (t == 0) {
      if (teacher.s == 0.f) store_nothing(a, row);
      else store_loss<TH>(a, row, w, red.loss, student);
    }
  }
  if (slices > 1) cluster_sync();   // no block leaves while another reads its shared memory
}

// The gradient from the stats: no exchange but the teacher's, and every block has its own slice of a row. Bound by memory:
// 4096 x 128256 bf16 in 315 us, 6.7 TB/s.
template <typename ZT, typename DT, int TH, bool VEC>
__global__ void __launch_bounds__(TH, blocks_of(TH)) distill_backward_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int GE = granule_of<ZT, DT>();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed<TH> red;
  const Teacher s = teacher_at(smem, a.K);
  const float c = a.inv_t * LOG2E;
  const int t = threadIdx.x;
  const long long row = blockIdx.x / a.slices;
  const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
  DT *dz = static_cast<DT *>(a.dz) + row * a.ldd;
  const Granules<GE> G = granules<GE, VEC>(row, a.ldz, a.V);
  const Slice S = slice_of(G, static_cast<int>(blockIdx.x - row * a.slices), a.slices);
  const int lo = max(G.first(S.g0), 0), hi = min(G.first(S.g1), a.V);
  const float w = weight_of(a, row);
  Entry e{};
  if (t < a.K) e = load_entry(a, row, t);
  if (w == 0.f) {
    zero_granules<DT, GE, TH, VEC>(dz, G, S);
    return;
  }
  if constexpr (TABLE<TH>) clear_table<TH>(a, s);
  Stream<ZT, GE, TH, VEC> stream(z, G, S);
  const float m = a.stats[2 * row], l = a.stats[2 * row + 1], up = a.grad != nullptr ? a.grad[row] : 1.f;
  if (t < a.K) e.z = entry_logit<ZT, false>(e, z, lo, hi);
  Soft teacher = put_teacher<ZT, TH, false>(a, row, z, s, lo, hi, c, e), student{-INFINITY, 0.f};
  merge_all<TH>(red, c, student, teacher);   // its barrier also ends the reads of z that dz may overwrite
  if (teacher.s == 0.f) {
    zero_granules<DT, GE, TH, VEC>(dz, G, S);
    return;
  }
  const float inv = expf(-l), scale = up * w * a.temp;
  if constexpr (TABLE<TH>) fill_table<TH>(a, s);
  stream.write_grad(dz, m, c, scale * inv);
  __syncthreads();
  subtract_teacher<TH>(a, s, dz, lo, hi, c, m, inv, scale, teacher);
}

// Loss and gradient: the forward kernel's pass, then the backward kernel's over the same row, out of L2. Memory sees each
// logit and each gradient once (8192 x 50304 bf16: 312 us, 5.3 TB/s), and what bounds it is the two passes' instructions:
// with a row kept in shared memory in between, and the next one on its way there, it took 400 us.
template <typename ZT, typename DT, int TH, bool VEC>
__global__ void __launch_bounds__(TH, blocks_of(TH)) distill_joint_kernel(const DistillArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int GE = granule_of<ZT, DT>();
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ BlockRed<TH> red;
  __shared__ float2 put;
  const Teacher s = teacher_at(smem, a.K);
  const float c = a.inv_t * LOG2E;
  const int t = threadIdx.x, slices = a.slices, rank = slices > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const long long row = blockIdx.x / slices;
  const ZT *z = static_cast<const ZT *>(a.z) + row * a.ldz;
  DT *dz = static_cast<DT *>(a.dz) + row * a.ldd;
  const Granules<GE> G = granules<GE, VEC>(row, a.ldz, a.V);
  const Slice S = slice_of(G, rank, slices);
  const float w = weight_of(a, row);
  Entry e{};
  if (t < a.K) e = load_entry(a, row, t);
  if (w == 0.f) {   // the same for the whole cluster
    if (rank == 0 && t == 0) store_nothing(a, row);
    zero_granules<DT, GE, TH, VEC>(dz, G, S);
    return;
  }
  if constexpr (TABLE<TH>) clear_table<TH>(a, s);
  Run run;
  {
    Stream<ZT, GE, TH, VEC> stream(z, G, S);
    if (t < a.K) e.z = entry_logit<ZT, true>(e, z, 0, 0);
    auto add = [&](int, const Vals<GE> &o) { run.add(o, c); };
    stream.run(add, add);
  }
  // every block has all entries' logits before any block of the cluster writes its part of the gradient
  Soft student = run.soft(), teacher = put_teacher<ZT, TH, true>(a, row, z, s, 0, 0, c, e);
  merge_all<TH>(red, c, student, teacher);
  if (slices > 1) merge_cluster(&put, slices, c, student);
  if (teacher.s == 0.f) {
    if (rank == 0 && t == 0) store_nothing(a, row);
    zero_granules<DT, GE, TH, VEC>(dz, G, S);
  } else {
    no_softmax(student);
    Stream<ZT, GE, TH, VEC> stream(z, G, S);
    if (rank == 0) {
      const float part = loss_part<TH>(a, s, teacher, student.m, c);
      if (t % 32 == 0) red.loss[t / 32] = part;
    }
    const float scale = a.grad_scale * w * a.temp, inv = 1.f / student.s;
    if constexpr (TABLE<TH>) fill_table<TH>(a, s);
    stream.write_grad(dz, student.m, c, scale * inv);
    __syncthreads();
    if (rank == 0 && t == 0) store_loss<TH>(a, row, w, red.loss, student);
    subtract_teacher<TH>(a, s, dz, max(G.first(S.g0), 0), min(G.first(S.g1), a.V), c, student.m, inv, scale, teacher);
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
  a.bits = table_bits(a.K);
  a.grad_scale = 1.f;
  return a;
}

// A dependent launch of clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), long long blocks, int threads, int cluster, size_t smem,
                            cudaStream_t s, Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
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

// Blocks per row: 1, or as many as it takes to give every multiprocessor half of its blocks, each with at least 4096
// logits. To fill it, or a last wave, with smaller slices costs more than it gives, since a cluster starts only where all
// of its blocks fit, and its blocks wait for each other (300 x 50304 bf16, joint: 18 us, and 25 us when filled; 590 rows:
// 29 and 35 us; 1000 rows with the last wave filled: 61 us, and 48 us without clusters).
int row_slices(const DistillArgs &a, int TH) {
  const long long want = static_cast<long long>(device_sm_count()) * blocks_of(TH) / 2;
  int n = 1;
  while (n < MAX_CLUSTER && a.N * n < want && a.V / (2 * n) >= 4096) n *= 2;
  return n;
}

// Threads of a row's block: a warp for short rows, whose time is the chain of their loads and exchanges, so that as many
// rows as can be are on their way; 256 for long ones. (8192 x 50304 bf16, forward: 306, 186 and 145 us with 1024, 512 and
// 256 threads.)
int row_threads(int V) { return V < 4096 ? 32 : V < 16384 ? 128 : 256; }

// The joint form's second reading wants a row still in L2 (129 MB, and its gradient goes there too): wider blocks, and
// so fewer rows at once (608, 304 and 152), for rows of more than 131072 and 270000 bytes of logits. The limits lie
// between the lengths that were measured, 100608, 256512 and 513024 bytes, with a gradient of the logits' type; longer rows
// than those are more than L2 holds. (4096 x 128256 bf16: 464, 426 and 453 us with 256, 512 and 1024 threads;
// 2048 x 128256 fp32: 494, 460 and 425 us.)
int joint_threads(int V, size_t row_bytes) {
  return row_bytes <= 131072 ? row_threads(V) : row_bytes <= 270000 ? 512 : 1024;
}

// f with the thread count as a type
template <typename F>
cudaError_t with_threads(int TH, F &&f) {
  switch (TH) {
    case 32: return f(std::integral_constant<int, 32>());
    case 128: return f(std::integral_constant<int, 128>());
    case 256: return f(std::integral_constant<int, 256>());
    case 512: return f(std::integral_constant<int, 512>());
    default: return f(std::integral_constant<int, 1024>());
  }
}

template <typename ZT, bool VEC>
cudaError_t launch_fwd(DistillArgs a, cudaStream_t s) {
  return with_threads(row_threads(a.V), [&](auto th) {
    constexpr int TH = std::min(256, decltype(th)::value);
    a.slices = row_slices(a, TH);
    return launch_clusters(distill_forward_kernel<ZT, TH, VEC>, a.N * a.slices, TH, a.slices, teacher_bytes(a.K), s, a);
  });
}

template <typename ZT, typename DT, bool VEC>
cudaError_t launch_bwd(DistillArgs a, cudaStream_t s) {
  return with_threads(row_threads(a.V), [&](auto th) {
    constexpr int TH = std::min(256, decltype(th)::value);
    // slices of at most 65536 logits, so that the last blocks end close together
    a.slices = row_slices(a, TH);
    while (a.V / a.slices > 65536) a.slices *= 2;
    return launch_pdl(distill_backward_kernel<ZT, DT, TH, VEC>, dim3(static_cast<unsigned>(a.N * a.slices)), dim3(TH),
                      teacher_bytes(a.K) + (TABLE<TH> ? table_bytes(a.K) : 0), s, a);
  });
}

template <typename ZT, typename DT, bool VEC>
cudaError_t launch_step(DistillArgs a, cudaStream_t s) {
  // where a cluster shares a row the blocks are as in the forward kernel
  int threads = row_threads(a.V);
  a.slices = row_slices(a, threads);
  if (a.slices == 1) threads = joint_threads(a.V, static_cast<size_t>(a.V) * sizeof(ZT));
  return with_threads(threads, [&](auto th) {
    constexpr int TH = decltype(th)::value;
    return launch_clusters(distill_joint_kernel<ZT, DT, TH, VEC>, a.N * a.slices, TH, a.slices, teacher_bytes(a.K) + (TABLE<TH> ? table_bytes(a.K) : 0), s, a);
  });
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
  const bool vec = V >= 8 && aligned16(logits);
  launch_begin(KK_DISTILL_FWD, s);
  const cudaError_t e = zdt == MUON_F32 ? (vec ? launch_fwd<float, true>(a, s) : launch_fwd<float, false>(a, s))
                                        : (vec ? launch_fwd<__nv_bfloat16, true>(a, s) : launch_fwd<__nv_bfloat16, false>(a, s));
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
  const bool vec = V >= 8 && aligned16(logits) && aligned16(dlogits) && (ldz - ldd) % 8 == 0;
  launch_begin(KK_DISTILL_BWD, s);
  auto run = [&](auto z, auto d) {
    using ZT = decltype(z);
    using DT = decltype(d);
    return vec ? launch_bwd<ZT, DT, true>(a, s) : launch_bwd<ZT, DT, false>(a, s);
  };
  const __nv_bfloat16 h{};
  const cudaError_t e = zdt == MUON_F32 ? (ddt == MUON_F32 ? run(0.f, 0.f) : run(0.f, h))
                                        : (ddt == MUON_F32 ? run(h, 0.f) : run(h, h));
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
  const bool vec = V >= 8 && aligned16(logits) && aligned16(dlogits) && (ldz - ldd) % 8 == 0;
  launch_begin(KK_DISTILL_STEP, s);
  auto run = [&](auto z, auto d) {
    using ZT = decltype(z);
    using DT = decltype(d);
    return vec ? launch_step<ZT, DT, true>(a, s) : launch_step<ZT, DT, false>(a, s);
  };
  const __nv_bfloat16 h{};
  const cudaError_t e = zdt == MUON_F32 ? (ddt == MUON_F32 ? run(0.f, 0.f) : run(0.f, h))
                                        : (ddt == MUON_F32 ? run(h, 0.f) : run(h, h));
  launch_end(s);
  return status_of(e);
}

}  // extern "C"
