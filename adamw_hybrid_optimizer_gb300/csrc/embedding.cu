// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
//   out_i = scale * E[id_i]                         (an id outside [0, V) names no row: zeros)
//   dE_v  = scale * sum_{i : id_i = v} dout_i       (fp32 in a fixed order, rounded once at the end)
//
// The gradient sorts the ids with their positions (a stable radix sort, so that equal ids keep the order of
// their positions), and then sums each run of equal ids. No sum goes through an atomic: the same inputs give
// the same bits.
//
// Rows that do not all start on 16-byte boundaries (an odd width) still go through whole vectors: a lane's values come
// out of the two aligned granules around them, and lie where the granules of the row that is written are.
//
//   embedding_forward_kernel, embedding_forward_cut_kernel   a gather that reads and writes each byte once
//   embedding_prepare_kernel  one cluster sorts up to 131072 ids in its shared memory, while the other blocks zero the
//                             gradient (unless it accumulates).
//   embedding_zero_kernel     the zeroes alone, before a longer sort.
//   radix_*_kernel            one pass of a longer sort: digit counts per tile, their scan, the stable scatter.
//   embedding_sum_kernel      one warp per 16 or 32 sorted positions and 256 columns; the rows to come are in flight
//                             whether or not they belong to the id being summed, since most ids occur once or twice.
//   embedding_join_kernel     ids whose run covers the group after its first and goes on: adds the groups' sums, eighths of
//                             them at a time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int THREADS = 256;
constexpr int FWD_BLOCKS = 5, CUT_BLOCKS = 5;    // resident blocks of the lookup's kernels
constexpr int CUT_STAGES = 2;
constexpr int UNIT = 128;        // granules per warp and turn of the lookup: four per lane
constexpr int SUM_COLS = 256;    // columns per warp of the gradient's sums: 8 per lane
constexpr int SUM_BLOCKS = 3;    // resident blocks of the gradient's sums
// Sorted positions per warp of the gradient's sums: 32, or 16 with blocks of four warps where there are at most FEW_UNITS
// groups of 16 and 256 columns (152 multiprocessors, SUM_BLOCKS of 4 warps, twice).
constexpr int FEW_UNITS = 3648;
constexpr int group_of(int warps) { return 4 * warps; }
constexpr int SORT_TILE = 4096;  // keys per block of a sort pass
constexpr int MAX_DIGIT_BITS = 9;
constexpr unsigned NO_KEY = 0xffffffffu;

__device__ __forceinline__ long long load_id(const void *ids, int itype, long long i) {
  return itype == MUON_I32 ? static_cast<long long>(static_cast<const int *>(ids)[i])
                           : static_cast<const long long *>(ids)[i];
}

// ------------------------------------------------------------------------------------------ granules

// A granule is 8 values of bf16 or, where a matrix is fp32, 4: one access of 16 (8 for bf16 beside fp32) bytes.
template <typename A, typename B>
constexpr int granule_of() { return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4; }

// Values d .. d + GE - 1 of the 2 GE in lo and hi; d < GE is the same for the whole row.
template <typename T, int GE>
__device__ __forceinline__ Raw<T, GE> cut(const Raw<T, GE> &lo, const Raw<T, GE> &hi, int d) {
  constexpr int W = Raw<T, GE>::WORDS;
  unsigned w[2 * W];
#pragma unroll
  for (int i = 0; i < W; ++i) w[i] = lo.w[i], w[W + i] = hi.w[i];
  int words = sizeof(T) == 4 ? d : d / 2;
#pragma unroll
  for (int by = W / 2; by > 0; by /= 2)
    if (words & by) {
#pragma unroll
      for (int i = 0; i + by < 2 * W; ++i) w[i] = w[i + by];
    }
  Raw<T, GE> r;
#pragma unroll
  for (int i = 0; i < W; ++i) r.w[i] = sizeof(T) == 2 && (d & 1) ? __funnelshift_r(w[i], w[i + 1], 16) : w[i];
  return r;
}

// The granule of a matrix (`total` values from its first to its last) that starts at value `from`, on a boundary. Values
// outside the matrix are left 0.
template <typename T, int GE>
__device__ __forceinline__ void load_granule(const T *base, long long from, long long total, Raw<T, GE> &r) {
  if (from >= 0 && from + GE <= total) {
    r.load(base + from);
    return;
  }
  r.clear();
#pragma unroll
  for (int e = 0; e < GE; ++e)
    if (from + e >= 0 && from + e < total) r.put(e, base[from + e]);
}

// Values by which a base is past the boundary of a granule.
template <typename T, int GE>
int past(const void *base) { return static_cast<int>(reinterpret_cast<uintptr_t>(base) / sizeof(T) % GE); }

// Values [first, first + GE) of a row that has [0, D).
template <typename T, int GE>
__device__ __forceinline__ void store_edge(T *row, int first, int D, const Vals<GE> &o) {
#pragma unroll
  for (int e = 0; e < GE; ++e)
    if (first + e >= 0 && first + e < D) store1(row, first + e, e % 2 ? o.p[e / 2].y : o.p[e / 2].x);
}

// ------------------------------------------------------------------------------------------ lookup

struct LookupArgs {
  const void *ids, *table;
  void *out;
  long long ldt, ldo, n, V;
  int itype, D;
  float scale;
  int past_table, past_out;   // values by which the bases are past a granule's boundary
  int per_row;                // granules of a row, and 2^32 / per_row, rounded up
  unsigned inverse;
  int skip;                   // granules, and whole rows, from a warp's unit to its next one
  long long skip_rows;
};

// A warp's unit of work: it starts at granule `first` of row `row`, and rows have a.per_row granules.
struct LookupUnit {
  long long row;
  int first;
  struct Place {
    long long row;
    int granule;
  };
  __device__ __forceinline__ LookupUnit(const LookupArgs &a, long long granule)
      : row(granule / a.per_row), first(static_cast<int>(granule - row * a.per_row)) {}
  // granule i < UNIT of the unit. first + i < per_row + UNIT, so that the high half of its product with 2^32 / per_row,
  // rounded up, is the quotient
  __device__ __forceinline__ Place place(const LookupArgs &a, int i) const {
    const int at = first + i, rows = a.per_row == 1 ? at : static_cast<int>(__umulhi(at, a.inverse));
    return {row + rows, at - rows * a.per_row};
  }
  __device__ __forceinline__ void next(const LookupArgs &a) {
    row += a.skip_rows;
    first += a.skip;
    if (first >= a.per_row) ++row, first -= a.per_row;
  }
  // the ids of the lane's granules, -1 for what names no row
  __device__ __forceinline__ void ids(const LookupArgs &a, int lane, int *id) const {
#pragma unroll
    for (int q = 0; q < UNIT / 32; ++q) {
      const long long r = place(a, q * 32 + lane).row, v = r < a.n ? load_id(a.ids, a.itype, r) : -1;
      id[q] = v >= 0 && v < a.V ? static_cast<int>(v) : -1;
    }
  }
};

// Rows that start on a granule and have whole ones: warps take units of 128 granules in turn, four per lane, which follow
// each other through the rows (of any length, so that no lane is idle: 65536 rows of 768 bf16 take 24 us, and 29 us with
// units of whole rows). All loads of a unit are in flight before the first is used, and the ids of the next unit are loaded
// under them, so that a unit waits for one latency, not two. No one unit is at its limit (32768 of 4096 bf16 out of 50304:
// memory at 61% of its peak, L2 at 42%, instructions issued in 58% of the cycles): the time is the loads' latency with half
// of the warps that a multiprocessor can hold. 65536 of 4096 bf16 out of 128256: 139 us for 701 MB (distinct rows counted
// once), 5.0 TB/s.
template <typename TT, typename OT>
__global__ void __launch_bounds__(THREADS, FWD_BLOCKS) embedding_forward_kernel(const LookupArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int GE = granule_of<TT, OT>(), U = UNIT / 32;
  const int lane = threadIdx.x % 32;
  const TT *table = static_cast<const TT *>(a.table);
  LookupUnit u(a, (static_cast<long long>(blockIdx.x) * (THREADS / 32) + threadIdx.x / 32) * UNIT);
  int next[U];
  u.ids(a, lane, next);
  while (u.row < a.n) {
    int id[U];
    Raw<TT, GE> r[U];
#pragma unroll
    for (int q = 0; q < U; ++q) {
      id[q] = next[q];
      r[q].clear();
      if (id[q] >= 0) r[q].load(table + id[q] * a.ldt + u.place(a, q * 32 + lane).granule * GE);
    }
    LookupUnit then = u;
    then.next(a);
    then.ids(a, lane, next);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const auto p = u.place(a, q * 32 + lane);
      if (p.row >= a.n) continue;
      Vals<GE> o = r[q].get();
#pragma unroll
      for (int i = 0; i < GE / 2; ++i)
        o.p[i] = id[q] < 0 ? make_float2(0.f, 0.f) : __fmul2_rn(o.p[i], make_float2(a.scale, a.scale));
      store_vals(static_cast<OT *>(a.out) + p.row * a.ldo + p.granule * GE, o);
    }
    u = then;
  }
}

// Other rows: a row's granules are those of the table around the output's, one more than are written; each is copied to
// the warp's ring in shared memory, and an output granule is cut out of two. A unit's last granule is only copied: it is
// the next unit's first. The granules of the next units are on their way, and the ids of the one after on theirs, while a
// unit is stored. Bound by instructions, those that cut a granule out of two first (32768 of 1001 bf16: issued in 64% of the
// cycles, memory at 12% of its peak). (65536 rows of 771 bf16: 41 us, and 76 us with two loads per lane and granule into
// registers; but where rows are aligned the ring takes 194 us for 65536 rows of 4096, and registers 138 us.)
template <typename TT, typename OT>
__global__ void __launch_bounds__(THREADS, CUT_BLOCKS) embedding_forward_cut_kernel(const LookupArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int GE = granule_of<TT, OT>(), U = UNIT / 32, WARPS = THREADS / 32, S = CUT_STAGES;
  constexpr int B = Raw<TT, GE>::BYTES;
  extern __shared__ __align__(16) unsigned char shared[];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  unsigned char *ring = shared + w * (S * UNIT * B);
  int *kept = reinterpret_cast<int *>(shared + WARPS * S * UNIT * B) + threadIdx.x;   // the ids of units in the ring
  const long long total = (a.V - 1) * a.ldt + a.D;
  const TT *table = static_cast<const TT *>(a.table);
  // first column of a granule, in the output row's own granules
  auto column = [&](const LookupUnit::Place &p) {
    return p.granule * GE - static_cast<int>((p.row * a.ldo + a.past_out) & (GE - 1));
  };
  auto fetch = [&](const LookupUnit &u, int stage, const int *id) {
#pragma unroll
    for (int q = 0; q < U; ++q) {
      kept[(stage * U + q) * THREADS] = id[q];
      if (id[q] < 0) continue;
      const int c = column(u.place(a, q * 32 + lane));
      unsigned char *slot = ring + (stage * UNIT + q * 32 + lane) * B;
      const long long at = id[q] * a.ldt + c;
      if (c < a.D + GE) {
        const long long from = at - ((at + a.past_table) & (GE - 1));
        if (from >= 0 && from + GE <= total) {
          copy_async<B>(slot, table + from);
        } else {
          Raw<TT, GE> r;
          load_granule(table, from, total, r);
          r.store(reinterpret_cast<TT *>(slot));
        }
      }
    }
    copy_async_commit();
  };
  LookupUnit u(a, (static_cast<long long>(blockIdx.x) * WARPS + w) * (UNIT - 1)), ahead = u;
  int id[U];
#pragma unroll
  for (int k = 0; k < S - 1; ++k) {
    ahead.ids(a, lane, id);
    fetch(ahead, k, id);
    ahead.next(a);
  }
  ahead.ids(a, lane, id);
  int stage = 0;
  for (; u.row < a.n; u.next(a)) {
    copy_async_wait<S - 2>();
    __syncwarp();
    // the place of the unit before this one, which all lanes have read
    fetch(ahead, stage == 0 ? S - 1 : stage - 1, id);
    ahead.next(a);
    ahead.ids(a, lane, id);
#pragma unroll
    for (int q = 0; q < U; ++q) {
      const auto p = u.place(a, q * 32 + lane);
      const int c = column(p), at = kept[(stage * U + q) * THREADS];
      if (p.row >= a.n || c >= a.D || p.granule == a.per_row - 1 || q * 32 + lane == UNIT - 1) continue;
      const unsigned char *slot = ring + (stage * UNIT + q * 32 + lane) * B;
      Vals<GE> o;
#pragma unroll
      for (int i = 0; i < GE / 2; ++i) o.p[i] = make_float2(0.f, 0.f);
      if (at >= 0) {
        Raw<TT, GE> lo, hi;
        lo.load(reinterpret_cast<const TT *>(slot));
        hi.load(reinterpret_cast<const TT *>(slot + B));
        o = cut(lo, hi, static_cast<int>((at * a.ldt + c + a.past_table) & (GE - 1))).get();
#pragma unroll
        for (int i = 0; i < GE / 2; ++i) o.p[i] = __fmul2_rn(o.p[i], make_float2(a.scale, a.scale));
      }
      OT *dst = static_cast<OT *>(a.out) + p.row * a.ldo;
      if (c >= 0 && c + GE <= a.D) store_vals(dst + c, o);
      else store_edge(dst, c, a.D, o);
    }
    stage = stage == S - 1 ? 0 : stage + 1;
  }
}

// ------------------------------------------------------------------------------------------ sort

// Sort key of position i: its id, or V (after every id) where the id takes no gradient.
__device__ __forceinline__ unsigned key_of(const void *ids, int itype, long long i, long long V, long long padding) {
  const long long id = load_id(ids, itype, i);
  return static_cast<unsigned>(id < 0 || id >= V || id == padding ? V : id);
}

struct SortPass {
  const void *ids;            // first pass: the ids; later passes read keys / pos
  int itype;
  long long V, padding;
  const unsigned *key_in, *pos_in;
  unsigned *key_out, *pos_out;
  unsigned *hist;             // [digit][tile]: counts, then (after the scan) the first output index
  long long n;
  int tiles, shift, bits;
};

__device__ __forceinline__ unsigned pass_key(const SortPass &p, long long i) {
  return p.key_in != nullptr ? p.key_in[i] : key_of(p.ids, p.itype, i, p.V, p.padding);
}

__global__ void __launch_bounds__(THREADS) radix_count_kernel(const SortPass p) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ unsigned cnt[1 << MAX_DIGIT_BITS];
  const int bins = 1 << p.bits;
  for (int b = threadIdx.x; b < bins; b += THREADS) cnt[b] = 0;
  __syncthreads();
  const long long t0 = static_cast<long long>(blockIdx.x) * SORT_TILE;
  for (int k = threadIdx.x; k < SORT_TILE; k += THREADS)
    if (t0 + k < p.n) atomicAdd(&cnt[(pass_key(p, t0 + k) >> p.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += THREADS) p.hist[static_cast<long long>(b) * p.tiles + blockIdx.x] = cnt[b];
}

// Exclusive scan of the counts in place; also zeroes the list counter of the join kernel.
__global__ void __launch_bounds__(1024) radix_scan_kernel(unsigned *hist, long long total, unsigned *list_count) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ unsigned wsum[32];
  const int t = threadIdx.x, lane = t % 32;
  const long long per = (total + 1023) / 1024;
  const long long a = min(per * t, total), b = min(a + per, total);
  unsigned s = 0;
  for (long long i = a; i < b; ++i) s += hist[i];
  unsigned x = s;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) wsum[t / 32] = x;
  __syncthreads();
  if (t < 32) {
    unsigned w = wsum[t];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    wsum[t] = w;
  }
  __syncthreads();
  unsigned base = x - s + (t >= 32 ? wsum[t / 32 - 1] : 0u);
  for (long long i = a; i < b; ++i) {
    const unsigned v = hist[i];
    hist[i] = base;
    base += v;
  }
  if (t == 0) *list_count = 0;
}

// Warp w of a block takes the tile's keys [512 w, 512 w + 512) in order, 32 at a time; a key's place is its digit's
// first place in this tile, plus the keys of that digit in earlier warps, earlier rounds and lower lanes.
__global__ void __launch_bounds__(THREADS) radix_scatter_kernel(const SortPass p) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int WARPS = THREADS / 32, PER_WARP = SORT_TILE / WARPS;
  __shared__ unsigned place[WARPS][1 << MAX_DIGIT_BITS];
  const int bins = 1 << p.bits, w = threadIdx.x / 32, lane = threadIdx.x % 32;
  for (int k = threadIdx.x; k < WARPS * bins; k += THREADS) place[k / bins][k % bins] = 0;
  __syncthreads();
  const long long t0 = static_cast<long long>(blockIdx.x) * SORT_TILE + w * PER_WARP;
  for (int k = lane; k < PER_WARP; k += 32)
    if (t0 + k < p.n) atomicAdd(&place[w][(pass_key(p, t0 + k) >> p.shift) & (bins - 1)], 1u);
  __syncthreads();
  for (int b = threadIdx.x; b < bins; b += THREADS) {
    unsigned at = p.hist[static_cast<long long>(b) * p.tiles + blockIdx.x];
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const unsigned c = place[k][b];
      place[k][b] = at;
      at += c;
    }
  }
  __syncthreads();
  for (int k = lane; k < PER_WARP; k += 32) {
    const long long i = t0 + k;
    const bool in = i < p.n;
    const unsigned key = in ? pass_key(p, i) : NO_KEY;
    const unsigned pos = in ? (p.pos_in != nullptr ? p.pos_in[i] : static_cast<unsigned>(i)) : 0u;
    const int d = in ? static_cast<int>((key >> p.shift) & (bins - 1)) : bins;
    const unsigned same = __match_any_sync(0xffffffffu, d);
    const unsigned below = __popc(same & ((1u << lane) - 1u));
    unsigned first = 0;
    if (in) first = place[w][d];
    __syncwarp();
    if (in && below == 0) place[w][d] = first + __popc(same);
    __syncwarp();
    if (in) {
      p.key_out[first + below] = key;
      p.pos_out[first + below] = pos;
    }
  }
}

// What is to be zeroed: rows x `bytes` at a pitch (one row of everything where the rows leave no gaps).
struct ZeroArgs {
  unsigned char *g;
  long long pitch, rows, bytes;
};
constexpr long long ZERO_BLOCK = 256 * 1024;   // bytes of one row per block; of many rows, whole rows of about that

__device__ __forceinline__ void zero_stretch(unsigned char *p, long long bytes, int first, int threads) {
  const long long head = (16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15;
  const long long lead = head < bytes ? head : bytes, whole = (bytes - lead) / 16;
  uint4 *q = reinterpret_cast<uint4 *>(p + lead);
#pragma unroll 4
  for (long long i = first; i < whole; i += threads) q[i] = make_uint4(0, 0, 0, 0);
  for (long long i = first; i < lead; i += threads) p[i] = 0;
  for (long long i = lead + whole * 16 + first; i < bytes; i += threads) p[i] = 0;
}

__host__ __device__ __forceinline__ long long zero_rows_per_block(const ZeroArgs &z) {
  return z.bytes >= ZERO_BLOCK ? 1 : ZERO_BLOCK / z.bytes;
}
long long zero_blocks(const ZeroArgs &z) {
  if (z.rows == 1) return (z.bytes + ZERO_BLOCK - 1) / ZERO_BLOCK;
  return (z.rows + zero_rows_per_block(z) - 1) / zero_rows_per_block(z);
}

// The share of block b of zero_blocks().
__device__ __forceinline__ void zero_share(const ZeroArgs &z, long long b) {
  if (z.rows == 1) {
    const long long from = b * ZERO_BLOCK;
    if (from < z.bytes) zero_stretch(z.g + from, min(ZERO_BLOCK, z.bytes - from), threadIdx.x, blockDim.x);
  } else {   // warps take rows
    const long long per = zero_rows_per_block(z), end = min((b + 1) * per, z.rows);   // none past the last block
    for (long long r = b * per + threadIdx.x / 32; r < end; r += blockDim.x / 32)
      zero_stretch(z.g + r * z.pitch, z.bytes, threadIdx.x % 32, 32);
  }
}

__global__ void __launch_bounds__(THREADS) embedding_zero_kernel(const ZeroArgs z) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  zero_share(z, blockIdx.x);
}

// The whole sort in one cluster, for n <= 16 * 8192: block b holds the sorted positions [b * chunk, (b + 1) * chunk) in
// its shared memory, and a pass moves every item to its place in any block's. A thread keeps its items in registers
// while their places are computed, so one buffer is enough. Warp w of a block has the block's items [w * per, ...), 32
// at a time; an item's place is its digit's first place, plus the digit's items in earlier blocks, warps, rounds and
// lanes: stable, like the passes above. Bound by the latency of its rounds and of the cluster's barriers: two passes over
// 16384 ids take about 20 us, which the zeroes of 50304 x 768 bf16 (77 MB) hide half of, and those of 128256 x 4096 all.
constexpr int CS_THREADS = 512;
constexpr int CS_WARPS = CS_THREADS / 32;
constexpr int CS_ROUNDS = 16;                              // items per thread
constexpr int CS_CHUNK = CS_THREADS * CS_ROUNDS;           // items per block
constexpr int CS_BLOCKS = 16;

struct ClusterSort {
  const void *ids;
  int itype;
  long long V, padding;
  unsigned *key, *pos;      // sorted
  unsigned *list_count;
  int n, blocks, chunk, passes, bits;
  ZeroArgs zero;            // for the blocks after the first cluster
};

struct ClusterShared {
  unsigned short place[CS_WARPS][1 << MAX_DIGIT_BITS];
  unsigned count[2][1 << MAX_DIGIT_BITS];                   // the block's items of each digit; by parity of the pass
  unsigned first[1 << MAX_DIGIT_BITS];                      // where the block's first item of each digit goes
  unsigned warp_total[CS_WARPS];
  alignas(8) uint2 item[CS_CHUNK];                          // (key, position); only `chunk` of them are allocated
};

__global__ void __launch_bounds__(CS_THREADS, 2) embedding_prepare_kernel(const ClusterSort a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  if (blockIdx.x >= a.blocks) {   // whole clusters
    zero_share(a.zero, blockIdx.x - a.blocks);
    return;
  }
  extern __shared__ __align__(16) unsigned char cluster_smem[];
  ClusterShared &s = *reinterpret_cast<ClusterShared *>(cluster_smem);
  const int rank = a.blocks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int w = threadIdx.x / 32, lane = threadIdx.x % 32, bins = 1 << a.bits;
  const int base = rank * a.chunk, mine = min(a.chunk, a.n - base);      // may be <= 0 for the last blocks
  const int per = (a.chunk + CS_THREADS - 1) / CS_THREADS * 32, rounds = per / 32;
  for (int pass = 0; pass < a.passes; ++pass) {
    const int shift = pass * a.bits;
    for (int b = lane; b < bins; b += 32) s.place[w][b] = 0;
    __syncwarp();
    unsigned key[CS_ROUNDS], pos[CS_ROUNDS];   // pos: the position, and above its 17 bits the rank within the warp
#pragma unroll
    for (int r = 0; r < CS_ROUNDS; ++r) {
      if (r >= rounds) break;
      const int i = w * per + r * 32 + lane;
      const bool in = i < mine;
      if (pass == 0) {
        key[r] = in ? key_of(a.ids, a.itype, base + i, a.V, a.padding) : NO_KEY;
        pos[r] = static_cast<unsigned>(base + i);
      } else {
        const uint2 it = in ? s.item[i] : make_uint2(NO_KEY, 0u);
        key[r] = it.x;
        pos[r] = it.y;
      }
    }
#pragma unroll
    for (int r = 0; r < CS_ROUNDS; ++r) {
      if (r >= rounds) break;
      const bool in = w * per + r * 32 + lane < mine;
      const int d = in ? static_cast<int>((key[r] >> shift) & (bins - 1)) : bins;
      const unsigned same = __match_any_sync(0xffffffffu, d);
      const unsigned below = __popc(same & ((1u << lane) - 1u));
      const unsigned before = in ? s.place[w][d] : 0u;
      __syncwarp();
      if (in && below == 0) s.place[w][d] = static_cast<unsigned short>(before + __popc(same));
      __syncwarp();
      if (in) pos[r] |= (before + below) << 17;
    }
    __syncthreads();
    unsigned *count = s.count[pass & 1];
    for (int b = threadIdx.x; b < bins; b += CS_THREADS) {
      unsigned at = 0;
      for (int k = 0; k < CS_WARPS; ++k) {
        const unsigned c = s.place[k][b];
        s.place[k][b] = static_cast<unsigned short>(at);
        at += c;
      }
      count[b] = at;
    }
    if (a.blocks > 1) cluster_sync();
    else __syncthreads();
    // first place of each digit: all items of lower digits, and this digit's items in earlier blocks
    unsigned total = 0, earlier = 0;
    if (static_cast<int>(threadIdx.x) < bins) {
      if (a.blocks > 1) {
        const uint32_t at = smem_u32(count + threadIdx.x);
        for (int k = 0; k < a.blocks; ++k) {
          unsigned c;
          asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(c) : "r"(mapa_shared(at, k)) : "memory");
          total += c;
          if (k < rank) earlier += c;
        }
      } else {
        total = count[threadIdx.x];
      }
    }
    unsigned x = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s.warp_total[w] = x;
    __syncthreads();
    unsigned lower = x - total;
    for (int k = 0; k < w && k < bins / 32; ++k) lower += s.warp_total[k];
    if (static_cast<int>(threadIdx.x) < bins) s.first[threadIdx.x] = lower + earlier;
    __syncthreads();
    const bool last = pass + 1 == a.passes;
#pragma unroll
    for (int r = 0; r < CS_ROUNDS; ++r) {
      if (r >= rounds) break;
      if (w * per + r * 32 + lane >= mine) continue;
      const int d = static_cast<int>((key[r] >> shift) & (bins - 1));
      const unsigned to = s.first[d] + s.place[w][d] + (pos[r] >> 17), p = pos[r] & 0x1ffffu;
      if (last) {
        a.key[to] = key[r];
        a.pos[to] = p;
      } else if (a.blocks > 1) {
        const unsigned block = to / a.chunk;
        asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(
                         mapa_shared(smem_u32(&s.item[to - block * a.chunk]), block)),
                     "r"(key[r]), "r"(p)
                     : "memory");
      } else {
        s.item[to] = make_uint2(key[r], p);
      }
    }
    // the last pass: no block leaves while another reads its counts
    if (a.blocks > 1) cluster_sync();
    else __syncthreads();
  }
  if (rank == 0 && threadIdx.x == 0) *a.list_count = 0;
}

// ------------------------------------------------------------------------------------------ sums

struct SumArgs {
  const unsigned *key, *pos;   // sorted
  const void *dout;
  long long ldo;
  void *g;
  long long ldg;
  float *part;                 // [2 * groups][ldp]: sums of the runs that the join kernel finishes
  uint2 *list;                 // (group where such a run starts, groups that it touches)
  unsigned *list_count;
  long long n, V, ldp;
  int D, tiles, group, groups, accumulate, past_dout, past_g;   // past: values by which a base is past a boundary
  float scale;
};

// How the sums see memory. ALIGNED: every row of dout and dtable starts on a granule and has whole ones. CUT: not so;
// a lane's columns are those of its granules of the gradient row, which starts `shift` values past a boundary, and
// dout's values come out of the two granules around them.
enum Access { ALIGNED, CUT };

// The lane's eight of 256 columns of a tile, in granules that lie 32 apart: the first column of granule j.
template <int GE>
__device__ __forceinline__ int sum_col(int tile, int lane, int j, int shift) {
  return (tile * (SUM_COLS / GE) + j * 32 + lane) * GE - shift;
}

template <int ACCESS, int GE>
__device__ __forceinline__ int shift_of(const SumArgs &a, unsigned key) {
  return ACCESS == CUT ? static_cast<int>((static_cast<long long>(key) * a.ldg + a.past_g) & (GE - 1)) : 0;
}

// A row's 256 columns of a tile in the warp's ring: the granules of dout that hold them, in order (CUT: one more). ALIGNED:
// a lane copies what it reads itself.
template <typename OT, int GE, int ACCESS, int WARPS>
struct SumRing {
  static constexpr int B = Raw<OT, GE>::BYTES, P = SUM_COLS / GE;
  static constexpr int SLOTS = (sizeof(OT) == 2 ? 128 : 64) / WARPS;
  static constexpr int STRIDE = ACCESS == CUT ? (P * B + B + 15) / 16 * 16 : P * B;
  static constexpr int BYTES = SLOTS * STRIDE;   // per warp
  // the first of the tile's granules in dout, and by how many values the columns start past it
  static __device__ __forceinline__ long long start(const SumArgs &a, unsigned pos, int tile, int shift, int *d) {
    const long long first = static_cast<long long>(pos) * a.ldo + tile * SUM_COLS - shift;
    *d = ACCESS == CUT ? static_cast<int>((first + a.past_dout) & (GE - 1)) : 0;
    return first - *d;
  }
  static __device__ __forceinline__ void copy(const SumArgs &a, unsigned char *slot, unsigned pos, int tile, int lane,
                                              int shift) {
    const OT *base = static_cast<const OT *>(a.dout);
    int d;
    const long long from = start(a, pos, tile, shift, &d);
    if constexpr (ACCESS == ALIGNED) {
#pragma unroll
      for (int j = 0; j < 8 / GE; ++j) {
        const int p = j * 32 + lane;
        if (tile * SUM_COLS + p * GE < a.D) copy_async<B>(slot + p * B, base + from + p * GE);
      }
    } else {
      const long long total = (a.n - 1) * a.ldo + a.D, end = static_cast<long long>(pos) * a.ldo + a.D;
#pragma unroll
      for (int j = 0; j <= 8 / GE; ++j) {
        const int p = j * 32 + lane;
        const long long at = from + p * GE;
        if (p > P || at >= end) continue;
        if (at >= 0 && at + GE <= total) {
          copy_async<B>(slot + p * B, base + at);
        } else {
          Raw<OT, GE> r;
          load_granule(base, at, total, r);
          r.store(reinterpret_cast<OT *>(slot + p * B));
        }
      }
    }
  }
  static __device__ __forceinline__ void add(const SumArgs &a, const unsigned char *slot, unsigned pos, int tile, int lane,
                                             int shift, Vals<8> &acc) {
    int d = 0;
    if constexpr (ACCESS == CUT) start(a, pos, tile, shift, &d);
#pragma unroll
    for (int j = 0; j < 8 / GE; ++j) {
      Raw<OT, GE> r;
      const OT *at = reinterpret_cast<const OT *>(slot + (j * 32 + lane) * B);
      r.load(at);
      if constexpr (ACCESS == CUT) {
        Raw<OT, GE> hi;
        hi.load(at + GE);
        r = cut(r, hi, d);
      }
      const Vals<GE> v = r.get();
#pragma unroll
      for (int i = 0; i < GE / 2; ++i) acc.p[j * GE / 2 + i] = __fadd2_rn(acc.p[j * GE / 2 + i], v.p[i]);
    }
  }
};

// The gradient row's columns: scale * acc, added to what is there if asked.
template <typename GT, int GE, int ACCESS>
__device__ __forceinline__ void store_row(const SumArgs &a, unsigned key, int tile, int lane, const Vals<8> &acc) {
  GT *p = static_cast<GT *>(a.g) + static_cast<long long>(key) * a.ldg;
  const int shift = shift_of<ACCESS, GE>(a, key);
  const float2 s2 = make_float2(a.scale, a.scale);
#pragma unroll
  for (int j = 0; j < 8 / GE; ++j) {
    const int c = sum_col<GE>(tile, lane, j, shift);
    if (c >= a.D) continue;
    const bool whole = ACCESS == ALIGNED || (c >= 0 && c + GE <= a.D);
    Raw<GT, GE> r;
    r.clear();
    if (a.accumulate) {
      if (whole) {
        r.load(p + c);
      } else {
#pragma unroll
        for (int e = 0; e < GE; ++e)
          if (c + e >= 0 && c + e < a.D) r.put(e, p[c + e]);
      }
    }
    Vals<GE> o = r.get();
#pragma unroll
    for (int i = 0; i < GE / 2; ++i) o.p[i] = __ffma2_rn(acc.p[j * GE / 2 + i], s2, o.p[i]);
    if (whole) store_vals(p + c, o);
    else store_edge(p, c, a.D, o);
  }
}

// Partial sums keep the lane's own eight columns together: written and read by the same mapping.
__device__ __forceinline__ void store_part(float *p, int tile, int lane, const Vals<8> &acc) {
  store_vals(p + tile * SUM_COLS + lane * 8, acc);
}

// Groups that the long run of k which starts in group c touches: 32 probes at a time for the first group after c + 1
// whose first key is not k.
__device__ __forceinline__ unsigned run_groups(const SumArgs &a, long long c, unsigned k, int lane) {
  long long lo = c + 2, hi = a.groups;   // groups below lo are the run's, hi is not (or the end)
  while (lo < hi) {
    const long long stride = (hi - lo + 31) / 32, probe = lo + lane * stride;
    const unsigned yes = __ballot_sync(0xffffffffu, probe < hi && a.key[probe < hi ? probe * a.group : 0] == k);
    const int ok = __popc(yes);   // the run's probes are the first ones
    if (ok == 0) {
      hi = lo;
    } else {
      const long long limit = lo + ok * stride;
      lo += (ok - 1) * stride + 1;
      if (ok < 32 && limit < hi) hi = limit;
    }
  }
  return static_cast<unsigned>(lo - c);
}

// A run of equal ids that starts in group c belongs to it, unless the run covers the whole of the next group and
// goes on (a long run): then every group sums its own part, into part[2c + 1] where the run starts and part[2c]
// where it came from the group before, and the join kernel adds the parts. So a warp sums fewer positions than two
// groups have. The rows to come are on their way to the warp's ring in shared memory, whether or not they belong to
// one id. The loop is short on purpose: with a store for the end of a run unrolled into every place of a batch in
// registers, the code did not fit the instruction cache (131072 rows of 64: 45 us, and 27 us now). Bound by memory,
// dout read once and the rows that ids name written once, behind the sort and the zeroes: 32768 x 4096 bf16 in 64 us,
// 330 MB at 5.1 TB/s (memory at 64% of its peak, instructions issued in 65% of the cycles); the whole gradient of 128256
// rows in 212 us, 6.2 TB/s. Few tokens: by the latency of the
// positions of one warp, some 90 instructions each.
template <typename OT, typename GT, int ACCESS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, SUM_BLOCKS) embedding_sum_kernel(const SumArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int GE = granule_of<OT, GT>();
  using Ring = SumRing<OT, GE, ACCESS, WARPS>;
  constexpr int S = Ring::SLOTS, GROUP = group_of(WARPS);
  extern __shared__ __align__(16) unsigned char shared[];
  const int lane = threadIdx.x % 32;
  unsigned char *ring = shared + threadIdx.x / 32 * Ring::BYTES;
  const long long units = static_cast<long long>(a.groups) * a.tiles;
  const long long warps = static_cast<long long>(gridDim.x) * WARPS;
  const unsigned none = static_cast<unsigned>(a.V);
  for (long long u = static_cast<long long>(blockIdx.x) * WARPS + threadIdx.x / 32; u < units; u += warps) {
    const long long c = u / a.tiles;
    const int tile = static_cast<int>(u - c * a.tiles);
    const long long s = c * GROUP;
    auto key_at = [&](long long i) { return i >= 0 && i < a.n ? a.key[i] : NO_KEY; };
    const bool has = lane < GROUP;
    const unsigned k0 = has ? key_at(s + lane) : NO_KEY, k1 = has ? key_at(s + GROUP + lane) : NO_KEY;
    const unsigned p0 = has && s + lane < a.n ? a.pos[s + lane] : 0u;
    const unsigned p1 = has && s + GROUP + lane < a.n ? a.pos[s + GROUP + lane] : 0u;
    const unsigned before = key_at(s - 1), far_before = key_at(s - GROUP - 1), far_after = key_at(s + 2 * GROUP);
    const unsigned first = __shfl_sync(0xffffffffu, k0, 0), last = __shfl_sync(0xffffffffu, k0, GROUP - 1);
    const unsigned next = __shfl_sync(0xffffffffu, k1, 0);
    if (first >= none) continue;                       // only ids that take no gradient from here on
    int begin = 0;
    bool to_lead = false;                              // the leading run goes to part[2c]
    if (before == first) {
      if (far_before == first || next == first) to_lead = true;
      else begin = __popc(__ballot_sync(0xffffffffu, k0 == first));
    }
    int end = __popc(__ballot_sync(0xffffffffu, k0 < none));
    bool tail_part = false;                            // the last run goes to part[2c + 1]
    if (end == GROUP && next == last && before != last) {   // before == last: the one run covers the group
      tail_part = far_after == last;
      if (!tail_part) end += __popc(__ballot_sync(0xffffffffu, k1 == last));
    }
    if (tail_part && tile == 0) {
      const unsigned parts = run_groups(a, c, last, lane);
      if (lane == 0) a.list[atomicAdd(a.list_count, 1u)] = make_uint2(static_cast<unsigned>(c), parts);
    }
    if (begin >= end) continue;

    auto at = [&](unsigned lo, unsigned hi, int i) {
      return __shfl_sync(0xffffffffu, i < GROUP ? lo : hi, i % GROUP);
    };
    auto fetch = [&](int i) {
      if (i < end)
        Ring::copy(a, ring + i % S * Ring::STRIDE, at(p0, p1, i), tile, lane,
                   shift_of<ACCESS, GE>(a, ACCESS == CUT ? at(k0, k1, i) : 0u));
      copy_async_commit();
    };
    if (ACCESS == CUT) __syncwarp();   // the last unit's rows are read
    for (int i = 0; i < S - 1; ++i) fetch(begin + i);
    Vals<8> acc;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc.p[i] = make_float2(0.f, 0.f);
    unsigned cur = at(k0, k1, begin);
#pragma unroll 2
    for (int i = begin; i <= end; ++i) {
      const unsigned k = i < end ? at(k0, k1, i) : NO_KEY;
      if (k != cur) {
        if (to_lead) store_part(a.part + 2 * c * a.ldp, tile, lane, acc);
        else if (i == end && tail_part) store_part(a.part + (2 * c + 1) * a.ldp, tile, lane, acc);
        else store_row<GT, GE, ACCESS>(a, cur, tile, lane, acc);
        if (i == end) break;
        to_lead = false;
        cur = k;
#pragma unroll
        for (int h = 0; h < 4; ++h) acc.p[h] = make_float2(0.f, 0.f);
      }
      copy_async_wait<S - 2>();
      if (ACCESS == CUT) __syncwarp();   // all lanes' copies are there, and the row before this one is read
      fetch(i + S - 1);
      Ring::add(a, ring + i % S * Ring::STRIDE, at(p0, p1, i), tile, lane, shift_of<ACCESS, GE>(a, k), acc);
    }
  }
}

// One block per long run and 256 columns: warp w adds parts w, w + 8, ... of the run, and the warps' sums are added
// from warp 0 on. Bound by latency: 9 us for the 7 MB of 32768 ids.
template <typename OT, typename GT, int ACCESS>
__global__ void __launch_bounds__(THREADS) embedding_join_kernel(const SumArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int WARPS = THREADS / 32, GE = granule_of<OT, GT>();
  __shared__ float2 red[WARPS][SUM_COLS / 2];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const long long units = static_cast<long long>(*a.list_count) * a.tiles;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const uint2 run = a.list[u / a.tiles];
    const long long c = run.x, parts = run.y;
    const int tile = static_cast<int>(u % a.tiles);
    const unsigned k = a.key[(c + 1) * a.group - 1];
    Vals<8> acc;
#pragma unroll
    for (int i = 0; i < 4; ++i) acc.p[i] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (long long i = w; i < parts; i += WARPS) {
      Raw<float, 8> r;
      r.load(a.part + (i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.ldp + tile * SUM_COLS + lane * 8);
      const Vals<8> o = r.get();
#pragma unroll
      for (int q = 0; q < 4; ++q) acc.p[q] = __fadd2_rn(acc.p[q], o.p[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) red[w][q * 32 + lane] = acc.p[q];
    __syncthreads();
    if (w == 0) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 s = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < WARPS; ++i) s = __fadd2_rn(s, red[i][q * 32 + lane]);
        acc.p[q] = s;
      }
      store_row<GT, GE, ACCESS>(a, k, tile, lane, acc);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------ host

struct EmbeddingLayout {
  size_t key[2], pos[2], hist, list, part, total;
  long long groups, tiles, ldp;
  int group;
};

EmbeddingLayout embedding_layout(long long n, long long D) {
  EmbeddingLayout L{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 256);
    return a;
  };
  L.tiles = (n + SORT_TILE - 1) / SORT_TILE;
  L.ldp = (D + 7 + SUM_COLS - 1) / SUM_COLS * SUM_COLS;   // rows past a boundary reach up to 7 columns further
  L.group = group_of((n + 15) / 16 * ((D + SUM_COLS - 1) / SUM_COLS) <= FEW_UNITS ? 4 : 8);
  L.groups = (n + L.group - 1) / L.group;
  L.list = take(8 * (1 + static_cast<size_t>(L.groups)));   // the count, then the pairs
  for (int k = 0; k < 2; ++k) L.key[k] = take(4 * static_cast<size_t>(n));
  for (int k = 0; k < 2; ++k) L.pos[k] = take(4 * static_cast<size_t>(n));
  L.hist = take(4 * static_cast<size_t>(L.tiles) << MAX_DIGIT_BITS);
  L.part = take(8 * static_cast<size_t>(L.groups) * L.ldp);
  L.total = at;
  return L;
}

bool natural(const void *p, int dt) { return (reinterpret_cast<uintptr_t>(p) & (dt == MUON_F32 ? 3 : 1)) == 0; }

muon_status check_ids(const void *ids, muon_itype itype, int64_t n) {
  if (itype != MUON_I32 && itype != MUON_I64) return MUON_ERR_DTYPE;
  if (n > 0 && ids == nullptr) return MUON_ERR_INVALID_ARG;
  return (reinterpret_cast<uintptr_t>(ids) & (itype == MUON_I32 ? 3 : 7)) == 0 ? MUON_OK : MUON_ERR_ALIGNMENT;
}

muon_status check_embedding(const void *ids, muon_itype itype, const void *table, muon_dtype tdt, int64_t ldt,
                            const void *rows, muon_dtype rdt, int64_t ldr, int64_t n, int64_t V, int64_t D,
                            float scale) {
  if (table == nullptr || (n > 0 && rows == nullptr) || n < 0 || V < 1 || D < 1 || ldt < D || ldr < D ||
      !std::isfinite(scale))
    return MUON_ERR_INVALID_ARG;
  if (n > (1ll << 27) || V > (1ll << 30) || D > 65536) return MUON_ERR_SHAPE;
  if ((tdt != MUON_F32 && tdt != MUON_BF16) || (rdt != MUON_F32 && rdt != MUON_BF16)) return MUON_ERR_DTYPE;
  const muon_status st = check_ids(ids, itype, n);
  if (st != MUON_OK) return st;
  return natural(table, tdt) && natural(rows, rdt) ? MUON_OK : MUON_ERR_ALIGNMENT;
}

muon_status status_of(cudaError_t e) { return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA; }

template <typename TT, typename OT>
cudaError_t launch_lookup(LookupArgs a, cudaStream_t s) {
  constexpr int GE = granule_of<TT, OT>();
  const long long sms = device_sm_count();
  const dim3 block(THREADS);
  a.past_table = past<TT, GE>(a.table);
  a.past_out = past<OT, GE>(a.out);
  const bool aligned =
      a.D % GE == 0 && a.ldt % GE == 0 && a.ldo % GE == 0 && a.past_table == 0 && a.past_out == 0;
  // not aligned: the most granules that a row touches, and one more
  a.per_row = aligned ? a.D / GE : (a.D + 2 * (GE - 1)) / GE + 1;
  const long long unit = aligned ? UNIT : UNIT - 1, units = (a.n * a.per_row + unit - 1) / unit;
  const dim3 grid(static_cast<unsigned>(
      std::min((units + THREADS / 32 - 1) / (THREADS / 32), sms * (aligned ? FWD_BLOCKS : CUT_BLOCKS))));
  const long long skip = static_cast<long long>(grid.x) * (THREADS / 32) * unit;
  a.inverse = static_cast<unsigned>(((1ull << 32) + a.per_row - 1) / a.per_row);
  a.skip_rows = skip / a.per_row;
  a.skip = static_cast<int>(skip % a.per_row);
  if (aligned) return launch_pdl(embedding_forward_kernel<TT, OT>, grid, block, 0, s, a);
  constexpr size_t smem = THREADS * CUT_STAGES * (UNIT / 32) * (Raw<TT, GE>::BYTES + 4);
  static AttributesSet set;
  const cudaError_t allowed = set.once([] {
    return cudaFuncSetAttribute(embedding_forward_cut_kernel<TT, OT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(smem));
  });
  if (allowed != cudaSuccess) return allowed;
  return launch_pdl(embedding_forward_cut_kernel<TT, OT>, grid, block, smem, s, a);
}

muon_status launch_sort(const void *ids, int itype, long long n, long long V, long long padding, char *ws,
                        const EmbeddingLayout &L, const unsigned **key, const unsigned **pos, cudaStream_t s) {
  int key_bits = 1;
  while ((V >> key_bits) != 0) ++key_bits;
  const int passes = (key_bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
  SortPass p{};
  p.ids = ids;
  p.itype = itype;
  p.V = V;
  p.padding = padding;
  p.n = n;
  p.hist = reinterpret_cast<unsigned *>(ws + L.hist);
  p.tiles = static_cast<int>(L.tiles);
  p.bits = (key_bits + passes - 1) / passes;
  const dim3 grid(static_cast<unsigned>(L.tiles)), block(THREADS);
  muon_status st;
  for (int k = 0; k < passes; ++k) {
    p.shift = k * p.bits;
    p.key_out = reinterpret_cast<unsigned *>(ws + L.key[k & 1]);
    p.pos_out = reinterpret_cast<unsigned *>(ws + L.pos[k & 1]);
    launch_begin(KK_EMBED_SORT, s);
    st = status_of(launch_pdl(radix_count_kernel, grid, block, 0, s, p));
    launch_end(s);
    if (st != MUON_OK) return st;
    launch_begin(KK_EMBED_SORT, s);
    st = status_of(launch_pdl(radix_scan_kernel, dim3(1), dim3(1024), 0, s, p.hist, L.tiles << p.bits,
                              reinterpret_cast<unsigned *>(ws + L.list)));
    launch_end(s);
    if (st != MUON_OK) return st;
    launch_begin(KK_EMBED_SORT, s);
    st = status_of(launch_pdl(radix_scatter_kernel, grid, block, 0, s, p));
    launch_end(s);
    if (st != MUON_OK) return st;
    p.key_in = p.key_out;
    p.pos_in = p.pos_out;
  }
  *key = p.key_in;
  *pos = p.pos_in;
  return MUON_OK;
}

// The sort in one cluster (n <= CS_BLOCKS * CS_CHUNK) and the zeroes beside it (z.rows = 0: none). Blocks of up to 1024
// items each while there are sixteen of them: a block's rounds cost more than the cluster's barriers.
muon_status launch_prepare(const void *ids, int itype, long long n, long long V, long long padding, char *ws,
                           const EmbeddingLayout &L, const ZeroArgs &z, const unsigned **key, const unsigned **pos,
                           cudaStream_t s) {
  static AttributesSet set;
  const cudaError_t allowed = set.once([] {
    const cudaError_t e = cudaFuncSetAttribute(embedding_prepare_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(sizeof(ClusterShared)));
    if (e != cudaSuccess) return e;
    return cudaFuncSetAttribute(embedding_prepare_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);   // 16 blocks
  });
  if (allowed != cudaSuccess) return MUON_ERR_CUDA;
  int key_bits = 1;
  while ((V >> key_bits) != 0) ++key_bits;
  ClusterSort a{};
  a.ids = ids;
  a.itype = itype;
  a.V = V;
  a.padding = padding;
  a.key = reinterpret_cast<unsigned *>(ws + L.key[0]);
  a.pos = reinterpret_cast<unsigned *>(ws + L.pos[0]);
  a.list_count = reinterpret_cast<unsigned *>(ws + L.list);
  a.n = static_cast<int>(n);
  a.blocks = 1;
  while (a.blocks < CS_BLOCKS && a.blocks * 1024 < n) a.blocks *= 2;
  a.chunk = (a.n + a.blocks - 1) / a.blocks;
  a.passes = (key_bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
  a.bits = (key_bits + a.passes - 1) / a.passes;
  a.zero = z;
  const long long zeros = z.rows > 0 ? (zero_blocks(z) + a.blocks - 1) / a.blocks * a.blocks : 0;   // whole clusters
  if (zeros > (1ll << 30)) return MUON_ERR_SHAPE;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.blocks + zeros));
  cfg.blockDim = dim3(CS_THREADS);
  cfg.dynamicSmemBytes = offsetof(ClusterShared, item) + sizeof(uint2) * static_cast<size_t>(a.chunk);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(a.blocks);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.blocks > 1 ? 2 : 1;
  launch_begin(KK_EMBED_SORT, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, embedding_prepare_kernel, a);
  launch_end(s);
  *key = a.key;
  *pos = a.pos;
  return status_of(e);
}

muon_status launch_zero(const ZeroArgs &z, cudaStream_t s) {
  const long long blocks = zero_blocks(z);
  if (blocks > (1ll << 30)) return MUON_ERR_SHAPE;
  launch_begin(KK_EMBED_ZERO, s);
  const muon_status st =
      status_of(launch_pdl(embedding_zero_kernel, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, s, z));
  launch_end(s);
  return st;
}

template <typename OT, typename GT, int ACCESS, int WARPS>
muon_status launch_sum(const SumArgs &a, long long units, cudaStream_t s) {
  const auto kernel = embedding_sum_kernel<OT, GT, ACCESS, WARPS>;
  constexpr int smem = WARPS * SumRing<OT, granule_of<OT, GT>(), ACCESS, WARPS>::BYTES;
  static AttributesSet set;
  const cudaError_t allowed =
      set.once([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem); });
  if (allowed != cudaSuccess) return MUON_ERR_CUDA;
  const long long blocks = std::min((units + WARPS - 1) / WARPS, 4096ll * device_sm_count());
  launch_begin(KK_EMBED_SUM, s);
  const muon_status st =
      status_of(launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(WARPS * 32), smem, s, a));
  launch_end(s);
  return st;
}

template <typename OT, typename GT, int ACCESS>
muon_status launch_sums(SumArgs a, cudaStream_t s) {
  // CUT: a row reaches up to GE - 1 columns past its boundary
  a.tiles = (a.D + (ACCESS == CUT ? granule_of<OT, GT>() - 1 : 0) + SUM_COLS - 1) / SUM_COLS;
  const long long sms = device_sm_count();
  const long long units = static_cast<long long>(a.groups) * a.tiles;
  // few units: the time is that of one of them, which is shorter, and half the warps have twice the rows on their way
  // (8192 rows of 768 bf16: 28 us, and 33 us with groups of 32; 1024 rows: 23 and 27 us, and 31 us with eight warps too)
  muon_status st = a.group == group_of(4) ? launch_sum<OT, GT, ACCESS, 4>(a, units, s)
                                                 : launch_sum<OT, GT, ACCESS, 8>(a, units, s);
  if (st != MUON_OK || a.groups < 3) return st;   // no run can be long
  // no more long runs than a third of the groups
  const long long joins = std::min(static_cast<long long>(a.groups / 2 + 1) * a.tiles, sms * 4);
  launch_begin(KK_EMBED_JOIN, s);
  st = status_of(launch_pdl(embedding_join_kernel<OT, GT, ACCESS>, dim3(static_cast<unsigned>(joins)), dim3(THREADS), 0,
                            s, a));
  launch_end(s);
  return st;
}

template <typename OT, typename GT>
muon_status launch_sums_for(SumArgs a, cudaStream_t s) {
  constexpr int GE = granule_of<OT, GT>();
  a.past_dout = past<OT, GE>(a.dout);
  a.past_g = past<GT, GE>(a.g);
  const bool aligned = a.D % GE == 0 && a.ldo % GE == 0 && a.ldg % GE == 0 && a.past_dout == 0 && a.past_g == 0;
  return aligned ? launch_sums<OT, GT, ALIGNED>(a, s) : launch_sums<OT, GT, CUT>(a, s);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status embedding_forward(const void *ids, muon_itype itype, const void *table, muon_dtype tdt, int64_t ldt,
                              void *out, muon_dtype odt, int64_t ldo, int64_t n, int64_t V, int64_t D, float scale,
                              muon_stream_t stream) {
  muon_status st = check_embedding(ids, itype, table, tdt, ldt, out, odt, ldo, n, V, D, scale);
  if (st != MUON_OK) return st;
  if ((st = device_check()) != MUON_OK) return st;
  if (n == 0) return MUON_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  LookupArgs a{};
  a.ids = ids;
  a.table = table;
  a.out = out;
  a.ldt = ldt;
  a.ldo = ldo;
  a.n = n;
  a.V = V;
  a.itype = itype;
  a.D = static_cast<int>(D);
  a.scale = scale;
  launch_begin(KK_EMBED_FWD, s);
  cudaError_t e;
  if (tdt == MUON_F32)
    e = odt == MUON_F32 ? launch_lookup<float, float>(a, s) : launch_lookup<float, __nv_bfloat16>(a, s);
  else
    e = odt == MUON_F32 ? launch_lookup<__nv_bfloat16, float>(a, s) : launch_lookup<__nv_bfloat16, __nv_bfloat16>(a, s);
  launch_end(s);
  return status_of(e);
}

size_t embedding_workspace_bytes(int64_t n, int64_t V, int64_t D) {
  if (n < 0 || V < 1 || D < 1) return 0;
  return embedding_layout(n, D).total;
}

muon_status embedding_backward(const void *ids, muon_itype itype, const void *dout, muon_dtype odt, int64_t ldo,
                               void *dtable, muon_dtype gdt, int64_t ldg, int64_t n, int64_t V, int64_t D, float scale,
                               int64_t padding_idx, int accumulate, void *ws, size_t ws_bytes, muon_stream_t stream) {
  muon_status st = check_embedding(ids, itype, dtable, gdt, ldg, dout, odt, ldo, n, V, D, scale);
  if (st != MUON_OK) return st;
  if (ws == nullptr && n > 0) return MUON_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255) != 0) return MUON_ERR_ALIGNMENT;
  const EmbeddingLayout L = embedding_layout(n, D);
  if (n > 0 && ws_bytes < L.total) return MUON_ERR_WORKSPACE;
  if ((st = device_check()) != MUON_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int Di = static_cast<int>(D);
  ZeroArgs z{};
  if (!accumulate) {
    const long long size = gdt == MUON_F32 ? 4 : 2;
    const bool dense = ldg == D || V == 1;
    z = {static_cast<unsigned char *>(dtable), static_cast<long long>(ldg) * size, dense ? 1 : V, (dense ? V * D : D) * size};
  }
  const bool clustered = n > 0 && n <= CS_BLOCKS * CS_CHUNK;
  if (!clustered && z.rows > 0 && (st = launch_zero(z, s)) != MUON_OK) return st;
  if (n == 0) return MUON_OK;
  char *base = static_cast<char *>(ws);
  SumArgs a{};
  st = clustered ? launch_prepare(ids, itype, n, V, padding_idx, base, L, z, &a.key, &a.pos, s)
                 : launch_sort(ids, itype, n, V, padding_idx, base, L, &a.key, &a.pos, s);
  if (st != MUON_OK) return st;
  a.dout = dout;
  a.ldo = ldo;
  a.g = dtable;
  a.ldg = ldg;
  a.part = reinterpret_cast<float *>(base + L.part);
  a.list_count = reinterpret_cast<unsigned *>(base + L.list);
  a.list = reinterpret_cast<uint2 *>(a.list_count) + 1;
  a.n = n;
  a.V = V;
  a.ldp = L.ldp;
  a.D = Di;
  a.group = L.group;
  a.groups = static_cast<int>(L.groups);
  a.accumulate = accumulate != 0;
  a.scale = scale;
  if (odt == MUON_F32)
    return gdt == MUON_F32 ? launch_sums_for<float, float>(a, s) : launch_sums_for<float, __nv_bfloat16>(a, s);
  return gdt == MUON_F32 ? launch_sums_for<__nv_bfloat16, float>(a, s)
                         : launch_sums_for<__nv_bfloat16, __nv_bfloat16>(a, s);
}

}  // extern "C"
