// Embedding lookup with scaling, and the table's gradient by sorted tokens.
//
//   out_i = scale * E[id_i]                         (an id outside [0, V) names no row: zeros)
//   dE_v  = scale * sum_{i : id_i = v} dout_i       (in increasing i, fp32, rounded once at the end)
//
// The gradient sorts the ids with their positions (a stable radix sort, so that equal ids keep the order of
// their positions), and then sums each run of equal ids. No sum goes through an atomic: the same inputs give
// the same bits.
//
//   embedding_forward_kernel  one warp per row of up to 1024 columns: a gather that reads and writes each byte once.
//   embedding_zero_kernel     zeroes the gradient (not called when it accumulates).
//   embedding_cluster_sort_kernel  the sort of up to 65536 ids in one cluster's shared memory, under the zero kernel.
//   radix_*_kernel            one pass of a longer sort: digit counts per tile, their scan, the stable scatter.
//   embedding_sum_kernel      one warp per 32 sorted positions and 256 columns; rows of dout go to registers eight
//                             at a time whether or not they belong to one id, since most ids occur once or twice.
//   embedding_join_kernel     ids whose run spans a whole group of 32 or more: adds the groups' sums in order.
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
constexpr int FWD_COLS = 1024;   // columns per warp of the lookup
constexpr int fwd_blocks(size_t value) { return value == 2 ? 6 : 4; }   // resident blocks of the lookup
constexpr int SUM_COLS = 256;    // columns per warp of the gradient's sums: 8 per lane
constexpr int GROUP = 32;        // sorted positions per warp of the gradient's sums
constexpr int SORT_TILE = 4096;  // keys per block of a sort pass
constexpr int MAX_DIGIT_BITS = 9;
constexpr unsigned NO_KEY = 0xffffffffu;

__device__ __forceinline__ long long load_id(const void *ids, int itype, long long i) {
  return itype == MUON_I32 ? static_cast<long long>(static_cast<const int *>(ids)[i])
                           : static_cast<const long long *>(ids)[i];
}

// ------------------------------------------------------------------------------------------ lookup

// Warps take (row, 1024 columns) units in turn. A unit's four 16-byte loads per lane (of bf16) are all in flight before
// the first is used, and the id of the next unit is loaded under them, so that a unit waits for one latency, not two.
template <typename TT, typename OT, bool VEC>
__global__ void __launch_bounds__(THREADS, fwd_blocks(sizeof(TT))) embedding_forward_kernel(
    const void *ids, int itype, const TT *table, long long ldt, OT *out, long long ldo, long long n, long long V, int D,
    int tiles, float scale) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long units = n * tiles, warps = static_cast<long long>(gridDim.x) * (THREADS / 32);
  long long u = static_cast<long long>(blockIdx.x) * (THREADS / 32) + threadIdx.x / 32;
  long long i = u / tiles, next_id = u < units ? load_id(ids, itype, i) : 0;
  for (; u < units; u += warps) {
    const long long id = next_id, row = i;
    const int c0 = static_cast<int>(u - i * tiles) * FWD_COLS;
    const bool in = id >= 0 && id < V;
    const TT *src = table + (in ? id : 0) * ldt;
    OT *dst = out + row * ldo;
    i = (u + warps) / tiles;
    if constexpr (VEC) {
      Raw8<TT> r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + (k * 32 + lane) * 8;
        if (c < D) r[k].load(src + c);
      }
      if (u + warps < units) next_id = load_id(ids, itype, i);
      const float2 s2 = make_float2(scale, scale);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int c = c0 + (k * 32 + lane) * 8;
        Oct o = r[k].get();
#pragma unroll
        for (int q = 0; q < 4; ++q) o.p[q] = in ? __fmul2_rn(o.p[q], s2) : make_float2(0.f, 0.f);
        if (c < D) store_oct(dst + c, o);
      }
    } else {
      if (u + warps < units) next_id = load_id(ids, itype, i);
#pragma unroll 8
      for (int k = 0; k < FWD_COLS / 32; ++k) {
        const int c = c0 + k * 32 + lane;
        if (c < D) store1(dst, c, in ? load1(src, c) * scale : 0.f);
      }
    }
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

// The whole sort in one cluster, for n <= 8 * 8192: block b holds the sorted positions [b * chunk, (b + 1) * chunk) in
// its shared memory, and a pass moves every item to its place in any block's. A thread keeps its items in registers
// while their places are computed, so one buffer is enough. Warp w of a block has the block's items [w * per, ...), 32
// at a time; an item's place is its digit's first place, plus the digit's items in earlier blocks, warps, rounds and
// lanes: stable, like the passes above.
constexpr int CS_THREADS = 512;    // few enough registers to run beside the zero kernel's blocks
constexpr int CS_WARPS = CS_THREADS / 32;
constexpr int CS_ROUNDS = 16;                              // items per thread
constexpr int CS_CHUNK = CS_THREADS * CS_ROUNDS;           // items per block
constexpr int CS_BLOCKS = 8;

struct ClusterSort {
  const void *ids;
  int itype;
  long long V, padding;
  unsigned *key, *pos;      // sorted
  unsigned *list_count;
  int n, blocks, chunk, passes, bits;
  int after_zero;           // the launch before is the zero kernel, under which this one runs
};

struct ClusterShared {
  uint2 item[CS_CHUNK];                                     // (key, position)
  unsigned short place[CS_WARPS][1 << MAX_DIGIT_BITS];
  unsigned count[2][1 << MAX_DIGIT_BITS];                   // the block's items of each digit; by parity of the pass
  unsigned first[1 << MAX_DIGIT_BITS];                      // where the block's first item of each digit goes
  unsigned warp_total[CS_WARPS];
};

__global__ void __launch_bounds__(CS_THREADS, 2) embedding_cluster_sort_kernel(const ClusterSort a) {
  // The zero kernel passes its own wait before it lets this kernel start, so whatever came before it is complete; this
  // kernel waits for the zero kernel only at its end, so that the sums, which wait for this one, follow both.
  if (!a.after_zero) pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
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
  if (a.after_zero) pdl_wait();
}

// ------------------------------------------------------------------------------------------ sums

template <typename GT>
__global__ void __launch_bounds__(THREADS) embedding_zero_kernel(GT *g, long long ldg, long long V, int D, int vec) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const long long tid = static_cast<long long>(blockIdx.x) * THREADS + threadIdx.x;
  const long long stride = static_cast<long long>(gridDim.x) * THREADS;
  if (vec) {
    const int per = D / 8;
    const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (long long u = tid; u < V * per; u += stride) store8(g + u / per * ldg + u % per * 8, z);
  } else {
    for (long long u = tid; u < V * D; u += stride) store1(g, u / D * ldg + u % D, 0.f);
  }
}

struct SumArgs {
  const unsigned *key, *pos;   // sorted
  const void *dout;
  long long ldo;
  void *g;
  long long ldg;
  float *part;                 // [2 * groups][ldp]: sums of the runs that the join kernel finishes
  unsigned *list, *list_count; // groups where such a run starts
  long long n, V, ldp;
  int D, tiles, groups, accumulate;
  float scale;
};

// A lane's eight of a row's 256 columns: contiguous on the vector path (which needs a width of whole eights).
template <bool VEC>
__device__ __forceinline__ int sum_col(int c0, int lane, int e) {
  return VEC ? c0 + lane * 8 + e : c0 + e * 32 + lane;
}

template <typename T, bool VEC>
__device__ __forceinline__ void load_cols(const T *p, int c0, int lane, int D, Raw8<T> &r) {
  if constexpr (VEC) {
    if (c0 + lane * 8 < D) r.load(p + c0 + lane * 8);
  } else {
    T f[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = T(0.f);
      if (sum_col<false>(c0, lane, e) < D) f[e] = p[sum_col<false>(c0, lane, e)];
    }
    r.set(f);
  }
}

// The gradient row's columns: scale * acc, added to what is there if asked.
template <typename GT, bool VEC>
__device__ __forceinline__ void store_row(GT *p, int c0, int lane, int D, const Oct &acc, float scale,
                                          int accumulate) {
  if (VEC && c0 + lane * 8 >= D) return;
  Oct o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o.p[q] = make_float2(0.f, 0.f);
  if (accumulate) {
    Raw8<GT> r;
    load_cols<GT, VEC>(p, c0, lane, D, r);
    o = r.get();
  }
  const float2 s2 = make_float2(scale, scale);
#pragma unroll
  for (int q = 0; q < 4; ++q) o.p[q] = __ffma2_rn(acc.p[q], s2, o.p[q]);
  if constexpr (VEC) {
    store_oct(p + c0 + lane * 8, o);
  } else {
    const float f[8] = {o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y, o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y};
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (sum_col<false>(c0, lane, e) < D) store1(p, sum_col<false>(c0, lane, e), f[e]);
  }
}

// Partial sums keep the lane's own eight columns together whatever the path: written and read by the same mapping.
__device__ __forceinline__ void store_part(float *p, int c0, int lane, const Oct &acc) {
  store_oct(p + c0 + lane * 8, acc);
}

// A run of equal ids that starts in group c belongs to it, unless the run covers the whole of the next group and
// goes on (a long run): then every group sums its own part, into part[2c + 1] where the run starts and part[2c]
// where it came from the group before, and the join kernel adds the parts. So a warp sums at most 63 positions. While
// it adds four rows the loads of the next four are in flight, whether or not they belong to one id.
template <typename OT, typename GT, bool VEC>
__global__ void __launch_bounds__(THREADS, sizeof(OT) == 2 ? 3 : 2) embedding_sum_kernel(const SumArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long units = static_cast<long long>(a.groups) * a.tiles;
  const long long warps = static_cast<long long>(gridDim.x) * (THREADS / 32);
  const unsigned none = static_cast<unsigned>(a.V);
  for (long long u = static_cast<long long>(blockIdx.x) * (THREADS / 32) + threadIdx.x / 32; u < units; u += warps) {
    const long long c = u / a.tiles;
    const int tile = static_cast<int>(u - c * a.tiles), c0 = tile * SUM_COLS;
    const long long s = c * GROUP;
    auto key_at = [&](long long i) { return i >= 0 && i < a.n ? a.key[i] : NO_KEY; };
    const unsigned k0 = key_at(s + lane), k1 = key_at(s + GROUP + lane);
    const unsigned p0 = s + lane < a.n ? a.pos[s + lane] : 0u;
    const unsigned p1 = s + GROUP + lane < a.n ? a.pos[s + GROUP + lane] : 0u;
    const unsigned before = key_at(s - 1), far_before = key_at(s - GROUP - 1), far_after = key_at(s + 2 * GROUP);
    const unsigned first = __shfl_sync(0xffffffffu, k0, 0), last = __shfl_sync(0xffffffffu, k0, 31);
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
    if (tail_part && tile == 0 && lane == 0) a.list[atomicAdd(a.list_count, 1u)] = static_cast<unsigned>(c);
    if (begin >= end) continue;

    const OT *dout = static_cast<const OT *>(a.dout);
    GT *g = static_cast<GT *>(a.g);
    auto at = [&](unsigned lo, unsigned hi, int i) {
      return __shfl_sync(0xffffffffu, i < GROUP ? lo : hi, i % GROUP);
    };
    constexpr int U = 4;
    Raw8<OT> raw[2][U];
    auto fetch = [&](int i0, Raw8<OT> *r) {
#pragma unroll
      for (int q = 0; q < U; ++q)
        if (i0 + q < end)
          load_cols<OT, VEC>(dout + static_cast<long long>(at(p0, p1, i0 + q)) * a.ldo, c0, lane, a.D, r[q]);
    };
    Oct acc;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc.p[q] = make_float2(0.f, 0.f);
    unsigned cur = at(k0, k1, begin);
    auto flush = [&](bool tail) {
      if (to_lead) store_part(a.part + 2 * c * a.ldp, c0, lane, acc);
      else if (tail) store_part(a.part + (2 * c + 1) * a.ldp, c0, lane, acc);
      else store_row<GT, VEC>(g + static_cast<long long>(cur) * a.ldg, c0, lane, a.D, acc, a.scale, a.accumulate);
      to_lead = false;
    };
    auto add = [&](int i0, const Raw8<OT> *r) {
#pragma unroll
      for (int q = 0; q < U; ++q) {
        if (i0 + q >= end) break;
        const unsigned k = at(k0, k1, i0 + q);
        if (k != cur) {
          flush(false);
          cur = k;
#pragma unroll
          for (int h = 0; h < 4; ++h) acc.p[h] = make_float2(0.f, 0.f);
        }
        const Oct o = r[q].get();
#pragma unroll
        for (int h = 0; h < 4; ++h) acc.p[h] = __fadd2_rn(acc.p[h], o.p[h]);
      }
    };
    fetch(begin, raw[0]);
    for (int i0 = begin; i0 < end; i0 += 2 * U) {
      fetch(i0 + U, raw[1]);
      add(i0, raw[0]);
      fetch(i0 + 2 * U, raw[0]);
      add(i0 + U, raw[1]);
    }
    flush(tail_part);
  }
}

// One block per long run and 256 columns: warp w adds parts w, w + 8, ... of the run, and the warps' sums are added
// in order.
template <typename GT, bool VEC>
__global__ void __launch_bounds__(THREADS) embedding_join_kernel(const SumArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  constexpr int WARPS = THREADS / 32;
  __shared__ float2 red[WARPS][SUM_COLS / 2];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32;
  const long long units = static_cast<long long>(*a.list_count) * a.tiles;
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const long long c = a.list[u / a.tiles];
    const int c0 = static_cast<int>(u % a.tiles) * SUM_COLS;
    const unsigned k = a.key[c * GROUP + GROUP - 1];
    long long lo = c + 2, hi = a.groups;   // the first group after c + 1 whose first key is not k
    while (lo < hi) {
      const long long mid = (lo + hi) / 2;
      if (a.key[mid * GROUP] == k) lo = mid + 1;
      else hi = mid;
    }
    const long long parts = lo - c;
    Oct acc;
#pragma unroll
    for (int q = 0; q < 4; ++q) acc.p[q] = make_float2(0.f, 0.f);
#pragma unroll 4
    for (long long i = w; i < parts; i += WARPS) {
      Raw8<float> r;
      r.load(a.part + (i == 0 ? 2 * c + 1 : 2 * (c + i)) * a.ldp + c0 + lane * 8);
      const Oct o = r.get();
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
        for (int k2 = 0; k2 < WARPS; ++k2) s = __fadd2_rn(s, red[k2][q * 32 + lane]);
        acc.p[q] = s;
      }
      store_row<GT, VEC>(static_cast<GT *>(a.g) + static_cast<long long>(k) * a.ldg, c0, lane, a.D, acc, a.scale,
                         a.accumulate);
    }
    __syncthreads();
  }
}

// ------------------------------------------------------------------------------------------ host

struct EmbeddingLayout {
  size_t key[2], pos[2], hist, list, part, total;
  long long groups, tiles, ldp;
};

EmbeddingLayout embedding_layout(long long n, long long D) {
  EmbeddingLayout L{};
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t a = at;
    at += align_up(bytes, 256);
    return a;
  };
  L.groups = (n + GROUP - 1) / GROUP;
  L.tiles = (n + SORT_TILE - 1) / SORT_TILE;
  L.ldp = (D + SUM_COLS - 1) / SUM_COLS * SUM_COLS;
  L.list = take(4 * (1 + static_cast<size_t>(n) / GROUP));
  for (int k = 0; k < 2; ++k) L.key[k] = take(4 * static_cast<size_t>(n));
  for (int k = 0; k < 2; ++k) L.pos[k] = take(4 * static_cast<size_t>(n));
  L.hist = take(4 * static_cast<size_t>(L.tiles) << MAX_DIGIT_BITS);
  L.part = take(8 * static_cast<size_t>(L.groups) * L.ldp);
  L.total = at;
  return L;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
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
cudaError_t launch_forward(bool vec, dim3 grid, cudaStream_t s, const void *ids, int itype, const void *table,
                           long long ldt, void *out, long long ldo, long long n, long long V, int D, int tiles,
                           float scale) {
  const dim3 block(THREADS);
  const TT *t = static_cast<const TT *>(table);
  OT *o = static_cast<OT *>(out);
  return vec ? launch_pdl(embedding_forward_kernel<TT, OT, true>, grid, block, 0, s, ids, itype, t, ldt, o, ldo, n, V,
                          D, tiles, scale)
             : launch_pdl(embedding_forward_kernel<TT, OT, false>, grid, block, 0, s, ids, itype, t, ldt, o, ldo, n, V,
                          D, tiles, scale);
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

// The sort in one cluster (n <= CS_BLOCKS * CS_CHUNK). Blocks of 4096 items each up to eight of them: a block's rounds
// cost more than the cluster's barriers.
muon_status launch_cluster_sort(const void *ids, int itype, long long n, long long V, long long padding, char *ws,
                                const EmbeddingLayout &L, bool after_zero, const unsigned **key, const unsigned **pos,
                                cudaStream_t s) {
  static const cudaError_t allowed = cudaFuncSetAttribute(
      embedding_cluster_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(ClusterShared)));
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
  while (a.blocks < CS_BLOCKS && a.blocks * 4096 < n) a.blocks *= 2;
  a.chunk = (a.n + a.blocks - 1) / a.blocks;
  a.passes = (key_bits + MAX_DIGIT_BITS - 1) / MAX_DIGIT_BITS;
  a.bits = (key_bits + a.passes - 1) / a.passes;
  a.after_zero = after_zero ? 1 : 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.blocks));
  cfg.blockDim = dim3(CS_THREADS);
  cfg.dynamicSmemBytes = sizeof(ClusterShared);
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
  const cudaError_t e = cudaLaunchKernelEx(&cfg, embedding_cluster_sort_kernel, a);
  launch_end(s);
  *key = a.key;
  *pos = a.pos;
  return status_of(e);
}

template <typename OT, typename GT, bool VEC>
muon_status launch_sums(const SumArgs &a, cudaStream_t s) {
  const long long sms = device_sm_count();
  const long long units = static_cast<long long>(a.groups) * a.tiles;
  const long long blocks = std::min((units + THREADS / 32 - 1) / (THREADS / 32), sms * 4096);
  launch_begin(KK_EMBED_SUM, s);
  muon_status st = status_of(launch_pdl(embedding_sum_kernel<OT, GT, VEC>, dim3(static_cast<unsigned>(blocks)),
                                        dim3(THREADS), 0, s, a));
  launch_end(s);
  if (st != MUON_OK || a.groups < 3) return st;   // no run can be long
  launch_begin(KK_EMBED_JOIN, s);
  st = status_of(launch_pdl(embedding_join_kernel<GT, VEC>, dim3(static_cast<unsigned>(sms * 4)), dim3(THREADS), 0, s,
                            a));
  launch_end(s);
  return st;
}

template <typename OT, typename GT>
muon_status launch_sums_vec(bool vec, const SumArgs &a, cudaStream_t s) {
  return vec ? launch_sums<OT, GT, true>(a, s) : launch_sums<OT, GT, false>(a, s);
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
  const bool vec = aligned16(table) && aligned16(out) && ldt % 8 == 0 && ldo % 8 == 0 && D % 8 == 0;
  const int tiles = static_cast<int>((D + FWD_COLS - 1) / FWD_COLS), Di = static_cast<int>(D);
  const long long units = n * tiles, sms = device_sm_count();
  const dim3 grid(static_cast<unsigned>(std::min((units + THREADS / 32 - 1) / (THREADS / 32), sms * fwd_blocks(tdt == MUON_F32 ? 4 : 2))));
  launch_begin(KK_EMBED_FWD, s);
  cudaError_t e;
  if (tdt == MUON_F32 && odt == MUON_F32)
    e = launch_forward<float, float>(vec, grid, s, ids, itype, table, ldt, out, ldo, n, V, Di, tiles, scale);
  else if (tdt == MUON_F32)
    e = launch_forward<float, __nv_bfloat16>(vec, grid, s, ids, itype, table, ldt, out, ldo, n, V, Di, tiles, scale);
  else if (odt == MUON_F32)
    e = launch_forward<__nv_bfloat16, float>(vec, grid, s, ids, itype, table, ldt, out, ldo, n, V, Di, tiles, scale);
  else
    e = launch_forward<__nv_bfloat16, __nv_bfloat16>(vec, grid, s, ids, itype, table, ldt, out, ldo, n, V, Di, tiles,
                                                     scale);
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
  const long long sms = device_sm_count();
  const int Di = static_cast<int>(D);
  const bool gvec = aligned16(dtable) && ldg % 8 == 0 && D % 8 == 0;
  if (!accumulate) {
    const long long work = V * (gvec ? D / 8 : D);
    const dim3 grid(static_cast<unsigned>(std::min((work + THREADS - 1) / THREADS, sms * 4))), block(THREADS);   // room for the sort beside it
    launch_begin(KK_EMBED_ZERO, s);
    st = status_of(gdt == MUON_F32
                       ? launch_pdl(embedding_zero_kernel<float>, grid, block, 0, s, static_cast<float *>(dtable), ldg,
                                    V, Di, static_cast<int>(gvec))
                       : launch_pdl(embedding_zero_kernel<__nv_bfloat16>, grid, block, 0, s,
                                    static_cast<__nv_bfloat16 *>(dtable), ldg, V, Di, static_cast<int>(gvec)));
    launch_end(s);
    if (st != MUON_OK) return st;
  }
  if (n == 0) return MUON_OK;
  char *base = static_cast<char *>(ws);
  SumArgs a{};
  st = n <= CS_BLOCKS * CS_CHUNK
           ? launch_cluster_sort(ids, itype, n, V, padding_idx, base, L, !accumulate, &a.key, &a.pos, s)
           : launch_sort(ids, itype, n, V, padding_idx, base, L, &a.key, &a.pos, s);
  if (st != MUON_OK) return st;
  a.dout = dout;
  a.ldo = ldo;
  a.g = dtable;
  a.ldg = ldg;
  a.part = reinterpret_cast<float *>(base + L.part);
  a.list_count = reinterpret_cast<unsigned *>(base + L.list);
  a.list = a.list_count + 1;
  a.n = n;
  a.V = V;
  a.ldp = L.ldp;
  a.D = Di;
  a.tiles = static_cast<int>((D + SUM_COLS - 1) / SUM_COLS);
  a.groups = static_cast<int>(L.groups);
  a.accumulate = accumulate != 0;
  a.scale = scale;
  const bool vec = aligned16(dout) && ldo % 8 == 0 && aligned16(dtable) && ldg % 8 == 0 && D % 8 == 0;
  if (odt == MUON_F32)
    return gdt == MUON_F32 ? launch_sums_vec<float, float>(vec, a, s) : launch_sums_vec<float, __nv_bfloat16>(vec, a, s);
  return gdt == MUON_F32 ? launch_sums_vec<__nv_bfloat16, float>(vec, a, s)
                         : launch_sums_vec<__nv_bfloat16, __nv_bfloat16>(vec, a, s);
}

}  // extern "C"
