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

// How memory is accessed:
//   SCALAR   one value at a time: bases or pitches that fit neither of the others
//   ALIGNED  every row starts on a boundary of a granule, and the width is whole granules
//   FULL     ALIGNED, and the row gives every thread all of its granules, so that nothing is asked
//   SHIFTED  rows start past a boundary (an odd width): a row is a few single values up to the first boundary (the head),
//            whole granules, and a few single values (the tail). Sixteen threads have one of these each, beside their
//            granules. A block sees rows whose index differs by multiples of 8, which all start alike, so its threads' columns
//            stay the same, and its rows share the weights.
enum Mode { SCALAR, ALIGNED, SHIFTED, FULL };

// A granule is 8 values of bf16 or, where a matrix is fp32, 4: an access of one is 16 (8 for bf16 beside fp32) bytes,
// next to the neighbouring thread's.
template <typename A, typename B>
constexpr int granule_of() { return sizeof(A) == 2 && sizeof(B) == 2 ? 8 : 4; }

// The columns of thread t of the T that hold a row, eight to a chunk: PG granules, each T granules after the one
// before, or in SCALAR single columns T apart; and in SHIFTED, for some threads, the single column `extra` (else -1).
template <int MODE_, int GE_, int T_>
struct Cols {
  static constexpr int MODE = MODE_, GE = MODE_ == SCALAR ? 8 : GE_, PG = 8 / GE, T = T_;
  int t, D, head, mine, extra;   // mine: the thread's granules (SCALAR: its columns)
  // start: the row's first value's place, in values
  __device__ __forceinline__ Cols(int t_, int D_, long long start) : t(t_), D(D_), head(0), extra(-1) {
    if (MODE == SHIFTED) head = static_cast<int>(-start & (GE - 1));
    const int total = MODE == SCALAR ? D : (D - head) / GE;
    mine = max((total - t + T - 1) / T, 0);
    if (MODE == SHIFTED) {
      const int tail = head + total * GE;
      if (t < 8 && t < head) extra = t;
      if (t >= 8 && t < 16 && tail + t - 8 < D) extra = tail + t - 8;
    }
  }
  __device__ __forceinline__ int first(int k, int j) const { return ((k * PG + j) * T + t) * GE + head; }
  __device__ __forceinline__ int col(int k, int e) const {
    return MODE == SCALAR ? (8 * k + e) * T + t : first(k, e / GE) + e % GE;
  }
  __device__ __forceinline__ bool has(int k, int j) const {
    return MODE == FULL || (MODE == SCALAR ? 8 * k : k * PG + j) < mine;
  }
  __device__ __forceinline__ bool in(int k, int e) const {   // of a granule that the thread has
    return MODE == SCALAR ? 8 * k + e < mine : true;
  }
  // SCALAR: pair i of chunk k with zeros where the row has no column
  __device__ __forceinline__ float2 only(int k, int i, float2 v) const {
    if (MODE == SCALAR) {
      if (!in(k, 2 * i)) v.x = 0.f;
      if (!in(k, 2 * i + 1)) v.y = 0.f;
    }
    return v;
  }
  __device__ __forceinline__ int columns() const { return MODE == SCALAR ? mine : mine * GE + (extra >= 0 ? 1 : 0); }
};

// The single column of a thread of a SHIFTED row
template <typename XT, typename CT>
__device__ __forceinline__ float load_extra(const XT *p, const CT &c) {
  return CT::MODE == SHIFTED && c.extra >= 0 ? load1(p, c.extra) : 0.f;
}

// A chunk as it lies in memory.
template <typename XT, int GE>
struct RawChunk {
  Raw<XT, GE> g[8 / GE];
  __device__ __forceinline__ Vals<8> get() const {
    Vals<8> o;
#pragma unroll
    for (int j = 0; j < 8 / GE; ++j) {
      const Vals<GE> v = g[j].get();
#pragma unroll
      for (int i = 0; i < GE / 2; ++i) o.p[j * GE / 2 + i] = v.p[i];
    }
    return o;
  }
};

// Columns that the thread does not have read as 0.
template <typename XT, typename CT>
__device__ __forceinline__ void load_chunk(const XT *p, const CT &c, int k, RawChunk<XT, CT::GE> &r) {
#pragma unroll
  for (int j = 0; j < CT::PG; ++j) {
    if (CT::MODE != SCALAR && c.has(k, j)) {
      r.g[j].load(p + c.first(k, j));
    } else {
      r.g[j].clear();
      if constexpr (CT::MODE == SCALAR) {
#pragma unroll
        for (int e = 0; e < CT::GE; ++e)
          if (c.in(k, e)) r.g[j].put(e, p[c.col(k, e)]);
      }
    }
  }
}

template <typename XT, typename CT>
__device__ __forceinline__ void store_values(XT *p, const CT &c, int k, int j, const Vals<8> &o) {
#pragma unroll
  for (int e = 0; e < CT::GE; ++e) {
    const float2 v = o.p[(j * CT::GE + e) / 2];
    if (c.in(k, j * CT::GE + e)) store1(p, c.col(k, j * CT::GE + e), e % 2 ? v.y : v.x);
  }
}

template <typename XT, typename CT>
__device__ __forceinline__ void store_chunk(XT *p, const CT &c, int k, const Vals<8> &o) {
#pragma unroll
  for (int j = 0; j < CT::PG; ++j) {
    if (!c.has(k, j)) continue;
    if constexpr (CT::MODE == SCALAR) {
      store_values(p, c, k, j, o);
    } else {
      Vals<CT::GE> v;
#pragma unroll
      for (int i = 0; i < CT::GE / 2; ++i) v.p[i] = o.p[j * CT::GE / 2 + i];
      store_vals(p + c.first(k, j), v);
    }
  }
}

// fp32 sums of the thread's columns to a row that starts on a boundary itself
template <typename CT>
__device__ __forceinline__ void store_sums(float *p, const CT &c, int k, const Vals<8> &o) {
  if (CT::MODE == ALIGNED || CT::MODE == FULL) {
    store_chunk(p, c, k, o);
    return;
  }
#pragma unroll
  for (int j = 0; j < CT::PG; ++j)
    if (c.has(k, j)) store_values(p, c, k, j, o);
}

// The thread's weights (or biases): `absent` where there are none. wide: the vector may be read a granule at a time.
template <typename CT>
__device__ __forceinline__ Vals<8> param_chunk(const void *p, int dt, bool wide, const CT &c, int k, float absent) {
  Vals<8> o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = make_float2(absent, absent);
  if (p == nullptr) return o;
  if ((CT::MODE == ALIGNED || CT::MODE == FULL) && wide) {
    if (dt == MUON_F32) {
      RawChunk<float, CT::GE> r;
      load_chunk(static_cast<const float *>(p), c, k, r);
      return r.get();
    }
    RawChunk<__nv_bfloat16, CT::GE> r;
    load_chunk(static_cast<const __nv_bfloat16 *>(p), c, k, r);
    return r.get();
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c.has(k, e / CT::GE) && c.in(k, e)) (e % 2 ? o.p[e / 2].y : o.p[e / 2].x) = param_at(p, dt, c.col(k, e), absent);
  return o;
}

// The rows to come. In ALIGNED and SHIFTED they are copied into a ring of STAGES places in shared memory, of which
// every thread writes and reads its own columns only: its own wait orders them, and no registers hold them meanwhile.
// In SCALAR the next row's loads wait in registers. Layout: [stage][chunk][granule][thread].
template <typename XT, typename CT, int C, int THREADS>
struct Ring {
  using R = Raw<XT, CT::GE>;
  unsigned char *base;   // of this thread
  __device__ __forceinline__ unsigned char *at(int stage, int k, int j) const {
    return base + ((stage * C + k) * CT::PG + j) * (THREADS * R::BYTES);
  }
  __device__ __forceinline__ void fetch(const XT *row, const CT &c, int stage) const {
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int j = 0; j < CT::PG; ++j)
        if (c.has(k, j)) copy_async<R::BYTES>(at(stage, k, j), row + c.first(k, j));
  }
  __device__ __forceinline__ Vals<8> get(int k, int stage) const {
    RawChunk<XT, CT::GE> r;
#pragma unroll
    for (int j = 0; j < CT::PG; ++j) r.g[j].load(reinterpret_cast<const XT *>(at(stage, k, j)));
    return r.get();
  }
};

// A vector of weights (or biases), as each thread wants its own columns of it row after row: in registers where there
// is one chunk, as fp32 in shared memory where there are several and they fit beside the ring, and otherwise read (from
// cache) row after row. The block's rows share it.
template <typename CT, int C, bool SHARED>
struct Params {
  static constexpr int STRIDE = CT::T, BYTES = SHARED ? 32 * C * STRIDE : 0;
  const void *p;
  int dt;
  bool wide;
  float absent;
  float4 *base;   // SHARED: [2 chunk + half][STRIDE], of this thread
  Vals<8> one;
  // what the rows share is put by the threads of the block's first row, and read after a barrier
  __device__ __forceinline__ void init(const CT &c, int slot) {
    if constexpr (C == 1) one = param_chunk(p, dt, wide, c, 0, absent);
    if constexpr (SHARED) {
      if (slot != 0) return;
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const Vals<8> o = param_chunk(p, dt, wide, c, k, absent);
        base[(2 * k) * STRIDE] = make_float4(o.p[0].x, o.p[0].y, o.p[1].x, o.p[1].y);
        base[(2 * k + 1) * STRIDE] = make_float4(o.p[2].x, o.p[2].y, o.p[3].x, o.p[3].y);
      }
    }
  }
  __device__ __forceinline__ Vals<8> get(const CT &c, int k) const {
    if constexpr (C == 1) return one;
    if constexpr (SHARED) {
      const float4 u = base[(2 * k) * STRIDE], v = base[(2 * k + 1) * STRIDE];
      return {{make_float2(u.x, u.y), make_float2(u.z, u.w), make_float2(v.x, v.y), make_float2(v.z, v.w)}};
    }
    return param_chunk(p, dt, wide, c, k, absent);
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

// Row slot `slot` of the R that a block holds starts at first_row, and the block's slots are rows_apart from each other;
// the grid of SHIFTED is a multiple of eight blocks.
template <int MODE>
constexpr int rows_apart = MODE == SHIFTED ? 8 : 1;
template <int R, int MODE>
__device__ __forceinline__ long long first_row(int slot) {
  const long long b = blockIdx.x;
  return MODE == SHIFTED ? b % 8 + 8 * (b / 8 * R + slot) : b * R + slot;
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

// ------------------------------------------------------------------------------------------ host

constexpr int SM_SHARED = 227 * 1024;
constexpr int STATIC_SHARED = 12 * 1024;   // more than any kernel's static share

// Once for each kernel and device: it may take more than 48 KB, and the multiprocessor is to hold as many blocks of it as fit.
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

// An output that takes the place of an input has its dtype and pitch (of a single row: its dtype), so that every value is
// written where it was read.
inline bool in_place_ok(const void *in, int idt, long long ldi, const void *out, int odt, long long ldo, long long N) {
  return N == 0 || in != out || (idt == odt && (N == 1 || ldi == ldo));
}

// The mode for matrices whose bases are all 16-byte aligned (or not), the pitch of the first, and whether all pitches
// are the same modulo 8.
inline Mode mode_of(bool bases, bool pitches, long long ld, long long D) {
  if (!bases || !pitches || D < 8) return SCALAR;
  return ld % 8 == 0 && D % 8 == 0 ? ALIGNED : SHIFTED;
}

}  // namespace
}  // namespace muon
