// The cross entropy of a linear head, z = h W^T, without keeping the N x V logits, and its gradients.
//
//     lse_i = log sum_v exp z_iv,   loss_i = w_i (lse_i - z_it),   dz_iv = g_i w_i (exp(z_iv - lse_i) - [v = t_i])
//     dh = dz W,   dW = dz^T h
//
// Rows go through in pieces of up to 2^30 logits (plan()); of a piece, only gradients put its dz into memory. Per piece:
//   logits  z a tile of 256 x 256 at a time on the tensor cores; a tile's accumulators leave as one running maximum and sum
//           of exponentials for each row and half tile (online softmax) and the target's logit
//   combine the parts' pairs into lse and the loss; and h without the rows that have no part in the loss, for dw
//   dlogits dz = g w (exp(z - lse) - [v = t]), rounded to bf16 as an operand of the two products that follow, without a factor
//           that all rows share, which the products' sums take: the targets' -1, most of dz, is then exact. It comes
//           from the exponentials, which the logits' epilogue has kept, in the joint call of wide rows; else from the product,
//           computed again. For fp32 gradients dz is the sum of two bf16 terms, which holds 16 bits of it, and always from
//           the product
//   dh      dz W, the contraction over V cut into slices where the tiles alone would leave SMs without work
//   dw      dz^T h, added up over the pieces in fp32
//   reduce  adds slices in their order and rounds once
//
// One kernel computes all the products (ce_gemm_kernel), a persistent one of CTA pairs as the Newton-Schulz GEMMs of
// ns_gemm.cu are: tcgen05 cta_group::2 MMAs of 256 x 256 x 16 from operands that TMA brings in 64-deep stages, two
// accumulators in tensor memory so that one tile's epilogue runs under the next one's MMAs. Bound by the tensor cores
// wherever there are a few hundred rows, by the reading of W below that.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstring>

#include "internal.h"
#include "ptx.cuh"
#include "tensor_map.h"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int BM = 128;                      // accumulator rows per CTA: 256 per pair
constexpr int BK = 64;
__host__ __device__ constexpr int tile_rows(bool pair) { return pair ? 2 * BM : BM; }
__host__ __device__ constexpr int tile_cols(bool pair) { return pair ? 256 : 128; }
// How a product's rows are cut: pairs of CTAs share tiles of 256 rows, or a CTA has a tile of up to 128, or of up to
// FEW_ROWS, alone. See ce_gemm_kernel.
enum Shape : int { PAIRED = 0, ALONE = 1, FEW = 2 };
constexpr int FEW_ROWS = 32;
constexpr int B_COLS = 128;                  // of B in a CTA: half of a pair's tile
constexpr int B_BYTES = B_COLS * BK * 2;
constexpr int MAX_STAGES = 9;
__host__ __device__ constexpr int stages(int shape) { return shape == FEW ? MAX_STAGES : 6; }
__host__ __device__ constexpr int a_bytes(int shape) { return (shape == FEW ? FEW_ROWS : BM) * BK * 2; }
__host__ __device__ constexpr int stage_bytes(int shape) { return a_bytes(shape) + B_BYTES; }
constexpr int EPI_WARPS = 8;
constexpr int JOB_WARPS = 12;                // run a pass over memory beside the MMAs
constexpr int FIRST_JOB_WARP = 2 + EPI_WARPS;
__host__ __device__ constexpr int gemm_threads(bool job) { return 32 * (FIRST_JOB_WARP + (job ? JOB_WARPS : 0)); }
constexpr int BUF_BYTES = 32 * 128;          // an epilogue warp's staging: 32 rows of 128 bytes
// Widths from which on the joint call keeps the exponentials rather than computing the logits twice: what they cost in memory
// does not depend on the width (8192 x 32000: 541 us against 402 at 64, 672 and 620 at 384, 706 and 739 at 512; 8192 x 50304 x
// 768: 1382 and 1624 us).
constexpr int KEEP_WIDTH = 512;
constexpr int GROUP = 16;                    // row tiles that take a column of tiles together
constexpr float LOG2E = 1.4426950408889634f;
constexpr long long MAX_PITCH = 1ll << 37;   // elements: a tensor map's strides are below 2^40 bytes
constexpr long long PIECE_ELEMS = 1ll << 30; // of dz, or of h, in a piece
constexpr long long SMS = 152;               // of a GB300: slices are counted by it, so that sums have one order
constexpr int MAX_SPLIT = 64;
// An accumulator of the tensor cores loses up to a unit in the last place with each step of 16 products, always towards
// zero: over a contraction of 128256 that is 2e-5 of the result (dh, 1024 x 128256 x 4096). For fp32 gradients it therefore
// adds up all of the lower term's products, which are small, and then 8 steps of 64 of the upper one's; the epilogue's threads
// add that to sums of their own, rounding to nearest (add_segment). The sums' error is then 7e-7, less than the 2^-17 to which
// two terms hold dz. (2048 x 50304 x 768: 641 us with 32 steps, whose error is 2.5e-6, 657 with 16 and 1.3e-6, 679 with 8, 714
// with 4 and 4e-7.)
constexpr int SEGMENT = 8;

// LOGITS leaves statistics alone, LOGITS_EXP the tile's exponentials too (for the joint call).
enum Kind : int { LOGITS = 0, LOGITS_EXP = 1, DLOGITS = 2, DH = 3, DW = 4 };

struct Ctrl {
  uint64_t full[MAX_STAGES], empty[MAX_STAGES];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
};

constexpr size_t smem_bytes(int shape) {
  return static_cast<size_t>(stages(shape)) * stage_bytes(shape) + EPI_WARPS * BUF_BYTES + sizeof(Ctrl) + 1024;
}
static_assert(sizeof(Ctrl) <= 512 && smem_bytes(PAIRED) <= 232448 && smem_bytes(FEW) <= 232448, "shared memory over budget");

// What a row of exponentials needs to become dz: -lse log2(e), g w, and the target, -1 for a row that has no part in the
// loss. Four floats in memory, written by ce_combine_kernel.
struct RowState {
  float base, g;
  int target;
  static __device__ __forceinline__ RowState of(const float4 &v) { return RowState{v.x, v.y, __float_as_int(v.z)}; }
};

// dz from the exponentials that LOGITS_EXP kept, in their place: dz = g w (exp(m_part - lse) e - [v = t]).
struct ScaleJob {
  uint16_t *x;                 // rows of ld elements
  long long ld;
  const float2 *partials;      // [parts][rows]
  const float4 *row_state;
  int rows, cols, part_cols;
};

struct CeArgs {
  CUtensorMap map_a, map_b, map_out;   // map_out: dz, the exponentials in its place, or the output
  int rows, cols;                      // of the output
  int m_tiles, n_tiles;
  int a_box;                           // rows of A that a stage loads: all, or, for a CTA alone, those that there are
  int k_iters, k_low;                  // 64-deep steps, the first k_low of them over A's second plane (dz's lower term)
  int split, k_per;
  int k_seg;                           // steps past the lower term's that one accumulator adds up
  int planes;                          // DLOGITS: terms of dz
  long long total;                     // tile pairs times slices
  // LOGITS, LOGITS_EXP, DLOGITS
  const void *targets;
  int itype;
  const float *weights, *grad, *lse;
  float2 *partials;                    // [parts][rows]: maximum and sum of exponentials
  float *z_target;                     // [rows]
  // DH, DW
  void *out;
  long long ld_out, slice_stride;      // elements; slice s goes to out + s * slice_stride
  float factor;                        // of the products
  int out_f32, accumulate, vec, tma;
  ScaleJob job;
  uint32_t *err;
  unsigned long long timeout_ns;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ long long target_of(const void *t, int itype, long long i) {
  return itype == MUON_I32 ? static_cast<long long>(static_cast<const int *>(t)[i]) : static_cast<const long long *>(t)[i];
}

// The end of the segment that begins at step ks: the lower term's steps and k_seg others.
__device__ __forceinline__ int segment_end(const CeArgs &a, int ks, int k1) { return min(k1, max(ks, a.k_low) + a.k_seg); }

// Unit u: slice, then groups of GROUP row tiles, in a group column after column of tiles. A wave of 76 pairs then
// reads GROUP row tiles and five column tiles, which L2 holds, whatever the matrix' size.
__device__ __forceinline__ void decode(const CeArgs &a, long long u, int &slice, int &ti, int &tj) {
  const int tiles = a.m_tiles * a.n_tiles;
  slice = static_cast<int>(u / tiles);
  int r = static_cast<int>(u - static_cast<long long>(slice) * tiles);
  const int per_group = GROUP * a.n_tiles;
  const int g = r / per_group;
  r -= g * per_group;
  const int in_group = min(GROUP, a.m_tiles - g * GROUP);
  tj = r / in_group;
  ti = g * GROUP + (r - tj * in_group);
}

// The warp's staging buffer: line i holds 128 bytes of output row i, its 16-byte piece q at q ^ (i & 7), the order in
// which TMA reads a box of 128-byte rows with the 128-byte swizzle; rows and columns of pieces are free of bank conflicts.
__device__ __forceinline__ uint4 *piece(uint8_t *buf, int i, int q) {
  return reinterpret_cast<uint4 *>(buf + i * 128 + ((q ^ (i & 7)) << 4));
}

__device__ __forceinline__ unsigned pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const unsigned *>(&h);
}

// Exponentials are at most 1: kept in fp16 times 2^13, they have 11 bits down to 2^-27 of the part's largest and the last at
// 2^-37, for the gradients of columns that no row gives much. (Four times 2^13 is still finite: 1 is a power of 2 off by up to
// 2 where z is 2^25 and its product with log2(e) rounded.)
constexpr float KEPT = 8192.f;
__device__ __forceinline__ unsigned pack2_kept(float a, float b) {
  const float2 x = __fmul2_rn(make_float2(a, b), make_float2(KEPT, KEPT));
  const __half2 h = __floats2half2_rn(x.x, x.y);
  return *reinterpret_cast<const unsigned *>(&h);
}

// One tile's part of a warp (32 NC columns from col0) as its maximum and the sum of its exponentials relative to that, for
// each row; with KEEP the exponentials too, in fp16 (pack2_kept). The accumulators are read twice, since a thread has no room
// for a part's 128: 64 columns at a time, or 32 where warps beside the product leave 80 registers. Both add in the same order.
// (8192 x 32000 x 64, where there is little else to do: 91 us forward by 64 columns and in pairs, 115 us by 32 and one by one.)
template <bool KEEP, int NC>
__device__ __forceinline__ void epilogue_logits(const CeArgs &a, uint32_t tmem, int row, int warp_row0, int col0, int lane,
                                                uint8_t *buf) {
  constexpr int W = KEEP ? 32 : 64;
  if (col0 >= a.cols || warp_row0 >= a.rows) return;
  const long long t = row < a.rows ? target_of(a.targets, a.itype, row) : -1;
  float v[W];
  auto fetch = [&](int c) {   // columns W c .. of the part; -inf past the last
    uint32_t r[W / 32][32];
    __syncwarp();
#pragma unroll
    for (int q = 0; q < W / 32; ++q) tmem_ld_32x32b_x32_async(tmem + W * c + 32 * q, r[q]);
    tmem_ld_wait();
    const int left = a.cols - col0 - W * c;
#pragma unroll
    for (int j = 0; j < W; ++j) v[j] = __uint_as_float(r[j / 32][j % 32]);
    if (left < W) {
#pragma unroll
      for (int j = 0; j < W; ++j) v[j] = j < left ? v[j] : -INFINITY;
    }
  };
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int c = 0; c < 32 * NC / W; ++c) {
    fetch(c);
#pragma unroll
    for (int j = 0; j < W; ++j) top[j & 3] = fmaxf(top[j & 3], v[j]);
    const long long hit = t - col0 - W * c;
    if (__any_sync(0xffffffffu, hit >= 0 && hit < W)) {
      float z = 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j) z = hit == j ? v[j] : z;
      if (hit >= 0 && hit < W && t < a.cols) a.z_target[row] = z;
    }
  }
  const float m = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  const float ref = m == -INFINITY ? 0.f : m * LOG2E;   // nothing above -inf: exponentials of zero
  float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int c = 0; c < 32 * NC / W; ++c) {
    if (32 * NC > W) fetch(c);
#pragma unroll
    for (int j = 0; j < W; j += 2) {
      const float2 x = __ffma2_rn(make_float2(v[j], v[j + 1]), make_float2(LOG2E, LOG2E), make_float2(-ref, -ref));
      v[j] = exp2_fast(x.x);
      v[j + 1] = exp2_fast(x.y);
      sum[j / 2 % 2] = __fadd2_rn(sum[j / 2 % 2], make_float2(v[j], v[j + 1]));
    }
    if constexpr (KEEP) {
      if (c % 2 == 0) {
        if (lane == 0) bulk_wait_group_read<0>();   // the buffer's last store has read it
        __syncwarp();
      }
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *piece(buf, lane, 4 * (c & 1) + q) =
            make_uint4(pack2_kept(v[8 * q], v[8 * q + 1]), pack2_kept(v[8 * q + 2], v[8 * q + 3]),
                       pack2_kept(v[8 * q + 4], v[8 * q + 5]), pack2_kept(v[8 * q + 6], v[8 * q + 7]));
      if (c % 2 == 1) {
        const int c0 = col0 + 32 * (c - 1);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0 && c0 < a.cols) {
          tma_store_3d(&a.map_out, buf, c0, warp_row0, 0);
          bulk_commit_group();
        }
      }
    }
  }
  if (row < a.rows)
    a.partials[static_cast<long long>(col0 / (32 * NC)) * a.rows + row] =
        make_float2(m, (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y));
}

// One tile's part of a warp as dz, in bf16 terms, through the staging buffer and TMA (which leaves out what lies past the
// rows or columns).
template <int NC>
__device__ __forceinline__ void epilogue_dlogits(const CeArgs &a, uint32_t tmem, int row, int warp_row0, int col0, int lane,
                                                 uint8_t *buf) {
  long long t = -1;
  float scale = 0.f, base = 0.f;
  bool live = false;
  if (row < a.rows) {
    t = target_of(a.targets, a.itype, row);
    const float w = a.weights != nullptr ? a.weights[row] : 1.f;
    live = t >= 0 && t < a.cols && w != 0.f;
    scale = a.grad != nullptr ? w * a.grad[row] : w;
    base = -a.lse[row] * LOG2E;
  }
  if (warp_row0 >= a.rows) return;
#pragma unroll 1
  for (int c = 0; c < NC / 2; ++c) {
    const int c0 = col0 + 64 * c;
    if (c0 >= a.cols) break;
#pragma unroll 1
    for (int plane = 0; plane < a.planes; ++plane) {
      if (lane == 0) bulk_wait_group_read<0>();   // the buffer's last store has read it
      __syncwarp();
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        __syncwarp();
        tmem_ld_32x32b_x32(tmem + 64 * c + 32 * h, v);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = live ? scale * exp2_fast(fmaf(v[j], LOG2E, base)) : 0.f;
        const long long hit = t - (c0 + 32 * h);
        if (__any_sync(0xffffffffu, hit >= 0 && hit < 32)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = live && hit == j ? v[j] - scale : v[j];
        }
        if (plane > 0) {   // what the first term leaves
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] -= __bfloat162float(__float2bfloat16_rn(v[j]));
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *piece(buf, lane, 4 * h + q) = make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                                                    pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
      }
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        tma_store_3d(&a.map_out, buf, c0, warp_row0, plane);
        bulk_commit_group();
      }
    }
  }
}

// E elements of one output row from their fp32 values (stored as T), 16 bytes or singly.
template <typename T, int E>
__device__ __forceinline__ void store_piece(T *dst, float *f, int left, bool vec, bool accumulate) {
  if (vec && left >= E) {
    Raw<T, E> r;
    if (accumulate) {
      r.load(dst);
      const Vals<E> old = r.get();
#pragma unroll
      for (int e = 0; e < E / 2; ++e) f[2 * e] += old.p[e].x, f[2 * e + 1] += old.p[e].y;
    }
    Vals<E> o;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) o.p[e] = make_float2(f[2 * e], f[2 * e + 1]);
    store_vals(dst, o);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (e < left) store1(dst, e, accumulate ? load1(dst, e) + f[e] : f[e]);
  }
}

// One tile's part of a warp as rows of the output: lines of 128 bytes (64 bf16 or 32 fp32 values) through the staging
// buffer and TMA, where the output's rows are 16-byte aligned; TMA adds to fp32 values that are there.
template <int NC>
__device__ __forceinline__ void epilogue_out_tma(const CeArgs &a, uint32_t tmem, int slice, int warp_row0, int col0, int lane,
                                                 uint8_t *buf) {
  if (warp_row0 >= a.rows) return;
#pragma unroll 1
  for (int c = 0; c < NC; ++c) {
    const int c0 = col0 + 32 * c;
    if (c0 >= a.cols) break;
    float v[32];
    __syncwarp();
    tmem_ld_32x32b_x32(tmem + 32 * c, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) v[j] *= a.factor;
    if (a.out_f32 || c % 2 == 0) {
      if (lane == 0) bulk_wait_group_read<0>();   // the buffer's last store has read it
      __syncwarp();
    }
    if (a.out_f32) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *piece(buf, lane, q) = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                          __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
    } else {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *piece(buf, lane, 4 * (c & 1) + q) = make_uint4(pack2(v[8 * q], v[8 * q + 1]), pack2(v[8 * q + 2], v[8 * q + 3]),
                                                        pack2(v[8 * q + 4], v[8 * q + 5]), pack2(v[8 * q + 6], v[8 * q + 7]));
    }
    if (a.out_f32 || c % 2 == 1 || c0 + 32 >= a.cols) {
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) {
        const int x = a.out_f32 ? c0 : c0 - 32 * (c & 1);
        if (a.accumulate) tma_add_3d(&a.map_out, buf, x, warp_row0, slice);
        else tma_store_3d(&a.map_out, buf, x, warp_row0, slice);
        bulk_commit_group();
      }
    }
  }
}

// As above for any other output: 32 columns of fp32 at a time through the buffer, so that eight lanes write 128 bytes of a
// row (four lanes 64 as bf16).
template <int NC>
__device__ __forceinline__ void epilogue_out(const CeArgs &a, uint32_t tmem, int slice, int warp_row0, int col0, int lane,
                                             uint8_t *buf) {
  if (warp_row0 >= a.rows) return;
#pragma unroll 1
  for (int c = 0; c < NC; ++c) {
    const int c0 = col0 + 32 * c;
    if (c0 >= a.cols) break;
    {
      float v[32];
      __syncwarp();   // the buffer's last rows have been read
      tmem_ld_32x32b_x32(tmem + 32 * c, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] *= a.factor;
#pragma unroll
      for (int q = 0; q < 8; ++q)
        *piece(buf, lane, q) = make_uint4(__float_as_uint(v[4 * q]), __float_as_uint(v[4 * q + 1]),
                                          __float_as_uint(v[4 * q + 2]), __float_as_uint(v[4 * q + 3]));
    }
    __syncwarp();
    const int left0 = a.cols - c0;
    if (a.out_f32) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = 4 * k + (lane >> 3), q = lane & 7;
        const uint4 w = *piece(buf, i, q);
        float f[4] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w)};
        if (warp_row0 + i < a.rows)
          store_piece<float, 4>(static_cast<float *>(a.out) + slice * a.slice_stride +
                                    static_cast<long long>(warp_row0 + i) * a.ld_out + c0 + 4 * q,
                                f, left0 - 4 * q, a.vec, a.accumulate != 0);
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = 8 * k + (lane >> 2), q = lane & 3;
        const uint4 w = *piece(buf, i, 2 * q), x = *piece(buf, i, 2 * q + 1);
        float f[8] = {__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w),
                      __uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
        if (warp_row0 + i < a.rows)
          store_piece<__nv_bfloat16, 8>(static_cast<__nv_bfloat16 *>(a.out) +
                                            static_cast<long long>(warp_row0 + i) * a.ld_out + c0 + 8 * q,
                                        f, left0 - 8 * q, a.vec, a.accumulate != 0);
      }
    }
  }
}

// A segment's accumulators (32 NC columns) added to sum, rounding to nearest; with `put` the sums take their place in tensor
// memory, from where they go out as any tile does. (Added to the output segment by segment, through L2: 668 us with 32 steps,
// 737 with 16, for 2048 x 50304 x 768.)
template <int NC>
__device__ __forceinline__ void add_segment(float (&sum)[32 * NC], uint32_t tmem, bool put) {
#pragma unroll
  for (int c = 0; c < NC; ++c) {
    float v[32];
    __syncwarp();
    tmem_ld_32x32b_x32(tmem + 32 * c, v);
#pragma unroll
    for (int j = 0; j < 32; ++j) sum[32 * c + j] += v[j];
    if (put) tmem_st_32x32b_x32(tmem + 32 * c, &sum[32 * c]);
  }
}

// Units first, first + stride, ... by a group of threads: SCALE_ROWS rows (whose maxima lie next to each other) and 8 columns
// per thread. All of a unit's loads are on their way before anything is stored. Bound by HBM: 4 bytes per logit.
constexpr int SCALE_ROWS = 4;
__device__ __forceinline__ void scale_units(const ScaleJob &a, long long first, long long stride, int thread, int threads) {
  const int blocks = (a.cols + 8 * threads - 1) / (8 * threads);   // of columns
  const long long units = static_cast<long long>((a.rows + SCALE_ROWS - 1) / SCALE_ROWS) * blocks;
#pragma unroll 1
  for (long long u = first; u < units; u += stride) {
    const int group = static_cast<int>(u / blocks);
    const int c0 = (static_cast<int>(u - static_cast<long long>(group) * blocks) * threads + thread) * 8;
    if (c0 >= a.cols) continue;
    const int r0 = group * SCALE_ROWS;
    uint16_t *x = a.x + r0 * a.ld + c0;
    const float2 *part = a.partials + static_cast<long long>(c0 / a.part_cols) * a.rows;
    uint4 e[SCALE_ROWS];
    float4 state[SCALE_ROWS];
    float m[SCALE_ROWS];
#pragma unroll
    for (int i = 0; i < SCALE_ROWS; ++i) {
      const int own = min(r0 + i, a.rows - 1);   // the last row again where there is no further one
      e[i] = __ldcs(reinterpret_cast<const uint4 *>(a.x + own * a.ld + c0));
      m[i] = __ldg(&part[own].x);
      state[i] = __ldg(a.row_state + own);
    }
#pragma unroll
    for (int i = 0; i < SCALE_ROWS; ++i) {
      const RowState r = RowState::of(state[i]);
      const float f = r.g * (1.f / KEPT) * exp2_fast(fmaf(m[i], LOG2E, r.base));
      const int hit = r.target - c0;
      const unsigned in[4] = {e[i].x, e[i].y, e[i].z, e[i].w};
      unsigned out[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float2 y = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2 *>(&in[k])), make_float2(f, f));
        if (hit == 2 * k) y.x -= r.g;
        if (hit == 2 * k + 1) y.y -= r.g;
        out[k] = r.target < 0 ? 0u : pack2(y.x, y.y);   // zeros for a row without a part, whatever its exponentials are
      }
      if (r0 + i < a.rows) *reinterpret_cast<uint4 *>(x + i * a.ld) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
}

__global__ void __launch_bounds__(256) ce_scale_kernel(const ScaleJob a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  scale_units(a, blockIdx.x, gridDim.x, threadIdx.x, 256);
}

// A: h (K-major) for the logits, DH dz (K-major), DW dz (MN-major: dz^T). B: W (K-major) for the logits, DH W and DW h
// (MN-major). An MN-major operand is loaded as boxes of 64 columns x 64 steps.
//
// PAIRED: the two CTAs of a pair share a tile of 256 x 256, which halves what each reads of B. ALONE: a CTA has a tile of
// 128 x 128, for up to 128 rows, where half of a pair's MMAs would multiply rows that there are not. Its stages then hold only
// the rows of A that there are, in eights (a_box): TMA takes as long for 128-byte lines that it fills with zeros as for
// others, and W does not come in at full rate beside them (forward, 8 x 50304 x 768: 29.9 us by pairs, 18.5 us so;
// 1 x 128256 x 4096: 220 and 173 us). FEW: for up to 32 rows A's part of a stage is that small, and nine stages fit instead of
// six (1 x 128256 x 4096: 170 -> 164 us, 0.94 of the copy bandwidth). The MMA reads 128 rows of A in either case: past a_box
// it finds what else lies in the stage, which makes accumulator rows that nothing reads.
//
// SUMS: a tile's accumulators come in segments of the contraction (SEGMENT), whose sums 8 warps hold, 128 in a thread.
//
// JOB: more warps run a ScaleJob, which belongs to other rows than the product's, so that its HBM traffic passes under the
// MMAs (8192 x 50304 x 768: 1528 -> 1360 us, 4096 x 128256 x 4096: 8.16 -> 7.93 ms). Twelve of them, since each waits for
// its loads: 1666 us with four, 1358 with eight, 1335 with twelve on another box.
template <int KIND, int SHAPE, bool JOB, bool SUMS>
__global__ void __launch_bounds__(gemm_threads(JOB), 1) ce_gemm_kernel(const __grid_constant__ CeArgs args) {
  constexpr bool A_MN = KIND == DW, B_MN = KIND == DH || KIND == DW;
  constexpr bool PAIR = SHAPE == PAIRED;
  constexpr int STAGES = stages(SHAPE), STAGE_BYTES = stage_bytes(SHAPE), A_BYTES = a_bytes(SHAPE);
  constexpr int CTAS = PAIR ? 2 : 1, BN = tile_cols(PAIR), NC = BN / 64;   // NC: chunks of 32 columns per epilogue warp
  constexpr uint32_t TMEM_COLS = 2 * BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *staging = smem + STAGES * STAGE_BYTES;
  Ctrl *ctrl = reinterpret_cast<Ctrl *>(staging + EPI_WARPS * BUF_BYTES);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctrl->full[s], 1);
      mbar_init(&ctrl->empty[s], 1);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&ctrl->acc_full[s], 1);
      mbar_init(&ctrl->acc_empty[s], CTAS * EPI_WARPS);   // a pair's epilogue warps all use the even CTA's copy
    }
    mbar_init(&ctrl->drain, 1);
    ctrl->abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane < 2) tma_prefetch_desc(lane ? &args.map_b : &args.map_a);
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(&ctrl->tmem_base, TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&ctrl->tmem_base, TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncwarp();
  if constexpr (PAIR) cluster_sync();   // both CTAs' barriers are initialised before either signals the other
  else __syncthreads();
  tc_fence_after();
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const uint32_t tmem_base = ctrl->tmem_base;
  WaitCtl ctl{&ctrl->abort_flag, args.err, args.timeout_ns};
  const int rank = PAIR ? static_cast<int>(cluster_ctarank()) : 0;
  const long long first = blockIdx.x / CTAS, stride = gridDim.x / CTAS;
  // the even CTA's copy of a barrier, as a cluster address
  auto leader = [](uint64_t *bar) { return PAIR ? mapa_shared(smem_u32(bar), 0) : smem_u32(bar); };

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t leader_full0 = leader(&ctrl->full[0]);
      uint32_t stage = 0, phase = 0;
      int last_parity[STAGES];
      for (int s = 0; s < STAGES; ++s) last_parity[s] = -1;
      bool ok = true;
      for (long long u = first; ok && u < args.total; u += stride) {
        int slice, ti, tj;
        decode(args, u, slice, ti, tj);
        const int row0 = (CTAS * ti + rank) * BM, col0 = tj * BN + B_COLS * rank;
        const int k0 = slice * args.k_per, k1 = min(args.k_iters, k0 + args.k_per);
        for (int kk = k0; kk < k1; ++kk) {
          if (!wait_bounded(&ctrl->empty[stage], phase ^ 1u, ctl, ERR_WAIT_EMPTY)) {
            ok = false;
            break;
          }
          if (rank == 0) {   // a pair's copies complete on the even CTA's barrier
            mbar_arrive_expect_tx(&ctrl->full[stage], PAIR ? 2 * STAGE_BYTES : args.a_box * BK * 2 + B_BYTES);
            last_parity[stage] = static_cast<int>(phase);
          }
          uint8_t *sa = smem + stage * STAGE_BYTES, *sb = sa + A_BYTES;
          auto load = [&](uint8_t *dst, const CUtensorMap *map, int x, int y, int z) {
            if constexpr (PAIR)
              tma_load_3d_pair(dst, map, leader_full0 + stage * static_cast<uint32_t>(sizeof(uint64_t)), x, y, z);
            else
              tma_load_3d(dst, map, &ctrl->full[stage], x, y, z);
          };
          const int plane = kk < args.k_low ? 1 : 0;
          const int k = (plane ? kk : kk - args.k_low) * BK;
          if constexpr (A_MN) {
#pragma unroll
            for (int q = 0; q < 2; ++q) load(sa + q * (64 * BK * 2), &args.map_a, row0 + 64 * q, k, plane);
          } else {
            load(sa, &args.map_a, k, row0, plane);
          }
          if constexpr (B_MN) {
#pragma unroll
            for (int q = 0; q < 2; ++q) load(sb + q * (64 * BK * 2), &args.map_b, col0 + 64 * q, k, 0);
          } else {
            load(sb, &args.map_b, k, col0, 0);
          }
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      // every armed stage's copies have landed before the CTA may exit
      for (int s = 0; s < STAGES; ++s)
        if (last_parity[s] >= 0) drain_wait(&ctrl->full[s], static_cast<uint32_t>(last_parity[s]), ctl);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      constexpr uint32_t idesc = idesc_bf16_f32(CTAS * BM, BN, A_MN, B_MN);
      auto commit = [](uint64_t *bar) {
        if constexpr (PAIR) tc_commit_pair_mc(bar, 0x3);
        else tc_commit(bar);
      };
      uint32_t stage = 0, phase = 0, acc = 0, acc_phase = 0;
      bool ok = true, issued = false;
      for (long long u = first; ok && u < args.total; u += stride) {
        int slice, ti, tj;
        decode(args, u, slice, ti, tj);
        const int k0 = slice * args.k_per, k1 = min(args.k_iters, k0 + args.k_per);
        for (int ks = k0, ke; ok && ks < k1; ks = ke) {
          ke = segment_end(args, ks, k1);
          if (!wait_bounded(&ctrl->acc_empty[acc], acc_phase ^ 1u, ctl, ERR_WAIT_ACC_EMPTY)) {
            ok = false;
            break;
          }
          tc_fence_after();
          for (int kk = ks; kk < ke; ++kk) {
            if (!wait_bounded(&ctrl->full[stage], phase, ctl, ERR_WAIT_FULL)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t sa = smem_u32(smem + stage * STAGE_BYTES), sb = sa + A_BYTES;
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              const uint64_t adesc =
                  A_MN ? smem_desc_sw128(sa + k * 16 * 128, 64 * BK * 2, 1024) : smem_desc_sw128(sa + k * 32, 16, 1024);
              const uint64_t bdesc =
                  B_MN ? smem_desc_sw128(sb + k * 16 * 128, 64 * BK * 2, 1024) : smem_desc_sw128(sb + k * 32, 16, 1024);
              const uint32_t add = ((kk - ks) | k) != 0 ? 1u : 0u;
              if constexpr (PAIR) tc_mma_bf16_pair(tmem_base + acc * BN, adesc, bdesc, idesc, add);
              else tc_mma_bf16(tmem_base + acc * BN, adesc, bdesc, idesc, add);
            }
            issued = true;
            commit(&ctrl->empty[stage]);   // frees the stage, in both CTAs of a pair
            if (++stage == STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          commit(&ctrl->acc_full[acc]);
          acc ^= 1u;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      if (issued) {   // all MMAs have completed before tensor memory is released
        if constexpr (PAIR) tc_commit_pair_mc(&ctrl->drain, 0x1);
        else tc_commit(&ctrl->drain);
        drain_wait(&ctrl->drain, 0u, ctl);
      }
    }
  } else if (warp < FIRST_JOB_WARP) {
    const uint32_t leader_acc_empty0 = leader(&ctrl->acc_empty[0]);
    const int lane_base = (warp % 4) * 32;   // the lanes of tensor memory that this warp may read
    const int half = (warp - 2) / 4;         // of the tile's columns
    uint8_t *buf = staging + (warp - 2) * BUF_BYTES;
    uint32_t acc = 0, acc_phase = 0;
    bool ok = true;
    for (long long u = first; ok && u < args.total; u += stride) {
      int slice, ti, tj;
      decode(args, u, slice, ti, tj);
      const int k0 = slice * args.k_per, k1 = min(args.k_iters, k0 + args.k_per);
      const int warp_row0 = (CTAS * ti + rank) * BM + lane_base, col0 = tj * BN + 32 * NC * half;
      float sum[SUMS ? 32 * NC : 1];
#pragma unroll
      for (int j = 0; j < (SUMS ? 32 * NC : 1); ++j) sum[j] = 0.f;
      for (int ks = k0; ks < k1; ks = segment_end(args, ks, k1)) {
        ok = wait_bounded(&ctrl->acc_full[acc], acc_phase, ctl, ERR_WAIT_ACC_FULL);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const uint32_t tmem = tmem_base + acc * BN + (static_cast<uint32_t>(lane_base) << 16) + 32 * NC * half;
        const bool whole = !SUMS || segment_end(args, ks, k1) == k1;   // the tile's last segment
        if constexpr (SUMS) add_segment<NC>(sum, tmem, whole);
        if (!whole) {
        } else if constexpr (KIND == LOGITS || KIND == LOGITS_EXP)
          epilogue_logits<KIND == LOGITS_EXP, NC>(args, tmem, warp_row0 + lane, warp_row0, col0, lane, buf);
        else if constexpr (KIND == DLOGITS)
          epilogue_dlogits<NC>(args, tmem, warp_row0 + lane, warp_row0, col0, lane, buf);
        else if (args.tma)
          epilogue_out_tma<NC>(args, tmem, slice, warp_row0, col0, lane, buf);
        else
          epilogue_out<NC>(args, tmem, slice, warp_row0, col0, lane, buf);
        tc_fence_before();
        __syncwarp();
        // the MMA warp reads none of this warp's stores, so the signal need not wait for them
        if (lane == 0) mbar_arrive_cluster_relaxed(leader_acc_empty0 + acc * static_cast<uint32_t>(sizeof(uint64_t)));
        acc ^= 1u;
        if (acc == 0) acc_phase ^= 1u;
      }
    }
    if (lane == 0) bulk_wait_group_all();
  } else if constexpr (JOB) {
    scale_units(args.job, blockIdx.x, gridDim.x, threadIdx.x - 32 * FIRST_JOB_WARP, 32 * JOB_WARPS);
  }

  // neither CTA of a pair leaves while the other may still signal it
  tc_fence_before();
  __syncwarp();
  if constexpr (PAIR) cluster_sync();
  else __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, TMEM_COLS);
    else tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ------------------------------------------------------------------------------------------ the small kernels

struct RowsArgs {
  const __nv_bfloat16 *h;
  __nv_bfloat16 *out;
  long long ldh, ld_out, V;
  const void *targets;
  const float *weights;
  int itype, rows, D;
};

// h with zeros for the rows that have no part in the loss: dw's product multiplies every row, and a row of padding may
// hold NaN. One warp, 16 bytes per lane and turn (both pitches are multiples of 8; what lies past D is not read).
__device__ __forceinline__ void copy_live_row(const RowsArgs &a, long long row, int lane) {
  if (row >= a.rows) return;
  const long long t = target_of(a.targets, a.itype, row);
  const bool live = t >= 0 && t < a.V && (a.weights == nullptr || a.weights[row] != 0.f);
  const __nv_bfloat16 *src = a.h + row * a.ldh;
  __nv_bfloat16 *dst = a.out + row * a.ld_out;
#pragma unroll 4
  for (int c = 8 * lane; c + 8 <= a.D; c += 256)
    *reinterpret_cast<uint4 *>(dst + c) = live ? *reinterpret_cast<const uint4 *>(src + c) : make_uint4(0u, 0u, 0u, 0u);
  for (int c = a.D / 8 * 8 + lane; c < a.D; c += 32) dst[c] = live ? src[c] : __float2bfloat16_rn(0.f);
}

__global__ void __launch_bounds__(256) ce_rows_kernel(const RowsArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  copy_live_row(a, static_cast<long long>(blockIdx.x) * 8 + threadIdx.x / 32, threadIdx.x % 32);
}

struct CombineArgs {
  const float2 *partials;
  const float *z_target, *weights;
  const void *targets;
  int itype, parts, rows;
  long long V;
  float *losses, *lse;
  float4 *row_state;   // or null
  int own_blocks;      // blocks past these copy h's rows
  RowsArgs copy;
};

// Eight rows per block, whose pairs of one part fill a 32-byte sector; 32 threads share a row's parts.
// lse = m + log(sum of s_p exp(m_p - m)).
constexpr int COMBINE_ROWS = 8;
__global__ void __launch_bounds__(256) ce_combine_kernel(const __grid_constant__ CombineArgs a) {
  __shared__ float2 sh[8][COMBINE_ROWS];
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= a.own_blocks) {
    copy_live_row(a.copy, static_cast<long long>(blockIdx.x - a.own_blocks) * 8 + threadIdx.x / 32, threadIdx.x % 32);
    return;
  }
  const int own = threadIdx.x % COMBINE_ROWS, stream = threadIdx.x / COMBINE_ROWS;
  const int row = blockIdx.x * COMBINE_ROWS + own;
  float m = -INFINITY, s = 0.f;
  auto join = [&](float2 p) {
    const float mn = fmaxf(m, p.x);
    const float ref = mn == -INFINITY ? 0.f : mn;
    s = s * exp2_fast((m - ref) * LOG2E) + p.y * exp2_fast((p.x - ref) * LOG2E);
    m = mn;
  };
  if (row < a.rows) {
    const float2 *src = a.partials + row;
    for (int p = stream; p < a.parts; p += 8 * 32) {   // eight at once, the last ones again where there are no further ones
      float2 x[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) x[k] = src[static_cast<long long>(min(p + 32 * k, a.parts - 1)) * a.rows];
      float mn = m;
#pragma unroll
      for (int k = 0; k < 8; ++k) mn = fmaxf(mn, x[k].x);
      const float ref = mn == -INFINITY ? 0.f : mn;
      s *= exp2_fast((m - ref) * LOG2E);
#pragma unroll
      for (int k = 0; k < 8; ++k) s += p + 32 * k < a.parts ? x[k].y * exp2_fast((x[k].x - ref) * LOG2E) : 0.f;
      m = mn;
    }
  }
#pragma unroll
  for (int o = COMBINE_ROWS; o < 32; o *= 2)
    join(make_float2(__shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o)));
  if (threadIdx.x % 32 < COMBINE_ROWS) sh[threadIdx.x / 32][own] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x >= COMBINE_ROWS || row >= a.rows) return;
  for (int w = 1; w < 8; ++w) join(sh[w][own]);
  const long long t = target_of(a.targets, a.itype, row);
  const float w = a.weights != nullptr ? a.weights[row] : 1.f;
  const bool live = t >= 0 && t < a.V && w != 0.f;
  const float lse = m + logf(s);
  a.lse[row] = live ? lse : 0.f;
  a.losses[row] = live ? w * (lse - a.z_target[row]) : 0.f;
  if (a.row_state != nullptr)
    a.row_state[row] = make_float4(-lse * LOG2E, w, __int_as_float(live ? static_cast<int>(t) : -1), 0.f);
}

struct ReduceArgs {
  const float *parts;          // n of rows x ld_part, slice_stride apart
  long long slice_stride, ld_part, ld_out;
  int n, rows, cols, accumulate;
  void *out;
};

// out (+)= the slices in their order; n = 0: zeros. Four columns per thread.
template <typename T>
__global__ void __launch_bounds__(256) ce_reduce_kernel(const ReduceArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const long long per_row = (a.cols + 3) / 4, total = per_row * a.rows;
  const bool vec = (reinterpret_cast<uintptr_t>(a.out) & (4 * sizeof(T) - 1)) == 0 && a.ld_out % 4 == 0;
  for (long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; i < total;
       i += static_cast<long long>(gridDim.x) * 256) {
    const long long row = i / per_row, c = 4 * (i - row * per_row);
    float f[4] = {0.f, 0.f, 0.f, 0.f};
    const float *src = a.parts + row * a.ld_part + c;
#pragma unroll 4
    for (int k = 0; k < a.n; ++k) {   // the slices' rows are padded to whole 16 bytes
      const float4 q = *reinterpret_cast<const float4 *>(src + k * a.slice_stride);
      f[0] += q.x, f[1] += q.y, f[2] += q.z, f[3] += q.w;
    }
    store_piece<T, 4>(static_cast<T *>(a.out) + row * a.ld_out + c, f, static_cast<int>(min(4ll, a.cols - c)), vec,
                      a.accumulate != 0);
  }
}

// ------------------------------------------------------------------------------------------ plan

long long ceil_div(long long a, long long b) { return (a + b - 1) / b; }
long long round_up(long long a, long long b) { return ceil_div(a, b) * b; }

// Rows from which on the joint call goes by halves (Run::joint). Below, the halves' products lose more to their last wave of
// tiles than the scale pass costs: 1024 x 32000 x 1024 174 us whole and 200 us by halves, 2048 x 50304 x 768 396 and 391 us.
constexpr long long HALVES = 2048;

// Slices of a contraction of k 64-deep steps over `tiles` tile pairs: the count for which the longest SM pair's steps are
// fewest, each slice counted with TILE_STEPS more for its start and epilogue, and with what its sums' way through memory
// costs. From sizes alone.
constexpr int TILE_STEPS = 6;
int choose_split(bool pair, long long rows, long long cols, long long k) {
  const long long tiles = ceil_div(rows, tile_rows(pair)) * ceil_div(cols, tile_cols(pair)), at_once = pair ? SMS / 2 : SMS;
  if (tiles >= 4 * at_once) return 1;
  int best = 1;
  double best_cost = 0;
  for (int s = 1; s <= MAX_SPLIT && (s == 1 || k / s >= 8); ++s) {
    const long long per = (k + s - 1) / s, n = (k + per - 1) / per;
    const double waves = static_cast<double>(ceil_div(tiles * n, at_once));
    // a pair's tile is 256 KB written, mostly under MMAs, and read again: up to 0.08 us of the GPU's bandwidth, 0.2 steps
    const double way = n > 1 ? 0.2 * static_cast<double>(tiles * n) * (pair ? 1.0 : 0.25) + 12 : 0;
    const double cost = waves * static_cast<double>(per + TILE_STEPS) + way;
    if (s == 1 || cost < best_cost) {
      best = static_cast<int>(n);
      best_cost = cost;
    }
  }
  return best;
}

std::atomic<long long> g_piece_rows{0};   // muon_debug_loss_rows

struct Plan {
  long long rows, pieces, Vp, Dp;     // rows of a piece; pitches of dz and of fp32 scratch rows
  int planes, parts, part_cols;       // a part: the columns of a tile whose exponentials share a maximum
  int shape;                          // of the products over rows: logits, dlogits, dh
  long long half;                     // rows of a piece's first half in the joint call, or all
  int split_dh, split_half, split_dw;
  size_t partials, z_target, row_state, dz, h_live, slices, dw_sum, total;
};

Plan plan(int64_t N, int64_t V, int64_t D, int terms) {
  Plan p{};
  long long rows = g_piece_rows.load();
  p.Vp = round_up(V, 64);
  if (rows <= 0) rows = PIECE_ELEMS / std::max<long long>(p.Vp, round8(D));
  rows = std::max(256ll, rows / 256 * 256);
  p.rows = std::max<long long>(1, std::min<long long>(N, rows));
  p.pieces = ceil_div(N, p.rows);
  p.Dp = round_up(D, 4);
  p.planes = terms;
  p.shape = p.rows > BM ? PAIRED : p.rows > FEW_ROWS ? ALONE : FEW;
  p.part_cols = tile_cols(p.shape == PAIRED) / 2;
  p.parts = static_cast<int>(ceil_div(V, p.part_cols));
  size_t off = 1024;   // the control block
  auto take = [&](size_t &at, long long bytes) {
    at = off;
    off = align_up(off + static_cast<size_t>(bytes), 1024);
  };
  take(p.partials, 8ll * p.parts * p.rows);
  take(p.z_target, 4 * p.rows);
  if (terms > 0) {
    const long long kh = ceil_div(V, BK) * terms, kw = ceil_div(p.rows, BK) * terms;
    p.half = terms == 1 && p.rows >= HALVES ? round_up(p.rows / 2, tile_rows(true)) : p.rows;
    p.split_dh = choose_split(p.shape == PAIRED, p.rows, D, kh);
    p.split_half = choose_split(p.shape == PAIRED, p.half, D, kh);
    p.split_dw = choose_split(true, V, D, kw);
    take(p.row_state, 16 * p.rows);
    take(p.dz, 2ll * terms * p.rows * p.Vp);
    take(p.h_live, 2 * p.rows * round8(D));
    const long long dh =
        4 * p.Dp * std::max(p.split_dh > 1 ? p.split_dh * p.rows : 0, p.split_half > 1 ? p.split_half * p.half : 0);
    const long long dw = p.split_dw > 1 ? 4ll * p.split_dw * V * p.Dp : 0;
    take(p.slices, std::max(dh, dw));
    if (p.pieces > 1) take(p.dw_sum, 4ll * V * p.Dp);
  }
  p.total = off;
  return p;
}

// ------------------------------------------------------------------------------------------ launches

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

template <int KIND, int SHAPE, bool JOB, bool SUMS = false>
muon_status launch_gemm(CeArgs &a, int32_t kind, cudaStream_t s) {
  if (a.split < 1) a.split = 1;
  a.k_per = static_cast<int>(ceil_div(a.k_iters, a.split));
  a.split = static_cast<int>(ceil_div(a.k_iters, a.k_per));
  a.k_seg = SUMS ? SEGMENT : a.k_per;
  if constexpr ((KIND == DH || KIND == DW) && !JOB && !SUMS)   // more than one segment
    if (a.out_f32 && a.planes > 1 && a.k_per > SEGMENT && a.k_iters > a.k_low + SEGMENT)
      return launch_gemm<KIND, SHAPE, JOB, true>(a, kind, s);
  constexpr auto kernel = ce_gemm_kernel<KIND, SHAPE, JOB, SUMS>;
  constexpr bool PAIR = SHAPE == PAIRED;
  constexpr size_t SMEM = smem_bytes(SHAPE);
  static AttributesSet set;
  static std::atomic<int> clusters[64];
  if (set.once([] {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM));
      }) != cudaSuccess)
    return MUON_ERR_CUDA;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(gemm_threads(JOB));
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PAIR ? 2 : 1;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MUON_ERR_CUDA;
  int n = PAIR ? clusters[dev].load(std::memory_order_relaxed) : device_sm_count();   // CTAs or pairs that run at once
  if (n == 0) {
    cfg.gridDim = dim3(static_cast<unsigned>(2 * (device_sm_count() / 2)));
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) n = device_sm_count() / 2;
    clusters[dev].store(n, std::memory_order_relaxed);
  }
  a.m_tiles = static_cast<int>(ceil_div(a.rows, tile_rows(PAIR)));
  a.n_tiles = static_cast<int>(ceil_div(a.cols, tile_cols(PAIR)));
  if (KIND == DH || KIND == DW) {   // rows and columns past the output's are not stored; slices follow each other
    const long long apart = a.split > 1 ? a.slice_stride : a.ld_out;   // one slice has no next one
    if (a.tma && !(a.out_f32 ? make_f32_map(&a.map_out, a.out, a.cols, a.rows, a.split, a.ld_out, apart, 32)
                             : make_bf16_map(&a.map_out, a.out, a.cols, a.rows, a.split, a.ld_out, apart, 32)))
      return MUON_ERR_CUDA;
  }
  a.total = static_cast<long long>(a.m_tiles) * a.n_tiles * a.split;
  cfg.gridDim = dim3(static_cast<unsigned>((PAIR ? 2 : 1) * std::min<long long>(n, a.total)));
  launch_begin(kind, s);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  launch_end(s);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

template <int KIND>
muon_status launch_rows(int shape, CeArgs &a, int32_t kind, cudaStream_t s) {
  return shape == PAIRED  ? launch_gemm<KIND, PAIRED, false>(a, kind, s)
         : shape == ALONE ? launch_gemm<KIND, ALONE, false>(a, kind, s)
                          : launch_gemm<KIND, FEW, false>(a, kind, s);
}

// As launch_rows for a pair's tiles, with a job beside the product.
template <int KIND>
muon_status launch_beside(const ScaleJob *job, CeArgs &a, int32_t kind, cudaStream_t s) {
  a.job = *job;
  return launch_gemm<KIND, PAIRED, true>(a, kind, s);
}

muon_status launch_reduce(const ReduceArgs &r, int dtype, cudaStream_t s) {
  const long long work = ceil_div(r.cols, 4) * r.rows;
  const dim3 grid(static_cast<unsigned>(std::min<long long>(ceil_div(work, 256), 8ll * device_sm_count())));
  launch_begin(KK_CE_REDUCE, s);
  const cudaError_t e = dtype == MUON_F32 ? launch_pdl(ce_reduce_kernel<float>, grid, dim3(256), 0, s, r)
                                          : launch_pdl(ce_reduce_kernel<__nv_bfloat16>, grid, dim3(256), 0, s, r);
  launch_end(s);
  return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
}

// What a call has in hand.
struct Call {
  const char *h, *w;
  long long ldh, ldw;
  const void *targets;
  int itype;
  const float *weights;
  long long N, V, D;
  float *losses, *lse;
  const float *lse_in, *grad;
  float grad_scale;
  char *dh, *dw;
  int dhdt, dwdt;
  long long lddh, lddw;
  int accumulate;
  char *ws;
  bool forward, backward;
  int terms;
};

size_t size_of(int dt) { return dt == MUON_F32 ? 4 : 2; }

// Rows of a matrix of one row may have any pitch: none is used.
long long pitch8(long long ld, long long rows, long long cols) { return rows == 1 ? round8(cols) : ld; }

// One call's launches, a piece at a time.
class Run {
  const Call &c;
  const Plan &p;
  cudaStream_t s;
  CeArgs base_;
  long long r0_ = 0, rows_ = 0;      // the piece
  const char *h_ = nullptr;          // its rows
  long long ldh_, ldw_;
  float2 *partials_;
  float *z_target_, *slices_, *dw_sum_;
  float4 *row_state_;
  __nv_bfloat16 *dz_, *h_live_;

  template <typename T>
  T *at(size_t offset) const {
    return offset ? reinterpret_cast<T *>(c.ws + offset) : nullptr;
  }
  // the matrices as operands: rows [r, r + n) of the piece
  bool h_map(CUtensorMap *m, long long r, long long n) const {
    return make_bf16_map(m, h_ + r * ldh_ * 2, c.D, n, 1, ldh_, ldh_, a_box());
  }
  int a_box() const { return p.shape == PAIRED ? BM : static_cast<int>(round8(rows_)); }
  bool w_map(CUtensorMap *m, int box) const { return make_bf16_map(m, c.w, c.D, c.V, 1, ldw_, ldw_, box); }
  bool dz_map(CUtensorMap *m, long long r, long long n, int box) const {
    return make_bf16_map(m, dz_ + r * p.Vp, c.V, n, p.planes, p.Vp, p.Vp * rows_, box);
  }
  const void *targets(long long r) const {
    return static_cast<const char *>(c.targets) + (r0_ + r) * (c.itype == MUON_I32 ? 4 : 8);
  }
  const float *weights(long long r) const { return c.weights != nullptr ? c.weights + r0_ + r : nullptr; }
  RowsArgs copy_args(long long r, long long n) const {
    return RowsArgs{reinterpret_cast<const __nv_bfloat16 *>(h_ + r * ldh_ * 2), h_live_ + r * round8(c.D), ldh_, round8(c.D),
                    c.V, targets(r), weights(r), c.itype, static_cast<int>(n), static_cast<int>(c.D)};
  }
  // the statistics of rows [r, r + n) lie after those of the piece's earlier rows
  float2 *partials(long long r) const { return partials_ + r * p.parts; }
  ScaleJob job(long long r, long long n) const {
    return ScaleJob{reinterpret_cast<uint16_t *>(dz_ + r * p.Vp), p.Vp, partials(r), row_state_ + r, static_cast<int>(n),
                    static_cast<int>(c.V), p.part_cols};
  }
  bool product(CeArgs &f, long long r, long long n) const {
    f = base_;
    f.rows = static_cast<int>(n);
    f.cols = static_cast<int>(c.V);
    f.a_box = a_box();
    f.k_iters = static_cast<int>(ceil_div(c.D, BK));
    f.targets = targets(r);
    f.weights = weights(r);
    f.partials = partials(r);
    f.z_target = z_target_ + r;
    return h_map(&f.map_a, r, n) && w_map(&f.map_b, B_COLS);
  }

  // losses and lse of rows [r, r + n), the exponentials too if `keep`, with a job beside the product if there is one
  muon_status losses(long long r, long long n, bool keep, const ScaleJob *beside) {
    CeArgs f;
    if (!product(f, r, n) || (keep && !dz_map(&f.map_out, r, n, 32))) return MUON_ERR_CUDA;
    muon_status st = beside != nullptr ? launch_beside<LOGITS_EXP>(beside, f, KK_CE_LOGITS, s)
                     : keep            ? launch_rows<LOGITS_EXP>(p.shape, f, KK_CE_LOGITS, s)
                                       : launch_rows<LOGITS>(p.shape, f, KK_CE_LOGITS, s);
    if (st != MUON_OK) return st;
    const long long own = ceil_div(n, COMBINE_ROWS), copies = keep && c.dw != nullptr ? ceil_div(n, 8) : 0;
    const CombineArgs cb{partials(r),         z_target_ + r, weights(r),
                         targets(r),          c.itype,       p.parts,
                         static_cast<int>(n), c.V,           c.losses + r0_ + r,
                         c.lse + r0_ + r,     keep ? row_state_ + r : nullptr,
                         static_cast<int>(own), copies ? copy_args(r, n) : RowsArgs{}};
    return small(KK_CE_COMBINE, ce_combine_kernel, own + copies, cb);
  }

  template <typename Args, typename Given>
  muon_status small(int32_t kind, void (*kernel)(Args), long long blocks, const Given &args) {
    launch_begin(kind, s);
    const cudaError_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(256), 0, s, args);
    launch_end(s);
    return e == cudaSuccess ? MUON_OK : MUON_ERR_CUDA;
  }

  muon_status dlogits() {
    CeArgs f;
    if (!product(f, 0, rows_) || !dz_map(&f.map_out, 0, rows_, 32)) return MUON_ERR_CUDA;
    f.lse = (c.forward ? c.lse : c.lse_in) + r0_;
    f.grad = c.grad != nullptr ? c.grad + r0_ : nullptr;
    return launch_rows<DLOGITS>(p.shape, f, KK_CE_DLOGITS, s);
  }

  void output(CeArgs &f, void *out, int dtype, long long ld, bool cut, long long slice_rows, bool add) const {
    f.out = cut ? static_cast<void *>(slices_) : out;
    f.out_f32 = cut || dtype == MUON_F32;
    f.ld_out = cut ? p.Dp : ld;
    f.slice_stride = slice_rows * p.Dp;
    f.accumulate = cut ? 0 : add;
    const int piece = f.out_f32 ? 4 : 8;
    f.vec = aligned(f.out, 16) && f.ld_out % piece == 0;
    // TMA ends a row at a 16-byte boundary. What lies between a row's end and there is padding in scratch and the caller's
    // in dh and dw.
    const bool padded = c.D % piece == 0 || f.out == slices_ || f.out == dw_sum_;
    f.tma = f.vec && padded && (f.out_f32 || !f.accumulate) && f.ld_out <= MAX_PITCH;
  }

  muon_status dh(long long r, long long n, int split, const ScaleJob *beside) {
    char *out = c.dh + (r0_ + r) * c.lddh * static_cast<long long>(size_of(c.dhdt));
    CeArgs f = base_;
    f.rows = static_cast<int>(n);
    f.cols = static_cast<int>(c.D);
    f.k_iters = static_cast<int>(ceil_div(c.V, BK)) * p.planes;
    f.k_low = f.k_iters - f.k_iters / p.planes;
    f.split = split;
    f.a_box = a_box();
    if (!dz_map(&f.map_a, r, n, f.a_box) || !w_map(&f.map_b, BK)) return MUON_ERR_CUDA;
    const bool cut = split > 1;
    output(f, out, c.dhdt, c.lddh, cut, n, false);
    const muon_status st =
        beside != nullptr ? launch_beside<DH>(beside, f, KK_CE_DH, s) : launch_rows<DH>(p.shape, f, KK_CE_DH, s);
    if (st != MUON_OK || !cut) return st;
    return launch_reduce(ReduceArgs{slices_, f.slice_stride, p.Dp, c.lddh, f.split, f.rows, f.cols, 0, out}, c.dhdt, s);
  }

  muon_status dw() {
    CeArgs f = base_;
    f.rows = static_cast<int>(c.V);
    f.cols = static_cast<int>(c.D);
    f.k_iters = static_cast<int>(ceil_div(rows_, BK)) * p.planes;
    f.k_low = f.k_iters - f.k_iters / p.planes;
    f.split = p.split_dw;
    if (!dz_map(&f.map_a, 0, rows_, BK) ||
        !make_bf16_map(&f.map_b, h_live_, c.D, rows_, 1, round8(c.D), round8(c.D), BK))
      return MUON_ERR_CUDA;
    // several pieces add up in fp32: in the gradient itself, or in scratch that the last piece rounds
    void *sum = dw_sum_ != nullptr ? static_cast<void *>(dw_sum_) : c.dw;
    const long long ld = dw_sum_ != nullptr ? p.Dp : c.lddw;
    const int dt = dw_sum_ != nullptr ? static_cast<int>(MUON_F32) : c.dwdt;
    const bool add = r0_ > 0 || (dw_sum_ == nullptr && c.accumulate), cut = p.split_dw > 1;
    output(f, sum, dt, ld, cut, c.V, add);
    const muon_status st = launch_gemm<DW, PAIRED, false>(f, KK_CE_DW, s);
    if (st != MUON_OK || !cut) return st;
    return launch_reduce(ReduceArgs{slices_, f.slice_stride, p.Dp, ld, f.split, f.rows, f.cols, add, sum}, dt, s);
  }

  // dz of the piece (and h_live) from losses: by halves, so that the first half's exponentials become dz beside the second
  // half's logits, and the second half's beside the first half's dh.
  muon_status joint() {
    muon_status st;
    const long long a = p.half, b = rows_ - a;
    if (b < HALVES / 4 || c.dh == nullptr) {   // also a last piece with little more than a first half
      if ((st = losses(0, rows_, true, nullptr)) != MUON_OK) return st;
      const ScaleJob all = job(0, rows_);
      // a block per unit: blocks that take several in turn are 2 to 4 % slower
      const long long units = ceil_div(rows_, SCALE_ROWS) * ceil_div(c.V, 2048);
      if ((st = small(KK_CE_DLOGITS, ce_scale_kernel, std::min(units, 1ll << 30), all)) != MUON_OK) return st;
      return c.dh != nullptr ? dh(0, rows_, p.split_dh, nullptr) : MUON_OK;
    }
    const ScaleJob first = job(0, a), second = job(a, b);
    if ((st = losses(0, a, true, nullptr)) != MUON_OK || (st = losses(a, b, true, &first)) != MUON_OK ||
        (st = dh(0, a, p.split_half, &second)) != MUON_OK)
      return st;
    return dh(a, b, p.split_half, nullptr);
  }

  muon_status piece() {
    muon_status st;
    // the exponentials are kept in dz's place, or the logits are computed again
    const bool keep = c.forward && c.backward && p.planes == 1 && c.D >= KEEP_WIDTH;
    if (keep) {
      if ((st = joint()) != MUON_OK) return st;
    } else {
      if (c.forward && (st = losses(0, rows_, false, nullptr)) != MUON_OK) return st;
      if (!c.backward) return MUON_OK;
      if ((st = dlogits()) != MUON_OK) return st;
      if (c.dh != nullptr && (st = dh(0, rows_, p.split_dh, nullptr)) != MUON_OK) return st;
      if (c.dw != nullptr && (st = small(KK_CE_ROWS, ce_rows_kernel, ceil_div(rows_, 8), copy_args(0, rows_))) != MUON_OK)
        return st;
    }
    return c.dw != nullptr ? dw() : MUON_OK;
  }

 public:
  Run(const Call &call, const Plan &pl, cudaStream_t stream) : c(call), p(pl), s(stream) {
    memset(&base_, 0, sizeof(base_));
    base_.itype = c.itype;
    base_.factor = c.grad_scale;
    base_.planes = p.planes;
    base_.err = reinterpret_cast<uint32_t *>(c.ws);
    base_.timeout_ns = wait_timeout_ns();
    ldh_ = pitch8(c.ldh, c.N, c.D);
    ldw_ = pitch8(c.ldw, c.V, c.D);
    partials_ = at<float2>(p.partials);
    z_target_ = at<float>(p.z_target);
    row_state_ = at<float4>(p.row_state);
    dz_ = at<__nv_bfloat16>(p.dz);
    h_live_ = at<__nv_bfloat16>(p.h_live);
    slices_ = at<float>(p.slices);
    dw_sum_ = c.dw != nullptr && c.dwdt != MUON_F32 ? at<float>(p.dw_sum) : nullptr;
  }

  muon_status all() {
    const ReduceArgs last{dw_sum_, 0, p.Dp, c.lddw, 1, static_cast<int>(c.V), static_cast<int>(c.D), c.accumulate, c.dw};
    if (c.N == 0) {
      ReduceArgs zeros = last;
      zeros.n = 0;
      return c.dw != nullptr && !c.accumulate ? launch_reduce(zeros, c.dwdt, s) : MUON_OK;
    }
    for (r0_ = 0; r0_ < c.N; r0_ += p.rows) {
      rows_ = std::min(p.rows, c.N - r0_);
      h_ = c.h + r0_ * ldh_ * 2;
      const muon_status st = piece();
      if (st != MUON_OK) return st;
    }
    return c.dw != nullptr && dw_sum_ != nullptr ? launch_reduce(last, c.dwdt, s) : MUON_OK;
  }
};

// ------------------------------------------------------------------------------------------ checks

constexpr int64_t MAX_ROWS = 1 << 26, MAX_COLS = 1 << 26, MAX_D = 65536;

muon_status check_sizes(int64_t N, int64_t V, int64_t D) {
  if (N < 0 || V < 1 || D < 1) return MUON_ERR_INVALID_ARG;
  if (N > MAX_ROWS || V > MAX_COLS || D > MAX_D || N * V > (1ll << 40)) return MUON_ERR_SHAPE;
  return MUON_OK;
}

muon_status check_inputs(const void *h, muon_dtype hdt, int64_t ldh, const void *w, muon_dtype wdt, int64_t ldw,
                         const void *targets, muon_itype itype, const float *weights, int64_t N, int64_t V, int64_t D) {
  muon_status st = check_sizes(N, V, D);
  if (st != MUON_OK) return st;
  if (w == nullptr || (N > 0 && (h == nullptr || targets == nullptr)) || ldh < D || ldw < D) return MUON_ERR_INVALID_ARG;
  if (hdt != MUON_BF16 || wdt != MUON_BF16 || (itype != MUON_I32 && itype != MUON_I64)) return MUON_ERR_DTYPE;
  if ((N > 1 && ldh > MAX_PITCH) || (V > 1 && ldw > MAX_PITCH)) return MUON_ERR_SHAPE;
  if (!aligned(h, 16) || !aligned(w, 16) || (N > 1 && ldh % 8 != 0) || (V > 1 && ldw % 8 != 0) ||
      !aligned(targets, itype == MUON_I32 ? 4 : 8) || !aligned(weights, 4))
    return MUON_ERR_ALIGNMENT;
  return MUON_OK;
}

muon_status check_outputs(const void *h, const void *w, const void *dh, muon_dtype dhdt, int64_t lddh, const void *dw,
                          muon_dtype dwdt, int64_t lddw, int64_t N, int64_t D, int *terms) {
  if (dh == nullptr && dw == nullptr && N > 0) return MUON_ERR_INVALID_ARG;
  if (N > 0 && ((dh != nullptr && (dh == h || dh == w || dh == dw)) || (dw != nullptr && (dw == h || dw == w))))
    return MUON_ERR_INVALID_ARG;   // h and w are read again after the first gradient is written
  *terms = 1;
  if (dh != nullptr) {
    if (lddh < D) return MUON_ERR_INVALID_ARG;
    if (!valid_dtype(dhdt)) return MUON_ERR_DTYPE;
    if (!aligned(dh, size_of(dhdt))) return MUON_ERR_ALIGNMENT;
    if (dhdt == MUON_F32) *terms = 2;
  }
  if (dw != nullptr) {
    if (lddw < D) return MUON_ERR_INVALID_ARG;
    if (!valid_dtype(dwdt)) return MUON_ERR_DTYPE;
    if (!aligned(dw, size_of(dwdt))) return MUON_ERR_ALIGNMENT;
    if (dwdt == MUON_F32) *terms = 2;
  }
  return MUON_OK;
}

// The plan is made once: the sizes that the workspace is checked for are those that the launches use.
muon_status check_and_run(const Call &c, size_t ws_bytes, muon_stream_t stream) {
  if (c.ws == nullptr) return MUON_ERR_INVALID_ARG;
  if (!aligned(c.ws, 256)) return MUON_ERR_ALIGNMENT;
  const Plan p = plan(c.N, c.V, c.D, c.terms);
  if (ws_bytes < p.total) return MUON_ERR_WORKSPACE;
  const muon_status st = device_check();
  return st != MUON_OK ? st : Run(c, p, reinterpret_cast<cudaStream_t>(stream)).all();
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t linear_cross_entropy_workspace_bytes(int64_t N, int64_t V, int64_t D, int terms) {
  if (check_sizes(N, V, D) != MUON_OK || terms < 0 || terms > 2) return 0;
  size_t most = 0;   // a call with fewer terms splits differently: its slices can be more than dz saves
  for (int t = 0; t <= terms; ++t) most = std::max(most, plan(N, V, D, t).total);
  return most;
}

muon_status linear_cross_entropy_forward(const void *h, muon_dtype hdt, int64_t ldh, const void *w, muon_dtype wdt,
                                         int64_t ldw, const void *targets, muon_itype itype, const float *weights,
                                         float *losses, float *lse, int64_t N, int64_t V, int64_t D, void *ws,
                                         size_t ws_bytes, muon_stream_t stream) {
  muon_status st = check_inputs(h, hdt, ldh, w, wdt, ldw, targets, itype, weights, N, V, D);
  if (st != MUON_OK) return st;
  if (N > 0 && (losses == nullptr || lse == nullptr)) return MUON_ERR_INVALID_ARG;
  if (!aligned(losses, 4) || !aligned(lse, 4)) return MUON_ERR_ALIGNMENT;
  Call c{};
  c.h = static_cast<const char *>(h);
  c.w = static_cast<const char *>(w);
  c.ldh = ldh;
  c.ldw = ldw;
  c.targets = targets;
  c.itype = itype;
  c.weights = weights;
  c.N = N;
  c.V = V;
  c.D = D;
  c.losses = losses;
  c.lse = lse;
  c.ws = static_cast<char *>(ws);
  c.forward = true;
  return check_and_run(c, ws_bytes, stream);
}

muon_status linear_cross_entropy_backward(const void *h, muon_dtype hdt, int64_t ldh, const void *w, muon_dtype wdt,
                                          int64_t ldw, const void *targets, muon_itype itype, const float *weights,
                                          const float *lse, const float *grad, void *dh, muon_dtype dhdt, int64_t lddh,
                                          void *dw, muon_dtype dwdt, int64_t lddw, int accumulate, int64_t N, int64_t V,
                                          int64_t D, void *ws, size_t ws_bytes, muon_stream_t stream) {
  muon_status st = check_inputs(h, hdt, ldh, w, wdt, ldw, targets, itype, weights, N, V, D);
  if (st != MUON_OK) return st;
  Call c{};
  if (N > 0 && lse == nullptr) return MUON_ERR_INVALID_ARG;
  if (!aligned(lse, 4) || !aligned(grad, 4)) return MUON_ERR_ALIGNMENT;
  if ((st = check_outputs(h, w, dh, dhdt, lddh, dw, dwdt, lddw, N, D, &c.terms)) != MUON_OK) return st;
  c.h = static_cast<const char *>(h);
  c.w = static_cast<const char *>(w);
  c.ldh = ldh;
  c.ldw = ldw;
  c.targets = targets;
  c.itype = itype;
  c.weights = weights;
  c.N = N;
  c.V = V;
  c.D = D;
  c.lse_in = lse;
  c.grad = grad;
  c.grad_scale = 1.f;
  c.dh = static_cast<char *>(dh);
  c.dw = static_cast<char *>(dw);
  c.dhdt = dhdt;
  c.dwdt = dwdt;
  c.lddh = lddh;
  c.lddw = lddw;
  c.accumulate = accumulate != 0;
  c.ws = static_cast<char *>(ws);
  c.backward = true;
  return check_and_run(c, ws_bytes, stream);
}

muon_status linear_cross_entropy_forward_backward(const void *h, muon_dtype hdt, int64_t ldh, const void *w,
                                                  muon_dtype wdt, int64_t ldw, const void *targets, muon_itype itype,
                                                  const float *weights, float grad_scale, float *losses, float *lse,
                                                  void *dh, muon_dtype dhdt, int64_t lddh, void *dw, muon_dtype dwdt,
                                                  int64_t lddw, int accumulate, int64_t N, int64_t V, int64_t D, void *ws,
                                                  size_t ws_bytes, muon_stream_t stream) {
  muon_status st = check_inputs(h, hdt, ldh, w, wdt, ldw, targets, itype, weights, N, V, D);
  if (st != MUON_OK) return st;
  Call c{};
  if ((N > 0 && (losses == nullptr || lse == nullptr)) || !std::isfinite(grad_scale)) return MUON_ERR_INVALID_ARG;
  if (!aligned(losses, 4) || !aligned(lse, 4)) return MUON_ERR_ALIGNMENT;
  if ((st = check_outputs(h, w, dh, dhdt, lddh, dw, dwdt, lddw, N, D, &c.terms)) != MUON_OK) return st;
  c.h = static_cast<const char *>(h);
  c.w = static_cast<const char *>(w);
  c.ldh = ldh;
  c.ldw = ldw;
  c.targets = targets;
  c.itype = itype;
  c.weights = weights;
  c.N = N;
  c.V = V;
  c.D = D;
  c.losses = losses;
  c.lse = lse;
  c.grad_scale = grad_scale;
  c.dh = static_cast<char *>(dh);
  c.dw = static_cast<char *>(dw);
  c.dhdt = dhdt;
  c.dwdt = dwdt;
  c.lddh = lddh;
  c.lddw = lddw;
  c.accumulate = accumulate != 0;
  c.ws = static_cast<char *>(ws);
  c.forward = c.backward = true;
  return check_and_run(c, ws_bytes, stream);
}

muon_status muon_debug_loss_rows(int64_t rows) {
  if (rows < 0) return MUON_ERR_INVALID_ARG;
  g_piece_rows.store(rows);
  return MUON_OK;
}

}  // extern "C"
