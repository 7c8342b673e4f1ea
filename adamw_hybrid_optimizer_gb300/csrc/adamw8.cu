// AdamW over many tensors at once with both moments held in 8 bits.
//
// Per element, with the moments of ADAMW8_BLOCK consecutive elements sharing one scale each:
//     m = beta1 (sm cm) + (1 - beta1) g        cm: e4m3 code of the first moment, sm its block's scale
//     v = beta2 (sr cr)^2 + (1 - beta2) g^2    cr: e4m3 code of the root of the second moment, sr its block's scale
//     p as in AdamW from m and v, then  cm = e4m3(m / sm'), cr = e4m3(sqrt(v) / sr')  with sm', sr' from the new moments
// ("Optimizers: AdamW, Muon and the distributed optimizer", sections "AdamW: decoupled weight decay" and "The optimizer's
// memory budget", which the moments dominate). The root is what is held because it has half the range of v in powers of
// two, so that the 18 of e4m3 cover 36 of v, and because the step needs the root anyway.
//
// A scale is its block's largest magnitude / 448, so the largest moment of a block is exact up to fp32 and decays
// exactly; rounding to nearest. A second moment that is not zero never becomes zero. A moment that is not finite becomes
// NaN and leaves the others of its block alone.
//
// Bound by HBM: 10 bytes and a 16-byte pair of scales per 256 elements for bf16 weights and gradients (22 bytes with fp32
// moments). One warp takes a block: 8 elements per lane, so that the block's maxima are one register reduction each.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <vector>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int BLOCK = ADAMW8_BLOCK;
constexpr int THREADS = 128;
constexpr int BLOCKS_PER_SM = 8;
constexpr float TOP = 448.f;            // the largest e4m3 value
constexpr float LEAST = 0x1p-9f;        // the smallest above zero
// A block whose moments are all below this is scaled as if this were its largest, so that 448 / largest stays finite.
constexpr float FLOOR = 0x1p-100f;

// One tensor of a launch; its blocks are numbered from block_begin.
struct Tensor8 {
  void *p;
  const void *g;
  uint8_t *m, *r;
  float2 *scales;
  float *master;
  long long n, block_begin;
  int pdt, gdt, vec;
  AdamwConst c;
};

struct Group8 {
  Tensor8 t[ADAMW_GROUP_MAX];
  int ntensors, chunk;       // blocks a warp takes in one turn
  long long total_blocks;
};
static_assert(sizeof(Group8) <= 32764, "kernel parameter block too large");

__device__ __forceinline__ float2 decode2(unsigned short codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(codes, __NV_E4M3)));
}
__device__ __forceinline__ unsigned encode2(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// The largest of the warp's magnitudes; NaN counts as zero.
__device__ __forceinline__ float warp_largest(const float (&x)[8]) {
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) t = fmaxf(t, fabsf(x[k]));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t)));
}

// As warp_largest over the finite values; the infinite ones become NaN, which e4m3 holds.
__device__ __noinline__ float warp_largest_finite(float (&x)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (isinf(x[k])) x[k] = __uint_as_float(0x7fffffffu);
  return warp_largest(x);
}

// The update of one block: 8 elements per lane. Every rounding is spelled out, so that each way of loading the elements
// gives the same bits. pf: weights in and out; gf: gradients; cm, cr: codes in and out; s: scales in and out.
__device__ __forceinline__ void update(float (&pf)[8], float (&gf)[8], uint2 &cm, uint2 &cr, float2 &s,
                                       const AdamwConst &c) {
  if (c.l2) {
#pragma unroll
    for (int k = 0; k < 8; ++k) gf[k] = fmaf(c.l2_wd, pf[k], gf[k]);
  }
  float m[8], r[8];
  const float km = __fmul_rn(s.x, c.beta1), kr = __fmul_rn(__fmul_rn(s.y, s.y), c.beta2);
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const unsigned wm = k < 4 ? cm.x : cm.y, wr = k < 4 ? cr.x : cr.y;
    const float2 dm = decode2(static_cast<unsigned short>(wm >> (8 * (k & 2))));
    const float2 dr = decode2(static_cast<unsigned short>(wr >> (8 * (k & 2))));
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float g = gf[k + e], q = e ? dr.y : dr.x;
      m[k + e] = fmaf(km, e ? dm.y : dm.x, __fmul_rn(c.one_minus_beta1, g));
      const float v = fmaf(kr, __fmul_rn(q, q), __fmul_rn(__fmul_rn(c.one_minus_beta2, g), g));
      r[k + e] = __fsqrt_rn(v);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    pf[k] = fmaf(-c.step_size, __fdiv_rn(m[k], fmaf(r[k], c.inv_sqrt_bc2, c.eps)), __fmul_rn(pf[k], c.decay));
  float tm = warp_largest(m), tr = warp_largest(r);
  if (isinf(tm)) tm = warp_largest_finite(m);
  if (isinf(tr)) tr = warp_largest_finite(r);
  tm = fmaxf(tm, FLOOR);
  tr = fmaxf(tr, FLOOR);
  const float im = __fdiv_rn(TOP, tm), ir = __fdiv_rn(TOP, tr);
  s = make_float2(__fmul_rn(tm, 1.f / TOP), __fmul_rn(tr, 1.f / TOP));
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    m[k] = __fmul_rn(m[k], im);
    const float y = __fmul_rn(r[k], ir);
    r[k] = r[k] > 0.f ? fmaxf(y, LEAST) : y;
  }
  cm.x = encode2(m[0], m[1]) | encode2(m[2], m[3]) << 16;
  cm.y = encode2(m[4], m[5]) | encode2(m[6], m[7]) << 16;
  cr.x = encode2(r[0], r[1]) | encode2(r[2], r[3]) << 16;
  cr.y = encode2(r[4], r[5]) | encode2(r[6], r[7]) << 16;
}

// Blocks [b0, b1) of a tensor by one warp. Lane l of a full block of aligned arrays has its elements 8 l .. 8 l + 7, else
// elements l, l + 32, ...: the sums over a block are maxima, so both give the same bits.
template <typename PT, typename GT, bool MASTER>
__device__ __forceinline__ void span(const Tensor8 &d, long long b0, long long b1, int lane) {
  PT *p = static_cast<PT *>(d.p);
  const GT *g = static_cast<const GT *>(d.g);
  uint8_t *m = d.m, *r = d.r;
  float *ms = d.master;
  const long long n = d.n;
#pragma unroll 1
  for (long long b = b0; b < b1; ++b) {
    float pf[8], gf[8];
    uint2 cm, cr;
    float2 s = d.scales[b];
    if (d.vec && (b + 1) * BLOCK <= n) {
      const long long o = b * BLOCK + 8 * lane;
      if constexpr (MASTER) load8(ms + o, pf);
      else load8(p + o, pf);
      load8(g + o, gf);
      cm = *reinterpret_cast<const uint2 *>(m + o);
      cr = *reinterpret_cast<const uint2 *>(r + o);
      update(pf, gf, cm, cr, s, d.c);
      if constexpr (MASTER) store8(ms + o, pf);
      store8(p + o, pf);
      *reinterpret_cast<uint2 *>(m + o) = cm;
      *reinterpret_cast<uint2 *>(r + o) = cr;
    } else {
      const long long o = b * BLOCK + lane;
      cm = cr = make_uint2(0u, 0u);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const long long i = o + 32 * k;
        const bool in = i < n;
        pf[k] = !in ? 0.f : MASTER ? ms[i] : load1(p, i);
        gf[k] = in ? load1(g, i) : 0.f;
        const unsigned um = in ? m[i] : 0u, ur = in ? r[i] : 0u;
        (k < 4 ? cm.x : cm.y) |= um << (8 * (k & 3));
        (k < 4 ? cr.x : cr.y) |= ur << (8 * (k & 3));
      }
      update(pf, gf, cm, cr, s, d.c);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const long long i = o + 32 * k;
        if (i >= n) continue;
        if constexpr (MASTER) ms[i] = pf[k];
        store1(p, i, pf[k]);
        m[i] = static_cast<uint8_t>((k < 4 ? cm.x : cm.y) >> (8 * (k & 3)));
        r[i] = static_cast<uint8_t>((k < 4 ? cr.x : cr.y) >> (8 * (k & 3)));
      }
    }
    if (lane == 0) d.scales[b] = s;
  }
}

__global__ void __launch_bounds__(THREADS, BLOCKS_PER_SM) adamw8_kernel(const __grid_constant__ Group8 G) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long warp = static_cast<long long>(blockIdx.x) * (THREADS / 32) + threadIdx.x / 32;
  const long long stride = static_cast<long long>(gridDim.x) * (THREADS / 32) * G.chunk;
  for (long long first = warp * G.chunk; first < G.total_blocks; first += stride) {
    const long long last = min(first + G.chunk, G.total_blocks);
    int lo = 0, hi = G.ntensors - 1;   // the last tensor that begins at or before `first`
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (G.t[mid].block_begin <= first) lo = mid;
      else hi = mid - 1;
    }
    for (long long b = first; b < last; ++lo) {
      const Tensor8 &d = G.t[lo];
      const long long b0 = b - d.block_begin, b1 = min(last - d.block_begin, (d.n + BLOCK - 1) / BLOCK);
      if (d.master != nullptr) {
        if (d.gdt == MUON_F32) span<__nv_bfloat16, float, true>(d, b0, b1, lane);
        else span<__nv_bfloat16, __nv_bfloat16, true>(d, b0, b1, lane);
      } else if (d.pdt == MUON_F32) {
        if (d.gdt == MUON_F32) span<float, float, false>(d, b0, b1, lane);
        else span<float, __nv_bfloat16, false>(d, b0, b1, lane);
      } else {
        if (d.gdt == MUON_F32) span<__nv_bfloat16, float, false>(d, b0, b1, lane);
        else span<__nv_bfloat16, __nv_bfloat16, false>(d, b0, b1, lane);
      }
      b = d.block_begin + b1;
    }
  }
}

bool aligned(const void *p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }
uintptr_t bytes_of(int dt) { return dt == MUON_F32 ? 4 : 2; }

muon_status check_tensor8(const adamw8_tensor &x) {
  if (x.param == nullptr || x.grad == nullptr || x.exp_avg == nullptr || x.exp_avg_sq == nullptr || x.scales == nullptr ||
      x.hp == nullptr || x.n < 1)
    return MUON_ERR_INVALID_ARG;
  if (x.n > (1ll << 40)) return MUON_ERR_SHAPE;
  if (!valid_dtype(x.pdt) || !valid_dtype(x.gdt) || (x.master != nullptr && x.pdt != MUON_BF16)) return MUON_ERR_DTYPE;
  if (!aligned(x.param, bytes_of(x.pdt)) || !aligned(x.grad, bytes_of(x.gdt)) || !aligned(x.master, 4) ||
      !aligned(x.scales, 8))
    return MUON_ERR_ALIGNMENT;
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status adamw8_step_grouped(const adamw8_tensor *tensors, int64_t n, muon_stream_t stream) {
  if (tensors == nullptr || n < 1 || n > (1 << 20)) return MUON_ERR_INVALID_ARG;
  muon_status st;
  AdamwConst c{};
  for (int64_t i = 0; i < n; ++i)
    if ((st = check_tensor8(tensors[i])) != MUON_OK || (st = adamw_constants(tensors[i].hp, &c)) != MUON_OK) return st;
  if ((st = device_check()) != MUON_OK) return st;
  const long long warps = static_cast<long long>(device_sm_count()) * BLOCKS_PER_SM * (THREADS / 32);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  Group8 G;
  for (int64_t i = 0; i < n;) {
    G.ntensors = 0;
    G.total_blocks = 0;
    for (; i < n && G.ntensors < ADAMW_GROUP_MAX; ++i) {
      const adamw8_tensor &x = tensors[i];
      Tensor8 &d = G.t[G.ntensors++];
      adamw_constants(x.hp, &d.c);
      d.p = x.param;
      d.g = x.grad;
      d.m = static_cast<uint8_t *>(x.exp_avg);
      d.r = static_cast<uint8_t *>(x.exp_avg_sq);
      d.scales = reinterpret_cast<float2 *>(x.scales);
      d.master = x.master;
      d.n = x.n;
      d.block_begin = G.total_blocks;
      d.pdt = x.pdt;
      d.gdt = x.gdt;
      d.vec = aligned(x.param, 16) && aligned(x.grad, 16) && aligned(x.master, 16) && aligned(x.exp_avg, 8) &&
              aligned(x.exp_avg_sq, 8);
      G.total_blocks += (x.n + BLOCK - 1) / BLOCK;
    }
    // a few turns per warp, so that the last one is a small part of the pass
    G.chunk = static_cast<int>(std::min(8ll, std::max(1ll, G.total_blocks / (8 * warps))));
    const long long turns = (G.total_blocks + G.chunk - 1) / G.chunk;
    const long long blocks = std::min(warps / (THREADS / 32), (turns + THREADS / 32 - 1) / (THREADS / 32));
    launch_begin(KK_ADAMW8, s);
    const cudaError_t e = launch_pdl(adamw8_kernel, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, s, G);
    launch_end(s);
    if (e != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

}  // extern "C"
