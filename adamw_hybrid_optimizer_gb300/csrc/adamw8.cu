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
// exactly; rounding to nearest. A second moment that fp32 holds above zero keeps a code above zero. A moment that is not finite
// becomes NaN and leaves the others of its block alone.
//
// A first moment without a gradient has to end, since the step divides it by a root that shrinks with it: held at one smallest
// code it would move its weight by some 0.1 lr a step, always the same way. But 0.9 of up to five smallest codes rounds to as
// many. Where the gradient is zero, codes below 2^-6, whose steps are all 2^-9, are therefore rounded toward zero. (Steps above
// are at most 1/9 of a code, half of which beta1 up to 15/16 takes away.) Where a whole block has no gradient its scales shrink
// instead; with L2 the weight's own term is a gradient.
//
// Bound by HBM: 10 bytes and a 16-byte pair of scales per 256 elements for bf16 weights and gradients (22 bytes with fp32
// moments). One warp takes a block: 8 elements per lane, so that the block's maxima are one register reduction each.
#include <cuda_bf16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstring>
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"
#include "vec.cuh"

namespace muon {
namespace {

constexpr int BLOCK = ADAMW8_BLOCK;
// Resident blocks: 32 warps of 64 registers where weights and gradients are bf16, 24 of 80 where one is fp32 or there is a
// master. (1.05 G elements, bf16: 1692 us with 4 blocks, 1721 with 3, 1739 with 3.5, 2145 with 5; 77 M elements, fp32: 185 us with
// 3, 200 with 2, 203 with 3.5, 213 with 4. The kernels spill 20 and 36 bytes a thread so; with 5 and 4 blocks 164 and 244.)
constexpr int THREADS = 256;
constexpr int NARROW_BLOCKS = 4;
constexpr int WIDE_BLOCKS = 3;
constexpr float TOP = 448.f;            // the largest e4m3 value
constexpr float LEAST = 0x1p-9f;        // the smallest above zero
// A block whose moments are all below this is scaled as if this were its largest, so that 448 / largest stays finite.
constexpr float FLOOR = 0x1p-100f;
// From here on beta2 times the square of a scale is a normal number (for beta2 of 2^-26 or more).
constexpr float SMALL_SCALE = 0x1p-50f;

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
  int ntensors;
  long long total_blocks;
};
static_assert(sizeof(Group8) <= 32764, "kernel parameter block too large");

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float2 decode2(unsigned codes) {
  return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(static_cast<unsigned short>(codes), __NV_E4M3)));
}
__device__ __forceinline__ unsigned encode2(float2 x) { return __nv_cvt_float2_to_fp8x2(x, __NV_SATFINITE, __NV_E4M3); }

// The square root by one Newton step on an approximate one, in fma: with s = v y, y about 1 / sqrt(v), it is
// s + (v - s^2) y / 2, as close as fp32 gets in all but a few cases in a million. 0 and infinity, for which that is NaN, are
// their own roots.
__device__ __forceinline__ float2 root2(float2 v) {
  const float2 y = make_float2(rsqrtf(v.x), rsqrtf(v.y));
  const float2 s = __fmul2_rn(v, y);
  const float2 e = __ffma2_rn(make_float2(-s.x, -s.y), s, v);
  const float2 r = __ffma2_rn(e, __fmul2_rn(y, both(0.5f)), s);
  return make_float2(r.x == r.x ? r.x : v.x, r.y == r.y ? r.y : v.y);
}

// To two units in the last place: the weights take it times the learning rate.
__device__ __forceinline__ float quick_divide(float a, float b) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
  return a * y;
}

// The largest of the warp's magnitudes, NaN counting as zero.
__device__ __forceinline__ float warp_largest(const Vals<8> &x) {
  float t = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) t = fmaxf(t, fmaxf(fabsf(x.p[k].x), fabsf(x.p[k].y)));
  return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(t)));
}

// As above over the finite values: infinite ones become NaN, which e4m3 holds.
__device__ __forceinline__ float warp_largest_finite(Vals<8> &x) {
  const float t = warp_largest(x);
  if (!isinf(t)) return t;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (isinf(x.p[k].x)) x.p[k].x = __uint_as_float(0x7fffffffu);
    if (isinf(x.p[k].y)) x.p[k].y = __uint_as_float(0x7fffffffu);
  }
  return warp_largest(x);
}

// Whether a lane has an element without a gradient.
__device__ __forceinline__ bool any_zero(const Vals<8> &g) {
  float least = INFINITY;
#pragma unroll
  for (int k = 0; k < 4; ++k) least = fminf(least, fminf(fabsf(g.p[k].x), fabsf(g.p[k].y)));
  return least == 0.f;
}
__device__ __forceinline__ bool any_zero(const Raw<float, 8> &g) { return any_zero(g.get()); }
__device__ __forceinline__ bool any_zero(const Raw<__nv_bfloat16, 8> &g) {   // two values at a time
  auto pair = [&](int i) { return __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&g.w[i])); };
  const __nv_bfloat162 least = __hmin2(__hmin2(pair(0), pair(1)), __hmin2(pair(2), pair(3)));
  const unsigned bits = *reinterpret_cast<const unsigned *>(&least);
  return (bits & 0x7fffu) == 0 || bits < 0x10000u;
}

// A lane's first moments' codes again where its gradients g are zero and others of the block are not: rounded toward zero below
// 2^-6. held(): the old codes; km: beta1 times their scale; im: 1 / the new one. Apart from the update, which has no registers
// left (within it: 1701 us for 1.05 G elements, bf16, instead of 1688; 1648 without any of this. 128256 x 4096 with gradients in
// 3% of the rows: 840 us without, 913 with it).
template <typename Held>
__device__ __forceinline__ void fade(const Vals<8> &g, const Held &held, float km, float im, uint2 &cm) {
  bool each = true;
#pragma unroll
  for (int k = 0; k < 4; ++k) each = each && g.p[k].x == 0.f && g.p[k].y == 0.f;
  if (__all_sync(0xffffffffu, each)) return;
  const uint2 old = held();
  auto round = [](float x, float y) { return x == 0.f && fabsf(y) < 0x1p-6f ? truncf(y * 0x1p9f) * LEAST : y; };
  unsigned e[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int shift = 16 * (k & 1);
    const float2 y = __fmul2_rn(__fmul2_rn(both(km), decode2((k < 2 ? old.x : old.y) >> shift)), both(im));
    const unsigned now = encode2(make_float2(round(g.p[k].x, y.x), round(g.p[k].y, y.y)));
    const unsigned keep = (g.p[k].x == 0.f ? 0u : 0xffu) | (g.p[k].y == 0.f ? 0u : 0xff00u);
    e[k] = (now & ~keep) | ((k < 2 ? cm.x : cm.y) >> shift & keep);
  }
  cm = make_uint2(e[0] | e[1] << 16, e[2] | e[3] << 16);
}

// The update of one block: 8 elements per lane. Every rounding is spelled out, so that each way of loading the elements
// gives the same bits. w: weights in and out; g: gradients; cm, cr: codes in and out; s: scales in and out; inv: 1 / the first
// moments' new one. The old second moment is beta2 (scale code)^2: the square of a small scale underflows where that, up to 448^2
// times as much, does not. Such a scale therefore takes a power of two (up) that the codes give back (down), which changes no
// other rounding.
template <bool SCALED>
__device__ __forceinline__ void update_as(Vals<8> &w, Vals<8> &g, uint2 &cm, uint2 &cr, float2 &s, const AdamwConst &c,
                                          float up, float down, float &inv) {
  if (c.l2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) g.p[k] = __ffma2_rn(both(c.l2_wd), w.p[k], g.p[k]);
  }
  Vals<8> m, r;
  const float sr = SCALED ? __fmul_rn(s.y, up) : s.y;
  const float2 km = both(__fmul_rn(s.x, c.beta1)), kr = both(__fmul_rn(__fmul_rn(sr, sr), c.beta2));
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int shift = 16 * (k & 1);
    float2 q = decode2((k < 2 ? cr.x : cr.y) >> shift);
    if constexpr (SCALED) q = __fmul2_rn(q, both(down));
    m.p[k] = __ffma2_rn(km, decode2((k < 2 ? cm.x : cm.y) >> shift), __fmul2_rn(both(c.one_minus_beta1), g.p[k]));
    r.p[k] = root2(__ffma2_rn(kr, __fmul2_rn(q, q), __fmul2_rn(__fmul2_rn(both(c.one_minus_beta2), g.p[k]), g.p[k])));
    const float2 d = __ffma2_rn(r.p[k], both(c.inv_sqrt_bc2), both(c.eps));
    w.p[k] = __ffma2_rn(both(-c.step_size), make_float2(quick_divide(m.p[k].x, d.x), quick_divide(m.p[k].y, d.y)),
                        __fmul2_rn(w.p[k], both(c.decay)));
  }
  const float tm = fmaxf(warp_largest_finite(m), FLOOR), tr = fmaxf(warp_largest_finite(r), FLOOR);
  const float2 im = both(__fmul_rn(TOP, __frcp_rn(tm))), ir = both(__fmul_rn(TOP, __frcp_rn(tr)));
  s = make_float2(__fmul_rn(tm, 1.f / TOP), __fmul_rn(tr, 1.f / TOP));
  inv = im.x;
  unsigned em[4], er[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    em[k] = encode2(__fmul2_rn(m.p[k], im));
    float2 y = __fmul2_rn(r.p[k], ir);
    if (r.p[k].x > 0.f) y.x = fmaxf(y.x, LEAST);
    if (r.p[k].y > 0.f) y.y = fmaxf(y.y, LEAST);
    er[k] = encode2(y);
  }
  cm = make_uint2(em[0] | em[1] << 16, em[2] | em[3] << 16);
  cr = make_uint2(er[0] | er[1] << 16, er[2] | er[3] << 16);
}

// Wide types wait for memory and take the multiplication for every scale (77 M elements, fp32: 187 us, 192 with the branch);
// bf16 ones, which issue more than they load, branch (1.05 G elements: 1647 us, 1708 without).
template <bool WIDE>
__device__ __forceinline__ void update(Vals<8> &w, Vals<8> &g, uint2 &cm, uint2 &cr, float2 &s, const AdamwConst &c,
                                       float &inv) {
  const bool small = s.y < SMALL_SCALE;
  if constexpr (WIDE) update_as<true>(w, g, cm, cr, s, c, small ? 0x1p40f : 1.f, small ? 0x1p-40f : 1.f, inv);
  else if (small) update_as<true>(w, g, cm, cr, s, c, 0x1p40f, 0x1p-40f, inv);
  else update_as<false>(w, g, cm, cr, s, c, 1.f, 1.f, inv);
}

// A full block of aligned arrays as it lies in memory: lane l has elements 8 l .. 8 l + 7. W: the weights that take the
// update.
template <typename W, typename GT>
struct Block8 {
  Raw<W, 8> w;
  Raw<GT, 8> g;
  uint2 cm, cr;
  float2 s;
  __device__ __forceinline__ void load(const Tensor8 &d, const W *weights, long long b, int lane) {
    const long long o = b * BLOCK + 8 * lane;
    w.load(weights + o);
    g.load(static_cast<const GT *>(d.g) + o);
    cm = *reinterpret_cast<const uint2 *>(d.m + o);
    cr = *reinterpret_cast<const uint2 *>(d.r + o);
    s = d.scales[b];
  }
};

// Blocks b, b + stride, ... of a tensor by one warp; returns the first that is past its end. Full blocks of aligned arrays
// are loaded one turn ahead; a lane of any other has elements l, l + 32, ...: the sums over a block are maxima, so both give
// the same bits.
template <typename PT, typename GT, bool MASTER>
__device__ __forceinline__ long long span(const Tensor8 &d, long long b, long long stride, int lane) {
  using W = typename std::conditional<MASTER, float, PT>::type;
  constexpr bool WIDE = sizeof(W) == 4 || sizeof(GT) == 4;
  W *weights = MASTER ? reinterpret_cast<W *>(d.master) : static_cast<W *>(d.p);
  PT *p = static_cast<PT *>(d.p);
  const GT *g = static_cast<const GT *>(d.g);
  uint8_t *m = d.m, *r = d.r;
  const long long n = d.n, end = (n + BLOCK - 1) / BLOCK, whole = d.vec ? n / BLOCK : 0;
  if (b < whole) {
    Block8<W, GT> next;
    next.load(d, weights, b, lane);
#pragma unroll 1
    do {
      Block8<W, GT> x = next;
      const long long o = b * BLOCK + 8 * lane, at = b;
      b += stride;
      if (b < whole) next.load(d, weights, b, lane);
      Vals<8> w = x.w.get(), gv = x.g.get();
      const bool some_zero = any_zero(x.g) && !d.c.l2;
      const float km = __fmul_rn(x.s.x, d.c.beta1);
      float inv;
      update<WIDE>(w, gv, x.cm, x.cr, x.s, d.c, inv);
      if (__any_sync(0xffffffffu, some_zero)) {   // from memory: registers are short, and few blocks come here
        Raw<GT, 8> again;
        again.load(g + o);
        fade(again.get(), [&] { return *reinterpret_cast<const uint2 *>(m + o); }, km, inv, x.cm);
      }
      if constexpr (MASTER) store_vals(weights + o, w);
      store_vals(p + o, w);
      *reinterpret_cast<uint2 *>(m + o) = x.cm;
      *reinterpret_cast<uint2 *>(r + o) = x.cr;
      if (lane == 0) d.scales[at] = x.s;
    } while (b < whole);
  }
#pragma unroll 1
  for (; b < end; b += stride) {
    const long long o = b * BLOCK + lane;
    Vals<8> w, gv;
    uint2 cm = make_uint2(0u, 0u), cr = cm;
    float2 s = d.scales[b];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long long i = o + 32 * k;
      const bool in = i < n;
      (k & 1 ? w.p[k / 2].y : w.p[k / 2].x) = in ? load1(weights, i) : 0.f;
      (k & 1 ? gv.p[k / 2].y : gv.p[k / 2].x) = in ? load1(g, i) : 0.f;
      (k < 4 ? cm.x : cm.y) |= (in ? m[i] : 0u) << (8 * (k & 3));
      (k < 4 ? cr.x : cr.y) |= (in ? r[i] : 0u) << (8 * (k & 3));
    }
    const Vals<8> given = gv;
    const uint2 held = cm;
    const float km = __fmul_rn(s.x, d.c.beta1);
    float inv;
    update<WIDE>(w, gv, cm, cr, s, d.c, inv);
    if (!d.c.l2) fade(given, [&] { return held; }, km, inv, cm);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const long long i = o + 32 * k;
      if (i >= n) continue;
      const float x = k & 1 ? w.p[k / 2].y : w.p[k / 2].x;
      if constexpr (MASTER) store1(weights, i, x);
      store1(p, i, x);
      m[i] = static_cast<uint8_t>((k < 4 ? cm.x : cm.y) >> (8 * (k & 3)));
      r[i] = static_cast<uint8_t>((k < 4 ? cr.x : cr.y) >> (8 * (k & 3)));
    }
    if (lane == 0) d.scales[b] = s;
  }
  return b;
}

// Warps take the launch's blocks in turn, so that those in flight at any time lie next to each other.
template <bool WIDE>
__global__ void __launch_bounds__(THREADS, WIDE ? WIDE_BLOCKS : NARROW_BLOCKS) adamw8_kernel(const __grid_constant__ Group8 G) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  const int lane = threadIdx.x % 32;
  const long long stride = static_cast<long long>(gridDim.x) * (THREADS / 32);
  long long b = static_cast<long long>(blockIdx.x) * (THREADS / 32) + threadIdx.x / 32;
  while (b < G.total_blocks) {
    int lo = 0, hi = G.ntensors - 1;   // the last tensor that begins at or before b
    while (lo < hi) {
      const int mid = (lo + hi + 1) / 2;
      if (G.t[mid].block_begin <= b) lo = mid;
      else hi = mid - 1;
    }
    const Tensor8 &d = G.t[lo];
    long long own = b - d.block_begin;
    if constexpr (!WIDE) {
      own = span<__nv_bfloat16, __nv_bfloat16, false>(d, own, stride, lane);
    } else if (d.master != nullptr) {
      if (d.gdt == MUON_F32) own = span<__nv_bfloat16, float, true>(d, own, stride, lane);
      else own = span<__nv_bfloat16, __nv_bfloat16, true>(d, own, stride, lane);
    } else if (d.pdt == MUON_F32) {
      if (d.gdt == MUON_F32) own = span<float, float, false>(d, own, stride, lane);
      else own = span<float, __nv_bfloat16, false>(d, own, stride, lane);
    } else {
      own = span<__nv_bfloat16, float, false>(d, own, stride, lane);
    }
    b = d.block_begin + own;
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

// Constants of a call's tensors, most of which share their hyperparameters: two powers each otherwise.
class Constants {
  adamw_hparams hp_{};
  AdamwConst c_{};
  bool any_ = false;

 public:
  muon_status get(const adamw_hparams *hp, AdamwConst *out) {
    if (!any_ || memcmp(hp, &hp_, sizeof(hp_)) != 0) {
      const muon_status st = adamw_constants(hp, &c_);
      if (st != MUON_OK) return st;
      hp_ = *hp;
      any_ = true;
    }
    *out = c_;
    return MUON_OK;
  }
};

bool is_wide(const adamw8_tensor &x) { return x.master != nullptr || x.pdt == MUON_F32 || x.gdt == MUON_F32; }

// The tensors of one kind, ADAMW_GROUP_MAX a launch.
template <bool WIDE>
muon_status launch_kind(const adamw8_tensor *tensors, int64_t n, cudaStream_t s) {
  constexpr int PER_SM = WIDE ? WIDE_BLOCKS : NARROW_BLOCKS;
  Group8 G;
  Constants constants;
  for (int64_t i = 0; i < n;) {
    G.ntensors = 0;
    G.total_blocks = 0;
    for (; i < n && G.ntensors < ADAMW_GROUP_MAX; ++i) {
      const adamw8_tensor &x = tensors[i];
      if (is_wide(x) != WIDE) continue;
      Tensor8 &d = G.t[G.ntensors++];
      constants.get(x.hp, &d.c);   // checked by the caller
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
    if (G.ntensors == 0) break;
    const long long blocks = std::min<long long>(static_cast<long long>(device_sm_count()) * PER_SM,
                                                 (G.total_blocks + THREADS / 32 - 1) / (THREADS / 32));
    launch_begin(KK_ADAMW8, s);
    const cudaError_t e = launch_pdl(adamw8_kernel<WIDE>, dim3(static_cast<unsigned>(blocks)), dim3(THREADS), 0, s, G);
    launch_end(s);
    if (e != cudaSuccess) return MUON_ERR_CUDA;
  }
  return MUON_OK;
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status adamw8_check_grouped(const adamw8_tensor *tensors, int64_t n) {
  if (tensors == nullptr || n < 1 || n > (1 << 20)) return MUON_ERR_INVALID_ARG;
  muon_status st;
  AdamwConst c{};
  Constants constants;
  for (int64_t i = 0; i < n; ++i)
    if ((st = check_tensor8(tensors[i])) != MUON_OK || (st = constants.get(tensors[i].hp, &c)) != MUON_OK) return st;
  return MUON_OK;
}

muon_status adamw8_step_grouped(const adamw8_tensor *tensors, int64_t n, muon_stream_t stream) {
  muon_status st = adamw8_check_grouped(tensors, n);
  if (st != MUON_OK) return st;
  if ((st = device_check()) != MUON_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if ((st = launch_kind<false>(tensors, n, s)) != MUON_OK) return st;
  return launch_kind<true>(tensors, n, s);
}

}  // extern "C"
