// Layer norm's gradients.
//
//   xh = (x - mu) r, g = dy w,  dx = r (g - mean(g) - xh mean(g xh)),  dw = sum_rows dy xh,  db = sum_rows dy
//
// Bound by bandwidth: x and dy are read once and dx is written. Each thread keeps its columns of dw and db over all
// rows of its block, the block stores one partial row of each, and a second kernel adds the partial rows in block
// order: no atomics, so the same inputs give the same bits.
//
//   layernorm_backward_kernel  rows of up to 16384 columns
//   layernorm_dx_long_kernel, layernorm_columns_kernel  longer rows: a block per row, which it reads twice; dw and db
//                              by columns
//   layernorm_reduce_kernel    the partial rows' sum
#include "layernorm.cuh"

namespace muon {
namespace {

constexpr int REDUCE_COLS = 32;
constexpr int REDUCE_WARPS = 16;

struct BackwardArgs {
  const void *dy, *x, *w;
  void *dx;
  long long lddy, ldx, lddx, N;
  const float *mean, *rstd;
  float *part;      // [2][parts][ldp]: dw's partial rows, then db's; null: neither is wanted
  long long parts, ldp;
  int wdt, wide, D;
};

// Threads of a multiprocessor, by the registers that they need (131072 x 201 bf16: 51 us with 512, and 84 us with 768,
// which spill).
constexpr int resident_threads(int C, Mode mode) { return C == 1 && mode != SHIFTED ? 768 : 512; }

// Rows as in the forward kernel: R at a time, W warps each, with the next rows on their way. A thread's columns of dw
// and db are in registers, or in shared memory for rows of more than 8192 columns (1024 threads have 64 registers
// each), which leaves no room for a ring: the next row waits in registers there, where it fits them. 32768 x 4096 bf16: 131
// us with the sum of the partial rows, 6.2 TB/s; fp32 246 us, 6.6 TB/s; but 8192 x 16384 bf16 248 us, 3.2 TB/s, since
// reading and writing the sums in shared memory takes longer than the row's own bytes.
template <typename XT, typename YT, int C, int W, int R, int MODE>
struct Backward {
  static constexpr int T = W * 32, THREADS = T * R;
  using CT = Cols<MODE, granule_of<XT, YT>(), T>;
  static constexpr bool IN_SHARED = W == 32, RING = MODE != SCALAR && !IN_SHARED;
  static constexpr bool AHEAD = !IN_SHARED || sizeof(XT) + sizeof(YT) == 4;
  static constexpr bool SHARED = RING && C > 1;
  using PT = Params<CT, C, SHARED>;
  static constexpr int STAGES = C * T * 8 * (sizeof(XT) + sizeof(YT)) <= 16384 ? 3 : 2;
  static constexpr int RING_X = RING ? STAGES * C * 8 * sizeof(XT) * THREADS : 0;   // bytes
  static constexpr int RING_DY = RING ? STAGES * C * 8 * sizeof(YT) * THREADS : 0;
  static constexpr size_t LOOP = static_cast<size_t>(RING_X) + RING_DY + PT::BYTES +
                                 (IN_SHARED ? 64 * C * THREADS : 0);
  static constexpr size_t BYTES = std::max<size_t>(LOOP, R > 1 ? 32 * C * THREADS : 0);   // the rows' sums at the end
  static constexpr int BLOCKS = std::max(1, resident_threads(C, static_cast<Mode>(MODE)) / THREADS);
};

template <typename XT, typename YT, int C, int W, int R, int MODE>
__global__ void __launch_bounds__(W *R * 32, (Backward<XT, YT, C, W, R, MODE>::BLOCKS))
    layernorm_backward_kernel(const BackwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  using B = Backward<XT, YT, C, W, R, MODE>;
  using CT = typename B::CT;
  constexpr int T = B::T, STAGES = B::STAGES, THREADS = B::THREADS;
  extern __shared__ __align__(16) unsigned char shared[];
  __shared__ float2 red[2][R][W];
  const int slot = R == 1 ? 0 : threadIdx.x / T, t = threadIdx.x - slot * T, D = a.D;
  const long long step = static_cast<long long>(gridDim.x) * R;
  long long row = first_row<R, MODE>(slot);
  const CT c(t, D, row * a.ldx);
  Exchange<W, R> exchange{red, slot, t / 32, 0};
  const Ring<XT, CT, C, THREADS> ring_x{shared + threadIdx.x * Raw<XT, CT::GE>::BYTES};
  const Ring<YT, CT, C, THREADS> ring_dy{shared + B::RING_X + threadIdx.x * Raw<YT, CT::GE>::BYTES};
  using PT = typename B::PT;
  float4 *kept = reinterpret_cast<float4 *>(shared + B::RING_X + B::RING_DY) + t;
  PT weight{a.w, a.wdt, a.wide != 0, 1.f, kept};
  Vals<8> aw[C], ab[C];
#pragma unroll
  for (int k = 0; k < C; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) aw[k].p[i] = ab[k].p[i] = make_float2(0.f, 0.f);
  // IN_SHARED: [4 chunk + half] of dw, [4 chunk + 2 + half] of db, of this thread
  auto sums_get = [&](int k) {
    if constexpr (B::IN_SHARED) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 u = kept[(4 * k + h) * THREADS], v = kept[(4 * k + 2 + h) * THREADS];
        aw[k].p[2 * h] = make_float2(u.x, u.y);
        aw[k].p[2 * h + 1] = make_float2(u.z, u.w);
        ab[k].p[2 * h] = make_float2(v.x, v.y);
        ab[k].p[2 * h + 1] = make_float2(v.z, v.w);
      }
    }
  };
  auto sums_put = [&](int k) {
    if constexpr (B::IN_SHARED) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float2 u = aw[k].p[2 * h], u1 = aw[k].p[2 * h + 1], v = ab[k].p[2 * h], v1 = ab[k].p[2 * h + 1];
        kept[(4 * k + h) * THREADS] = make_float4(u.x, u.y, u1.x, u1.y);
        kept[(4 * k + 2 + h) * THREADS] = make_float4(v.x, v.y, v1.x, v1.y);
      }
    }
  };
#pragma unroll
  for (int k = 0; k < C; ++k) sums_put(k);
  const float inv = 1.f / static_cast<float>(D);
  const long long x_step = step * a.ldx, dy_step = step * a.lddy, dx_step = step * a.lddx;
  const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;   // x and dy: the next row to fetch
  const YT *dy = static_cast<const YT *>(a.dy) + row * a.lddy;
  XT *dx = a.dx != nullptr ? static_cast<XT *>(a.dx) + row * a.lddx : nullptr;
  long long fetched = row;
  RawChunk<XT, CT::GE> rx[B::RING ? 1 : C];
  RawChunk<YT, CT::GE> rdy[B::RING ? 1 : C];
  auto fetch = [&](int stage) {
    if (fetched < a.N) {
      if constexpr (B::RING) {
        ring_x.fetch(x, c, stage);
        ring_dy.fetch(dy, c, stage);
      } else {
#pragma unroll
        for (int k = 0; k < C; ++k) {
          load_chunk(x, c, k, rx[k]);
          load_chunk(dy, c, k, rdy[k]);
        }
      }
    }
    if constexpr (B::RING) copy_async_commit();
    fetched += step;
    x += x_step;
    dy += dy_step;
  };
  const float w_extra = MODE == SHIFTED && c.extra >= 0 ? param_at(a.w, a.wdt, c.extra, 1.f) : 0.f;
  float aw_extra = 0.f, ab_extra = 0.f;
  const XT *x_row = x;
  const YT *dy_row = dy;
  float mean = 0.f, rstd = 0.f, x_next = 0.f, dy_next = 0.f;
  if (row < a.N) {
    mean = a.mean[row];
    rstd = a.rstd[row];
    x_next = load_extra(x_row, c);
    dy_next = load_extra(dy_row, c);
  }
  if constexpr (B::AHEAD) fetch(0);
  if constexpr (B::RING && STAGES == 3) fetch(1);
  weight.init(c, slot);
  if constexpr (B::SHARED && R > 1) __syncthreads();
  int stage = 0;
  for (; row - rows_apart<MODE> * slot < a.N; row += step) {   // the same count for the whole block
    const bool live = R == 1 || row < a.N;
    if constexpr (!B::AHEAD) fetch(0);
    const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
    const float x_extra = x_next, dy_extra = dy_next;
    x_row += x_step;
    dy_row += dy_step;
    if (row + step < a.N) {
      mean = a.mean[row + step];
      rstd = a.rstd[row + step];
      if (MODE == SHIFTED) {
        x_next = load_extra(x_row, c);
        dy_next = load_extra(dy_row, c);
      }
    }
    Vals<8> xh[C], g[C];
    if constexpr (B::RING) {
      copy_async_wait<STAGES - 2>();
#pragma unroll
      for (int k = 0; k < C; ++k) {
        xh[k] = ring_x.get(k, stage);
        g[k] = ring_dy.get(k, stage);
      }
      // the place of the row before this one, whose values are long used, takes the row STAGES - 1 ahead
      fetch(stage == 0 ? STAGES - 1 : stage - 1);
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) {
        xh[k] = rx[k].get();
        g[k] = rdy[k].get();
      }
      if constexpr (B::AHEAD) fetch(0);
    }
    float2 s1 = make_float2(0.f, 0.f), s2 = make_float2(0.f, 0.f);
    float xh_extra = 0.f, g_extra = 0.f;
    if (live) {
      if (MODE == SHIFTED && c.extra >= 0) {
        xh_extra = (x_extra + m2.x) * r2.x;
        aw_extra = fmaf(dy_extra, xh_extra, aw_extra);
        ab_extra += dy_extra;
        g_extra = dy_extra * w_extra;
        s1.x = g_extra;
        s2.x = g_extra * xh_extra;
      }
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const Vals<8> w = weight.get(c, k);
        sums_get(k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (!c.has(k, 2 * i / CT::GE)) continue;
          const float2 h = c.only(k, i, __fmul2_rn(__fadd2_rn(xh[k].p[i], m2), r2)), d = c.only(k, i, g[k].p[i]);
          xh[k].p[i] = h;
          aw[k].p[i] = __ffma2_rn(d, h, aw[k].p[i]);
          ab[k].p[i] = __fadd2_rn(ab[k].p[i], d);
          g[k].p[i] = __fmul2_rn(d, w.p[i]);
          s1 = __fadd2_rn(s1, g[k].p[i]);
          s2 = __ffma2_rn(g[k].p[i], h, s2);
        }
        sums_put(k);
      }
    }
    float2 sum = lanes_sum2<32>(make_float2(s1.x + s1.y, s2.x + s2.y));
    if constexpr (W > 1) sum = lanes_sum2<Exchange<W, R>::LANES>(exchange.put_get(sum.x, sum.y));
    if (a.dx != nullptr) {
      if (live) {
        const float2 c1 = make_float2(-sum.x * inv, -sum.x * inv), c2 = make_float2(-sum.y * inv, -sum.y * inv);
#pragma unroll
        for (int k = 0; k < C; ++k) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            g[k].p[i] = __fmul2_rn(__ffma2_rn(xh[k].p[i], c2, __fadd2_rn(g[k].p[i], c1)), r2);
          store_chunk(dx, c, k, g[k]);
        }
        if (MODE == SHIFTED && c.extra >= 0) store1(dx, c.extra, fmaf(xh_extra, c2.x, g_extra + c1.x) * r2.x);
      }
      dx += dx_step;
    }
  }
  if (a.part == nullptr) return;
  float *pw = a.part + static_cast<long long>(blockIdx.x) * a.ldp;
  float *pb = a.part + (a.parts + blockIdx.x) * a.ldp;
  if constexpr (R == 1) {
#pragma unroll
    for (int k = 0; k < C; ++k) {
      sums_get(k);
      store_sums(pw, c, k, aw[k]);
      store_sums(pb, c, k, ab[k]);
    }
    if (MODE == SHIFTED && c.extra >= 0) {
      pw[c.extra] = aw_extra;
      pb[c.extra] = ab_extra;
    }
  } else {   // the block's rows are added in order, where the ring was
    float *join = reinterpret_cast<float *>(shared);
    const int pitch = (D + 3) & ~3;
    if constexpr (B::RING) copy_async_wait<0>();
    for (int z = 0; z < 2; ++z) {
      __syncthreads();
#pragma unroll
      for (int k = 0; k < C; ++k) store_sums(join + slot * pitch, c, k, z == 0 ? aw[k] : ab[k]);
      if (MODE == SHIFTED && c.extra >= 0) join[slot * pitch + c.extra] = z == 0 ? aw_extra : ab_extra;
      __syncthreads();
      for (int j = threadIdx.x; j < D; j += THREADS) {
        float s = 0.f;
#pragma unroll
        for (int r = 0; r < R; ++r) s += join[r * pitch + j];
        (z == 0 ? pw : pb)[j] = s;
      }
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

// dw and db of long rows: block (b, z) sums 256 columns over row slice z, one column per thread. Reads x and dy again.
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

// dw (blockIdx.y = 0) and db (1): 32 columns per block, warp w adds partial rows w, w + 16, ... Bound by latency (7 us for
// the 10 MB of 304 partial rows of 4096 columns), which the rows are few for.
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
#pragma unroll 16
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

// Chunks per thread, warps per row and rows per block for D columns: a warp per row up to 768 columns, then as few
// warps as two or three chunks of eight columns per thread allow (the sums of dw and db take 16 registers for each). Two
// at most in SHIFTED, whose single columns take the registers of the third (65536 x 1501 bf16: 147 us, and 230 us with
// three).
struct Shape {
  int C, W, R;
};
Shape shape_of(long long D, Mode mode) {
  if (mode == SCALAR) return D <= 1024 ? Shape{1, 4, 2} : Shape{2, D <= 8192 ? 16 : 32, 1};
  if (D <= 256) return {1, 1, 8};
  if (D <= 512) return {2, 1, 8};
  if (D <= 768 && mode != SHIFTED) return {3, 1, 8};
  if (D <= 1024) return {2, 2, 4};
  if (D <= 1536 && mode != SHIFTED) return {3, 2, 4};
  for (int W : {4, 8, 16}) if (D <= 512 * W) return {2, W, 1};
  return {2, 32, 1};
}

// Blocks of the backward pass, each of which leaves one partial row of dw and db: as many as the registers of SMS
// multiprocessors hold at once, so that there are few partial rows to add. The count goes by the shape alone, since the
// workspace is sized by it; where that many rings do not fit the shared memory (fp32: one of two blocks fits at 513 to
// 768 columns and at 1025 to 1536 of whole granules, three of four up to 2048) the others are a second wave. In SHIFTED a
// block's rows lie multiples of eight apart.
constexpr long long SMS = 152;
long long parts_for(long long N, long long D, Mode mode) {
  if (D > MAX_ROW) return std::max(1LL, std::min(N, 64LL));
  const Shape h = shape_of(D, mode);
  const long long resident = std::max(1, resident_threads(h.C, mode) / (h.W * h.R * 32));
  const long long blocks = std::max(1LL, std::min((N + h.R - 1) / h.R, SMS * resident));
  return mode == SHIFTED ? (blocks + 7) / 8 * 8 : blocks;
}
long long part_pitch(long long D) { return (D + 7) / 8 * 8; }

template <typename XT, typename YT, int C, int W, int R, int MODE>
cudaError_t backward_launch(const BackwardArgs &a, cudaStream_t s) {
  using B = Backward<XT, YT, C, W, R, MODE>;
  auto kernel = layernorm_backward_kernel<XT, YT, C, W, R, MODE>;
  static AttributesSet set;
  const cudaError_t allowed = set.once([&] { return allow_shared(kernel); });
  if (allowed != cudaSuccess) return allowed;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(a.parts)), dim3(B::THREADS), B::BYTES, s, a);
}

template <typename XT, typename YT, int C, int W, int R, int MODE>
cudaError_t backward_shape(const BackwardArgs &a, cudaStream_t s) {
  if (MODE == ALIGNED && a.D == 256 * C * W) return backward_launch<XT, YT, C, W, R, FULL>(a, s);
  return backward_launch<XT, YT, C, W, R, MODE>(a, s);
}

template <typename XT, typename YT, int MODE>
cudaError_t backward_route_mode(const BackwardArgs &a, cudaStream_t s) {
  const Shape h = shape_of(a.D, static_cast<Mode>(MODE));
  if constexpr (MODE != SHIFTED)
    if (h.C == 3)
      return h.W == 1 ? backward_shape<XT, YT, 3, 1, 8, MODE>(a, s) : backward_shape<XT, YT, 3, 2, 4, MODE>(a, s);
  switch (h.W) {
    case 1: return h.C == 1 ? backward_shape<XT, YT, 1, 1, 8, MODE>(a, s) : backward_shape<XT, YT, 2, 1, 8, MODE>(a, s);
    case 2: return backward_shape<XT, YT, 2, 2, 4, MODE>(a, s);
    case 4: return backward_shape<XT, YT, 2, 4, 1, MODE>(a, s);
    case 8: return backward_shape<XT, YT, 2, 8, 1, MODE>(a, s);
    case 16: return backward_shape<XT, YT, 2, 16, 1, MODE>(a, s);
    default: return backward_shape<XT, YT, 2, 32, 1, MODE>(a, s);
  }
}

template <typename XT, typename YT>
cudaError_t backward_route(const BackwardArgs &a, Mode mode, cudaStream_t s) {
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
  if (mode == ALIGNED) return backward_route_mode<XT, YT, ALIGNED>(a, s);
  if (mode == SHIFTED) return backward_route_mode<XT, YT, SHIFTED>(a, s);
  switch (shape_of(a.D, mode).W) {
    case 4: return backward_launch<XT, YT, 1, 4, 2, SCALAR>(a, s);
    case 16: return backward_launch<XT, YT, 2, 16, 1, SCALAR>(a, s);
    default: return backward_launch<XT, YT, 2, 32, 1, SCALAR>(a, s);
  }
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

size_t layernorm_workspace_bytes(int64_t N, int64_t D) {
  if (N < 0 || D < 1) return 0;
  long long parts = 0;
  for (Mode mode : {SCALAR, ALIGNED, SHIFTED}) parts = std::max(parts, parts_for(N, D, mode));
  return align_up(static_cast<size_t>(8) * parts * part_pitch(D), 256);
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
  if (dx != nullptr && (!in_place_ok(dy, ydt, lddy, dx, xdt, lddx, N) || !in_place_ok(x, xdt, ldx, dx, xdt, lddx, N)))
    return MUON_ERR_INVALID_ARG;
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
  const Mode mode = mode_of(aligned16(dy) && aligned16(x) && aligned16(dx),
                            (ldx - lddy) % 8 == 0 && (dx == nullptr || (ldx - lddx) % 8 == 0), ldx, D);
  BackwardArgs a{dy, x, weight, dx, lddy, ldx, lddx, N, mean, rstd, sums ? static_cast<float *>(ws) : nullptr,
                 parts_for(N, D, mode), part_pitch(D), wdt, aligned16(weight) ? 1 : 0, static_cast<int>(D)};
  if (N == 0) a.parts = 0;
  if (N > 0) {
    launch_begin(KK_LN_BWD, s);
    cudaError_t e;
    if (xdt == MUON_F32)
      e = ydt == MUON_F32 ? backward_route<float, float>(a, mode, s) : backward_route<float, __nv_bfloat16>(a, mode, s);
    else
      e = ydt == MUON_F32 ? backward_route<__nv_bfloat16, float>(a, mode, s)
                          : backward_route<__nv_bfloat16, __nv_bfloat16>(a, mode, s);
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
