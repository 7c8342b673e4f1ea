// Layer norm over the rows of an N x D matrix, forward.
//
//   mu = mean(x), v = mean((x - mu)^2), r = 1 / sqrt(v + eps), y = (x - mu) r w + b
//
// Bound by bandwidth: a row is read once into registers (as fp32), its sums are exchanged between the warps that hold
// it, and the result is stored. The variance is taken around a mean, so no E[x^2] - mu^2 cancels.
//
//   layernorm_forward_kernel       rows of up to 16384 columns
//   layernorm_forward_long_kernel  longer rows: a block per row, re-reading it (from L2) for each sweep
#include "layernorm.cuh"

namespace muon {
namespace {

struct ForwardArgs {
  const void *x, *w, *b;
  void *y;
  long long ldx, ldy, N;
  float *mean, *rstd;
  float eps;
  int wdt, wide, D;
};

// R rows at a time, W warps each, with the next rows on their way. Mean and variance take one exchange: each warp sums
// its own columns and their squared distances from the warp's own mean, and
//   sum (x - mean)^2 = sum over warps of (own squares + n_w (mean_w - mean)^2).
// 65536 x 4096 bf16: 161 us, 6.7 TB/s; 65536 x 768: 35 us, 5.7 TB/s; 65536 x 1023: 49 us, 5.5 TB/s.
template <typename XT, typename YT, int C, int W, int R, int MODE>
struct Forward {
  static constexpr int T = W * 32, THREADS = T * R;
  using CT = Cols<MODE, granule_of<XT, YT>(), T>;
  static constexpr bool RING = MODE != SCALAR;
  static constexpr int STAGES = C * T * 8 * sizeof(XT) <= 16384 ? 3 : 2;
  static constexpr int ROWS = RING ? STAGES * C * 8 * sizeof(XT) * THREADS : 0;   // bytes of the ring
  static constexpr bool SHARED = RING && C > 1 && ROWS + 64 * C * T <= 200 * 1024;   // the weights, beside the ring
  using PT = Params<CT, C, SHARED>;
  static constexpr size_t BYTES = static_cast<size_t>(ROWS) + 2 * PT::BYTES;
  static constexpr int by_registers = C >= 3 ? 768 : 1024;   // threads
  static constexpr int BLOCKS = std::max(1, by_registers / THREADS);   // of a multiprocessor
};

template <typename XT, typename YT, int C, int W, int R, int MODE>
__global__ void __launch_bounds__(W *R * 32, (Forward<XT, YT, C, W, R, MODE>::BLOCKS))
    layernorm_forward_kernel(const ForwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  using F = Forward<XT, YT, C, W, R, MODE>;
  using CT = typename F::CT;
  constexpr int T = F::T, STAGES = F::STAGES;
  extern __shared__ __align__(16) unsigned char shared[];
  __shared__ float2 red[2][R][W];
  const int slot = R == 1 ? 0 : threadIdx.x / T, t = threadIdx.x - slot * T;
  const long long step = static_cast<long long>(gridDim.x) * R;
  long long row = first_row<R, MODE>(slot);
  const CT c(t, a.D, row * a.ldx);
  Exchange<W, R> exchange{red, slot, t / 32, 0};
  const Ring<XT, CT, C, F::THREADS> ring{shared + threadIdx.x * Raw<XT, CT::GE>::BYTES};
  using PT = typename F::PT;
  float4 *kept = reinterpret_cast<float4 *>(shared + F::ROWS) + t;
  PT weight{a.w, a.wdt, a.wide != 0, 1.f, kept}, bias{a.b, a.wdt, a.wide != 0, 0.f, kept + PT::BYTES / 16};
  const long long x_step = step * a.ldx, y_step = step * a.ldy;
  const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;   // the next row to fetch
  YT *y = static_cast<YT *>(a.y) + row * a.ldy;
  long long fetched = row;
  RawChunk<XT, CT::GE> raw[F::RING ? 1 : C];
  auto fetch = [&](int stage) {
    if (fetched < a.N) {
      if constexpr (F::RING) {
        ring.fetch(x, c, stage);
      } else {
#pragma unroll
        for (int k = 0; k < C; ++k) load_chunk(x, c, k, raw[k]);
      }
    }
    if constexpr (F::RING) copy_async_commit();
    fetched += step;
    x += x_step;
  };
  const float w_extra = MODE == SHIFTED && c.extra >= 0 ? param_at(a.w, a.wdt, c.extra, 1.f) : 0.f;
  const float b_extra = MODE == SHIFTED && c.extra >= 0 ? param_at(a.b, a.wdt, c.extra, 0.f) : 0.f;
  const XT *x_row = x;
  float x_next = row < a.N ? load_extra(x_row, c) : 0.f;
  fetch(0);
  if constexpr (F::RING && STAGES == 3) fetch(1);
  weight.init(c, slot);
  bias.init(c, slot);
  if constexpr (F::SHARED && R > 1) __syncthreads();
  const float inv = 1.f / static_cast<float>(a.D);
  // columns of this warp, and of the warp whose pair this lane reads in the exchange
  const float n_w = warp_sum(static_cast<float>(c.columns())), inv_n = n_w > 0.f ? 1.f / n_w : 0.f;
  float n_lane = n_w;
  if constexpr (W > 1) n_lane = exchange.put_get(n_w, 0.f).x;
  int stage = 0;
  for (; row - rows_apart<MODE> * slot < a.N; row += step) {   // the same count for the whole block
    const bool live = R == 1 || row < a.N;
    Vals<8> v[C];
    if constexpr (F::RING) {
      copy_async_wait<STAGES - 2>();
#pragma unroll
      for (int k = 0; k < C; ++k) v[k] = ring.get(k, stage);
      // the place of the row before this one, whose values are long used, takes the row STAGES - 1 ahead
      fetch(stage == 0 ? STAGES - 1 : stage - 1);
      stage = stage == STAGES - 1 ? 0 : stage + 1;
    } else {
#pragma unroll
      for (int k = 0; k < C; ++k) v[k] = raw[k].get();
      fetch(0);
    }
    const float x_extra = x_next;
    x_row += x_step;
    if (MODE == SHIFTED && row + step < a.N) x_next = load_extra(x_row, c);
    float2 s = make_float2(x_extra, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c.has(k, 2 * i / CT::GE)) s = __fadd2_rn(s, c.only(k, i, v[k].p[i]));
    const float own = warp_sum(s.x + s.y) * inv_n;
    const float d_extra = MODE == SHIFTED && c.extra >= 0 ? x_extra - own : 0.f;
    float2 q = make_float2(d_extra * d_extra, 0.f);
#pragma unroll
    for (int k = 0; k < C; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (c.has(k, 2 * i / CT::GE)) {
          const float2 d = c.only(k, i, __fadd2_rn(v[k].p[i], make_float2(-own, -own)));
          q = __ffma2_rn(d, d, q);
        }
    float sq = warp_sum(q.x + q.y), mean = own;
    if constexpr (W > 1) {
      const float2 r = exchange.put_get(own, sq);
      mean = lanes_sum<Exchange<W, R>::LANES>(n_lane * r.x) * inv;
      const float d = r.x - mean;
      sq = lanes_sum<Exchange<W, R>::LANES>(fmaf(n_lane * d, d, r.y));
    }
    const float rstd = rsqrtf(sq * inv + a.eps);   // within 2 units in the last place
    if (live) {
      if (t == 0) {
        if (a.mean != nullptr) a.mean[row] = mean;
        if (a.rstd != nullptr) a.rstd[row] = rstd;
      }
      const float2 m2 = make_float2(-mean, -mean), r2 = make_float2(rstd, rstd);
#pragma unroll
      for (int k = 0; k < C; ++k) {
        const Vals<8> w = weight.get(c, k), b = bias.get(c, k);
#pragma unroll
        for (int i = 0; i < 4; ++i)
          v[k].p[i] = __ffma2_rn(__fmul2_rn(__fadd2_rn(v[k].p[i], m2), r2), w.p[i], b.p[i]);
        store_chunk(y, c, k, v[k]);
      }
      if (MODE == SHIFTED && c.extra >= 0) store1(y, c.extra, fmaf((x_extra - mean) * rstd, w_extra, b_extra));
    }
    y += y_step;
  }
}

template <typename XT, typename YT>
__global__ void __launch_bounds__(LONG_THREADS) layernorm_forward_long_kernel(const ForwardArgs a) {
  pdl_wait();
  if (threadIdx.x == 0) pdl_launch_dependents();
  __shared__ float red[2][32];
  int turn = 0;
  const float inv = 1.f / static_cast<float>(a.D);
  for (long long row = blockIdx.x; row < a.N; row += gridDim.x) {
    const XT *x = static_cast<const XT *>(a.x) + row * a.ldx;
    YT *y = static_cast<YT *>(a.y) + row * a.ldy;
    float s = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) s += load1(x, c);
    const float mean = block_sum(s, red, turn) * inv;
    float q = 0.f;
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS) {
      const float d = load1(x, c) - mean;
      q = fmaf(d, d, q);
    }
    const float rstd = 1.f / sqrtf(block_sum(q, red, turn) * inv + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean != nullptr) a.mean[row] = mean;
      if (a.rstd != nullptr) a.rstd[row] = rstd;
    }
#pragma unroll 4
    for (int c = threadIdx.x; c < a.D; c += LONG_THREADS)
      store1(y, c, fmaf((load1(x, c) - mean) * rstd, param_at(a.w, a.wdt, c, 1.f), param_at(a.b, a.wdt, c, 0.f)));
  }
}

// ------------------------------------------------------------------------------------------ host

template <typename XT, typename YT, int C, int W, int R, int MODE>
cudaError_t forward_launch(const ForwardArgs &a, cudaStream_t s) {
  using F = Forward<XT, YT, C, W, R, MODE>;
  auto kernel = layernorm_forward_kernel<XT, YT, C, W, R, MODE>;
  static AttributesSet set;
  const cudaError_t allowed = set.once([&] { return allow_shared(kernel); });
  if (allowed != cudaSuccess) return allowed;
  const long long resident = std::max<long long>(1, std::min<long long>(F::BLOCKS, SM_SHARED / (F::BYTES + 2048)));
  long long blocks = std::min((a.N + R - 1) / R, device_sm_count() * resident);
  if (MODE == SHIFTED) blocks = (blocks + 7) / 8 * 8;   // a block's rows lie multiples of eight apart
  return launch_pdl(kernel, dim3(static_cast<unsigned>(blocks)), dim3(F::THREADS), F::BYTES, s, a);
}

template <typename XT, typename YT, int C, int W, int R, int MODE>
cudaError_t forward_shape(const ForwardArgs &a, cudaStream_t s) {
  if (MODE == ALIGNED && a.D == 256 * C * W) return forward_launch<XT, YT, C, W, R, FULL>(a, s);
  return forward_launch<XT, YT, C, W, R, MODE>(a, s);
}

// Rows of up to 1024 columns: a warp each, eight to a block, since the shuffles and the exchange of a row cost a thread
// the same whatever it holds (65536 x 768 bf16: 36 us, and 41 us with three warps to a row). Longer rows: two chunks of
// eight columns per thread, or three up to 12288 (65536 x 4096 bf16: 161 us with two, 164 to 195 us with four, which leave
// a multiprocessor half the warps beside the weights in shared memory; 8192 x 12000 bf16: 79 us with three chunks, 84 us
// with two and 32 warps, and 128 us with four and the weights from L2; 8192 x 16384: 95 us, and 131 us with four).
template <typename XT, typename YT, int MODE>
cudaError_t forward_route_mode(const ForwardArgs &a, cudaStream_t s) {
  const int D = a.D;
  if (D <= 256) return forward_shape<XT, YT, 1, 1, 8, MODE>(a, s);
  if (D <= 512) return forward_shape<XT, YT, 2, 1, 8, MODE>(a, s);
  if (D <= 768) return forward_shape<XT, YT, 3, 1, 8, MODE>(a, s);
  if (D <= 1024) return forward_shape<XT, YT, 4, 1, 8, MODE>(a, s);
  if (D <= 1536) return forward_shape<XT, YT, 3, 2, 4, MODE>(a, s);
  if (D <= 2048) return forward_shape<XT, YT, 2, 4, 1, MODE>(a, s);
  if (D <= 4096) return forward_shape<XT, YT, 2, 8, 1, MODE>(a, s);
  if (D <= 8192) return forward_shape<XT, YT, 2, 16, 1, MODE>(a, s);
  if (D <= 12288) return forward_shape<XT, YT, 3, 16, 1, MODE>(a, s);
  return forward_shape<XT, YT, 2, 32, 1, MODE>(a, s);
}

template <typename XT, typename YT>
cudaError_t forward_route(const ForwardArgs &a, Mode mode, cudaStream_t s) {
  if (a.D > MAX_ROW) {
    const dim3 grid(static_cast<unsigned>(std::min<long long>(a.N, device_sm_count() * 2))), block(LONG_THREADS);
    return launch_pdl(layernorm_forward_long_kernel<XT, YT>, grid, block, 0, s, a);
  }
  if (mode == ALIGNED) return forward_route_mode<XT, YT, ALIGNED>(a, s);
  if (mode == SHIFTED) return forward_route_mode<XT, YT, SHIFTED>(a, s);
  if (a.D <= 1024) return forward_launch<XT, YT, 1, 4, 2, SCALAR>(a, s);
  if (a.D <= 8192) return forward_launch<XT, YT, 2, 16, 1, SCALAR>(a, s);
  return forward_launch<XT, YT, 2, 32, 1, SCALAR>(a, s);
}

}  // namespace
}  // namespace muon

using namespace muon;

extern "C" {

muon_status layernorm_forward(const void *x, muon_dtype xdt, int64_t ldx, const void *weight, const void *bias,
                              muon_dtype wdt, void *y, muon_dtype ydt, int64_t ldy, float *mean, float *rstd, int64_t N,
                              int64_t D, float eps, muon_stream_t stream) {
  if (N > 0 && (x == nullptr || y == nullptr)) return MUON_ERR_INVALID_ARG;
  muon_status st = check_dims(N, D);
  if (st != MUON_OK) return st;
  if (ldx < D || ldy < D || !std::isfinite(eps) || eps < 0.f) return MUON_ERR_INVALID_ARG;
  if (!dtype_ok(xdt) || !dtype_ok(ydt) || !dtype_ok(wdt)) return MUON_ERR_DTYPE;
  if (!in_place_ok(x, xdt, ldx, y, ydt, ldy, N)) return MUON_ERR_INVALID_ARG;
  if (!natural(x, xdt) || !natural(y, ydt) || !natural(weight, wdt) || !natural(bias, wdt) ||
      !natural(mean, MUON_F32) || !natural(rstd, MUON_F32))
    return MUON_ERR_ALIGNMENT;
  if ((st = device_check()) != MUON_OK) return st;
  if (N == 0) return MUON_OK;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool wide = aligned16(weight) && aligned16(bias);
  const ForwardArgs a{x, weight, bias, y, ldx, ldy, N, mean, rstd, eps, wdt, wide ? 1 : 0, static_cast<int>(D)};
  const Mode mode = mode_of(aligned16(x) && aligned16(y), (ldx - ldy) % 8 == 0, ldx, D);
  launch_begin(KK_LN_FWD, s);
  cudaError_t e;
  if (xdt == MUON_F32)
    e = ydt == MUON_F32 ? forward_route<float, float>(a, mode, s) : forward_route<float, __nv_bfloat16>(a, mode, s);
  else
    e = ydt == MUON_F32 ? forward_route<__nv_bfloat16, float>(a, mode, s)
                        : forward_route<__nv_bfloat16, __nv_bfloat16>(a, mode, s);
  launch_end(s);
  return status_of(e);
}

}  // extern "C"
