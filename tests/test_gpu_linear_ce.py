"""linear_cross_entropy_* on the GPU against the fp64 oracle (oracle/operators.py).

Tolerances, element by element. A logit is an fp32 sum of bf16 products: off by at most 1e-5 of the sum of their magnitudes
(gpu_common). lse moves by at most as much as the logits do (a), plus the roundings of its own sum and logarithm (1e-5 and
2^-22 of its size); a loss by both. dz = g w (exp(z - lse) - [v = t]) then has an error of |g w| p (2 a + 2e-5), and one rounding
to bf16, 2^-8 of its size (two terms: 2^-16). dh and dw are sums of dz's errors times the other factor's magnitudes, 1e-5 of the
products' magnitudes for the fp32 sum, and a rounding of their own (2^-8 as bf16, 2^-23 as fp32 after an addition)."""
import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.gpu_common import DEV, build_lib, f64

pytestmark = pytest.mark.gpu
BF, F = torch.bfloat16, torch.float32
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    return build_lib()


def pitched(x, extra=0):
    """x on the device, rows on 16-byte boundaries; what lies between the rows is NaN."""
    rows, cols = x.shape
    buf = torch.full((rows, (cols + 7) // 8 * 8 + extra), NAN, dtype=x.dtype, device=DEV)
    buf[:, :cols] = x.to(DEV)
    return buf[:, :cols]


class Case:
    def __init__(self, N, V, D, seed=0, itype=torch.int64, weighted=True, padding=True, spread=1.0, extra=0):
        gen = torch.Generator().manual_seed(77 + seed)
        self.N, self.V, self.D = N, V, D
        self.h = pitched((torch.randn((N, D), generator=gen) * spread).to(BF), extra)
        self.w = pitched((torch.randn((V, D), generator=gen) * 1.5 / D ** 0.5).to(BF), extra)
        t = torch.randint(0, V, (N,), generator=gen)
        wt = torch.rand(N, generator=gen) + 0.25
        if padding and N > 3:
            t[::5] = -100
            t[2::7] = V
            wt[3::6] = 0.0
        self.t = t.to(itype).to(DEV)
        self.weights = wt.to(DEV) if weighted else None
        self.grad = (torch.rand(N, generator=gen) + 0.5).to(DEV)
        self.losses, self.lse = (torch.full((N,), NAN, device=DEV) for _ in range(2))

    def oracle(self, grad=None):
        return ops.linear_cross_entropy(f64(self.h), f64(self.w), self.t.cpu().numpy(),
                                        None if self.weights is None else f64(self.weights),
                                        None if grad is None else grad)

    def ws(self, L, terms):
        return torch.zeros(L.linear_cross_entropy_workspace_bytes(self.N, self.V, self.D, terms), dtype=torch.uint8,
                           device=DEV)


def outputs(c, hdt=BF, wdt=BF, extra=0):
    empty = lambda rows, dt: torch.full((rows, c.D + extra), NAN, dtype=dt, device=DEV)[:, :c.D]  # noqa: E731
    return empty(c.N, hdt), empty(c.V, wdt)


def scales(c, up):
    """Per row: |g w| where the row counts, and the logits' error bound."""
    t = c.t.cpu().numpy()
    wt = np.ones(c.N) if c.weights is None else f64(c.weights)
    live = (t >= 0) & (t < c.V) & (wt != 0)
    mag = np.abs(np.nan_to_num(f64(c.h))) @ np.abs(f64(c.w)).T
    return np.where(live, np.abs(wt * up), 0.0), 1e-5 * mag.max(1), live


def check_forward(c, ref):
    s, a, live = scales(c, 1.0)
    tol = a + 1e-5 + 2.0 ** -22 * np.abs(ref["lse"])
    assert np.all(np.abs(f64(c.lse) - ref["lse"]) <= np.where(live, tol, 0.0))
    assert np.all(np.abs(f64(c.losses) - ref["losses"]) <= s * (2 * tol + 2.0 ** -22 * np.abs(ref["lse"])))


def check_gradients(c, ref, up, dh, dw, terms, old=None):
    s, a, live = scales(c, up)
    p = np.where(live[:, None], np.exp(ref["logits"] - ref["lse"][:, None]), 0.0)
    err = s[:, None] * p * (2 * a + 2e-5)[:, None] + np.abs(ref["dz"]) * (2.0 ** -8 if terms == 1 else 2.0 ** -16)
    H, W = np.abs(np.where(live[:, None], f64(c.h), 0.0)), np.abs(f64(c.w))
    Z = np.abs(ref["dz"])
    for got, want, tol in ((dh, ref["dh"], err @ W + 1e-5 * (Z @ W)), (dw, ref["dw"], err.T @ H + 1e-5 * (Z.T @ H))):
        if got is None:
            continue
        if old is not None and got is dw:
            want = want + old
        own = 2.0 ** -8 if got.dtype == BF else 2.0 ** -23
        assert np.all(np.abs(f64(got) - want) <= tol * (1 + own) + own * np.abs(want) + 1e-38)


SIZES = [(1, 1, 1), (1, 5, 7), (2, 64, 8), (31, 63, 64), (33, 127, 65), (127, 129, 63), (128, 256, 64), (129, 255, 130),
         (256, 257, 128), (300, 1000, 72), (520, 2051, 200), (5, 30011, 96), (64, 513, 1030)]


@pytest.mark.parametrize("N,V,D", SIZES)
def test_forward(L, N, V, D):
    c = Case(N, V, D, seed=N)
    ws = c.ws(L, 0)
    L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
    torch.cuda.synchronize()
    assert L.muon_check(ws) == L.MUON_OK
    check_forward(c, c.oracle())


@pytest.mark.parametrize("N,V,D", SIZES)
@pytest.mark.parametrize("hdt,wdt", [(BF, BF), (F, F), (BF, F)])
def test_backward(L, N, V, D, hdt, wdt):
    c = Case(N, V, D, seed=N + 1)
    up = f64(c.grad)
    ref = c.oracle(up)
    c.lse.copy_(torch.from_numpy(ref["lse"]).float())
    dh, dw = outputs(c, hdt, wdt)
    terms = 2 if F in (hdt, wdt) else 1
    ws = c.ws(L, terms)
    L.linear_cross_entropy_backward(c.h, c.w, c.t, c.weights, c.lse, c.grad, dh, dw, ws)
    torch.cuda.synchronize()
    assert L.muon_check(ws) == L.MUON_OK
    check_gradients(c, ref, up, dh, dw, terms)


@pytest.mark.parametrize("N,V,D", [(1, 3, 8), (37, 300, 64), (300, 1000, 72), (130, 700, 264)])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
@pytest.mark.parametrize("weighted", [True, False])
def test_both_in_one_call(L, N, V, D, itype, weighted):
    """Against the oracle, and against the two calls."""
    c = Case(N, V, D, seed=N + 2, itype=itype, weighted=weighted)
    ref = c.oracle(np.full(N, 0.125))
    dh, dw = outputs(c)
    ws = c.ws(L, 1)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 0.125, c.losses, c.lse, dh, dw, ws)
    torch.cuda.synchronize()
    assert L.muon_check(ws) == L.MUON_OK
    check_forward(c, ref)
    check_gradients(c, ref, 0.125, dh, dw, 1)
    losses, lse = c.losses.clone(), c.lse.clone()
    L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
    assert torch.equal(losses, c.losses) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("N", [256, 257, 700, 1024])
@pytest.mark.parametrize("dts", [(BF, BF), (F, F)])
def test_pieces(L, N, dts):
    """Pieces of 256 rows: dw adds up over them in fp32, and is rounded once."""
    c = Case(N, 901, 136, seed=N)
    ref = c.oracle(np.full(N, 2.0))
    dh, dw = outputs(c, *dts)
    terms = 2 if F in dts else 1
    try:
        L.muon_debug_loss_rows(256)
        ws = c.ws(L, terms)
        L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 2.0, c.losses, c.lse, dh, dw, ws)
        torch.cuda.synchronize()
        check_forward(c, ref)
        check_gradients(c, ref, 2.0, dh, dw, terms)
        old = f64(dw)
        L.linear_cross_entropy_backward(c.h, c.w, c.t, c.weights, c.lse, None, None, dw, ws, accumulate=True)
        torch.cuda.synchronize()
        check_gradients(c, c.oracle(), 1.0, None, dw, terms, old)
    finally:
        L.muon_debug_loss_rows(0)


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("N,V", [(70, 400), (4, 20011)])
def test_accumulate(L, dt, N, V):
    c = Case(N, V, 64, seed=3)
    dh, dw = outputs(c, dt, dt)
    dw.copy_(torch.randn(dw.shape, generator=torch.Generator().manual_seed(1)))
    old = f64(dw)
    terms = 2 if dt == F else 1
    c.lse.copy_(torch.from_numpy(c.oracle()["lse"]).float())
    L.linear_cross_entropy_backward(c.h, c.w, c.t, c.weights, c.lse, None, dh, dw, c.ws(L, terms), accumulate=True)
    torch.cuda.synchronize()
    check_gradients(c, c.oracle(), 1.0, dh, dw, terms, old)


def test_long_contractions_are_cut(L):
    """Few tiles and a long vocabulary (dh), or many rows and a short one (dw): sums of slices, the same bits every time."""
    for N, V, D in ((40, 50001, 64), (3000, 60, 72)):
        c = Case(N, V, D, seed=V)
        ref = c.oracle()
        runs = []
        for _ in range(2):
            dh, dw = outputs(c)
            ws = c.ws(L, 1)
            L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, ws)
            torch.cuda.synchronize()
            runs.append((dh, dw, c.losses.clone()))
        check_forward(c, ref)
        check_gradients(c, ref, 1.0, dh, dw, 1)
        for x, y in zip(*runs):
            assert torch.equal(x, y)


def test_padding_may_hold_anything(L):
    """Rows without a part in the loss: NaN in h, and no trace of them."""
    c = Case(200, 333, 80, seed=5)
    _, _, live = scales(c, 1.0)
    dead = torch.from_numpy(~live).to(DEV)
    assert dead.any() and not dead.all()
    c.h[dead] = NAN
    ref = c.oracle()
    dh, dw = outputs(c)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, c.ws(L, 1))
    torch.cuda.synchronize()
    check_forward(c, ref)
    check_gradients(c, ref, 1.0, dh, dw, 1)
    assert not dh[dead].any() and not c.losses[dead].any() and not c.lse[dead].any()


def test_no_row_counts(L):
    c = Case(70, 300, 64, seed=6)
    c.t.fill_(-1)
    dh, dw = outputs(c)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, c.ws(L, 1))
    torch.cuda.synchronize()
    for x in (c.losses, c.lse, dh, dw):
        assert not x.any()


def test_no_rows(L):
    w = torch.randn((30, 16), device=DEV).to(BF)
    h = torch.empty((0, 16), dtype=BF, device=DEV)
    t = torch.empty(0, dtype=torch.int64, device=DEV)
    e = torch.empty(0, device=DEV)
    for dt in (BF, F):
        dw = torch.full((30, 16), NAN, dtype=dt, device=DEV)
        ws = torch.zeros(L.linear_cross_entropy_workspace_bytes(0, 30, 16, 2), dtype=torch.uint8, device=DEV)
        L.linear_cross_entropy_forward(h, w, t, None, e, e, ws)
        L.linear_cross_entropy_forward_backward(h, w, t, None, 1.0, e, e, torch.empty((0, 16), dtype=dt, device=DEV), dw,
                                                ws)
        assert not dw.any()
        dw.fill_(3.0)
        L.linear_cross_entropy_backward(h, w, t, None, e, None, None, dw, ws, accumulate=True)
        assert (dw == 3.0).all()


@pytest.mark.parametrize("shift", [30.0, 300.0])
def test_large_logits(L, shift):
    """Logits far beyond what exp can take, the target far below the largest, and one far above all others."""
    c = Case(60, 500, 64, seed=8, spread=shift)
    ref = c.oracle()
    dh, dw = outputs(c)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, c.ws(L, 1))
    torch.cuda.synchronize()
    check_forward(c, ref)
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("extra,off", [(0, 1), (3, 0), (5, 3), (8, 8)])
def test_outputs_of_any_pitch_and_place(L, dt, extra, off):
    """Only the gradients' elements are written."""
    c = Case(150, 270, 76, seed=9, extra=8)
    bufs, views = [], []
    for rows in (c.N, c.V):
        b = torch.full((rows * (c.D + extra) + 64,), 7.0, dtype=dt, device=DEV)
        bufs.append(b)
        views.append(b[off:off + rows * (c.D + extra)].view(rows, c.D + extra)[:, :c.D])
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, *views,
                                            c.ws(L, 2 if dt == F else 1))
    torch.cuda.synchronize()
    check_gradients(c, c.oracle(), 1.0, *views, 2 if dt == F else 1)
    for b, v in zip(bufs, views):
        v.fill_(7.0)
        assert (b == 7.0).all()


@pytest.mark.parametrize("dt", [BF, F])
@pytest.mark.parametrize("N,V", [(6, 29), (150, 270), (3, 20011)])
@pytest.mark.parametrize("D,pitch", [(1, 8), (3, 8), (5, 8), (8, 16), (9, 16), (77, 80), (76, 88), (259, 264)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_what_lies_between_aligned_rows_stays(L, dt, N, V, D, pitch, accumulate):
    """Rows on 16-byte boundaries whose width is no multiple of 16 bytes: their padding belongs to the caller."""
    c = Case(N, V, D, seed=D)
    bufs = [torch.full((rows, pitch), 7.0, dtype=dt, device=DEV) for rows in (N, V)]
    dh, dw = (b[:, :D] for b in bufs)
    terms = 2 if dt == F else 1
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, c.ws(L, terms),
                                            accumulate=accumulate)
    torch.cuda.synchronize()
    check_gradients(c, c.oracle(), 1.0, dh, dw, terms, np.full((V, D), 7.0) if accumulate else None)
    for b in bufs:
        b[:, :D] = 7.0
        assert (b == 7.0).all()


@pytest.mark.parametrize("N", [40, 300])
@pytest.mark.parametrize("below", [8.0, 16.0])
def test_joint_gradient_of_a_column_that_no_row_gives_much(L, N, below):
    """Column 7's logits lie about `below` under the others', whose largest is near 3: for 16 its exponentials are 2^-26.4 to
    2^-30.5 of the largest beside them. h is positive, so nothing cancels in its gradient. Three roundings of at most half a
    step: the exponential's, whose last bit is 2^-37, so 2^-7.5 of the smallest; dz's and the output's in bf16. And 2^-12 for
    the logits."""
    V, D = 500, 512
    g = torch.Generator().manual_seed(N)
    h = (torch.rand((N, D), generator=g) + 0.5).to(DEV, BF)
    w = (torch.randn((V, D), generator=g) * 0.05).to(DEV, BF)
    w[7] = -below / D
    t = torch.randint(8, V, (N,), generator=g).to(DEV)
    losses, lse = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    ws = torch.zeros(L.linear_cross_entropy_workspace_bytes(N, V, D, 1), dtype=torch.uint8, device=DEV)
    L.linear_cross_entropy_forward_backward(h, w, t, None, 1.0, losses, lse, dh, dw, ws)
    p = torch.softmax(h.double() @ w.double().t(), 1)[:, 7]
    want = p @ h.double()
    err = ((dw[7].double() - want) / want).abs().max().item()
    assert p.max().item() < 1e-3 and err <= 2.0 ** -7.5 + 2 * 2.0 ** -8 + 2.0 ** -12


def test_the_shared_factor_is_no_part_of_the_roundings_of_dz(L):
    """Where no contraction is cut, fp32 gradients are their sum times grad_scale, rounded once."""
    c = Case(300, 200, 70, weighted=False)
    got = []
    for scale in (1.0, 1 / 300):
        dh, dw = (torch.full((rows, 70), 9.0, device=DEV) for rows in (300, 200))
        L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, None, scale, c.losses, c.lse, dh, dw, c.ws(L, 2))
        got.append((dh, dw))
    factor = torch.tensor(1 / 300, device=DEV)
    for whole, part in zip(*got):
        assert torch.equal(part, whole * factor)


def test_one_gradient_of_the_two(L):
    c = Case(90, 411, 64, seed=10)
    ref = c.oracle()
    ws = c.ws(L, 1)
    dh, dw = outputs(c)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, None, ws)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, None, dw, ws)
    torch.cuda.synchronize()
    check_gradients(c, ref, 1.0, dh, dw, 1)


def test_against_differences(L):
    """The loss along a direction, in fp32 by the forward pass, against the gradients' product with it."""
    c = Case(120, 600, 96, seed=11)
    dh, dw = outputs(c, F, F)
    ws = c.ws(L, 2)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, ws)
    gen = torch.Generator().manual_seed(2)
    for x, g in ((c.h, dh), (c.w, dw)):
        d = torch.sign(torch.randn(x.shape, generator=gen)).to(DEV) * 2.0 ** -6
        keep, total, moved = x.clone(), [], []
        for s in (1.0, -1.0):
            x.copy_((keep.float() + s * d).to(BF))
            moved.append(x.float() - keep.float())
            L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
            total.append(c.losses.double().sum().item())
        x.copy_(keep)
        # (f(x + a) - f(x + b)) = g (a - b) + second order; a and b differ from +-d by bf16's rounding alone
        want = (g.double() * (moved[0] - moved[1]).double()).sum().item()
        size = (g.double() * (moved[0] - moved[1]).double()).abs().sum().item()
        assert abs(total[0] - total[1] - want) <= 2e-2 * size


def test_another_stream_and_a_captured_call(L):
    c = Case(260, 700, 128, seed=12)
    want = outputs(c)
    ws = c.ws(L, 1)
    args = lambda dh, dw: (c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, ws)  # noqa: E731
    L.linear_cross_entropy_forward_backward(*args(*want))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = outputs(c)
    L.linear_cross_entropy_forward_backward(*args(*got), stream=s)
    s.synchronize()
    for x, y in zip(want, got):
        assert torch.equal(x, y)
    got = outputs(c)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        L.linear_cross_entropy_forward_backward(*args(*got))
    for _ in range(2):
        for x in got:
            x.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, got):
            assert torch.equal(x, y)
    assert L.muon_check(ws) == L.MUON_OK


def test_wide_rows(L):
    """Tiles in groups of rows: more row tiles than a group takes, and a last group that is not full."""
    c = Case(4700, 700, 40, seed=13)
    ref = c.oracle()
    dh, dw = outputs(c)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, c.ws(L, 1))
    torch.cuda.synchronize()
    check_forward(c, ref)
    check_gradients(c, ref, 1.0, dh, dw, 1)


def test_two_streams_at_once(L):
    """Calls with workspaces of their own, in flight together."""
    cases = [Case(300, 3001, 96, seed=20), Case(90, 2500, 128, seed=21)]
    want, got, spaces = [], [], []
    for c in cases:
        spaces.append(c.ws(L, 1))
        want.append(outputs(c))
        L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, *want[-1], spaces[-1])
        got.append(outputs(c))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        for c, s, g, ws in zip(cases, streams, got, spaces):
            L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, *g, ws, stream=s)
    torch.cuda.synchronize()
    for w, g, ws in zip(want, got, spaces):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1]) and L.muon_check(ws) == L.MUON_OK


@pytest.mark.parametrize("N", [2047, 2048, 2305, 2600, 4100])
def test_halves(L, N):
    """From 2048 rows on the joint call goes by halves, the second of them short or left out; the losses are those of the
    forward call, bit for bit."""
    c = Case(N, 1030, 72, seed=N)
    ref = c.oracle(np.full(N, 0.5))
    dh, dw = outputs(c)
    ws = c.ws(L, 1)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 0.5, c.losses, c.lse, dh, dw, ws)
    torch.cuda.synchronize()
    check_forward(c, ref)
    check_gradients(c, ref, 0.5, dh, dw, 1)
    losses = c.losses.clone()
    L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
    assert torch.equal(losses, c.losses)
    alone = outputs(c)[1]
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 0.5, c.losses, c.lse, None, alone, ws)
    assert torch.equal(alone, dw)


@pytest.mark.parametrize("N", [1, 7, 8, 9, 64, 127, 128, 129])
@pytest.mark.parametrize("V,D", [(3, 200), (64, 64), (65, 72), (5003, 40)])
def test_few_rows(L, N, V, D):
    """A CTA alone, whose stages hold only the rows that there are, and the first size of the other kind."""
    c = Case(N, V, D, seed=N + V)
    ref = c.oracle(f64(c.grad))
    c.lse.copy_(torch.from_numpy(ref["lse"]).float())
    for dt in (BF, F):
        terms = 2 if dt == F else 1
        ws = c.ws(L, terms)
        dh, dw = outputs(c, dt, dt)
        L.linear_cross_entropy_backward(c.h, c.w, c.t, c.weights, c.lse, c.grad, dh, dw, ws)
        torch.cuda.synchronize()
        check_gradients(c, ref, f64(c.grad), dh, dw, terms)
    dh, dw = outputs(c)
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, dh, dw, ws)
    torch.cuda.synchronize()
    ref = c.oracle()
    check_forward(c, ref)
    check_gradients(c, ref, 1.0, dh, dw, 1)


def test_another_device_is_refused(L):
    c = Case(20, 30, 16, seed=1)
    with pytest.raises(ValueError):
        L.linear_cross_entropy_forward(c.h, c.w.cpu(), c.t, c.weights, c.losses, c.lse, c.ws(L, 0))
