"""linear_cross_entropy_forward_backward from a width of 512 on with bf16 gradients, where it keeps the exponentials instead of
computing the logits twice, against the fp64 oracle (oracle/operators.py).

Tolerances are those of test_gpu_linear_ce.py, and what keeping an exponential in fp16 times 2^13 adds to it: relative 2^-11 (half
a step of fp16), and half of its last bit below 2^-27 of its part's largest, 2^-38 of that, which is at most the row's largest."""
import numpy as np
import pytest
import torch

from tests.gpu_common import DEV, build_lib, f64
from tests.test_gpu_linear_ce import BF, NAN, Case, check_forward, outputs, scales

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return build_lib()


def joint(L, c, scale, dh, dw, ws, **kw):
    L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, scale, c.losses, c.lse, dh, dw, ws, **kw)
    torch.cuda.synchronize()
    assert L.muon_check(ws) == L.MUON_OK


def check_kept(c, ref, scale, dh, dw, old=None):
    """ref: the oracle's with a gradient of 1 for each row's loss."""
    s, a, live = scales(c, 1.0)
    p = np.where(live[:, None], np.exp(ref["logits"] - ref["lse"][:, None]), 0.0)
    kept = p * 2.0 ** -11 + p.max(1, keepdims=True) * 2.0 ** -38
    err = s[:, None] * (p * (2 * a + 2e-5)[:, None] + kept)
    Z = np.abs(ref["dz"])
    err = err + 2.0 ** -8 * (Z + err)
    H, W = np.abs(np.where(live[:, None], f64(c.h), 0.0)), np.abs(f64(c.w))
    for got, want, tol in ((dh, ref["dh"], err @ W + 1e-5 * (Z @ W)), (dw, ref["dw"], err.T @ H + 1e-5 * (Z.T @ H))):
        if got is None:
            continue
        want, tol = scale * want, abs(scale) * tol
        if old is not None and got is dw:
            want = want + old
        assert np.all(np.abs(f64(got) - want) <= tol * (1 + 2.0 ** -8) + 2.0 ** -8 * np.abs(want) + 1e-38)


SIZES = [(1, 1, 512), (2, 5, 513), (33, 131, 520), (128, 64, 512), (129, 257, 515), (300, 1000, 768), (520, 2049, 512),
         (7, 30011, 512)]


@pytest.mark.parametrize("N,V,D", SIZES)
@pytest.mark.parametrize("itype,weighted,scale", [(torch.int64, True, 0.37), (torch.int32, False, 1.0)])
def test_against_the_oracle(L, N, V, D, itype, weighted, scale):
    """Rows that have no part in the loss hold NaN. The losses are the forward call's, bit for bit."""
    c = Case(N, V, D, seed=N + 31, itype=itype, weighted=weighted)
    _, _, live = scales(c, 1.0)
    c.h[torch.from_numpy(~live).to(DEV)] = NAN
    ref = c.oracle()
    ws = c.ws(L, 1)
    dh, dw = outputs(c)
    joint(L, c, scale, dh, dw, ws)
    check_forward(c, ref)
    check_kept(c, ref, scale, dh, dw)
    dead = torch.from_numpy(~live).to(DEV)
    assert not dh[dead].any() and not c.losses[dead].any() and not c.lse[dead].any()
    losses, lse = c.losses.clone(), c.lse.clone()
    L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
    assert torch.equal(losses, c.losses) and torch.equal(lse, c.lse)


@pytest.mark.parametrize("N", [2047, 2048, 2305, 2560, 2600, 4100])
@pytest.mark.parametrize("V,D", [(1030, 512), (901, 520)])
def test_by_halves(L, N, V, D):
    """From 2048 rows on by halves, one's exponentials becoming dz beside the other's products; the second half may be short,
    or too short to go alone. Without dh everything goes whole: the same dw. What the workspace held changes no bit."""
    c = Case(N, V, D, seed=N)
    _, _, live = scales(c, 1.0)
    c.h[torch.from_numpy(~live).to(DEV)] = NAN
    ref = c.oracle()
    ws = c.ws(L, 1)
    dh, dw = outputs(c)
    joint(L, c, 0.5, dh, dw, ws)
    check_forward(c, ref)
    check_kept(c, ref, 0.5, dh, dw)
    losses, lse = c.losses.clone(), c.lse.clone()
    L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
    assert torch.equal(losses, c.losses) and torch.equal(lse, c.lse)
    for byte in (255, 127):
        ws[256:] = byte
        again = outputs(c)
        joint(L, c, 0.5, *again, ws)
        assert torch.equal(again[0], dh) and torch.equal(again[1], dw) and torch.equal(losses, c.losses)
    alone = outputs(c)
    joint(L, c, 0.5, None, alone[1], ws)
    assert torch.equal(alone[1], dw)
    joint(L, c, 0.5, alone[0], None, ws)
    assert torch.equal(alone[0], dh)


@pytest.mark.parametrize("rows,N", [(256, 256), (256, 257), (256, 700), (2304, 5000), (2304, 4700)])
def test_pieces(L, rows, N):
    """dw adds up over the pieces in fp32 and is rounded once; pieces of 2304 rows go by halves, a last one of few rows whole."""
    c = Case(N, 500, 520, seed=N)
    ref = c.oracle()
    try:
        L.muon_debug_loss_rows(rows)
        ws = c.ws(L, 1)
        dh, dw = outputs(c)
        joint(L, c, 2.0, dh, dw, ws)
        check_forward(c, ref)
        check_kept(c, ref, 2.0, dh, dw)
        old = f64(dw)
        joint(L, c, -1.0, dh, dw, ws, accumulate=True)
        check_kept(c, ref, -1.0, dh, dw, old)
    finally:
        L.muon_debug_loss_rows(0)


@pytest.mark.parametrize("N,V", [(70, 400), (2100, 300), (4, 20011)])
def test_accumulate(L, N, V):
    c = Case(N, V, 512, seed=3)
    dh, dw = outputs(c)
    dw.copy_(torch.randn(dw.shape, generator=torch.Generator().manual_seed(1)))
    old = f64(dw)
    joint(L, c, 1.0, dh, dw, c.ws(L, 1), accumulate=True)
    check_kept(c, c.oracle(), 1.0, dh, dw, old)


@pytest.mark.parametrize("N", [40, 300, 2500])
def test_no_row_counts(L, N):
    c = Case(N, 300, 512, seed=6)
    c.t.fill_(-1)
    c.h.fill_(NAN)
    dh, dw = outputs(c)
    joint(L, c, 1.0, dh, dw, c.ws(L, 1))
    for x in (c.losses, c.lse, dh, dw):
        assert not x.any()


@pytest.mark.parametrize("N", [60, 2100])
def test_large_logits(L, N):
    """Logits far beyond what exp can take. Where a row's largest logit, of about 1000, leads by 60 and is not the target's, dz is 1
    there and -1 at the target: the probability is off by the roundings of two arguments of exp2, 2^-13 each, and so rounds to
    1 in bf16. dh is then the difference of two of w's rows, exact but for its own rounding and an fp32 sum."""
    c = Case(N, 500, 512, seed=8, spread=300.0, weighted=False)
    ref = c.oracle()
    dh, dw = outputs(c)
    joint(L, c, 1.0, dh, dw, c.ws(L, 1))
    check_forward(c, ref)
    assert torch.isfinite(dh).all() and torch.isfinite(dw).all()
    _, a, live = scales(c, 1.0)
    top2 = np.sort(ref["logits"], 1)[:, -2:]
    sure = live & (top2[:, 1] - top2[:, 0] > 60 + 2 * a) & (ref["logits"].argmax(1) != c.t.cpu().numpy())
    assert sure.sum() > N // 4
    want = ref["dh"][sure]
    assert np.all(np.abs(f64(dh)[sure] - want) <= 2.0 ** -8 * np.abs(want) + 1e-5 * 2 * np.abs(f64(c.w)).max())


@pytest.mark.parametrize("N,V,D,pitch", [(33, 270, 515, 520), (300, 401, 516, 528), (2100, 300, 517, 520), (2100, 300, 512, 528)])
def test_what_lies_between_rows_stays(L, N, V, D, pitch):
    c = Case(N, V, D, seed=D)
    bufs = [torch.full((rows, pitch), 7.0, dtype=BF, device=DEV) for rows in (N, V)]
    dh, dw = (b[:, :D] for b in bufs)
    joint(L, c, 1.0, dh, dw, c.ws(L, 1))
    check_kept(c, c.oracle(), 1.0, dh, dw)
    for b in bufs:
        b[:, :D] = 7.0
        assert (b == 7.0).all()


def test_streams_and_a_captured_call(L):
    """Two calls at once with workspaces of their own, and a captured one replayed."""
    cases = [Case(2300, 901, 520, seed=20), Case(90, 2500, 512, seed=21)]
    want, spaces = [], []
    for c in cases:
        spaces.append(c.ws(L, 1))
        want.append(outputs(c))
        joint(L, c, 1.0, *want[-1], spaces[-1])
    streams = [torch.cuda.Stream() for _ in cases]
    got = [outputs(c) for c in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s, g, ws in zip(cases, streams, got, spaces):
            L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, *g, ws, stream=s)
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert torch.equal(w[0], g[0]) and torch.equal(w[1], g[1])
    c, ws = cases[0], spaces[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        L.linear_cross_entropy_forward_backward(c.h, c.w, c.t, c.weights, 1.0, c.losses, c.lse, *got[0], ws)
    for _ in range(2):
        for x in got[0]:
            x.fill_(NAN)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0][0], got[0][0]) and torch.equal(want[0][1], got[0][1])
    assert L.muon_check(ws) == L.MUON_OK


@pytest.mark.parametrize("N,V,D,rows", [(5, 3001, 40, 0), (300, 901, 136, 0), (700, 500, 72, 256), (40, 20011, 64, 0)])
@pytest.mark.parametrize("dt", [BF, torch.float32])
def test_what_the_workspace_held_changes_no_bit(L, N, V, D, rows, dt):
    """Of the other forms: only the control block has to be zero."""
    c = Case(N, V, D, seed=N)
    terms = 1 if dt == BF else 2
    try:
        L.muon_debug_loss_rows(rows)
        ws = c.ws(L, terms)
        want = None
        for byte in (0, 255, 127):
            ws[256:] = byte
            got = [*outputs(c, dt, dt), *outputs(c, dt, dt)]
            joint(L, c, 0.5, *got[:2], ws)
            ws[256:] = byte
            L.linear_cross_entropy_backward(c.h, c.w, c.t, c.weights, c.lse, c.grad, *got[2:], ws)
            got += [c.losses.clone(), c.lse.clone()]
            ws[256:] = byte
            L.linear_cross_entropy_forward(c.h, c.w, c.t, c.weights, c.losses, c.lse, ws)
            torch.cuda.synchronize()
            assert torch.equal(got[-2], c.losses) and torch.equal(got[-1], c.lse)
            want = want or got
            for x, y in zip(want, got):
                assert torch.equal(x, y)
    finally:
        L.muon_debug_loss_rows(0)


@pytest.mark.parametrize("N", [40, 300])
def test_a_column_too_far_below_the_others(L, N):
    """Column 7's logits lie 30 or so under the others' largest: its exponentials are below 2^-38 of that, zero where they are
    kept, and computed again by the backward call. h is positive, so nothing cancels: two roundings to bf16, and 2^-12 for the
    logits."""
    V, D = 500, 512
    g = torch.Generator().manual_seed(N)
    h = (torch.rand((N, D), generator=g) + 0.5).to(DEV, BF)
    w = (torch.randn((V, D), generator=g) * 0.05).to(DEV, BF)
    w[7] = -30.0 / D
    t = torch.randint(8, V, (N,), generator=g).to(DEV)
    losses, lse = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    ws = torch.zeros(L.linear_cross_entropy_workspace_bytes(N, V, D, 1), dtype=torch.uint8, device=DEV)
    kept, again = torch.empty_like(w), torch.empty_like(w)
    L.linear_cross_entropy_forward_backward(h, w, t, None, 1.0, losses, lse, None, kept, ws)
    L.linear_cross_entropy_backward(h, w, t, None, lse, None, None, again, ws)
    z = h.double() @ w.double().t()
    assert (z[:, 7] - z[:, :64].max(1).values).max().item() < -38 * np.log(2.0)
    want = torch.softmax(z, 1)[:, 7] @ h.double()
    assert not kept[7].any()
    assert ((again[7].double() - want) / want).abs().max().item() <= 2 * 2.0 ** -8 + 2.0 ** -12
