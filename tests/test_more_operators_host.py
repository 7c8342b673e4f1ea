"""The linear head's cross entropy and AdamW with 8-bit moments without a GPU: the oracle's gradients against differences,
the e4m3 rounding against torch's, and the argument checks (which return before anything touches CUDA)."""
import ctypes

import numpy as np
import pytest
import torch

from adamw_hybrid_optimizer_gb300 import libmuon as L
from oracle import adamw as o32
from oracle import adamw8 as o8
from oracle import operators as ops
from tests.test_operators_checks import OnDevice as OnSomeDevice
from tests.test_operators_devices import fake, objects  # noqa: F401

FAKE = 1 << 20
NAN, INF = float("nan"), float("inf")
BF, F = L.MUON_BF16, L.MUON_F32


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


class OnDevice(OnSomeDevice):
    def __init__(self, *shape, device=0, **kw):
        super().__init__(*shape, **kw)
        self.device = device

    def get_device(self):
        return self.device


@pytest.fixture
def calls(monkeypatch):
    """Notes which operators' calls would reach the library, and makes none of them."""
    real, made = L.lib(), []

    class Recorder:
        def __getattr__(self, name):
            if not name.startswith("linear_cross_entropy") or name.endswith("workspace_bytes"):
                return getattr(real, name)
            return lambda *args: made.append((name, args)) or L.MUON_OK

    monkeypatch.setattr(L, "lib", lambda: Recorder())
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    return made


# ---------------------------------------------------------------------------------------- the oracle

def test_oracle_cross_entropy_gradients_match_differences():
    rng = np.random.default_rng(0)
    h, w = rng.standard_normal((6, 5)), rng.standard_normal((9, 5))
    t, wt, up = np.array([3, -100, 8, 9, 0, 4]), np.array([1.0, 1.0, 0.5, 1.0, 2.0, 0.0]), rng.random(6)
    r = ops.linear_cross_entropy(h, w, t, wt, up)
    f = lambda hh, ww: (ops.linear_cross_entropy(hh, ww, t, wt)["losses"] * up).sum()  # noqa: E731
    d, e, step = rng.standard_normal(h.shape), rng.standard_normal(w.shape), 1e-5
    assert abs((r["dh"] * d).sum() - (f(h + step * d, w) - f(h - step * d, w)) / (2 * step)) < 1e-8
    assert abs((r["dw"] * e).sum() - (f(h, w + step * e) - f(h, w - step * e)) / (2 * step)) < 1e-8
    for i in (1, 3, 5):
        assert r["losses"][i] == 0 and r["lse"][i] == 0 and not r["dh"][i].any()
    want = torch.nn.functional.cross_entropy(torch.from_numpy(h @ w.T)[[0, 2, 4]], torch.tensor([3, 8, 0]), reduction="none")
    assert np.allclose(r["losses"][[0, 2, 4]], want.numpy() * wt[[0, 2, 4]], rtol=1e-12)


def test_oracle_codes_are_e4m3():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    codes = codes[torch.isfinite(codes)].double().numpy()
    assert np.array_equal(o8.nearest_code(codes), codes)
    rng = np.random.default_rng(1)
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.uniform(-0.05, 0.05, 4000), [2.0 ** -10, 3 * 2.0 ** -10, 0.0]])
    y = y.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o8.nearest_code(y), want)


def test_oracle_update_is_adamw():
    rng = np.random.default_rng(2)
    p, g, m, v = rng.standard_normal(50), rng.standard_normal(50), rng.standard_normal(50), rng.random(50)
    hp = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1)
    got = o8.update(p, g, m, np.sqrt(v), 4, **hp)
    ref = o32.adamw_update(p, g, m, v, 4, **hp)
    for x, y in zip((got[0], got[1], got[2] ** 2), ref):
        assert np.allclose(x, y, rtol=1e-6, atol=1e-7)


def test_oracle_scales_follow_the_largest_and_leave_out_what_is_not_finite():
    x = np.zeros(600)
    x[3], x[300], x[301], x[599] = -7.0, INF, 2.0, 1e-40
    codes, scales = o8.quantise(x)
    assert scales[0] == 7.0 / 448 and codes[3] == -448 and scales[1] == 2.0 / 448 and np.isnan(codes[300])
    assert scales[2] == o8.FLOOR / 448 and codes[301] == 448
    codes, _ = o8.quantise(np.array([1.0, 1e-9, 0.0]), root=True)
    assert list(codes) == [448.0, o8.LEAST, 0.0]


# ---------------------------------------------------------------------------------------- cross entropy: refusals

def _ce(form, h=FAKE, hdt=BF, ldh=16, w=2 * FAKE, wdt=BF, ldw=16, t=FAKE, it=0, wt=FAKE, losses=FAKE, lse=FAKE, grad=FAKE,
        dh=3 * FAKE, dhdt=BF, lddh=16, dw=4 * FAKE, dwdt=BF, lddw=16, acc=0, N=4, V=30, D=16, ws=FAKE, nb=None, scale=1.0):
    lib = L.lib()
    terms = 0 if form == "fwd" else 2 if F in (dhdt, dwdt) else 1
    nb = lib.linear_cross_entropy_workspace_bytes(max(N, 0), max(V, 1), max(D, 1), terms) if nb is None else nb
    head = (h, hdt, ldh, w, wdt, ldw, t, it, wt)
    if form == "fwd":
        return lib.linear_cross_entropy_forward(*head, losses, lse, N, V, D, ws, nb, None)
    out = (dh, dhdt, lddh, dw, dwdt, lddw, acc, N, V, D, ws, nb, None)
    if form == "bwd":
        return lib.linear_cross_entropy_backward(*head, lse, grad, *out)
    return lib.linear_cross_entropy_forward_backward(*head, scale, losses, lse, *out)


def _need(N=4, V=30, D=16, terms=0):
    return L.linear_cross_entropy_workspace_bytes(N, V, D, terms)


@pytest.mark.parametrize("N,V,D", [(2330, 2529, 843), (2400, 2940, 1257), (16, 32000, 1024), (1, 1, 1), (9000, 100, 8)])
def test_cross_entropy_workspace_serves_calls_with_fewer_terms(N, V, D):
    need = [_need(N, V, D, terms) for terms in range(3)]
    assert 0 < need[0] <= need[1] <= need[2]


@pytest.mark.parametrize("form", ["fwd", "bwd", "step"])
def test_cross_entropy_refusals(form):
    f = lambda **kw: _ce(form, **kw)  # noqa: E731
    for bad in ("h", "w", "t", "lse", "ws"):
        assert f(**{bad: None}) == L.MUON_ERR_INVALID_ARG
    assert f(N=-1) == L.MUON_ERR_INVALID_ARG and f(V=0) == L.MUON_ERR_INVALID_ARG and f(D=0) == L.MUON_ERR_INVALID_ARG
    assert f(ldh=15) == L.MUON_ERR_INVALID_ARG and f(ldw=8) == L.MUON_ERR_INVALID_ARG
    assert f(D=17) == L.MUON_ERR_INVALID_ARG
    assert f(ldh=1 << 40) == L.MUON_ERR_SHAPE and f(ldw=1 << 40) == L.MUON_ERR_SHAPE
    assert f(N=1 << 27) == L.MUON_ERR_SHAPE and f(V=1 << 27) == L.MUON_ERR_SHAPE
    assert f(N=1 << 22, V=1 << 22) == L.MUON_ERR_SHAPE
    assert f(D=70000, ldh=70000, ldw=70000, lddh=70000, lddw=70000) == L.MUON_ERR_SHAPE
    assert f(hdt=F) == L.MUON_ERR_DTYPE and f(wdt=F) == L.MUON_ERR_DTYPE and f(it=2) == L.MUON_ERR_DTYPE
    for kw in (dict(h=FAKE + 8), dict(w=FAKE + 2), dict(ldh=20), dict(ldw=20), dict(t=FAKE + 2), dict(it=1, t=FAKE + 4),
               dict(wt=FAKE + 2), dict(lse=FAKE + 2), dict(ws=FAKE + 128)):
        assert f(**kw) == L.MUON_ERR_ALIGNMENT, kw
    terms = 0 if form == "fwd" else 1
    assert f(nb=_need(terms=terms) - 1) == L.MUON_ERR_WORKSPACE
    if form != "bwd":
        assert f(losses=None) == L.MUON_ERR_INVALID_ARG and f(losses=FAKE + 1) == L.MUON_ERR_ALIGNMENT
    if form != "fwd":
        assert f(dh=None, dw=None) == L.MUON_ERR_INVALID_ARG
        for kw in (dict(dh=FAKE), dict(dw=FAKE), dict(dh=2 * FAKE), dict(dw=2 * FAKE), dict(dw=3 * FAKE)):   # in place
            assert f(**kw) == L.MUON_ERR_INVALID_ARG
        assert f(lddh=15) == L.MUON_ERR_INVALID_ARG and f(lddw=15) == L.MUON_ERR_INVALID_ARG
        assert f(dhdt=3) == L.MUON_ERR_DTYPE and f(dwdt=3) == L.MUON_ERR_DTYPE
        assert f(dh=FAKE + 1) == L.MUON_ERR_ALIGNMENT and f(dw=FAKE + 2, dwdt=F) == L.MUON_ERR_ALIGNMENT
        assert f(dhdt=F, nb=_need(terms=2) - 1) == L.MUON_ERR_WORKSPACE
    if form == "bwd":
        assert f(grad=FAKE + 2) == L.MUON_ERR_ALIGNMENT
    if form == "step":
        assert f(scale=NAN) == L.MUON_ERR_INVALID_ARG and f(scale=INF) == L.MUON_ERR_INVALID_ARG


def test_cross_entropy_workspace_sizes():
    assert _need(-1) == 0 and _need(V=0) == 0 and _need(D=0) == 0 and _need(terms=3) == 0 and _need(terms=-1) == 0
    assert _need(1 << 27) == 0
    N, V, D = 8192, 128256, 4096
    assert _need(N, V, D, 0) < 100 << 20                              # nothing of the logits' size
    # with gradients: one or two bf16 terms of each logit, 8 bytes for each 128 of them, h again, and fp32 sums of dh by slices
    # of the contraction (half of the rows at a time, or all of them with two terms): eight at most here
    one, two = _need(N, V, D, 1), _need(N, V, D, 2)
    assert 2 * N * V <= one <= 2 * N * V + N * V // 16 + 2 * N * D + 8 * 4 * N // 2 * D + (1 << 20)
    assert 4 * N * V <= two <= 4 * N * V + N * V // 16 + 2 * N * D + 8 * 4 * N * D + (1 << 20)
    # beyond a piece only fp32 sums of dw come on top
    assert _need(16 * N, V, D, 1) <= one + 4 * V * D + (64 << 20)
    # a short vocabulary or a wide h: rows of a piece are bounded by whichever is larger
    assert _need(1 << 26, 1, 8, 1) < 32 << 30 and _need(1 << 22, 100, 65536, 1) < 16 << 30
    # the call without gradients takes a workspace of any kind
    for n in (1, 100, 5000):
        assert _need(n, 5000, 64, 0) <= min(_need(n, 5000, 64, 1), _need(n, 5000, 64, 2))


def test_pieces_switch():
    lib = L.lib()
    assert lib.muon_debug_loss_rows(-1) == L.MUON_ERR_INVALID_ARG
    big = _need(4096, 5000, 64, 1)
    assert lib.muon_debug_loss_rows(512) == L.MUON_OK
    small = _need(4096, 5000, 64, 1)
    assert lib.muon_debug_loss_rows(0) == L.MUON_OK
    assert small < big == _need(4096, 5000, 64, 1)


def test_cross_entropy_binding_refuses_what_the_c_call_cannot_see(calls):
    f, b, i = torch.float32, torch.bfloat16, torch.int64
    t = lambda *s, dtype=b, **kw: OnDevice(*s, dtype=dtype, **kw)  # noqa: E731
    ok = dict(h=t(4, 16), w=t(30, 16), targets=t(4, dtype=i), weights=t(4, dtype=f), losses=t(4, dtype=f), lse=t(4, dtype=f),
              ws=t(1 << 20, dtype=torch.uint8))

    def go(**kw):
        a = {**ok, **kw}
        L.linear_cross_entropy_forward(a["h"], a["w"], a["targets"], a["weights"], a["losses"], a["lse"], a["ws"], stream=0)

    for bad in (dict(w=t(30, 8)), dict(targets=t(5, dtype=i)), dict(weights=t(4)), dict(losses=t(3, dtype=f)),
                dict(h=t(4, 16, is_cuda=False)), dict(ws=t(9, dtype=torch.uint8, is_cuda=False)), dict(lse=t(4, dtype=i)),
                dict(w=t(30, 16, device=1)), dict(ws=t(1 << 20, dtype=torch.uint8, device=1))):
        with pytest.raises((ValueError, L.MuonError)):
            go(**bad)
    with pytest.raises(L.MuonError):
        go(targets=t(4, dtype=f))
    assert calls == []
    with pytest.raises(ValueError, match="current"):
        L.linear_cross_entropy_forward(*(t(*x.shape, dtype=x.dtype, device=2) for x in ok.values()), stream=0)
    assert calls == []
    go()
    go(weights=None)
    assert [name for name, _ in calls] == ["linear_cross_entropy_forward"] * 2
    with pytest.raises(ValueError):
        L.linear_cross_entropy_backward(ok["h"], ok["w"], ok["targets"], None, ok["lse"], None, t(4, 8), None, ok["ws"],
                                        stream=0)
    with pytest.raises(ValueError):
        L.linear_cross_entropy_forward_backward(ok["h"], ok["w"], ok["targets"], None, 1.0, ok["losses"], ok["lse"], None,
                                                t(31, 16), ok["ws"], stream=0)


# ---------------------------------------------------------------------------------------- AdamW in 8 bits: refusals

def _tensor(param=FAKE, grad=FAKE, m=FAKE, r=FAKE, scales=FAKE, master=None, n=1000, pdt=BF, gdt=BF, hp=None):
    hp = L.make_adamw_hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1) if hp is None else hp
    t = L.adamw8_tensor(param, grad, m, r, scales, master, n, pdt, gdt, ctypes.pointer(hp) if hp is not False else None)
    t._hp = hp
    return t


def _step8(*ts, n=None, lib=None):
    arr = (L.adamw8_tensor * max(len(ts), 1))(*ts)
    return (lib or L.lib()).adamw8_step_grouped(arr, len(ts) if n is None else n, None)


def test_adamw8_struct_layout():
    assert ctypes.sizeof(L.adamw8_tensor) == 72
    assert L.adamw8_tensor.n.offset == 48 and L.adamw8_tensor.pdt.offset == 56 and L.adamw8_tensor.hp.offset == 64


def test_adamw8_refusals():
    good = _tensor()
    assert L.lib().adamw8_step_grouped(None, 1, None) == L.MUON_ERR_INVALID_ARG
    assert _step8(good, n=0) == L.MUON_ERR_INVALID_ARG and _step8(good, n=(1 << 20) + 1) == L.MUON_ERR_INVALID_ARG
    for bad in ("param", "grad", "m", "r", "scales"):
        assert _step8(good, _tensor(**{bad: None})) == L.MUON_ERR_INVALID_ARG
    assert _step8(good, _tensor(hp=False)) == L.MUON_ERR_INVALID_ARG
    assert _step8(good, _tensor(n=0)) == L.MUON_ERR_INVALID_ARG
    assert _step8(good, _tensor(n=1 << 41)) == L.MUON_ERR_SHAPE
    assert _step8(good, _tensor(pdt=2)) == L.MUON_ERR_DTYPE and _step8(good, _tensor(gdt=7)) == L.MUON_ERR_DTYPE
    assert _step8(good, _tensor(master=FAKE, pdt=F)) == L.MUON_ERR_DTYPE
    for kw in (dict(param=FAKE + 1), dict(param=FAKE + 2, pdt=F), dict(grad=FAKE + 2, gdt=F), dict(scales=FAKE + 4),
               dict(master=FAKE + 2)):
        assert _step8(good, _tensor(**kw)) == L.MUON_ERR_ALIGNMENT, kw
    for hp in ((1e-3, 1.0, 0.95, 1e-8, 0.1, 1), (1e-3, 0.9, 0.95, 1e-8, 0.1, 0), (NAN, 0.9, 0.95, 1e-8, 0.1, 1)):
        assert _step8(good, _tensor(hp=L.make_adamw_hparams(*hp))) == L.MUON_ERR_INVALID_ARG
    if not torch.cuda.is_available():
        assert _step8(good, _tensor(m=FAKE + 1, r=FAKE + 3)) in (L.MUON_ERR_CUDA, L.MUON_ERR_UNSUPPORTED_DEVICE)


def test_adamw8_launches_and_devices(fake):  # noqa: F811
    """One launch per 96 tensors of bf16 throughout, and per 96 others, on whichever device is current."""
    for device in (0, 3, 1):
        fake.fake_use_device(device)
        for narrow, wide, want in ((1, 0, 1), (0, 1, 1), (96, 96, 2), (97, 0, 2), (5, 200, 4)):
            before = fake.fake_launches()
            ts = [_tensor() for _ in range(narrow)] + [_tensor(gdt=F) for _ in range(wide)]
            assert _step8(*ts, lib=fake) == L.MUON_OK
            assert fake.fake_launches() - before == want


def test_adamw8_binding_refuses_what_the_c_call_cannot_see(monkeypatch):
    f8, b, f = torch.float8_e4m3fn, torch.bfloat16, torch.float32
    t = lambda *s, dtype=b, **kw: OnDevice(*s, dtype=dtype, **kw)  # noqa: E731
    hp = L.make_adamw_hparams(1e-3, 0.9, 0.95, 1e-8, 0.1, 1)
    ok = [t(300), t(300), t(300, dtype=f8), t(300, dtype=f8), t(2, 2, dtype=f), hp]
    arr = L.make_adamw8_tensors([ok])
    assert arr[0].n == 300 and len(arr.tensors) == 6
    for k, bad in ((1, t(299)), (2, t(300, dtype=torch.uint8)), (3, t(300)), (3, t(301, dtype=f8)), (4, t(3, 2, dtype=f)),
                   (4, t(2, 2)), (0, t(300, contiguous=False)), (1, t(300, is_cuda=False))):
        with pytest.raises(ValueError):
            L.make_adamw8_tensors([ok[:k] + [bad] + ok[k + 1:]])
    for bad in ((t(300, dtype=b),), (t(299, dtype=f),)):
        with pytest.raises(ValueError):
            L.make_adamw8_tensors([ok + list(bad)])
    with pytest.raises(ValueError, match="devices"):
        L.make_adamw8_tensors([ok, ok[:1] + [t(300, device=1)] + ok[2:]])
    monkeypatch.setattr(L, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="current"):
        L.adamw8_step_grouped(arr, stream=0)
    with pytest.raises(ValueError):        # a master goes with bf16 weights
        L.make_adamw8_tensors([[t(300, dtype=f)] + ok[1:] + [t(300, dtype=f)]])
