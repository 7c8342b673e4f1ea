"""Embedding, layer norm and distillation without a GPU: the oracle's gradients against differences of its own
forward pass, and the argument checks of the C calls (which return before anything touches CUDA)."""
import ctypes

import numpy as np
import pytest

from adamw_hybrid_optimizer_gb300 import libmuon as L
from oracle import operators as ops

FAKE = 1 << 20
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _difference(f, x, d, h=1e-5):
    return (f(x + h * d) - f(x - h * d)) / (2 * h)


def test_oracle_embedding_gradient_matches_differences():
    rng = np.random.default_rng(0)
    ids = np.array([3, 1, 3, -1, 7, 0, 3])
    E, dout, d = rng.standard_normal((7, 5)), rng.standard_normal((7, 5)), rng.standard_normal((7, 5))
    g, count, _ = ops.embedding_backward(ids, dout, 7, 2.5)
    num = _difference(lambda e: (ops.embedding_forward(ids, e, 2.5) * dout).sum(), E, d)
    assert abs((g * d).sum() - num) < 1e-8
    assert list(count) == [1, 1, 0, 3, 0, 0, 0]
    padded, _, _ = ops.embedding_backward(ids, dout, 7, 2.5, padding_idx=3)
    assert not padded[3].any() and np.array_equal(padded[:3], g[:3])


def test_oracle_layernorm_gradients_match_differences():
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((4, 9)), rng.standard_normal(9), rng.standard_normal(9)
    dy, d, dwd = rng.standard_normal((4, 9)), rng.standard_normal((4, 9)), rng.standard_normal(9)
    _, mean, rstd = ops.layernorm_forward(x, w, b, 1e-5)
    dx, dw, db = ops.layernorm_backward(dy, x, w, mean, rstd)
    f = lambda xx, ww=w, bb=b: (ops.layernorm_forward(xx, ww, bb, 1e-5)[0] * dy).sum()  # noqa: E731
    assert abs((dx * d).sum() - _difference(f, x, d)) < 1e-7
    assert abs((dw * dwd).sum() - _difference(lambda ww: f(x, ww), w, dwd)) < 1e-7
    assert abs((db * dwd).sum() - _difference(lambda bb: f(x, w, bb), b, dwd)) < 1e-7


@pytest.mark.parametrize("T", [1.0, 3.0])
def test_oracle_distill_gradient_matches_differences(T):
    rng = np.random.default_rng(2)
    z, d = rng.standard_normal((5, 11)) * 3, rng.standard_normal((5, 11))
    idx = np.array([[0, 4, 9], [1, 1, 2], [-1, 5, 11], [-1, -1, 20], [3, 7, 10]])
    t = rng.standard_normal((5, 3)) * 2
    w = np.array([1.0, 0.5, 2.0, 1.0, 0.0])
    r = ops.distill(z, idx, t, T, w)
    num = _difference(lambda zz: ops.distill(zz, idx, t, T, w)["losses"].sum(), z, d)
    assert abs((r["dlogits"] * d).sum() - num) < 1e-7
    assert r["losses"][3] == 0 and not r["dlogits"][3].any() and not r["dlogits"][4].any()
    assert np.all(r["losses"] >= 0)


def _embed_fwd(ids=FAKE, it=0, table=FAKE, tdt=0, ldt=8, out=FAKE, odt=0, ldo=8, n=4, V=5, D=8, scale=1.0):
    return L.lib().embedding_forward(ids, it, table, tdt, ldt, out, odt, ldo, n, V, D, scale, None)


def _embed_bwd(ids=FAKE, it=0, dout=FAKE, odt=0, ldo=8, g=FAKE, gdt=0, ldg=8, n=4, V=5, D=8, scale=1.0, ws=FAKE,
               nb=None):
    nb = L.embedding_workspace_bytes(max(n, 0), max(V, 1), max(D, 1)) if nb is None else nb
    return L.lib().embedding_backward(ids, it, dout, odt, ldo, g, gdt, ldg, n, V, D, scale, -1, 0, ws, nb, None)


def test_embedding_refusals():
    for f in (_embed_fwd, _embed_bwd):
        assert f(ids=None) == L.MUON_ERR_INVALID_ARG
        assert f(n=-1) == L.MUON_ERR_INVALID_ARG
        assert f(V=0) == L.MUON_ERR_INVALID_ARG
        assert f(D=0) == L.MUON_ERR_INVALID_ARG
        assert f(D=9) == L.MUON_ERR_INVALID_ARG        # pitches below the width
        assert f(scale=NAN) == L.MUON_ERR_INVALID_ARG
        assert f(it=2) == L.MUON_ERR_DTYPE
        assert f(odt=3) == L.MUON_ERR_DTYPE
        assert f(ids=FAKE + 2) == L.MUON_ERR_ALIGNMENT
        assert f(it=1, ids=FAKE + 4) == L.MUON_ERR_ALIGNMENT
        assert f(n=1 << 28) == L.MUON_ERR_SHAPE
        assert f(V=1 << 31) == L.MUON_ERR_SHAPE
    assert _embed_fwd(table=None) == L.MUON_ERR_INVALID_ARG
    assert _embed_fwd(out=None) == L.MUON_ERR_INVALID_ARG
    assert _embed_fwd(tdt=1, table=FAKE + 1) == L.MUON_ERR_ALIGNMENT
    assert _embed_fwd(D=70000, ldt=70000, ldo=70000) == L.MUON_ERR_SHAPE
    assert _embed_bwd(g=None) == L.MUON_ERR_INVALID_ARG
    assert _embed_bwd(dout=None) == L.MUON_ERR_INVALID_ARG
    assert _embed_bwd(ws=None) == L.MUON_ERR_INVALID_ARG
    assert _embed_bwd(ws=FAKE + 128) == L.MUON_ERR_ALIGNMENT
    assert _embed_bwd(nb=L.embedding_workspace_bytes(4, 5, 8) - 1) == L.MUON_ERR_WORKSPACE
    assert L.embedding_workspace_bytes(-1, 5, 8) == 0 and L.embedding_workspace_bytes(1, 0, 8) == 0
    assert L.embedding_workspace_bytes(1, 5, 0) == 0
    assert L.embedding_workspace_bytes(100, 5, 8) >= 4 * 100 * 4


def _ln_fwd(x=FAKE, xdt=0, ldx=8, w=FAKE, b=FAKE, wdt=0, y=FAKE, ydt=0, ldy=8, mean=FAKE, rstd=FAKE, N=4, D=8,
            eps=1e-5):
    return L.lib().layernorm_forward(x, xdt, ldx, w, b, wdt, y, ydt, ldy, mean, rstd, N, D, eps, None)


def _ln_bwd(dy=FAKE, ydt=0, lddy=8, x=FAKE, xdt=0, ldx=8, w=FAKE, wdt=0, mean=FAKE, rstd=FAKE, dx=FAKE, lddx=8,
            dw=FAKE, db=FAKE, gdt=0, N=4, D=8, ws=FAKE, nb=None):
    nb = L.layernorm_workspace_bytes(max(N, 0), max(D, 1)) if nb is None else nb
    return L.lib().layernorm_backward(dy, ydt, lddy, x, xdt, ldx, w, wdt, mean, rstd, dx, lddx, dw, db, gdt, 0, N, D,
                                      ws, nb, None)


def test_layernorm_refusals():
    for f in (_ln_fwd, _ln_bwd):
        assert f(x=None) == L.MUON_ERR_INVALID_ARG
        assert f(N=-1) == L.MUON_ERR_INVALID_ARG
        assert f(D=0) == L.MUON_ERR_INVALID_ARG
        assert f(D=9) == L.MUON_ERR_INVALID_ARG
        assert f(N=1 << 31) == L.MUON_ERR_SHAPE
        assert f(xdt=2) == L.MUON_ERR_DTYPE
        assert f(ydt=2) == L.MUON_ERR_DTYPE
        assert f(wdt=2) == L.MUON_ERR_DTYPE
        assert f(x=FAKE + 2) == L.MUON_ERR_ALIGNMENT
        assert f(w=FAKE + 1) == L.MUON_ERR_ALIGNMENT
        assert f(mean=FAKE + 2) == L.MUON_ERR_ALIGNMENT
    assert _ln_fwd(y=None) == L.MUON_ERR_INVALID_ARG
    assert _ln_fwd(eps=-1.0) == L.MUON_ERR_INVALID_ARG
    assert _ln_fwd(eps=NAN) == L.MUON_ERR_INVALID_ARG
    assert _ln_fwd(D=1 << 21, ldx=1 << 21, ldy=1 << 21) == L.MUON_ERR_SHAPE
    assert _ln_bwd(dy=None) == L.MUON_ERR_INVALID_ARG
    assert _ln_bwd(mean=None) == L.MUON_ERR_INVALID_ARG
    assert _ln_bwd(rstd=None) == L.MUON_ERR_INVALID_ARG
    assert _ln_bwd(dx=None, dw=None, db=None) == L.MUON_ERR_INVALID_ARG
    assert _ln_bwd(gdt=5) == L.MUON_ERR_DTYPE
    assert _ln_bwd(lddx=7) == L.MUON_ERR_INVALID_ARG
    assert _ln_bwd(ws=None) == L.MUON_ERR_INVALID_ARG
    assert _ln_bwd(ws=FAKE + 64) == L.MUON_ERR_ALIGNMENT
    assert _ln_bwd(nb=L.layernorm_workspace_bytes(4, 8) - 1) == L.MUON_ERR_WORKSPACE
    assert L.layernorm_workspace_bytes(-1, 8) == 0 and L.layernorm_workspace_bytes(4, 0) == 0
    assert L.layernorm_workspace_bytes(0, 8) > 0


def _d(form, z=FAKE, zdt=0, ldz=16, idx=FAKE, it=0, val=FAKE, tdt=0, w=FAKE, losses=FAKE, stats=FAKE, grad=FAKE,
       dz=FAKE + 4096, ddt=0, ldd=16, N=4, V=16, K=3, T=1.0, scale=1.0):
    lib = L.lib()
    if form == "fwd":
        return lib.distill_forward(z, zdt, ldz, idx, it, val, tdt, w, losses, stats, N, V, K, T, None)
    if form == "bwd":
        return lib.distill_backward(z, zdt, ldz, idx, it, val, tdt, w, stats, grad, dz, ddt, ldd, N, V, K, T, None)
    return lib.distill_forward_backward(z, zdt, ldz, idx, it, val, tdt, w, scale, losses, stats, dz, ddt, ldd, N, V, K,
                                        T, None)


def test_distill_refusals():
    for f in ("fwd", "bwd", "step"):
        assert _d(f, z=None) == L.MUON_ERR_INVALID_ARG
        assert _d(f, idx=None) == L.MUON_ERR_INVALID_ARG
        assert _d(f, val=None) == L.MUON_ERR_INVALID_ARG
        assert _d(f, stats=None) == L.MUON_ERR_INVALID_ARG
        assert _d(f, N=-1) == L.MUON_ERR_INVALID_ARG
        assert _d(f, V=0) == L.MUON_ERR_INVALID_ARG
        assert _d(f, K=0) == L.MUON_ERR_INVALID_ARG
        assert _d(f, V=17) == L.MUON_ERR_INVALID_ARG
        for T in (0.0, -1.0, NAN, float("inf"), 1e-5, 1e5):
            assert _d(f, T=T) == L.MUON_ERR_INVALID_ARG
        assert _d(f, K=1025) == L.MUON_ERR_SHAPE
        assert _d(f, N=1 << 31) == L.MUON_ERR_SHAPE
        assert _d(f, zdt=4) == L.MUON_ERR_DTYPE
        assert _d(f, tdt=4) == L.MUON_ERR_DTYPE
        assert _d(f, it=4) == L.MUON_ERR_DTYPE
        assert _d(f, z=FAKE + 2) == L.MUON_ERR_ALIGNMENT
        assert _d(f, it=1, idx=FAKE + 4) == L.MUON_ERR_ALIGNMENT
        assert _d(f, stats=FAKE + 2) == L.MUON_ERR_ALIGNMENT
    for f in ("bwd", "step"):
        assert _d(f, dz=None) == L.MUON_ERR_INVALID_ARG
        assert _d(f, ldd=15) == L.MUON_ERR_INVALID_ARG
        assert _d(f, ddt=9) == L.MUON_ERR_DTYPE
        assert _d(f, dz=FAKE, ddt=1) == L.MUON_ERR_INVALID_ARG      # in place needs one dtype and pitch
        assert _d(f, dz=FAKE, ldd=24) == L.MUON_ERR_INVALID_ARG
    assert _d("fwd", losses=None) == L.MUON_ERR_INVALID_ARG
    assert _d("step", losses=None) == L.MUON_ERR_INVALID_ARG
    assert _d("step", scale=NAN) == L.MUON_ERR_INVALID_ARG
    assert _d("bwd", grad=FAKE + 1) == L.MUON_ERR_ALIGNMENT


def test_valid_arguments_reach_the_device_check():
    import torch
    if not torch.cuda.is_available():
        for st in (_embed_fwd(), _embed_bwd(), _ln_fwd(), _ln_bwd(), _d("fwd"), _d("bwd"), _d("step")):
            assert st in (L.MUON_ERR_CUDA, L.MUON_ERR_UNSUPPORTED_DEVICE)


def test_binding_refuses_shapes_the_c_calls_cannot_see():
    import torch
    ids, t, o = torch.zeros(3, dtype=torch.int64), torch.zeros(4, 8), torch.zeros(3, 8)
    with pytest.raises(ValueError):                       # not on the GPU
        L.embedding_forward(ids, t, o)
    with pytest.raises(ValueError):
        L.layernorm_forward(o, None, None, torch.zeros(3, 8), None, None)
    with pytest.raises(ValueError):                       # teacher arrays of two shapes
        L.distill_forward(torch.zeros(2, 8), torch.zeros(2, 3, dtype=torch.int32), torch.zeros(2, 4), 1.0, None,
                          torch.zeros(2), torch.zeros(2, 2))
    assert ctypes.sizeof(ctypes.c_int) == 4
