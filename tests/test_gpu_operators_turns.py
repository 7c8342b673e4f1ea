"""Calls whose blocks come round more than once: several turns of rows for every layout of layer norm, so that the places of
rows on their way are used again, and the table gradient's sort of more ids than one cluster takes, over wide keys. Against
the formulas in 64 bits, in PyTorch on the GPU; tolerances as in test_gpu_operators.py, from the same counts of roundings."""
import pytest
import torch

from tests.gpu_common import DEV, build_lib

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
K_LN = 128 * U            # adds of a thread's columns and of the exchange between warps
EPS = 1e-5
EPS64 = float(torch.tensor(EPS, dtype=torch.float32))   # as the call gets it
BF, F = torch.bfloat16, torch.float32
DTYPES = [(F, F), (BF, BF), (F, BF), (BF, F)]


@pytest.fixture(scope="module")
def L():
    return build_lib()


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(*shape, seed, dt=F):
    return torch.randn(shape, generator=gen(seed), device=DEV).to(dt)


def store_tol(ref, dt):
    return ref.abs() * (2.0 ** -8 if dt == BF else 2 * U) + 1e-37


def byte_ws(n):
    return torch.full((max(n, 256),), 0xCD, dtype=torch.uint8, device=DEV)


def blank(rows, cols, dt, ld=0, offset=0):
    """A NaN-filled matrix with a row pitch of ld (0: its width) from an element offset."""
    ld = ld or cols
    buf = torch.full((offset + rows * ld,), float("nan"), dtype=dt, device=DEV)
    return buf[offset:].as_strided((rows, cols), (ld, 1))


def place(t, ld=0, offset=0):
    return blank(*t.shape, t.dtype, ld, offset).copy_(t)


# N, D, offset: the largest launch holds 152 x 1024 / (threads of a row) rows at once (152 blocks of one row above 8192
# columns); four turns of it and a part of one. Whole granules with and without idle threads, rows that start past a
# boundary, and from an offset of one value rows of single values.
TURNS = [(20011, 256, 0), (20011, 200, 0), (20011, 201, 0), (20003, 512, 0), (20003, 300, 0), (15001, 768, 0),
         (15001, 771, 0), (15001, 1000, 0), (7301, 1200, 0), (7301, 1201, 0), (5003, 2048, 0), (5003, 1900, 0),
         (2601, 4096, 0), (2601, 2051, 0), (1301, 8192, 0), (1301, 5003, 0), (701, 12000, 0), (701, 12007, 0), (701, 16384, 0),
         (701, 16001, 0),
         (5001, 700, 1), (1301, 5000, 1), (701, 12000, 1),
         (700, 16400, 0), (701, 20001, 0)]


def ln_case(N, D, offset, xdt, ydt):
    wdt = BF if (N + D) % 4 < 2 else F
    x = (randn(N, D, seed=1) * 2 + randn(N, 1, seed=2)).to(xdt)
    w, b = (randn(D, seed=3) * 0.2 + 1).to(wdt), (randn(D, seed=4) * 0.2).to(wdt)
    return x, w, b, randn(N, D, seed=5, dt=ydt)


@pytest.mark.parametrize("N,D,offset", TURNS)
@pytest.mark.parametrize("xdt,ydt", DTYPES)
def test_layernorm_forward_turns(L, N, D, offset, xdt, ydt):
    x, w, b, _ = ln_case(N, D, offset, xdt, ydt)
    px, y = place(x, 0, offset), blank(N, D, ydt, 0, offset)
    mean, rstd = (torch.full((N,), float("nan"), device=DEV) for _ in range(2))
    L.layernorm_forward(px, w, b, y, mean, rstd, EPS)
    X, W, B = x.double(), w.double(), b.double()
    mu = X.mean(1)
    r = ((X - mu[:, None]).square().mean(1) + EPS64).rsqrt()
    xh = (X - mu[:, None]) * r[:, None]
    ref = xh * W + B
    e_mean = K_LN * X.abs().mean(1) + 1e-37
    e_r = K_LN + 0.5 * (e_mean * r).square()
    assert bool(((mean.double() - mu).abs() <= e_mean).all())
    assert bool(((rstd.double() - r).abs() <= e_r * r).all())
    tol = ((e_mean * r)[:, None] + (e_r + 4 * U)[:, None] * xh.abs() + 2 * U * X.abs() * r[:, None]) * W.abs() \
        + 4 * U * ref.abs() + 2 * U * B.abs()
    assert bool(((y.double() - ref).abs() <= store_tol(ref, ydt) + tol).all())
    if xdt == ydt:
        L.layernorm_forward(px, w, b, px, None, None, EPS)
        assert torch.equal(px, y)


@pytest.mark.parametrize("N,D,offset", TURNS)
@pytest.mark.parametrize("xdt,ydt", DTYPES)
def test_layernorm_backward_turns(L, N, D, offset, xdt, ydt):
    gdt = F if (N + D) % 4 < 2 else BF
    x, w, _, dy = ln_case(N, D, offset, xdt, ydt)
    mean = x.double().mean(1).float()
    rstd = ((x.double() - mean.double()[:, None]).square().mean(1) + EPS64).rsqrt().float()
    px, pdy, dx = place(x, 0, offset), place(dy, 0, offset), blank(N, D, xdt, 0, offset)
    dw, db = (torch.full((D,), float("nan"), dtype=gdt, device=DEV) for _ in range(2))
    ws = byte_ws(L.layernorm_workspace_bytes(N, D))
    L.layernorm_backward(pdy, px, w, mean, rstd, dx, dw, db, ws)
    X, R, DY = x.double(), rstd.double()[:, None], dy.double()
    xh = (X - mean.double()[:, None]) * R
    g = DY * w.double()
    rdx = R * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    exh = xh.abs() + 2 * X.abs() * R                  # xh's own rounding scales with these
    tol = K_LN * R * (g.abs() + g.abs().mean(1, keepdim=True) + exh * (g.abs() * exh).mean(1, keepdim=True))
    assert bool(((dx.double() - rdx).abs() <= store_tol(rdx, xdt) + tol).all())
    chain = (200 + N / 64) * U
    for got, ref, e in ((dw, (DY * xh).sum(0), chain * (DY.abs() * exh).sum(0)), (db, DY.sum(0), chain * DY.abs().sum(0))):
        assert bool(((got.double() - ref).abs() <= store_tol(ref, gdt) + e).all())
    for out in ([px, pdy] if xdt == ydt else [px]):   # in the place of x, and of dy
        px.copy_(x)
        pdy.copy_(dy)
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        L.layernorm_backward(pdy, px, w, mean, rstd, out, dw2, db2, ws)
        assert torch.equal(out, dx) and torch.equal(dw, dw2) and torch.equal(db, db2)


# n, V, D, gap between dtable's rows: digits of 7 bits in three passes, of 9 in two and three, of 7 in four, and one pass;
# more ids than the cluster takes, and (the last two) its largest
LONG_SORT = [(140001, 300000, 5, 3), (200000, 128256, 24, 8), (131073, 90_000_000, 1, 0), (150000, 200_000_000, 1, 0),
             (300000, 200, 33, 2), (1_000_003, 50304, 8, 0), (131072, 300000, 9, 1), (131071, 128256, 24, 0)]


@pytest.mark.parametrize("n,V,D,gap", LONG_SORT)
@pytest.mark.parametrize("odt,gdt", [(F, F), (BF, BF)])
def test_embedding_backward_long_sort(L, n, V, D, gap, odt, gdt):
    u = torch.rand(n, generator=gen(6), device=DEV, dtype=torch.float64)
    ids = (u.pow(3) * V).long().clamp_(0, V - 1)      # low ids are the frequent ones
    some = torch.rand(n, generator=gen(7), device=DEV) < 0.02
    ids[some] = torch.where(torch.rand(int(some.sum()), generator=gen(8), device=DEV) < 0.5, -1, V)
    dout = randn(n, D, seed=9, dt=odt)
    pad = 1
    live = (ids >= 0) & (ids < V) & (ids != pad)
    at = ids[live]
    scale = float(torch.tensor(0.3, dtype=torch.float32))
    zero = lambda: torch.zeros((V, D), dtype=torch.float64, device=DEV)  # noqa: E731
    ref = zero().index_add_(0, at, dout[live].double(), alpha=scale)
    mag = zero().index_add_(0, at, dout[live].double().abs(), alpha=scale)
    count = torch.bincount(at, minlength=V)
    tol = (count[:, None] + 2) * U * mag
    ws = byte_ws(L.embedding_workspace_bytes(n, V, D))
    g = blank(V, D, gdt, D + gap)
    L.embedding_backward(ids, dout, g, ws, 0.3, padding_idx=pad)
    assert bool(((g.double() - ref).abs() <= store_tol(ref, gdt) + tol).all())
    if gap:
        assert bool(torch.isnan(g.as_strided((V - 1, gap), (D + gap, 1), D)).all())
    again = blank(V, D, gdt, D + gap)
    L.embedding_backward(ids.int(), dout, again, ws, 0.3, padding_idx=pad)
    assert torch.equal(g, again)
    old = randn(V, D, seed=10, dt=gdt)
    acc = place(old, D + gap)
    L.embedding_backward(ids, dout, acc, ws, 0.3, padding_idx=pad, accumulate=True)
    want = ref + old.double()
    assert bool(((acc.double() - want).abs() <= store_tol(want, gdt) + tol + 2 * U * (old.double().abs() + mag)).all())
    assert torch.equal(acc[count == 0], old[count == 0])
