"""GPU parity of the embedding, layer norm and distillation operators against the fp64 oracle, through the C ABI.

Tolerances, from the arithmetic (u = 2^-24, the fp32 unit roundoff):
  * a stored result: 2^-8 of its value in bf16, 2 u in fp32, plus the error of the fp32 value it is rounded from;
  * an fp32 sum of n terms in whatever order the kernel takes has error at most (adds in its longest chain) * u * the
    sum of the terms' magnitudes. Embedding: the id's count. Layer norm: 128 adds cover a thread's columns and the
    exchange between warps; over rows 200 + N / 64. Distillation: V / 512 + 64;
  * exp2 within 2 ulp of its rounded argument, whose rounding adds 2 u of |argument| to the result's relative error.
"""
import numpy as np
import pytest
import torch

from oracle import operators as ops
from tests.gpu_common import DEV, build_lib, f64

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF, F = torch.bfloat16, torch.float32
DTYPES = [(F, F), (BF, BF), (F, BF), (BF, F)]


@pytest.fixture(scope="module")
def L():
    return build_lib()


def store_tol(ref, dt):
    return np.abs(ref) * (2.0 ** -8 if dt == BF else 2 * U) + 1e-37


def gen(seed):
    return torch.Generator().manual_seed(seed)


def place(t, ld=0, offset=0):
    """The matrix on the GPU with a row pitch of ld (0: its width) from an element offset; the gaps hold NaN."""
    rows, cols = t.shape
    ld = ld or cols
    buf = torch.full((offset + max(rows, 1) * ld,), float("nan"), dtype=t.dtype, device=DEV)
    m = buf[offset:].as_strided((rows, cols), (ld, 1))
    m.copy_(t)
    return m


def blank(rows, cols, dt, ld=0, offset=0):
    return place(torch.full((rows, cols), float("nan"), dtype=dt), ld, offset)


def gaps_untouched(m):
    """Nothing was written between the rows."""
    rows, cols = m.shape
    ld = m.stride(0)
    if rows < 2 or ld == cols:
        return True
    gap = m.as_strided((rows - 1, ld - cols), (ld, 1), m.storage_offset() + cols)
    return bool(torch.isnan(gap).all())


def byte_ws(n):
    return torch.full((max(n, 256),), 0xCD, dtype=torch.uint8, device=DEV)   # workspaces need no initialisation


# ------------------------------------------------------------------------------------------------ embedding

# n, V, D: none; one; odd widths on either side of a warp's 256 and 1024 columns; a few ids that fill many groups of
# 32 sorted positions; a vocabulary of three digits; runs that end on group boundaries
EMBED = [(0, 7, 5), (1, 1, 1), (3, 5, 7), (33, 10, 256), (65, 2, 40), (257, 50, 300), (1000, 3, 776), (5000, 17, 24),
         (4097, 600, 130), (70000, 40, 8), (9000, 300000, 16), (8192, 1000, 1030), (96, 1, 64), (140000, 900, 8), (100000, 5000, 72),
         (600, 90, 133), (3000, 40, 1337), (60000, 300, 513), (30000, 200, 776)]


def make_ids(n, V, seed, it):
    g = gen(seed)
    u = torch.rand(n, generator=g, dtype=torch.float64)
    ids = torch.floor(u * u * u * V).to(torch.int64).clamp_(0, V - 1)   # low ids are the frequent ones
    some = torch.rand(n, generator=g) < 0.03
    ids[some] = torch.tensor([-1, V, -100, V + 5])[torch.randint(0, 4, (int(some.sum()),), generator=g)]
    return ids.to(it)


@pytest.mark.parametrize("n,V,D", EMBED)
@pytest.mark.parametrize("tdt,odt", DTYPES)
def test_embedding_forward(L, n, V, D, tdt, odt):
    it = torch.int32 if (n + D) % 2 else torch.int64
    ids = make_ids(n, V, n + D, it)
    table = torch.randn((V, D), generator=gen(1)).to(tdt)
    out = blank(n, D, odt)
    L.embedding_forward(ids.to(DEV), place(table), out, 1.7)
    ref = ops.embedding_forward(ids.numpy(), f64(table), np.float64(np.float32(1.7)))
    assert np.all(np.abs(f64(out) - ref) <= store_tol(ref, odt))


@pytest.mark.parametrize("ld,offset", [(0, 1), (304, 0), (303, 0), (304, 4), (320, 8)])
@pytest.mark.parametrize("tdt,odt", DTYPES)
def test_embedding_strides_and_alignment(L, ld, offset, tdt, odt):
    n, V, D = 130, 21, 300
    ids = make_ids(n, V, 3, torch.int64)
    table, dout = torch.randn((V, D), generator=gen(2)).to(tdt), torch.randn((n, D), generator=gen(4)).to(odt)
    out = blank(n, D, odt, ld, offset)
    L.embedding_forward(ids.to(DEV), place(table, ld, offset), out)
    ref = ops.embedding_forward(ids.numpy(), f64(table), 1.0)
    assert np.all(np.abs(f64(out) - ref) <= store_tol(ref, odt)) and gaps_untouched(out)
    g = blank(V, D, tdt, ld, offset)
    L.embedding_backward(ids.to(DEV), place(dout, ld, offset), g, byte_ws(L.embedding_workspace_bytes(n, V, D)))
    ref, count, mag = ops.embedding_backward(ids.numpy(), f64(dout), V, 1.0)
    assert np.all(np.abs(f64(g) - ref) <= store_tol(ref, tdt) + (count[:, None] + 2) * U * mag) and gaps_untouched(g)


@pytest.mark.parametrize("n,V,D", EMBED)
@pytest.mark.parametrize("odt,gdt", DTYPES)
def test_embedding_backward(L, n, V, D, odt, gdt):
    it = torch.int64 if (n + D) % 2 else torch.int32
    ids = make_ids(n, V, n + 7 * D, it)
    dout = torch.randn((n, D), generator=gen(5)).to(odt)
    scale = np.float64(np.float32(0.3))
    ws = byte_ws(L.embedding_workspace_bytes(n, V, D))
    g = blank(V, D, gdt)
    dids, ddout = ids.to(DEV), place(dout)
    L.embedding_backward(dids, ddout, g, ws, 0.3, padding_idx=1)
    ref, count, mag = ops.embedding_backward(ids.numpy(), f64(dout), V, scale, padding_idx=1)
    tol = (count[:, None] + 2) * U * mag
    assert np.all(np.abs(f64(g) - ref) <= store_tol(ref, gdt) + tol)
    again = blank(V, D, gdt)
    L.embedding_backward(dids, ddout, again, ws, 0.3, padding_idx=1)
    assert torch.equal(g, again)                      # the same inputs give the same bits
    old = torch.randn((V, D), generator=gen(6)).to(gdt)
    acc = place(old)
    L.embedding_backward(dids, ddout, acc, ws, 0.3, padding_idx=1, accumulate=True)
    want = ref + f64(old)
    assert np.all(np.abs(f64(acc) - want) <= store_tol(want, gdt) + tol + 2 * U * (np.abs(f64(old)) + mag))
    assert torch.equal(acc.cpu()[count == 0], old[count == 0])


def test_embedding_rows_past_32_bit_offsets(L):
    V, D = 600_000, 4096                              # 2.46 G elements
    ids = torch.tensor([599_999, 0, 524_288, 599_999, 12, 524_287], dtype=torch.int64)
    table = torch.empty((V, D), dtype=BF, device=DEV)
    rows = torch.randn((6, D), generator=gen(8)).to(BF)
    for i, v in enumerate(ids.tolist()):
        table[v] = rows[i].to(DEV)
    out = torch.empty((6, D), dtype=BF, device=DEV)
    L.embedding_forward(ids.to(DEV), table, out)
    last = {v: i for i, v in enumerate(ids.tolist())}
    assert torch.equal(out.cpu(), rows[[last[v] for v in ids.tolist()]])
    L.embedding_backward(ids.to(DEV), rows.to(DEV), table, byte_ws(L.embedding_workspace_bytes(6, V, D)))
    ref, _, _ = ops.embedding_backward(np.array([0, 1, 2, 0, 3, 4]), f64(rows), 5, 1.0)
    for k, v in enumerate([599_999, 0, 524_288, 12, 524_287]):
        assert np.all(np.abs(f64(table[v]) - ref[k]) <= store_tol(ref[k], BF) + 4 * U * np.abs(f64(rows)).max())
    assert int((table != 0).any(1).sum()) == 5


# ------------------------------------------------------------------------------------------------ layer norm

# widths on either side of every layout's limit, odd ones, one column, one row, and rows too long for registers
LN = [(0, 16), (2, 9), (37, 1021), (9, 1030), (700, 771), (12, 8190), (10, 12001), (6, 16380), (1, 1), (5, 7), (9, 255), (4, 256), (33, 300), (17, 512), (300, 768), (13, 769), (70, 1000), (8, 1023),
      (6, 1024), (11, 1025), (5, 2048), (21, 3000), (40, 4096), (3, 4097), (5, 8192), (3, 10007), (4, 16384),
      (3, 16385), (5, 20000), (2, 65537)]
K_LN = 128 * U


def ln_inputs(N, D, xdt, wdt, seed, offset=0.0):
    g = gen(seed)
    x = (torch.randn((N, D), generator=g) * 2 + torch.randn((N, 1), generator=g) + offset).to(xdt)
    w = (torch.randn(D, generator=g) * 0.2 + 1).to(wdt)
    b = (torch.randn(D, generator=g) * 0.2).to(wdt)
    return x, w, b


def check_ln_forward(x, w, b, eps, y, mean, rstd, ydt):
    ref, rm, rr = ops.layernorm_forward(f64(x), None if w is None else f64(w), None if b is None else f64(b), eps)
    mag = np.abs(f64(x)).mean(1)
    e_mean = K_LN * mag + 1e-37
    assert np.all(np.abs(f64(mean) - rm) <= e_mean)
    # the variance is off by its own sum's error and by the mean's error squared
    e_r = K_LN + 0.5 * (e_mean * rr) ** 2
    assert np.all(np.abs(f64(rstd) - rr) <= e_r * rr)
    wa = np.ones(x.shape[1]) if w is None else np.abs(f64(w))
    xh = np.abs((f64(x) - rm[:, None]) * rr[:, None])
    tol = ((e_mean * rr)[:, None] + (e_r + 4 * U)[:, None] * xh + 2 * U * np.abs(f64(x)) * rr[:, None]) * wa \
        + 4 * U * np.abs(ref) + (0 if b is None else 2 * U * np.abs(f64(b)))
    assert np.all(np.abs(f64(y) - ref) <= store_tol(ref, ydt) + tol)


@pytest.mark.parametrize("N,D", LN)
@pytest.mark.parametrize("xdt,ydt", DTYPES)
def test_layernorm_forward(L, N, D, xdt, ydt):
    wdt = BF if (N + D) % 2 else F
    x, w, b = ln_inputs(N, D, xdt, wdt, N + D)
    y, mean, rstd = blank(N, D, ydt), *(torch.full((N,), float("nan"), device=DEV) for _ in range(2))
    L.layernorm_forward(place(x), w.to(DEV), b.to(DEV), y, mean, rstd, 1e-5)
    check_ln_forward(x, w, b, np.float64(np.float32(1e-5)), y, mean, rstd, ydt)


@pytest.mark.parametrize("N,D", LN)
@pytest.mark.parametrize("xdt,ydt", DTYPES)
def test_layernorm_backward(L, N, D, xdt, ydt):
    wdt, gdt = (BF, F) if (N + D) % 2 else (F, BF)
    x, w, _ = ln_inputs(N, D, xdt, wdt, 3 * N + D)
    dy = torch.randn((N, D), generator=gen(9)).to(ydt)
    _, rm, rr = ops.layernorm_forward(f64(x), None, None, 1e-5)
    mean, rstd = (torch.from_numpy(v).to(F) for v in (rm, rr))
    ws = byte_ws(L.layernorm_workspace_bytes(N, D))
    args = (place(dy), place(x), w.to(DEV), mean.to(DEV), rstd.to(DEV))
    dx = blank(N, D, xdt)
    dw, db = (torch.full((D,), float("nan"), dtype=gdt, device=DEV) for _ in range(2))
    L.layernorm_backward(*args, dx, dw, db, ws)
    rdx, rdw, rdb = ops.layernorm_backward(f64(dy), f64(x), f64(w), f64(mean), f64(rstd))
    xh = (f64(x) - f64(mean)[:, None]) * f64(rstd)[:, None]
    exh = np.abs(xh) + 2 * np.abs(f64(x)) * f64(rstd)[:, None]      # xh's own rounding scales with these
    g = np.abs(f64(dy) * f64(w))
    tol = K_LN * f64(rstd)[:, None] * (g + (g.mean(1) if N else np.zeros(0))[:, None]
                                       + exh * (g * exh).mean(1)[:, None])
    assert np.all(np.abs(f64(dx) - rdx) <= store_tol(rdx, xdt) + tol)
    chain = (200 + N / 64) * U
    ew, eb = chain * (np.abs(f64(dy)) * exh).sum(0), chain * np.abs(f64(dy)).sum(0)
    assert np.all(np.abs(f64(dw) - rdw) <= store_tol(rdw, gdt) + ew)
    assert np.all(np.abs(f64(db) - rdb) <= store_tol(rdb, gdt) + eb)
    # the same inputs, the same bits; without one output or the other; added to what is there
    dx2, dw2 = blank(N, D, xdt), torch.empty_like(dw)
    L.layernorm_backward(*args, dx2, dw2, None, ws)
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)
    db2 = torch.empty_like(db)
    L.layernorm_backward(*args, None, None, db2, ws)
    assert torch.equal(db, db2)
    if N:
        dx2.fill_(float("nan"))
        L.layernorm_backward(*args, dx2, None, None, None)
        assert torch.equal(dx, dx2)
    old = torch.randn(D, generator=gen(10)).to(gdt)
    aw, ab = old.to(DEV), old.to(DEV)
    L.layernorm_backward(*args, dx, aw, ab, ws, accumulate=True)
    for got, ref, e in ((aw, rdw, ew), (ab, rdb, eb)):
        want = ref + f64(old)
        assert np.all(np.abs(f64(got) - want) <= store_tol(want, gdt) + e + 2 * U * (np.abs(f64(old)) + np.abs(ref)))


@pytest.mark.parametrize("ld,offset", [(0, 1), (776, 0), (771, 0), (776, 4), (784, 8)])
@pytest.mark.parametrize("D", [768, 770])
def test_layernorm_strides_alignment_and_missing_weights(L, ld, offset, D):
    N = 37
    x, w, b = ln_inputs(N, D, BF, BF, 11)
    y, mean, rstd = blank(N, D, BF, ld, offset), *(torch.empty(N, device=DEV) for _ in range(2))
    px = place(x, ld, offset)
    for ww, bb in ((w, b), (w, None), (None, b), (None, None)):
        L.layernorm_forward(px, None if ww is None else ww.to(DEV), None if bb is None else bb.to(DEV), y, mean, rstd)
        check_ln_forward(x, ww, bb, np.float64(np.float32(1e-5)), y, mean, rstd, BF)
        assert gaps_untouched(y)
    dense = blank(N, D, BF)
    L.layernorm_forward(px, None, None, dense, None, None)
    assert torch.equal(dense, y)
    dy = torch.randn((N, D), generator=gen(12)).to(BF)
    dx = blank(N, D, BF, ld, offset)
    pdy = place(dy, ld, offset)
    L.layernorm_backward(pdy, px, None, mean, rstd, dx, None, None, None)
    rdx, _, _ = ops.layernorm_backward(f64(dy), f64(x), None, f64(mean), f64(rstd))
    assert np.all(np.abs(f64(dx) - rdx) <= store_tol(rdx, BF) + 1e-4) and gaps_untouched(dx)
    L.layernorm_backward(pdy, px, None, mean, rstd, pdy, None, None, None)     # dx in the place of dy
    assert torch.equal(pdy, dx)
    L.layernorm_forward(px, None, None, px, None, None)                        # y in the place of x
    assert torch.equal(px, y)


@pytest.mark.parametrize("D", [300, 4096, 20000])
def test_layernorm_large_offset_and_constant_rows(L, D):
    """A mean of 500 standard deviations, and rows of one value: the variance is taken around the mean."""
    x, w, b = ln_inputs(6, D, F, F, 13, offset=1000.0)
    x[4:] = 3.25
    y, mean, rstd = blank(6, D, F), *(torch.empty(6, device=DEV) for _ in range(2))
    L.layernorm_forward(place(x), w.to(DEV), b.to(DEV), y, mean, rstd, 1e-3)
    check_ln_forward(x, w, b, np.float64(np.float32(1e-3)), y, mean, rstd, F)


def test_layernorm_nan_stays_in_its_row(L):
    x, w, b = ln_inputs(9, 768, F, F, 14)
    x[4, 100], x[6, 3] = float("nan"), float("inf")
    y, mean, rstd = blank(9, 768, F), *(torch.empty(9, device=DEV) for _ in range(2))
    L.layernorm_forward(place(x), w.to(DEV), b.to(DEV), y, mean, rstd)
    bad = torch.isnan(y).any(1).cpu()
    assert bad.tolist() == [i in (4, 6) for i in range(9)]


@pytest.mark.parametrize("D", [24, 2100])
def test_layernorm_gradients_match_differences(L, D):
    """fp32 gradients along random directions against central differences of the fp64 forward pass: the step of 1e-5
    leaves a relative error below 1e-7 in the difference, and the sums of 7 D terms one of 200 u of their size."""
    N = 7
    x, w, b = ln_inputs(N, D, F, F, 15)
    dy = torch.randn((N, D), generator=gen(16))
    mean, rstd = torch.empty(N, device=DEV), torch.empty(N, device=DEV)
    y, dx = blank(N, D, F), blank(N, D, F)
    dw, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    L.layernorm_forward(place(x), w.to(DEV), b.to(DEV), y, mean, rstd)
    L.layernorm_backward(place(dy), place(x), w.to(DEV), mean, rstd, dx, dw, db,
                         byte_ws(L.layernorm_workspace_bytes(N, D)))
    rng = np.random.default_rng(17)
    f = lambda xx, ww, bb: (ops.layernorm_forward(xx, ww, bb, np.float64(np.float32(1e-5)))[0] * f64(dy)).sum()  # noqa: E731
    X, W, B = f64(x), f64(w), f64(b)
    for got, at in ((dx, 0), (dw, 1), (db, 2)):
        base = [X, W, B]
        d = rng.standard_normal(base[at].shape)
        lo, hi = list(base), list(base)
        lo[at], hi[at] = base[at] - 1e-5 * d, base[at] + 1e-5 * d
        num = (f(*hi) - f(*lo)) / 2e-5
        size = (np.abs(f64(got)) * np.abs(d)).sum()
        assert abs((f64(got) * d).sum() - num) <= 1e-6 * size + 1e-6


# ------------------------------------------------------------------------------------------------ distillation

# N, V, K: one logit; one row; fewer logits than a block's step and more; odd widths; the largest K; more entries than logits
DISTILL = [(0, 10, 2), (1, 1, 1), (3, 5, 4), (7, 100, 1), (5, 1000, 33), (4, 4096, 64), (9, 5003, 20), (2, 32003, 128),
           (1, 50304, 64), (3, 20000, 1024), (200, 700, 8), (1, 128256, 64), (2, 260001, 16), (2, 600011, 16),
           (400, 9001, 40), (3, 420001, 8), (300, 16001, 12), (5, 16384, 700), (9, 31, 5),
           (40, 3001, 1024), (40, 600, 1024), (33, 2000, 200)]


def distill_inputs(N, V, K, zdt, tdt, it, seed):
    g = gen(seed)
    z = (torch.randn((N, V), generator=g) * 3).to(zdt)
    idx = torch.stack([torch.randperm(V, generator=g)[:K] if V >= K else torch.randint(0, V, (K,), generator=g)
                       for _ in range(N)]) if N else torch.zeros((0, K), dtype=torch.int64)
    t = (torch.randn((N, K), generator=g) * 2 + 5).to(tdt)
    for i in range(N):                      # a little of the teacher in the student
        z[i, idx[i]] = (z[i, idx[i]].float() + 0.5 * t[i].float()).to(zdt)
    w = torch.rand(N, generator=g) + 0.25
    if N > 2:
        w[1] = 0.0
    if K > 1 and N:
        idx[N - 1, 0] = -1                  # absent entries
        idx[N // 2, K - 1] = V
        t[N // 2, 0] = -float("inf")
    return z, idx.to(it), t, w


def distill_tols(r, z, idx, t, T, w, V):
    """Bounds on the losses', the stats' and the gradients' fp32 errors of live rows."""
    rel = (V / 512 + 64) * U
    with np.errstate(invalid="ignore"):
        x = np.abs(f64(z) - r["stats"][:, :1]) / T
    x = np.where(np.isfinite(x), x, 0)
    e_l = rel + 8 * U + (r["p"] * (x + 1)).sum(1) * 4 * U + 4 * U * np.abs(r["stats"][:, 1])
    lq = np.where(r["q"] > 0, np.log(np.where(r["q"] > 0, r["q"], 1)), 0)
    terms = (r["q"] * (np.abs(lq) + x + 30 / T)).sum(1)
    e_loss = w * T * T * (e_l + (idx.shape[1] / 512 + 64) * U * terms)
    e_q = 1e-5                              # the teacher's exponents and sum: |t| below 16, at most 1024 entries
    e_d = (r["p"] * (e_l[:, None] + 4 * U * (x + 2)) + r["q"] * e_q) * (w * T)[:, None]
    return e_loss + 1e-37, e_l, e_d + 1e-37


@pytest.mark.parametrize("N,V,K", DISTILL)
@pytest.mark.parametrize("zdt,ddt", DTYPES)
def test_distill(L, N, V, K, zdt, ddt):
    T = [1.0, 2.0, 0.5][(N + V) % 3]
    it, tdt = (torch.int32, F) if (N + K) % 2 else (torch.int64, BF)
    z, idx, t, w = distill_inputs(N, V, K, zdt, tdt, it, N + V + K)
    r = ops.distill(f64(z), idx.numpy(), f64(t), T, f64(w))
    e_loss, e_l, e_d = distill_tols(r, z, idx, t, T, f64(w), V)
    dz_, di, dt_, dw_ = place(z), idx.to(DEV), t.to(DEV), w.to(DEV)
    losses, stats = torch.full((N,), float("nan"), device=DEV), torch.full((N, 2), float("nan"), device=DEV)
    L.distill_forward(dz_, di, dt_, T, dw_, losses, stats)
    assert np.all(np.abs(f64(losses) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    assert np.array_equal(f64(stats)[:, 0], r["stats"][:, 0])
    assert np.all(np.abs(f64(stats)[:, 1] - r["stats"][:, 1]) <= e_l)
    # backward, with a gradient for each row
    up = torch.rand(N, generator=gen(20)) + 0.5
    d = blank(N, V, ddt)
    L.distill_backward(dz_, di, dt_, T, dw_, stats, up.to(DEV), d)
    ref = r["dlogits"] * f64(up)[:, None]
    assert np.all(np.abs(f64(d) - ref) <= store_tol(ref, ddt) + 2 * e_d * f64(up)[:, None])
    # both in one call
    d2, l2, s2 = blank(N, V, ddt), torch.empty(N, device=DEV), torch.empty((N, 2), device=DEV)
    L.distill_forward_backward(dz_, di, dt_, T, dw_, 0.75, l2, s2, d2)
    assert np.all(np.abs(f64(l2) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    assert np.all(np.abs(f64(s2)[:, 1] - r["stats"][:, 1]) <= e_l)
    ref = r["dlogits"] * 0.75
    assert np.all(np.abs(f64(d2) - ref) <= store_tol(ref, ddt) + 2 * e_d)
    d3, l3 = blank(N, V, ddt), torch.empty(N, device=DEV)
    L.distill_forward_backward(dz_, di, dt_, T, dw_, 0.75, l3, s2, d3)
    assert torch.equal(d2, d3) and torch.equal(l2, l3)     # the same inputs give the same bits
    if zdt == ddt:                                          # the gradient in the place of the logits
        zz = place(z)
        L.distill_backward(zz, di, dt_, T, dw_, stats, up.to(DEV), zz)
        assert torch.equal(zz, d)
        zz = place(z)
        L.distill_forward_backward(zz, di, dt_, T, dw_, 0.75, l3, s2, zz)
        assert torch.equal(zz, d2) and torch.equal(l2, l3)
    # weights absent: all 1
    L.distill_forward(dz_, di, dt_, T, None, l2, s2)
    r1 = ops.distill(f64(z), idx.numpy(), f64(t), T)
    e1, _, _ = distill_tols(r1, z, idx, t, T, np.ones(N), V)
    assert np.all(np.abs(f64(l2) - r1["losses"]) <= e1 + 4 * U * np.abs(r1["losses"]))


@pytest.mark.parametrize("ld,offset", [(0, 1), (5008, 0), (5005, 0), (5008, 4), (5016, 8)])
@pytest.mark.parametrize("zdt", [F, BF])
def test_distill_strides_and_alignment(L, ld, offset, zdt):
    N, V, K = 6, 5003, 12
    z, idx, t, w = distill_inputs(N, V, K, zdt, F, torch.int64, 31)
    r = ops.distill(f64(z), idx.numpy(), f64(t), 2.0, f64(w))
    e_loss, e_l, e_d = distill_tols(r, z, idx, t, 2.0, f64(w), V)
    pz, d = place(z, ld, offset), blank(N, V, zdt, ld, offset)
    losses, stats = torch.empty(N, device=DEV), torch.empty((N, 2), device=DEV)
    args = (idx.to(DEV), t.to(DEV), 2.0, w.to(DEV))
    L.distill_forward(pz, *args, losses, stats)
    assert np.all(np.abs(f64(losses) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    L.distill_backward(pz, *args, stats, None, d)
    assert np.all(np.abs(f64(d) - r["dlogits"]) <= store_tol(r["dlogits"], zdt) + 2 * e_d) and gaps_untouched(d)
    d = blank(N, V, zdt, ld, offset)
    L.distill_forward_backward(pz, *args, 1.0, losses, stats, d)
    assert np.all(np.abs(f64(d) - r["dlogits"]) <= store_tol(r["dlogits"], zdt) + 2 * e_d) and gaps_untouched(d)


@pytest.mark.parametrize("V", [700, 40000])
def test_distill_masks_and_special_values(L, V):
    N, K, T = 12, 6, 1.5
    z, idx, t, _ = distill_inputs(N, V, K, F, F, torch.int64, 41)
    idx = torch.stack([torch.randperm(V, generator=gen(42))[:K] for _ in range(N)])
    t = torch.randn((N, K), generator=gen(43))
    low, inf = torch.finfo(F).min, float("inf")
    w = torch.ones(N)
    z[0], w[0] = float("nan"), 0.0                       # padding: its logits do not matter
    z[1], idx[1] = float("nan"), -1                      # no entry: nor do these
    z[2], t[2] = inf, -inf                               # nor these
    half = torch.ones(V, dtype=torch.bool)
    half[::2] = False
    half[idx[3]] = False
    z[3][half] = -inf                                    # masked vocabulary, the teacher's entries kept
    z[4][half & ~torch.isin(torch.arange(V), idx[4])] = low
    z[5][:V // 2] = -inf                                 # whole stretches masked, one teacher entry among them
    idx[5] = torch.arange(V - K, V)
    idx[5, 0], t[5, 0] = 3, -inf
    t[6] = low                                           # the type's lowest value everywhere: equal shares
    idx[7] = idx[7, 0]                                   # one index K times
    idx[8, 1] = idx[8, 4]
    z[9] = low                                           # equal logits
    z[10] = z[10] * 1e30                                 # one logit has all the weight
    idx[10, 0], t[10, 1:] = int(z[10].argmax()), -inf
    z[11] = 12345.0 + z[11] * 0.25                       # large values, small differences
    r = ops.distill(f64(z), idx.numpy(), f64(t), T, f64(w))
    assert np.all(np.isfinite(r["losses"]))
    e_loss, e_l, e_d = distill_tols(r, z, idx, t, T, f64(w), V)
    losses, stats, d = torch.empty(N, device=DEV), torch.empty((N, 2), device=DEV), blank(N, V, F)
    args = (place(z), idx.to(DEV), t.to(DEV), T, w.to(DEV))
    L.distill_forward(*args, losses, stats)
    assert np.all(np.abs(f64(losses) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    assert not f64(stats)[:3].any()
    for joint in (False, True):
        if joint:
            L.distill_forward_backward(*args, 1.0, losses, stats, d)
        else:
            L.distill_backward(*args, stats, None, d)
        assert np.all(np.abs(f64(d) - r["dlogits"]) <= store_tol(r["dlogits"], F) + 2 * e_d)
        assert not f64(d)[:3].any()
    # a teacher entry on a masked logit: infinite loss, finite gradient; a row of nothing else, or a NaN: NaN
    z[3][idx[3, 2]] = -inf
    z[4] = -inf
    z[5][V - 1] = float("nan")
    z[6][5] = inf
    args = (place(z), *args[1:])
    L.distill_forward_backward(*args, 1.0, losses, stats, d)
    got = f64(losses)
    assert got[3] == np.inf and np.isfinite(f64(d)[3]).all()
    assert np.isnan(got[4:7]).all() and np.isnan(f64(d)[4:7]).any(1).all()
    others = [0, 1, 2, 7, 8, 9, 10, 11]
    assert np.isfinite(got[others]).all() and np.isfinite(f64(d)[others]).all()


# V, K and how often a dozen rows are repeated: a multiprocessor has several rows of each of these sizes
@pytest.mark.parametrize("V,K,times", [(700, 6, 850), (1000, 64, 420), (1003, 64, 420), (9001, 33, 110), (14000, 300, 110),
                                       (20011, 64, 60), (33000, 40, 30), (50304, 64, 30), (50303, 1024, 15)])
@pytest.mark.parametrize("zdt,ddt", DTYPES)
def test_distill_many_rows(L, V, K, times, zdt, ddt):
    N, T = 12, 2.0
    z, idx, t, w = distill_inputs(N, V, K, zdt, F, torch.int64, 71)
    z[3], w[3] = float("nan"), 0.0
    z[4], idx[4] = float("inf"), -1
    z[5][K:] = -float("inf")
    idx[5] = torch.arange(K)
    z[5][:K] = torch.arange(K) % 7
    r = ops.distill(f64(z), idx.numpy(), f64(t), T, f64(w))
    e_loss, e_l, e_d = distill_tols(r, z, idx, t, T, f64(w), V)
    args = (idx.to(DEV).repeat(times, 1), t.to(DEV).repeat(times, 1), T, w.to(DEV).repeat(times), 1.0)
    ld = V if V % 8 else V + 8
    buf = torch.full((N * times, ld), float("nan"), dtype=zdt, device=DEV)
    pz = buf[:, :V]
    pz.copy_(z.to(DEV).repeat(times, 1))
    d = torch.full((N * times, ld), float("nan"), dtype=ddt, device=DEV)[:, :V]
    losses, stats = torch.empty(N * times, device=DEV), torch.empty((N * times, 2), device=DEV)
    L.distill_forward_backward(pz, *args, losses, stats, d)
    assert np.all(np.abs(f64(losses[:N]) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    assert np.all(np.abs(f64(stats[:N])[:, 1] - r["stats"][:, 1]) <= e_l)
    assert np.all(np.abs(f64(d[:N]) - r["dlogits"]) <= store_tol(r["dlogits"], ddt) + 2 * e_d) and gaps_untouched(d)
    last = (times - 1) * N                # elsewhere a row may start elsewhere past a boundary, and sum in another order
    assert np.all(np.abs(f64(losses).reshape(times, N) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    for i in (N, last // 2 // N * N, last):
        assert np.all(np.abs(f64(d[i:i + N]) - r["dlogits"]) <= store_tol(r["dlogits"], ddt) + 2 * e_d)
    if zdt == ddt:
        again, s2 = torch.empty_like(losses), torch.empty_like(stats)
        L.distill_forward_backward(pz, *args, again, s2, pz)
        assert torch.equal(pz, d) and torch.equal(again, losses) and torch.equal(s2, stats)


def test_distill_gradient_matches_differences(L):
    """fp32 gradient along a random direction against central differences of the fp64 loss."""
    N, V, K, T = 5, 300, 7, 2.0
    z, idx, t, w = distill_inputs(N, V, K, F, F, torch.int32, 51)
    losses, stats, d = torch.empty(N, device=DEV), torch.empty((N, 2), device=DEV), blank(N, V, F)
    L.distill_forward_backward(place(z), idx.to(DEV), t.to(DEV), T, w.to(DEV), 1.0, losses, stats, d)
    v = np.random.default_rng(52).standard_normal((N, V))
    f = lambda zz: ops.distill(zz, idx.numpy(), f64(t), T, f64(w))["losses"].sum()  # noqa: E731
    num = (f(f64(z) + 1e-5 * v) - f(f64(z) - 1e-5 * v)) / 2e-5
    assert abs((f64(d) * v).sum() - num) <= 1e-5 * (np.abs(f64(d)) * np.abs(v)).sum() + 1e-8


def test_distill_rows_past_32_bit_offsets(L):
    N, V, K = 17000, 128256, 4                            # 2.18 G elements
    z = torch.zeros((N, V), dtype=BF, device=DEV)
    rows = [0, 16743, 16744, N - 1]
    zr, idx4, t4, _ = distill_inputs(4, V, K, BF, F, torch.int32, 61)
    idx, t, w = torch.zeros((N, K), dtype=torch.int32), torch.zeros((N, K)), torch.zeros(N)
    for k, i in enumerate(rows):
        z[i], idx[i], t[i], w[i] = zr[k].to(DEV), idx4[k], t4[k], 1.0
    r = ops.distill(f64(zr), idx4.numpy(), f64(t4), 1.0)
    e_loss, _, e_d = distill_tols(r, zr, idx4, t4, 1.0, np.ones(4), V)
    losses, stats = torch.empty(N, device=DEV), torch.empty((N, 2), device=DEV)
    L.distill_forward_backward(z, idx.to(DEV), t.to(DEV), 1.0, w.to(DEV), 1.0, losses, stats, z)
    assert np.all(np.abs(f64(losses[rows]) - r["losses"]) <= e_loss + 4 * U * np.abs(r["losses"]))
    assert np.all(np.abs(f64(z[rows]) - r["dlogits"]) <= store_tol(r["dlogits"], BF) + 2 * e_d)
    keep = torch.ones(N, dtype=torch.bool)
    keep[rows] = False
    assert not bool(losses[keep.to(DEV)].any()) and not bool(z[1:16743].any()) and not bool(z[16745:N - 1].any())


# ------------------------------------------------------------------------------------------------ streams, graphs

def test_operators_follow_their_stream_and_replay_in_a_graph(L):
    """Inputs made on a side stream, the calls on the same stream; then the same calls captured and replayed on new
    values of the same buffers."""
    n, V, D, K = 300, 97, 64, 5
    s = torch.cuda.Stream()
    ids, idx = make_ids(n, V, 71, torch.int64).to(DEV), torch.randint(0, V, (n, K), generator=gen(72)).to(DEV)
    t = torch.randn((n, K), generator=gen(73)).to(DEV)
    E, h, y, dx, g = (torch.empty(sh, device=DEV) for sh in ((V, D), (n, D), (n, D), (n, D), (V, D)))
    z, mean, rstd, losses, stats = (torch.empty(sh, device=DEV) for sh in ((n, V), (n,), (n,), (n,), (n, 2)))
    dw, db = torch.empty(D, device=DEV), torch.empty(D, device=DEV)
    ews = byte_ws(L.embedding_workspace_bytes(n, V, D))
    lws = byte_ws(L.layernorm_workspace_bytes(n, D))
    zero = torch.zeros(n, V, device=DEV)

    def calls():
        L.embedding_forward(ids, E, h, 2.0)
        L.layernorm_forward(h, None, None, y, mean, rstd)
        z.copy_(zero)
        z[:, :D].copy_(y)
        L.distill_forward_backward(z, idx, t, 1.0, None, 1.0, losses, stats, z)
        L.layernorm_backward(z[:, :D], h, None, mean, rstd, dx, dw, db, lws)
        L.embedding_backward(ids, dx, g, ews, 2.0)

    def reference():
        e = f64(E)
        hh = ops.embedding_forward(ids.cpu().numpy(), e, 2.0)
        yy, m, r = ops.layernorm_forward(hh, None, None, 1e-5)
        zz = np.zeros((n, V))
        zz[:, :D] = yy
        q = ops.distill(zz, idx.cpu().numpy(), f64(t), 1.0)
        rx, _, rb = ops.layernorm_backward(q["dlogits"][:, :D], hh, None, m, r)
        return q["losses"], rb, ops.embedding_backward(ids.cpu().numpy(), rx, V, 2.0)[0]

    def close(got, ref):        # fp32 all the way: 1e-5 of the largest value covers every tolerance above
        return np.max(np.abs(f64(got) - ref)) <= 1e-5 * np.max(np.abs(ref)) + 1e-6

    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)               # the values arrive late on this stream
        E.copy_(torch.randn((V, D), generator=gen(74)).to(DEV))
        calls()
    s.synchronize()
    rl, rb, rg = reference()
    assert close(losses, rl) and close(db, rb) and close(g, rg)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    E.copy_(torch.randn((V, D), generator=gen(75)).to(DEV))
    graph.replay()
    torch.cuda.synchronize()
    rl, rb, rg = reference()
    assert close(losses, rl) and close(db, rb) and close(g, rg)
