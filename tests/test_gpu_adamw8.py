"""adamw8_step_grouped on the GPU against the fp64 oracle (oracle/adamw8.py).

Tolerances. m and v are sums of two products, each rounded once to fp32, then r = sqrt(v): with u = 2^-24 the errors are at most
3 u of the terms' magnitudes for m and 4 u of r. A code is off from the exact moment by half a step: 2^-4 of the value, or
2^-10 of the scale below 2^-6, and the fp32 errors of the moment and of the scaling (3 u) on top: 1e-6 of the terms covers them.
The weights get lr * m / r with a few roundings each (1e-6 of the update's size) and one rounding of their own."""
import numpy as np
import pytest
import torch

from oracle import adamw8 as o8
from tests.gpu_common import DEV, build_lib, f64

pytestmark = pytest.mark.gpu
HP = dict(lr=float(np.float32(1e-2)), beta1=float(np.float32(0.9)), beta2=float(np.float32(0.95)), eps=float(np.float32(1e-8)),
          weight_decay=float(np.float32(0.1)))
F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def L():
    return build_lib()


def blocks(n):
    return (n + o8.BLOCK - 1) // o8.BLOCK


class State:
    """One tensor and its state; `off` puts every array that many elements past a 16-byte boundary."""

    def __init__(self, n, pdt="bf16", gdt="bf16", master=False, off=0, seed=0, zero=False):
        gen = torch.Generator().manual_seed(1000 + seed)

        def place(x, pad=off):
            buf = torch.zeros(n + 32, dtype=torch.float32).to(x.dtype) if x.dtype != F8 else torch.zeros(
                n + 32, dtype=torch.uint8).view(F8)
            buf = buf.to(DEV)
            buf.view(torch.uint8)[pad * x.element_size():(pad + n) * x.element_size()] = x.to(DEV).view(torch.uint8)
            return buf[pad:pad + n]

        rnd = lambda: torch.randn(n, generator=gen, dtype=torch.float64)  # noqa: E731
        size = torch.exp(2.0 * rnd()) * 1e-3
        self.n = n
        self.w64 = rnd() * 0.1
        self.p = place(self.w64.to(DT[pdt]))
        self.master = place(self.w64.float()) if master else None
        self.g = place((rnd() * size).to(DT[gdt]))
        m, r = (np.zeros(n), np.zeros(n)) if zero else ((rnd() * size * 0.3).numpy(), size.numpy())
        (cm, sm), (cr, sr) = o8.quantise(m), o8.quantise(r, True)
        self.m, self.r = (place(torch.from_numpy(c).float().to(F8)) for c in (cm, cr))
        s = np.zeros((blocks(n), 2)) if zero else np.stack([sm, sr], 1)
        self.s = torch.from_numpy(s).float().to(DEV)

    def spec(self, hp):
        return (self.p, self.g, self.m, self.r, self.s, hp) + ((self.master,) if self.master is not None else ())

    def values(self):
        s = f64(self.s)
        return (f64(self.master if self.master is not None else self.p), f64(self.g),
                f64(self.m.float()) * o8.spread(s[:, 0], self.n), f64(self.r.float()) * o8.spread(s[:, 1], self.n))

    def bits(self):
        out = [self.p, self.m, self.r, self.s] + ([self.master] if self.master is not None else [])
        return [t.contiguous().view(torch.uint8).clone() for t in out]


def step(L, states, t=3, l2=False, hp=HP):
    h = L.make_adamw_hparams(hp["lr"], hp["beta1"], hp["beta2"], hp["eps"], hp["weight_decay"], t, l2)
    L.adamw8_step_grouped(L.make_adamw8_tensors([s.spec(h) for s in states]))
    torch.cuda.synchronize()


def check(state, before, t=3, l2=False, hp=HP):
    p0, g, m0, r0 = before
    p, m, r = o8.update(p0, g, m0, r0, t, l2=l2, **hp)
    gm = np.abs(g) + (hp["weight_decay"] * np.abs(p0) if l2 else 0.0)
    got_p, _, got_m, got_r = state.values()
    s = f64(state.s)
    sm, sr = o8.spread(s[:, 0], state.n), o8.spread(s[:, 1], state.n)
    for k, x, terms in ((0, m, np.abs(m0) + gm), (1, r, r0 + gm)):
        for b in range(blocks(state.n)):
            at = slice(b * o8.BLOCK, (b + 1) * o8.BLOCK)
            top = max(np.abs(x[at]).max(), o8.FLOOR)
            assert abs(s[b, k] * o8.TOP - top) <= 1e-6 * max(terms[at].max(), o8.FLOOR)
    half = lambda x, sc: np.maximum(np.abs(x) * 2.0 ** -4, sc * 2.0 ** -10)  # noqa: E731
    assert np.all(np.abs(got_m - m) <= half(m, sm) * (1 + 1e-6) + 1e-6 * (np.abs(m0) + gm))
    least = np.where(r > 0, sr * o8.LEAST, 0.0)        # a root above zero is held as the smallest code at least
    assert np.all((np.abs(got_r - r) <= half(r, sr) * (1 + 1e-6) + 1e-6 * (r0 + gm)) | ((got_r == least) & (r < least)))
    assert np.all(got_r[r > sr * 1e-30] > 0)
    upd = np.abs(p - p0) + hp["lr"] * (np.abs(m0) + gm) / (r + hp["eps"])
    tol = 2e-6 * upd + 2.0 ** -23 * np.abs(p0)
    if state.master is not None:
        assert torch.equal(state.p, state.master.to(torch.bfloat16))
    elif state.p.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(p)
    assert np.all(np.abs(got_p - p) <= tol)


@pytest.mark.parametrize("n", [1, 7, 31, 255, 256, 257, 511, 1000, 4096, 70001])
@pytest.mark.parametrize("pdt,gdt,master", [("bf16", "bf16", False), ("f32", "f32", False), ("bf16", "f32", True)])
@pytest.mark.parametrize("l2", [False, True])
def test_one_tensor(L, n, pdt, gdt, master, l2):
    st = State(n, pdt, gdt, master, seed=n)
    before = st.values()
    step(L, [st], l2=l2)
    check(st, before, l2=l2)


@pytest.mark.parametrize("pdt,gdt,master", [("bf16", "f32", False), ("f32", "bf16", False), ("bf16", "bf16", True)])
def test_the_other_types(L, pdt, gdt, master):
    st = State(5003, pdt, gdt, master, seed=4)
    before = st.values()
    step(L, [st])
    check(st, before)


@pytest.mark.parametrize("pdt,gdt,master", [("bf16", "bf16", False), ("f32", "f32", False), ("bf16", "f32", True)])
@pytest.mark.parametrize("off", [1, 2, 4, 5])
def test_alignment_changes_no_bit(L, pdt, gdt, master, off):
    a, b = (State(3000, pdt, gdt, master, off=o, seed=9) for o in (0, off))
    for t in (1, 2, 3):
        step(L, [a], t)
        step(L, [b], t)
    for x, y in zip(a.bits(), b.bits()):
        assert torch.equal(x, y)


def test_many_tensors_are_as_many_calls(L):
    """More than a launch takes, of all types and lengths, and what lies around them stays."""
    kinds = [("bf16", "bf16", False), ("f32", "f32", False), ("bf16", "f32", True), ("f32", "bf16", False)]
    lens = [1 + (i * i * 37) % 2500 for i in range(210)] + [300001]
    make = lambda: [State(n, *kinds[i % 4], off=(i % 3) * 4, seed=i) for i, n in enumerate(lens)]  # noqa: E731
    together, alone = make(), make()
    for t in (1, 2):
        step(L, together, t)
        for s in alone:
            step(L, [s], t)
    for s, a in zip(together, alone):
        for x, y in zip(s.bits(), a.bits()):
            assert torch.equal(x, y)


def test_from_zero_over_many_steps(L):
    """The first step from all zeros, then twenty with new gradients: each step against the oracle from the state held."""
    st = State(1300, "f32", "f32", zero=True, seed=5)
    gen = torch.Generator().manual_seed(6)
    for t in range(1, 21):
        st.g.copy_(torch.randn(st.n, generator=gen) * 10.0 ** (t % 5 - 4))
        before = st.values()
        step(L, [st], t)
        check(st, before, t)


def test_blocks_of_zeros_and_tiny_values(L):
    st = State(1024, "f32", "f32", zero=True, seed=7)
    st.g.zero_()
    st.g[256:512] = 1e-30
    st.g[512:768] = 1e-12
    st.g[768] = 1.0                         # one large element among zeros
    st.g[900] = 1e-9                        # and one that the block's scale leaves at the smallest code
    before = st.values()
    step(L, [st], 1)
    p, m, r = o8.update(*before, 1, **HP)
    got_p, _, got_m, got_r = st.values()
    assert np.isfinite(got_p).all() and np.isfinite(got_m).all() and np.isfinite(got_r).all()
    assert not got_m[:256].any() and not got_r[:256].any()
    assert (got_r[512:768] > 0).all() and got_r[900] == f64(st.s)[3, 1] * o8.LEAST
    assert np.all(np.abs(got_p - p) <= 1e-6 * (np.abs(before[0]) + HP["lr"]))


def test_not_finite_stays_with_its_element(L):
    good, bad = State(800, "f32", "f32", seed=8), State(800, "f32", "f32", seed=8)
    at = [3, 290, 511, 799]
    for s in (good, bad):
        s.g[at] = 0.0
        s.m.view(torch.uint8)[at] = 0
        s.r.view(torch.uint8)[at] = 0
    for i, v in zip(at, (float("nan"), float("inf"), -float("inf"), 1e30)):
        bad.g[i] = v
    for t in (1, 2):
        step(L, [good], t)
        step(L, [bad], t)
    gp, _, gm, gr = good.values()
    p, _, m, r = bad.values()
    for i in at[:3]:
        assert np.isnan(m[i]) and np.isnan(r[i]) and np.isnan(p[i])
    assert np.isfinite(m[799]) and np.isnan(r[799])   # 1e30 squared is not finite
    other = np.ones(800, bool)
    other[at] = False
    for x, y in ((gp, p), (gm, m), (gr, r)):
        assert np.array_equal(x[:512][other[:512]], y[:512][other[:512]])
    # in the last block the large first moment sets the scale
    assert np.isfinite(m[other]).all() and np.isfinite(r[other]).all() and np.isfinite(p[other]).all()


def test_another_stream_and_a_captured_call(L):
    a, b = State(5000, seed=11), State(5000, seed=11)
    h = L.make_adamw_hparams(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], 5)
    ts = L.make_adamw8_tensors([a.spec(h)])
    for _ in range(3):
        L.adamw8_step_grouped(ts)
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    tb = L.make_adamw8_tensors([b.spec(h)])
    L.adamw8_step_grouped(tb, stream=other)
    other.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=other):
        L.adamw8_step_grouped(tb)
    graph.replay()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip(a.bits(), b.bits()):
        assert torch.equal(x, y)


def test_long_tensor_offsets(L):
    """Elements beyond 2^31: the last block of a tensor of 2^31 + 1000 elements is updated as a short tensor's is."""
    n, tail = (1 << 31) + 1000, 1000
    one = State(tail, "bf16", "bf16", seed=12)
    p, g = (torch.zeros(n, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    m, r = (torch.zeros(n, dtype=torch.uint8, device=DEV).view(F8) for _ in range(2))
    s = torch.zeros((blocks(n), 2), dtype=torch.float32, device=DEV)
    p[-tail:], g[-tail:] = one.p, one.g
    m.view(torch.uint8)[-tail:], r.view(torch.uint8)[-tail:] = one.m.view(torch.uint8), one.r.view(torch.uint8)
    s[-blocks(tail):] = one.s
    h = L.make_adamw_hparams(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], 3)
    L.adamw8_step_grouped(L.make_adamw8_tensors([(p, g, m, r, s, h)]))
    step(L, [one], 3)
    assert torch.equal(p[-tail:], one.p) and torch.equal(s[-blocks(tail):], one.s)
    assert torch.equal(m.view(torch.uint8)[-tail:], one.m.view(torch.uint8))
    assert torch.equal(r.view(torch.uint8)[-tail:], one.r.view(torch.uint8))
    assert not p[:-tail].any() and not m.view(torch.uint8)[:-tail].any()
