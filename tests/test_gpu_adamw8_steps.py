"""adamw8_step_grouped over many steps: what the held moments do as steps add up."""
import numpy as np
import pytest
import torch

from oracle import adamw8 as o8
from tests.gpu_common import DEV, build_lib, f64
from tests.test_gpu_adamw8 import HP, State, step

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    return build_lib()


@pytest.mark.parametrize("x", [1e-17, 1e-18, 1e-19, 3e-20, 2e-21])
@pytest.mark.parametrize("off", [0, 1])
def test_small_roots_decay(L, x, off):
    """One gradient of x and then none, with an eps below all roots. A block's largest root is held to fp32, so its square, v,
    follows beta2 v from step to step: an fma of relative 2e-6, and the last bit of fp32's subnormal numbers, 2^-149, once for
    the gradient's square (two roundings) and once for the sum. The others lie within half a step of a code. The weights then
    get m / r, off by half of v's relative error."""
    hp = dict(HP, eps=float(np.float32(1e-37)), weight_decay=0.0)
    st = State(700, "f32", "f32", zero=True, seed=3, off=off)
    st.g.copy_(torch.linspace(0.5, 1.0, st.n) * x)
    for t in range(1, 21):
        p0, g, m0, r0 = st.values()
        step(L, [st], t, hp=hp)
        p, m, r = o8.update(p0, g, m0, r0, t, **hp)
        got_p, _, _, got_r = st.values()
        err = 2e-6 + 2 * 2.0 ** -149 / r ** 2                         # of v
        for a in range(0, st.n, o8.BLOCK):
            own = slice(a, min(st.n, a + o8.BLOCK))
            i = a + int(np.argmax(r[own]))
            assert abs(got_r[i] ** 2 - r[i] ** 2) <= err[i] * r[i] ** 2
        assert np.all(got_r > 0)
        assert np.all(np.abs(got_r - r) <= r * (2.0 ** -4 * (1 + err) + err))
        assert np.all(np.abs(got_p - p) <= (2e-6 + err) * np.abs(p - p0) + 2.0 ** -23 * np.abs(p0))
        st.g.zero_()


def moving(t, n, gen):
    """Gradients of step t: sizes of a factor of 1.2 or so around 1e-3, and none for every second element from step 41 on."""
    g = torch.randn(n, generator=gen) * 1e-3 * torch.exp(0.2 * torch.randn(n, generator=torch.Generator().manual_seed(7)))
    if t > 40:
        g[::2] = 0.0
    return g


@pytest.mark.parametrize("pdt,gdt,master,off", [("bf16", "bf16", False, 0), ("bf16", "bf16", False, 1), ("f32", "f32", False, 0),
                                                ("bf16", "f32", True, 0)])
def test_a_moment_without_gradients_ends(L, pdt, gdt, master, off):
    """Beside elements that go on: codes above 2^-6 lose more than half a step (beta1 is 0.9), those below a whole one, at every
    step, so that 18 binades of at most 8 codes each are gone after 18 * 8 steps; the block's scale, of normal gradients, moves too,
    which may put them back by a part of a code. Each step's codes are the oracle's of what was held, to half a step (a whole one
    toward zero). The weights of such elements, without decay, then stay."""
    hp = dict(HP, weight_decay=0.0)
    n = 1100
    st = State(n, pdt, gdt, master, off=off, zero=True, seed=4)
    gen = torch.Generator().manual_seed(5)
    for t in range(1, 361):
        st.g.copy_(moving(t, n, gen))
        before = st.values()
        step(L, [st], t, hp=hp)
        p0, g, m0, r0 = before
        _, m, _ = o8.update(p0, g, m0, r0, t, **hp)
        _, _, got, _ = st.values()
        sm = o8.spread(f64(st.s)[:, 0], n)
        faint = (g == 0) & (np.abs(m) < sm * 2.0 ** -6 * (1 - 1e-6))
        half = np.maximum(np.abs(m) * 2.0 ** -4, sm * 2.0 ** -10) * (1 + 1e-6) + 1e-6 * (np.abs(m0) + np.abs(g))
        assert np.all(np.abs(got - m)[~faint] <= half[~faint])
        lost = np.abs(m) - np.abs(got)
        assert np.all(lost[faint] >= -1e-6 * np.abs(m[faint])) and np.all(lost[faint] <= (sm * 2.0 ** -9 * (1 + 1e-5))[faint])
        if t == 300:
            kept = st.values()[0]
    now, _, m, r = st.values()
    assert not m[::2].any() and (r > 0).all() and m[1::2].any()
    assert np.array_equal(now[::2], kept[::2]) and not np.array_equal(now[1::2], kept[1::2])


@pytest.mark.parametrize("off", [0, 1])
def test_a_block_without_gradients_shrinks_as_one(L, off):
    """Its codes stay, since all of its moments take the same factor; its scales take it, to fp32's rounding (once for the product
    and once for each scaling). Codes are compared as values: a moment of -0 becomes 0."""
    hp = dict(HP, weight_decay=0.0)
    st = State(1000, "bf16", "bf16", seed=6, off=off)
    st.g[256:512] = 0.0
    st.g[900:] = 0.0
    cm, cr = st.m[256:512].float(), st.r[256:512].float()
    for t in range(1, 30):
        s0 = f64(st.s)
        step(L, [st], t, hp=hp)
        assert torch.equal(st.m[256:512].float(), cm) and torch.equal(st.r[256:512].float(), cr)
        s1 = f64(st.s)
        assert np.allclose(s1[1], s0[1] * [HP["beta1"], HP["beta2"] ** 0.5], rtol=4e-7, atol=0)


def test_roots_follow_those_of_fp32(L):
    """400 steps of normal gradients of one size, at the default betas: within the bounds that the oracle keeps over 1000."""
    n = 16384
    st = State(n, "f32", "f32", zero=True, seed=8)
    gen = torch.Generator().manual_seed(9)
    v = np.zeros(n)
    for t in range(1, 401):
        st.g.copy_(torch.randn(n, generator=gen) * 1e-3)
        v = HP["beta2"] * v + (1.0 - HP["beta2"]) * f64(st.g) ** 2
        step(L, [st], t)
    low, median, high = np.percentile(st.values()[3] / np.sqrt(v), (5, 50, 95))
    assert 0.85 < low and 0.97 < median < 1.12 and high < 1.3


@pytest.mark.parametrize("pdt,gdt,master", [("bf16", "bf16", False), ("f32", "f32", False), ("bf16", "f32", True), ("bf16", "f32", False),
                                            ("f32", "bf16", False)])
@pytest.mark.parametrize("l2", [False, True])
def test_alignment_changes_no_bit_of_sparse_and_small_gradients(L, pdt, gdt, master, l2):
    """Full aligned blocks and single elements go different ways, and bf16 blocks branch where a scale is small or some element
    has no gradient: the same bits."""
    n = 3000
    a, b = (State(n, pdt, gdt, master, off=o, zero=True, seed=10) for o in (0, 1))
    gen = torch.Generator().manual_seed(11)
    size = torch.ones(n) * 1e-3
    size[256:1100] = 1e-21          # roots whose square fp32 holds, of scales whose square it does not
    size[1100:1400] = 1e-17
    for t in range(1, 41):
        g = torch.randn(n, generator=gen) * size
        g[torch.rand(n, generator=gen) < (0.0, 0.1, 0.9)[t % 3]] = 0.0
        g[512:768] = 0.0 if t % 2 else g[512:768]
        for s in (a, b):
            s.g.copy_(g)
            step(L, [s], t, l2=l2)
    for x, y in zip(a.bits(), b.bits()):
        assert torch.equal(x, y)
