"""What moments held in 8 bits do over many steps, by the oracle (oracle/adamw8.py)."""
import numpy as np
import pytest

from adamw_hybrid_optimizer_gb300 import HybridMuonAdamW
from adamw_hybrid_optimizer_gb300.optim import ADAMW_DEFAULTS, BETAS8
from oracle import adamw8 as o8

HP = dict(lr=1e-2, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.0)


def run(gradients, beta1=0.9, beta2=0.95, fade=True):
    """Weights, moments held and fp32's, and the mean size of the update over the last half, as they are and in fp32."""
    n = len(gradients[0])
    p, m, r, m32, v32 = (np.zeros(n) for _ in range(5))
    moved, moved32, hp = [], [], dict(HP, beta1=beta1, beta2=beta2)
    weights = []
    for t, g in enumerate(gradients, 1):
        p, m, r = o8.update(p, g, m, r, t, **hp)
        m32, v32 = beta1 * m32 + (1 - beta1) * g, beta2 * v32 + (1 - beta2) * g * g
        if 2 * t > len(gradients):
            moved.append(np.abs(m / (r + 1e-12)).mean())
            moved32.append(np.abs(m32 / (np.sqrt(v32) + 1e-12)).mean())
        codes, s = o8.quantise(m, still=(g == 0) if fade else None)
        m = codes * o8.spread(s, n)
        codes, s = o8.quantise(r, True)
        r = codes * o8.spread(s, n)
        weights.append(p)
    return weights, m, r, m32, np.sqrt(v32), np.mean(moved) / np.mean(moved32)


def normal(n, steps, spread, seed=0):
    rng = np.random.default_rng(seed)
    size = 1e-3 * np.exp(spread * rng.standard_normal(n))
    return [rng.standard_normal(n) * size for _ in range(steps)]


def test_a_moment_without_gradients_ends():
    """Rounded to the nearest code it does not: it stays at a few of the smallest, and its weight goes on, the faster the further
    the root has shrunk (0.003 lr a step after these 400, 0.1 lr after 1700)."""
    g = normal(1024, 500, 0.2)
    for x in g[100:]:
        x[::2] = 0.0
    for fade in (True, False):
        weights, m, _, m32, _, _ = run(g, fade=fade)
        still = np.abs(weights[-1] - weights[-101])[::2]
        assert np.abs(m32[::2]).max() < 1e-15
        if fade:
            assert not m[::2].any() and not still.any()
        else:
            assert m[::2].all() and still.all()


def shrinking(n, steps, spread):
    g = normal(n, steps, spread, seed=1)
    for x in g[steps // 2:]:
        x[::2] *= 0.1
    return g


@pytest.mark.parametrize("spread", [0.0, 0.2, 1.0])
def test_roots_follow_those_of_fp32_up_to_the_limit(spread):
    """Held roots over fp32's: how far rounding to nearest lets them be after 1000 steps, at the largest betas that are taken."""
    for gradients in (normal(2048, 1000, spread), shrinking(2048, 1000, spread)):
        _, _, r, _, r32, update = run(gradients, *BETAS8)
        low, median, high = np.percentile(r / r32, (5, 50, 95))
        assert 0.85 < low and 0.97 < median < 1.12 and high < 1.3 and 0.9 < update < 1.05


def test_beyond_the_limit_they_do_not():
    _, _, r, _, r32, update = run(normal(2048, 1000, 0.0), 0.9, 0.98)
    assert np.median(r / r32) > 1.5 and update < 0.75
    _, _, r, _, r32, _ = run(shrinking(2048, 1000, 0.0), 0.9, 0.98)
    assert np.median((r / r32)[::2]) > 5
    # a first moment: 0.95 of a code that the block's scale does not move is the same code
    g = [np.full(512, 1e-3) for _ in range(300)]
    for x in g[100:]:
        x[::2] = 0.0
    assert run(g, 0.95, 0.95)[1][::2].all() and not run(g, *BETAS8)[1][::2].any()


@pytest.mark.parametrize("betas", [(0.9, 0.96), (0.9, 0.98), (0.9, 0.999), (0.95, 0.95)])
def test_the_optimizer_takes_betas_up_to_the_limit(betas):
    group = {"params": [], "kind": "adamw", "betas": betas}
    with pytest.raises(ValueError, match="betas"):
        HybridMuonAdamW([{**group, "state_bits": 8}])
    HybridMuonAdamW([group])
    opt = HybridMuonAdamW([{**group, "state_bits": 8, "betas": BETAS8}])
    opt.param_groups[0]["betas"] = betas
    with pytest.raises(ValueError, match="betas"):
        opt.step()
    assert opt.param_groups[0]["step"] == 0
    assert all(b <= top for b, top in zip(ADAMW_DEFAULTS["betas"], BETAS8))
