"""What moments held in 8 bits do over many steps, by the oracle (oracle/adamw8.py)."""
import numpy as np

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
