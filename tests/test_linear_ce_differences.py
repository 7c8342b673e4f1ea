"""What the check of the linear cross entropy's gradients against differences can tell (test_gpu_linear_ce_differences.py uses it),
by the fp64 oracle. The direction is the gradient's own signs, along which its product with the step is as large as the
tolerance's measure: along random signs it is a hundredth of that, and wrong gradients pass."""
import numpy as np
import pytest
import torch

from oracle import operators as ops

STEP = {"h": 2.0 ** -6, "w": 2.0 ** -8}
# Of the product of gradient and step. The difference's own error is the loss' third derivative along the step, 0.1% here; the
# kernels' losses are off by 1e-6 of themselves, together 1e-4 of the difference or less.
TOLERANCE = 0.01


def inputs(N=120, V=600, D=96, seed=5):
    """Rounded to bf16; one row in five has no part in the loss."""
    gen = torch.Generator().manual_seed(seed)
    h = torch.randn((N, D), generator=gen).to(torch.bfloat16)
    w = (torch.randn((V, D), generator=gen) * 1.5 / D ** 0.5).to(torch.bfloat16)
    t = torch.randint(0, V, (N,), generator=gen)
    t[::5] = -100
    return h, w, t, torch.rand(N, generator=gen) + 0.25


def both_ways(x, gradient, step):
    """x moved by the step along the gradient's signs and against them, in bf16."""
    d = step * torch.sign(gradient).float()
    return (x.float() + d).to(torch.bfloat16), (x.float() - d).to(torch.bfloat16)


def agrees(gradient, difference, ahead, behind):
    """Whether the losses' difference is the gradient's product with the way between the two points."""
    moved = ahead.double() - behind.double()
    return abs(difference - (gradient.double() * moved).sum().item()) <= TOLERANCE * (gradient.double() * moved).abs().sum().item()


def oracle(h, w, t, wt):
    f = lambda x: x.double().numpy()  # noqa: E731
    return ops.linear_cross_entropy(f(h), f(w), t.numpy(), f(wt))


@pytest.mark.parametrize("which", ["h", "w"])
def test_it_tells_wrong_gradients(which):
    h, w, t, wt = inputs()
    ref = oracle(h, w, t, wt)
    live = ref["dz"] != 0
    target = np.zeros_like(ref["dz"])
    rows = np.flatnonzero((t >= 0).numpy())
    target[rows, t.numpy()[rows]] = -f64(wt)[rows]
    assert np.all(live[rows])
    product = lambda dz: torch.from_numpy(dz @ f64(w) if which == "h" else dz.T @ f64(h))  # noqa: E731
    right = product(ref["dz"])
    ahead, behind = both_ways(h if which == "h" else w, right, STEP[which])
    ends = [oracle(x, w, t, wt) if which == "h" else oracle(h, x, t, wt) for x in (ahead, behind)]
    difference = ends[0]["losses"].sum() - ends[1]["losses"].sum()
    moved = ahead.double() - behind.double()
    assert abs(difference / (right * moved).sum().item() - 1.0) < 0.002
    assert agrees(right, difference, ahead, behind)
    for wrong in (-right, 0.5 * right, 3.0 * right, 1.03 * right, product(target), product(ref["dz"] - target),
                  torch.roll(right, 1, 0)):
        assert not agrees(wrong, difference, ahead, behind)


def f64(x):
    return x.double().numpy()
