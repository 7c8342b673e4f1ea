"""The example that runs the operators and the optimizer together: its gradients against the same model in 64 bits, and
its loss over a short run."""
import math

import pytest
import torch
import torch.nn.functional as TF

from tests.gpu_common import DEV, build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    build_lib()
    from examples import distill
    return distill


def reference_grads(ex, m, ids, idx, val, T, w):
    p64 = {id(p): p.detach().double().requires_grad_() for p in m.parameters()}
    g = lambda p: p64[id(p)]  # noqa: E731
    norm = lambda x, w, b: TF.layer_norm(x, x.shape[-1:], g(w), g(b), ex.EPS)  # noqa: E731
    inside = ids >= 0
    x = g(m.table)[ids.clamp(min=0)] * inside[:, None] * math.sqrt(m.table.shape[1])
    for nw, nb, up, down in m.blocks:
        x = x + TF.silu(norm(x, nw, nb) @ g(up).t()) @ g(down).t()
    z = norm(x, *m.norm) @ g(m.head).t()
    q, lp = torch.softmax(val.double() / T, 1), torch.log_softmax(z / T, 1).gather(1, idx)
    loss = (w.double() * T * T * (q * (q.log() - lp)).sum(1)).mean()
    loss.backward()
    return loss.item(), [g(p).grad for p in m.parameters()]


def test_gradients_match_the_model_in_64_bits(example):
    """Activations and their gradients are rounded to bf16 about a dozen times on a path, each 2^-9 of a tensor's norm at
    most: 2.4%, and as much again for what the roundings do to the layers after them."""
    n, V, K, T = 300, 611, 16, 2.0
    m = example.Model(V, 128, 2, 5, DEV, True)
    gen = torch.Generator().manual_seed(6)
    ids = torch.randint(0, V, (n,), generator=gen)
    ids[::9] = -1
    idx = torch.stack([torch.randperm(V, generator=gen)[:K] for _ in range(n)])
    val = torch.randn((n, K), generator=gen) * 3
    w = torch.rand(n, generator=gen)
    w[::9] = 0.0
    ids, idx, val, w = (t.to(DEV) for t in (ids, idx, val, w))
    loss = example.DistillLoss.apply(m.logits(ids), idx, val, T, w)
    loss.backward()
    ref, grads = reference_grads(example, m, ids, idx, val, T, w)
    assert abs(loss.item() - ref) <= 0.01 * ref
    for p, r in zip(m.parameters(), grads):
        assert (p.grad.double() - r).norm() <= 0.05 * r.norm()


def test_training_lowers_the_loss(example):
    losses, model = example.train(steps=40, tokens=1024, vocab=1003, width=128, kept=16)
    assert all(math.isfinite(x) for x in losses)
    assert sum(losses[-5:]) < 0.6 * sum(losses[:5])
    assert all(bool(torch.isfinite(p).all()) for p in model.parameters())
