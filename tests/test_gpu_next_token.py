"""The linear head's cross entropy and AdamW with 8-bit moments as they are used together (examples/next_token.py): the
gradients against the same model in 64 bits, and a run of steps."""
import math

import pytest
import torch
import torch.nn.functional as TF

from tests.gpu_common import DEV, build_lib

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    build_lib()
    from examples import next_token
    return next_token


def test_gradients_match_the_model_in_64_bits(example):
    """As for the distillation example: a dozen roundings to bf16 on a path, 2^-9 of a tensor's norm at most each, and as
    much again for what they do to the layers after them."""
    from examples import distill
    n, V = 300, 611
    m = example.Model(V, 128, 2, 5, DEV, True)
    gen = torch.Generator().manual_seed(6)
    ids, targets = (t.to(DEV) for t in example.batch(n, V, gen))
    w = torch.rand(n, generator=gen).to(DEV)
    loss = example.LinearCrossEntropy.apply(example.hidden(m, ids), m.head, targets, w)
    (2.0 * loss).backward()
    p64 = {id(p): p.detach().double().requires_grad_() for p in m.parameters()}
    g = lambda p: p64[id(p)]  # noqa: E731
    norm = lambda x, a, b: TF.layer_norm(x, x.shape[-1:], g(a), g(b), distill.EPS)  # noqa: E731
    x = g(m.table)[ids] * math.sqrt(m.table.shape[1])
    for nw, nb, up, down in m.blocks:
        x = x + TF.silu(norm(x, nw, nb) @ g(up).t()) @ g(down).t()
    each = TF.cross_entropy(norm(x, *m.norm) @ g(m.head).t(), targets, ignore_index=-100, reduction="none")
    ref = (w.double() * each).sum() / n
    (2.0 * ref).backward()
    assert abs(loss.item() - ref.item()) <= 0.01 * ref.item()
    for p in m.parameters():
        assert (p.grad.double() - g(p).grad).norm() <= 0.05 * g(p).grad.norm()


def test_a_run_of_steps(example):
    losses, model, opt = example.train(steps=8, tokens=700, vocab=1003, width=128)
    assert len(losses) == 8 and all(math.isfinite(x) for x in losses)
    assert all(bool(torch.isfinite(p).all()) for p in model.parameters())
    head = opt.state[model.head]
    assert head["exp_avg"].dtype == head["exp_avg_sq"].dtype == torch.float8_e4m3fn
    assert head["exp_avg_sq"].float().max() > 0


def test_a_second_derivative_is_refused(example):
    h = torch.randn((16, 64), device=DEV).to(torch.bfloat16).requires_grad_()
    w = torch.randn((40, 64), device=DEV).to(torch.bfloat16)
    t = torch.randint(0, 40, (16,), device=DEV)
    with pytest.raises(RuntimeError, match="second derivative"):
        g, = torch.autograd.grad(example.LinearCrossEntropy.apply(h, w, t, None), h, create_graph=True)
        torch.autograd.grad((g * h).sum(), h)
