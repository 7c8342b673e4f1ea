"""LinearCrossEntropy of examples/next_token.py without a GPU, over plain versions of the calls that it makes."""
import pytest
import torch

from examples import next_token as ex

N, V, D = 7, 9, 5


@pytest.fixture(autouse=True)
def calls(monkeypatch):
    """The operators in PyTorch, noted by name and by the gradients that they were asked for."""
    made = []

    def losses_of(h, w, t, weights):
        z = h.detach() @ w.detach().t()
        live = (t >= 0) & (t < w.shape[0])
        lse = torch.where(live, torch.logsumexp(z, 1), torch.zeros(()))
        each = lse - z.gather(1, torch.where(live, t, 0)[:, None])[:, 0]
        wt = torch.where(live, torch.ones(len(t)) if weights is None else weights, torch.zeros(()))
        return z, lse, wt * each * live, wt

    def forward(h, w, t, weights, losses, lse, ws):
        made.append("forward")
        assert not ws[:256].any()
        _, norm, each, _ = losses_of(h, w, t, weights)
        losses.copy_(each), lse.copy_(norm)

    def forward_backward(h, w, t, weights, scale, losses, lse, dh, dw, ws):
        made.append(("dh" if dh is not None else "") + ("dw" if dw is not None else ""))
        assert not ws[:256].any()
        z, norm, each, wt = losses_of(h, w, t, weights)
        losses.copy_(each), lse.copy_(norm)
        dz = torch.softmax(z, 1)
        dz[torch.arange(len(t)), t.clamp(0, w.shape[0] - 1)] -= 1.0
        dz *= (wt * scale)[:, None]
        if dh is not None:
            dh.copy_(dz @ w.detach())
        if dw is not None:
            dw.copy_(dz.t() @ h.detach())

    monkeypatch.setattr(ex.L, "linear_cross_entropy_workspace_bytes", lambda *a: 4096)
    monkeypatch.setattr(ex.L, "linear_cross_entropy_forward", forward)
    monkeypatch.setattr(ex.L, "linear_cross_entropy_forward_backward", forward_backward)
    return made


def case(n=N):
    gen = torch.Generator().manual_seed(2)
    t = torch.randint(0, V, (n,), generator=gen)
    t[::3] = -100
    return (torch.randn((n, D), generator=gen).requires_grad_(), torch.randn((V, D), generator=gen).requires_grad_(), t,
            torch.rand(n, generator=gen) + 0.5)


def reference(h, w, t, weights):
    each = torch.nn.functional.cross_entropy(h @ w.t(), t, ignore_index=-100, reduction="none")
    return (weights * each).sum() / len(t)


def test_gradients_are_those_of_the_plain_loss(calls):
    h, w, t, wt = case()
    got = torch.autograd.grad(3.0 * ex.LinearCrossEntropy.apply(h, w, t, wt), (h, w))
    want = torch.autograd.grad(3.0 * reference(h, w, t, wt), (h, w))
    for x, y in zip(got, want):
        assert torch.allclose(x, y, rtol=1e-5, atol=1e-6)
    assert calls == ["dhdw"]


def test_a_graph_that_is_kept_goes_back_twice():
    h, w, t, wt = case()
    loss = ex.LinearCrossEntropy.apply(h, w, t, wt)
    (2.0 * loss).backward(retain_graph=True)
    loss.backward()
    for x, y in zip((h, w), torch.autograd.grad(3.0 * reference(h, w, t, wt), (h, w))):
        assert torch.allclose(x.grad, y, rtol=1e-5, atol=1e-6)
    with pytest.raises(RuntimeError, match="second time"):
        loss.backward()


def test_only_what_is_wanted_is_computed(calls):
    h, w, t, wt = case()
    for a, b in ((h, w.detach()), (h.detach(), w)):
        want, = torch.autograd.grad(reference(a, b, t, wt), a if a.requires_grad else b)
        got, = torch.autograd.grad(ex.LinearCrossEntropy.apply(a, b, t, wt), a if a.requires_grad else b)
        assert torch.allclose(got, want, rtol=1e-5, atol=1e-6)
    loss = ex.LinearCrossEntropy.apply(h.detach(), w.detach(), t, wt)
    assert not loss.requires_grad and torch.allclose(loss, reference(h, w, t, wt).detach(), rtol=1e-5)
    assert calls == ["dh", "dw", "forward"]


def test_no_rows():
    h, w, t, wt = case(0)
    loss = ex.LinearCrossEntropy.apply(h, w, t, wt)
    loss.backward()
    assert loss.item() == 0.0 and not w.grad.any()


def test_a_second_derivative_is_refused():
    h, w, t, wt = case()
    with pytest.raises(RuntimeError, match="second derivative"):
        g, = torch.autograd.grad(ex.LinearCrossEntropy.apply(h, w, t, wt), h, create_graph=True)
        torch.autograd.grad((g * h).sum(), h)
