"""The example's autograd functions without a GPU, over plain versions of the calls that they make: what autograd has to
be told so that a wrong use is an error and not a wrong gradient."""
import pytest
import torch

from examples import distill as ex


@pytest.fixture(autouse=True)
def plain(monkeypatch):
    """The operators in PyTorch, writing their outputs behind autograd's back as the kernels do."""
    def put(dst, src):
        dst.detach().numpy()[...] = src.detach().numpy()

    def embedding_forward(ids, table, out, scale):
        put(out, scale * table[ids])

    def embedding_backward(ids, dout, grad, ws, scale):
        put(grad, torch.zeros_like(grad).index_add_(0, ids, scale * dout))

    def normed(x, eps):
        mean = x.mean(1)
        rstd = (x.var(1, correction=0) + eps).rsqrt()
        return mean, rstd, (x - mean[:, None]) * rstd[:, None]

    def layernorm_forward(x, weight, bias, y, mean, rstd, eps):
        m, r, xh = normed(x, eps)
        put(mean, m), put(rstd, r), put(y, xh * weight + bias)

    def layernorm_backward(dy, x, weight, mean, rstd, dx, dw, db, ws):
        xh, g = (x - mean[:, None]) * rstd[:, None], dy * weight
        put(dx, rstd[:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True)))
        put(dw, (dy * xh).sum(0)), put(db, dy.sum(0))

    def distill_forward_backward(z, idx, t, T, w, scale, losses, stats, dz):
        q = torch.softmax(t / T, 1)
        lp = torch.log_softmax(z.detach() / T, 1)
        put(losses, w * T * T * (q * (q.log() - lp.gather(1, idx))).sum(1))
        put(dz, (lp.exp().scatter_add(1, idx, -q)) * (scale * w * T)[:, None])

    for f in (embedding_forward, embedding_backward, layernorm_forward, layernorm_backward, distill_forward_backward):
        monkeypatch.setattr(ex.L, f.__name__, f)
    monkeypatch.setattr(ex.L, "embedding_workspace_bytes", lambda *a: 0)
    monkeypatch.setattr(ex.L, "layernorm_workspace_bytes", lambda *a: 0)


N, V, K, D, T = 6, 9, 3, 5, 2.0


def rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed))


def teacher():
    return torch.stack([torch.randperm(V)[:K] for _ in range(N)]), rand(N, K, seed=1), torch.rand(N) + 0.5


def functions():
    """Name -> (a leaf whose gradient is wanted, a scalar of it)."""
    table, x = rand(V, D, seed=2).requires_grad_(), rand(N, D, seed=3).requires_grad_()
    w, b = rand(D, seed=4).requires_grad_(), rand(D, seed=5).requires_grad_()
    z, (idx, t, weights) = rand(N, V, seed=6).requires_grad_(), teacher()
    return {"Embedding": (table, lambda: ex.Embedding.apply(torch.arange(N) % V, table, 2.0).square().sum()),
            "LayerNorm": (x, lambda: ex.LayerNorm.apply(x, w, b).square().sum()),
            "DistillLoss": (z, lambda: ex.DistillLoss.apply(z * 1.0, idx, t, T, weights))}


@pytest.mark.parametrize("name", ["Embedding", "LayerNorm", "DistillLoss"])
def test_a_second_derivative_is_refused(name):
    """The gradients come from kernels, through which no second derivative goes: one that takes them as constants would be
    wrong."""
    leaf, f = functions()[name]
    with pytest.raises(RuntimeError, match="second derivative"):
        grad, = torch.autograd.grad(f(), leaf, create_graph=True)
        torch.autograd.grad((grad * leaf).sum(), leaf)


@pytest.mark.parametrize("name", ["Embedding", "LayerNorm"])
def test_first_derivatives_are_those_of_the_plain_model(name):
    leaf, f = functions()[name]
    got, = torch.autograd.grad(f(), leaf)
    table, x = rand(V, D, seed=2).requires_grad_(), rand(N, D, seed=3).requires_grad_()
    w, b = rand(D, seed=4), rand(D, seed=5)
    ref, of = {"Embedding": ((2.0 * table[torch.arange(N) % V]).square().sum(), table),
               "LayerNorm": (torch.nn.functional.layer_norm(x, (D,), w, b, ex.EPS).square().sum(), x)}[name]
    want, = torch.autograd.grad(ref, of)
    assert torch.allclose(got, want, rtol=1e-4, atol=1e-5)


def test_distill_gradient_is_that_of_the_plain_loss():
    idx, t, weights = teacher()
    z, z2 = (rand(N, V, seed=6).requires_grad_() for _ in range(2))
    got, = torch.autograd.grad(3.0 * ex.DistillLoss.apply(z * 1.0, idx, t, T, weights), z)
    q, lp = torch.softmax(t / T, 1), torch.log_softmax(z2 / T, 1).gather(1, idx)
    want, = torch.autograd.grad(3.0 * (weights * T * T * (q * (q.log() - lp)).sum(1)).mean(), z2)
    assert torch.allclose(got, want, rtol=1e-4, atol=1e-6)


def test_logits_kept_for_another_gradient_are_an_error():
    """The logits' memory holds their gradient after the loss: what another operation had kept of them is gone."""
    idx, t, weights = teacher()
    z = rand(N, V, seed=6).requires_grad_()
    logits = z * 1.0
    other = logits.square().sum()           # keeps the logits for its own gradient
    ex.DistillLoss.apply(logits, idx, t, T, weights)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        other.backward()


def test_logits_that_are_a_leaf_are_refused():
    """A leaf's values would be its own gradient from then on."""
    idx, t, weights = teacher()
    z = rand(N, V, seed=6).requires_grad_()
    before = z.detach().clone()
    with pytest.raises(RuntimeError):
        ex.DistillLoss.apply(z, idx, t, T, weights)
    assert torch.equal(z.detach(), before)
