"""A small language model trained to predict the next token, without fp32 moments, and without logits beyond a bounded piece.

The model is that of examples/distill.py (embedding lookup, residual blocks of layer norm and a two-layer MLP, a last
norm). Its loss is the cross entropy of the vocabulary head, taken with both gradients in one call from the hidden states
and the head's weights (linear_cross_entropy_forward_backward). The hidden matrices take Muon; the table and the head take
AdamW with moments in 8 bits, the norms' vectors AdamW with fp32 ones, in one HybridMuonAdamW.step().

    python examples/next_token.py [--steps 60] [--tokens 2048] [--vocab 2003] [--width 256]
"""
import argparse
import math
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from adamw_hybrid_optimizer_gb300 import HybridMuonAdamW, libmuon as L  # noqa: E402
from examples.distill import Embedding, LayerNorm, Model, first_derivative_only  # noqa: E402


class LinearCrossEntropy(torch.autograd.Function):
    """Mean over the rows of weights * cross entropy of the head h w^T; targets outside the vocabulary count for nothing. The
    gradients are made with the loss, of those inputs that require one (detach them where no gradient is wanted)."""

    @staticmethod
    def forward(ctx, h, w, targets, weights):
        n, V = h.shape[0], w.shape[0]
        losses, lse = (torch.empty(n, dtype=torch.float32, device=h.device) for _ in range(2))
        dh, dw = (torch.empty_like(x) if wanted else None for x, wanted in zip((h, w), ctx.needs_input_grad))
        some = dh is not None or dw is not None
        ws = torch.empty(L.linear_cross_entropy_workspace_bytes(n, V, h.shape[1], int(some)), dtype=torch.uint8, device=h.device)
        ws[:256].zero_()   # the control block
        if some:
            L.linear_cross_entropy_forward_backward(h, w, targets, weights, 1.0 / max(n, 1), losses, lse, dh, dw, ws)
        else:
            L.linear_cross_entropy_forward(h, w, targets, weights, losses, lse, ws)
        ctx.save_for_backward(dh, dw)
        return losses.sum() / max(n, 1)

    @staticmethod
    def backward(ctx, upstream):
        first_derivative_only("LinearCrossEntropy")
        dh, dw = (None if g is None else g * upstream for g in ctx.saved_tensors)
        return dh, dw, None, None


def hidden(model, ids):
    """The normalised hidden states that the head takes."""
    x = Embedding.apply(ids, model.table, math.sqrt(model.table.shape[1]))
    for w, b, up, down in model.blocks:
        x = x + torch.nn.functional.silu(LayerNorm.apply(x, w, b) @ up.t()) @ down.t()
    return LayerNorm.apply(x, *model.norm)


def batch(tokens, vocab, gen):
    """Ids as rare as those of text, and targets that follow from them two times out of three; the last sixteenth is padding."""
    ids = ((vocab + 1.0) ** torch.rand(tokens, generator=gen)).long().sub_(1).clamp_(0, vocab - 1)
    other = torch.randint(0, vocab, (tokens,), generator=gen)
    targets = torch.where(torch.rand(tokens, generator=gen) < 2 / 3, (ids * 7 + 3) % vocab, other)
    targets[tokens - tokens // 16:] = -100
    return ids, targets


def train(steps=60, tokens=2048, vocab=2003, width=256, device="cuda:0"):
    """Returns the loss of every step, the model and the optimizer."""
    device = torch.device(device)
    model = Model(vocab, width, 2, 1, device, True)
    vectors = [*model.norm, *(v for block in model.blocks for v in block[:2])]
    opt = HybridMuonAdamW([{"params": model.hidden_matrices(), "kind": "muon", "lr": 0.02},
                           {"params": [model.table, model.head], "kind": "adamw", "lr": 3e-3, "weight_decay": 0.0,
                            "state_bits": 8},
                           {"params": vectors, "kind": "adamw", "lr": 3e-3, "weight_decay": 0.0}])
    gen = torch.Generator().manual_seed(3)
    losses = []
    for _ in range(steps):
        ids, targets = (t.to(device) for t in batch(tokens, vocab, gen))
        opt.zero_grad()
        loss = LinearCrossEntropy.apply(hidden(model, ids), model.head, targets, None)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), model, opt


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 60), ("tokens", 2048), ("vocab", 2003), ("width", 256)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    losses, _, _ = train(**vars(args))
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
