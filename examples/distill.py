"""A small language model trained to a teacher's top logits, from token ids to the optimizer step.

Each step looks the tokens up (embedding_forward), goes through residual blocks of layer norm and a two-layer MLP,
takes the loss against the teacher's K kept logits and its gradient in one call in the logits' own memory
(distill_forward_backward), and goes back through layernorm_backward and embedding_backward. The hidden matrices then
take Muon and the table, the head and the norms AdamW, in one HybridMuonAdamW.step(). The matrix products between
are torch's. The teacher is a second model with fixed random weights, its logits cut to the K largest as a stored
teacher's would be.

    python examples/distill.py [--steps 60] [--tokens 2048] [--vocab 2003] [--width 256] [--kept 32]
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

EPS = 1e-5


def first_derivative_only(name):
    """For backward: under create_graph gradients are recorded, and the kernels' would pass for constants."""
    if torch.is_grad_enabled():
        raise RuntimeError(f"{name} has no second derivative")


class Embedding(torch.autograd.Function):
    """scale * table[ids]; the gradient is summed by sorted tokens, the same bits for the same inputs."""

    @staticmethod
    def forward(ctx, ids, table, scale):
        out = torch.empty((ids.numel(), table.shape[1]), dtype=table.dtype, device=table.device)
        L.embedding_forward(ids, table, out, scale)
        ctx.save_for_backward(ids, table)
        ctx.scale = scale
        return out

    @staticmethod
    def backward(ctx, dout):
        first_derivative_only("Embedding")
        ids, table = ctx.saved_tensors
        grad = torch.empty_like(table)
        ws = torch.empty(L.embedding_workspace_bytes(ids.numel(), *table.shape), dtype=torch.uint8, device=table.device)
        L.embedding_backward(ids, dout.contiguous(), grad, ws, ctx.scale)
        return None, grad, None


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        y = torch.empty_like(x)
        mean = torch.empty(x.shape[0], dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
        L.layernorm_forward(x, weight, bias, y, mean, rstd, EPS)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    def backward(ctx, dy):
        first_derivative_only("LayerNorm")
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = torch.empty_like(x), torch.empty_like(weight), torch.empty_like(weight)
        ws = torch.empty(L.layernorm_workspace_bytes(*x.shape), dtype=torch.uint8, device=x.device)
        L.layernorm_backward(dy.contiguous(), x, weight, mean, rstd, dx, dw, db, ws)
        return dx, dw, db


class DistillLoss(torch.autograd.Function):
    """Mean over the rows of weights * T^2 KL(teacher || student). The logits' memory becomes their gradient's, so
    they must be used for nothing else: a leaf is refused, and what another operation has kept of them for its own gradient
    is an error there."""

    @staticmethod
    def forward(ctx, logits, t_idx, t_val, temperature, weights):
        if logits.is_leaf and logits.requires_grad:
            raise RuntimeError("DistillLoss overwrites its logits, which are a leaf that requires a gradient")
        n = logits.shape[0]
        losses = torch.empty(n, dtype=torch.float32, device=logits.device)
        stats = torch.empty((n, 2), dtype=torch.float32, device=logits.device)
        L.distill_forward_backward(logits, t_idx, t_val, temperature, weights, 1.0 / n, losses, stats, logits)
        torch.autograd.graph.increment_version(logits)   # autograd does not see what a kernel writes
        ctx.dlogits = logits.detach()
        return losses.sum() / n

    @staticmethod
    def backward(ctx, upstream):
        first_derivative_only("DistillLoss")
        dlogits, ctx.dlogits = ctx.dlogits, None
        return dlogits.mul_(upstream), None, None, None, None


class Model:
    def __init__(self, vocab, width, blocks, seed, device, trained):
        gen = torch.Generator().manual_seed(seed)

        def matrix(rows, cols, std):
            w = (torch.randn((rows, cols), generator=gen) * std).to(torch.bfloat16)
            return w.to(device).requires_grad_(trained)

        def vector(value):
            return torch.full((width,), value, dtype=torch.bfloat16, device=device).requires_grad_(trained)

        self.table = matrix(vocab, width, 0.02)
        self.head = matrix(vocab, width, 1 / math.sqrt(width))
        self.blocks = [(vector(1.0), vector(0.0), matrix(2 * width, width, 1 / math.sqrt(width)),
                        matrix(width, 2 * width, 0.5 / math.sqrt(width))) for _ in range(blocks)]
        self.norm = (vector(1.0), vector(0.0))

    def logits(self, ids):
        x = Embedding.apply(ids, self.table, math.sqrt(self.table.shape[1]))
        for w, b, up, down in self.blocks:
            x = x + torch.nn.functional.silu(LayerNorm.apply(x, w, b) @ up.t()) @ down.t()
        return LayerNorm.apply(x, *self.norm) @ self.head.t()

    def hidden_matrices(self):
        return [m for block in self.blocks for m in block[2:]]

    def others(self):
        return [self.table, self.head, *self.norm, *(v for block in self.blocks for v in block[:2])]

    def parameters(self):
        return self.hidden_matrices() + self.others()


def train(steps=60, tokens=2048, vocab=2003, width=256, kept=32, temperature=2.0, device="cuda:0"):
    """Returns the loss of every step, and the student."""
    device = torch.device(device)
    student = Model(vocab, width, 2, 1, device, True)
    teacher = Model(vocab, width, 2, 2, device, False)
    opt = HybridMuonAdamW([{"params": student.hidden_matrices(), "kind": "muon", "lr": 0.02},
                           {"params": student.others(), "kind": "adamw", "lr": 3e-3, "weight_decay": 0.0}])
    gen = torch.Generator().manual_seed(3)
    losses = []
    for _ in range(steps):
        # the ids of text are far from uniform; the last sixteenth of the batch is padding
        ids = ((vocab + 1.0) ** torch.rand(tokens, generator=gen)).long().sub_(1).clamp_(0, vocab - 1)
        weights = torch.ones(tokens)
        ids[tokens - tokens // 16:], weights[tokens - tokens // 16:] = -1, 0.0
        ids, weights = ids.to(device), weights.to(device)
        with torch.no_grad():
            t_val, t_idx = teacher.logits(ids).float().topk(kept, dim=1)
        for p in student.parameters():
            p.grad = None
        loss = DistillLoss.apply(student.logits(ids), t_idx, t_val, temperature, weights)
        loss.backward()
        opt.step()
        losses.append(loss.detach())
    return torch.stack(losses).tolist(), student


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, value in (("steps", 60), ("tokens", 2048), ("vocab", 2003), ("width", 256), ("kept", 32)):
        ap.add_argument(f"--{name}", type=int, default=value)
    args = ap.parse_args()
    losses, _ = train(**vars(args))
    for i in range(0, len(losses), max(1, len(losses) // 10)):
        print(f"step {i:4d}  loss {losses[i]:.4f}")
    print(f"step {len(losses) - 1:4d}  loss {losses[-1]:.4f}")


if __name__ == "__main__":
    main()
