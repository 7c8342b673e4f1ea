"""Timed cases of what trains the vocabulary head without its two largest arrays: the cross entropy of a linear head, whose
logits are never kept, with its gradients, and the AdamW step of many tensors whose moments are held in 8 bits.

With ``own`` false, ``run`` computes a case in elementary torch operations in 32 bits; with ``own`` true it makes the
library's calls. Sizes come from the optimizer's workloads (width 768 with a vocabulary of 50304, width 4096 with
128256), beside odd ones.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}
BLOCK = 256                 # elements that share a scale of their moments
TOP = 448.0                 # the largest e4m3 value, where a block's largest moment lies
LEAST = 2.0 ** -9           # the smallest e4m3 value above zero
FLOOR = 2.0 ** -100         # a block whose moments are all smaller is scaled as if this were its largest
HP = dict(lr=3e-4, beta1=0.9, beta2=0.95, eps=1e-8, weight_decay=0.1, step=1000)


def listed():
    return [
        # the loss of eight positions on the small model's head (an evaluation of short answers): latency, and the
        # head's weights read once
        dict(name="head_fwd_few", op="head_fwd", N=8, V=50304, D=768, idt="i64"),
        # an evaluation batch on the wide model
        dict(name="head_fwd_4096", op="head_fwd", N=4096, V=128256, D=4096, idt="i64"),
        # a small model's training batch: loss and gradients in one call
        dict(name="head_step_768", op="head_step", N=8192, V=50304, D=768, gdt="bf16", idt="i64"),
        # the wide model's training batch
        dict(name="head_step_4096", op="head_step", N=4096, V=128256, D=4096, gdt="bf16", idt="i32"),
        # few positions of a long vocabulary (the answers of a tuning set): the weights' gradient is most of what moves
        dict(name="head_step_few", op="head_step", N=200, V=128256, D=2048, gdt="bf16", idt="i32"),
        # the gradients alone, from the forward pass's normalisers and a gradient for each row; nothing is a multiple
        # of a tile
        dict(name="head_bwd_odd", op="head_bwd", N=1001, V=32003, D=1000, gdt="bf16", idt="i64"),
        # a model's vectors (norms, biases): many short tensors of odd lengths, latency alone
        dict(name="adamw8_vectors", op="adamw8", many=72, n=768, few=0, big=0, pdt="bf16", gdt="bf16", master=False,
             l2=False),
        # the small model's table, head and norms
        dict(name="adamw8_768", op="adamw8", many=24, n=768, few=2, big=50304 * 768, pdt="bf16", gdt="bf16",
             master=False, l2=False),
        # the same, fp32 throughout, with L2 instead of decoupled decay
        dict(name="adamw8_f32", op="adamw8", many=24, n=768, few=2, big=50257 * 768, pdt="f32", gdt="f32", master=False,
             l2=True),
        # a head of 32003 x 1001 kept with fp32 master weights, and fp32 gradients
        dict(name="adamw8_master", op="adamw8", many=7, n=1001, few=1, big=32003 * 1001, pdt="bf16", gdt="f32",
             master=True, l2=False),
        # the wide model's table and head: 1.05 G elements
        dict(name="adamw8_4096", op="adamw8", many=65, n=4096, few=2, big=128256 * 4096, pdt="bf16", gdt="bf16",
             master=False, l2=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = {kind: max(_cost(c) for c in listed() if c["op"].startswith(kind)) for kind in ("head", "adamw8")}
    while True:
        if rng.random() < 0.6:
            # rows start on 16-byte boundaries: the width's pitch is a multiple of 8, the width need not be
            c = dict(op=rng.choice(["head_fwd", "head_bwd", "head_step"]), N=_log(rng, 1, 16384),
                     V=rng.choice([50304, 128256, _log(rng, 1000, 260000)]),
                     D=rng.choice([768, 4096, 8 * _log(rng, 8, 768), _log(rng, 65, 6000)]), idt=rng.choice(["i32", "i64"]))
            if c["op"] != "head_fwd":
                c["gdt"] = "bf16"
            if _cost(c) <= most["head"] and c["N"] * c["V"] <= 1 << 29:
                return c
        else:
            c = dict(op="adamw8", many=_log(rng, 1, 200), n=_log(rng, 1, 20000), few=rng.choice([0, 1, 2, 3]),
                     big=_log(rng, 20000, 500000000), pdt=rng.choice(["bf16", "bf16", "f32"]),
                     gdt=rng.choice(["bf16", "bf16", "f32"]), master=rng.random() < 0.3, l2=rng.random() < 0.3)
            if c["master"]:
                c["pdt"] = "bf16"
            if _cost(c) <= most["adamw8"]:
                return c


def _lengths(c):
    """Lengths of the tensors: the few long ones, and the many short ones, of which no two are alike."""
    return [c["big"]] * c["few"] + [c["n"] + i for i in range(c["many"])]


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 280)


def work(c):
    if c["op"] == "adamw8":
        p, g = SIZE[c["pdt"]], SIZE[c["gdt"]]
        each = (8 + p if c["master"] else 2 * p) + g + 4       # weights read and written, gradient, two codes each way
        lens = _lengths(c)
        blocks = sum((n + BLOCK - 1) // BLOCK for n in lens)
        return {"bytes": sum(lens) * each + 16 * blocks, "flops": 16 * sum(lens)}
    N, V, D = c["N"], c["V"], c["D"]
    moved = 2 * D * (N + V) + N * (SIZE[c["idt"]] + 4)
    if c["op"] == "head_fwd":
        return {"bytes": moved + 8 * N, "flops": 2 * N * V * D}
    # the logits' product and the two of the gradients, whichever form
    return {"bytes": moved + 8 * N + SIZE[c["gdt"]] * D * (N + V), "flops": 6 * N * V * D}


def _ids(n, V, g):
    """Token ids as text has them: the id of rank r with a probability of about 1 / r, ranks spread over the ids."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    rank = torch.clamp(torch.floor(torch.exp(u * math.log(V + 1.0))).to(torch.int64) - 1, 0, V - 1)
    step = 7919
    while math.gcd(step, V) != 1:
        step += 2
    return (rank * step + 13) % V


def _pitched(rows, cols, dt):
    """A matrix whose rows start on 16-byte boundaries."""
    per = 16 // SIZE[dt]
    return torch.empty((rows, (cols + per - 1) // per * per), dtype=DT[dt], device=DEV)[:, :cols]


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return _prepare_adamw8(c, g) if c["op"] == "adamw8" else _prepare_head(c, g)


def _prepare_head(c, g):
    s = dict(c)
    N, V, D = c["N"], c["V"], c["D"]
    W = torch.randn((V, D), generator=g, device=DEV) * (1.5 / math.sqrt(D))
    t = _ids(N, V, g)
    # the hidden states of a model that has learned part of its task: normalised rows that lean towards the target's
    h = torch.randn((N, D), generator=g, device=DEV)
    h += W[t] * (2.0 * torch.rand((N, 1), generator=g, device=DEV))
    s["w"], s["h"] = _pitched(V, D, "bf16"), _pitched(N, D, "bf16")
    s["w"].copy_(W)
    s["h"].copy_(h)
    # one position in twenty is padding, which a weight of zero or a target outside the vocabulary marks
    keep = torch.rand(N, generator=g, device=DEV)
    s["weights"] = (keep >= 0.03).float() / N
    s["targets"] = torch.where((keep >= 0.03) & (keep < 0.05), torch.full_like(t, -100), t).to(
        torch.int32 if c["idt"] == "i32" else torch.int64)
    s["losses"], s["lse"] = (torch.empty(N, dtype=torch.float32, device=DEV) for _ in range(2))
    if c["op"] != "head_fwd":
        s["dh"], s["dw"] = _pitched(N, D, c["gdt"]), _pitched(V, D, c["gdt"])
    if c["op"] == "head_bwd":
        # what the forward pass left, and the gradient that reaches each row's loss
        wf = s["w"].float()
        for i in range(0, N, 2048):
            s["lse"][i:i + 2048] = torch.logsumexp(s["h"][i:i + 2048].float() @ wf.t(), 1)
        s["lse"].masked_fill_(keep < 0.05, 0.0)
        s["grad"] = torch.rand(N, generator=g, device=DEV) + 0.5
    return s


def _prepare_adamw8(c, g):
    s = dict(c)
    lens = _lengths(c)
    starts = np.cumsum([0] + [(n + BLOCK - 1) // BLOCK * BLOCK for n in lens])
    total = int(starts[-1])
    s["spans"] = [(int(a), n) for a, n in zip(starts, lens)]
    inside = torch.zeros(total, dtype=torch.bool, device=DEV)   # what lies between the tensors belongs to none
    for a, n in s["spans"]:
        inside[a:a + n] = True

    def normal(std):
        return (torch.randn(total, generator=g, device=DEV) * std).mul_(inside)

    # gradients of one element differ from those of another by powers of ten; the moments are those of earlier ones
    size = torch.exp(normal(1.0)).mul_(1e-3)
    s["grad"] = normal(1.0).mul_(size).to(DT[c["gdt"]])
    m, r = normal(0.3).mul_(size), size.mul_(inside)
    del size
    w = normal(0.05 if c["pdt"] == "bf16" else 1.0)
    s["param"] = w.to(DT[c["pdt"]])
    s["master"] = w if c["master"] else None
    s["scales"] = torch.empty((total // BLOCK, 2), dtype=torch.float32, device=DEV)
    for k, (name, x) in enumerate((("exp_avg", m), ("exp_avg_sq", r))):
        x = x.view(-1, BLOCK)
        scale = x.abs().amax(1).clamp_(min=FLOOR) / TOP
        s["scales"][:, k] = scale
        s[name] = (x / scale[:, None]).clamp_(-TOP, TOP).to(torch.float8_e4m3fn).view(-1)
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from adamw_hybrid_optimizer_gb300 import libmuon as L
    op = s["op"]
    if op == "adamw8":
        if "call" not in s:
            hp = L.make_adamw_hparams(HP["lr"], HP["beta1"], HP["beta2"], HP["eps"], HP["weight_decay"], HP["step"],
                                      s["l2"])
            part = lambda name, a, n: s[name][a:a + n]  # noqa: E731
            specs = [(part("param", a, n), part("grad", a, n), part("exp_avg", a, n), part("exp_avg_sq", a, n),
                      s["scales"][a // BLOCK:(a + n + BLOCK - 1) // BLOCK], hp)
                     + ((part("master", a, n),) if s["master"] is not None else ()) for a, n in s["spans"]]
            s["call"] = L.make_adamw8_tensors(specs)
        L.adamw8_step_grouped(s["call"])
        return _adamw8_outputs(s)
    if "ws" not in s:
        terms = 0 if op == "head_fwd" else 1 if s["gdt"] == "bf16" else 2
        s["ws"] = torch.zeros(L.linear_cross_entropy_workspace_bytes(s["N"], s["V"], s["D"], terms), dtype=torch.uint8,
                              device=DEV)
    if op == "head_fwd":
        L.linear_cross_entropy_forward(s["h"], s["w"], s["targets"], s["weights"], s["losses"], s["lse"], s["ws"])
        return {"losses": s["losses"], "lse": s["lse"]}
    if op == "head_bwd":
        L.linear_cross_entropy_backward(s["h"], s["w"], s["targets"], s["weights"], s["lse"], s["grad"], s["dh"],
                                        s["dw"], s["ws"])
        return {"dh": s["dh"], "dw": s["dw"]}
    L.linear_cross_entropy_forward_backward(s["h"], s["w"], s["targets"], s["weights"], 1.0, s["losses"], s["lse"],
                                            s["dh"], s["dw"], s["ws"])
    return {"losses": s["losses"], "lse": s["lse"], "dh": s["dh"], "dw": s["dw"]}


def _adamw8_outputs(s):
    """The codes as the 8-bit values that they are, beside their scales."""
    out = {k: s[k] for k in ("param", "exp_avg", "exp_avg_sq", "scales")}
    if s["master"] is not None:
        out["master"] = s["master"]
    return out


def _plain(s):
    return _plain_adamw8(s) if s["op"] == "adamw8" else _plain_head(s)


def _plain_head(s):
    op, N = s["op"], s["N"]
    h, w = s["h"].float(), s["w"].float()
    t = s["targets"].long()
    live = (t >= 0) & (t < s["V"]) & (s["weights"] != 0)
    at = torch.where(live, t, 0)[:, None]
    z = h @ w.t()
    if op == "head_bwd":
        lse, scale = s["lse"], s["grad"] * s["weights"]
    else:
        top = z.max(1, keepdim=True).values
        lse = (top + torch.exp(z - top).sum(1, keepdim=True).log())[:, 0]
        losses = torch.where(live, s["weights"] * (lse - z.gather(1, at)[:, 0]), 0.0)
        lse, scale = torch.where(live, lse, 0.0), s["weights"]
        if op == "head_fwd":
            return {"losses": losses, "lse": lse}
    p = torch.exp(z.sub_(lse[:, None]))
    p.scatter_add_(1, at, torch.full((N, 1), -1.0, device=DEV))
    dz = torch.where(live[:, None], p * scale[:, None], 0.0)
    dh, dw = (dz @ w).to(DT[s["gdt"]]), (dz.t() @ h).to(DT[s["gdt"]])
    return {"dh": dh, "dw": dw} if op == "head_bwd" else {"losses": losses, "lse": lse, "dh": dh, "dw": dw}


def _constants(l2):
    """The step's constants as floats, from hyperparameters that are floats."""
    f = np.float32
    lr, b1, b2, wd = (float(f(HP[k])) for k in ("lr", "beta1", "beta2", "weight_decay"))
    bc1, bc2 = 1.0 - b1 ** HP["step"], 1.0 - b2 ** HP["step"]
    return (b1, float(f(1.0 - b1)), b2, float(f(1.0 - b2)), 1.0 if l2 else float(f(1.0 - lr * wd)), wd if l2 else 0.0,
            float(f(lr / bc1)), float(f(1.0 / math.sqrt(bc2))), float(f(HP["eps"])))


def _fma(a, b, c):
    """a * b + c in 32 bits with one rounding (the product of two floats is exact in 64 bits): a moment next to the border
    between two codes has to come out on one side."""
    return (a.double() * b.double()).add_(c).float()


def _plain_adamw8(s):
    b1, omb1, b2, omb2, decay, l2_wd, step, ibc2, eps = _constants(s["l2"])
    w = s["master"] if s["master"] is not None else s["param"]
    p, g = w.float().view(-1, BLOCK), s["grad"].float().view(-1, BLOCK)
    if l2_wd:
        g = _fma(p, torch.full_like(p[:1, :1], l2_wd), g)
    old = s["scales"]
    code = s["exp_avg"].float().view(-1, BLOCK)
    m = _fma(old[:, :1] * b1, code, g * omb1)
    code = s["exp_avg_sq"].float().view(-1, BLOCK)
    v = _fma(old[:, 1:] * old[:, 1:] * b2, code * code, g * omb2 * g)
    r = torch.sqrt(v)
    p = p * decay - step * (m / (r * ibc2 + eps))
    w.copy_(p.view(-1))
    if s["master"] is not None:
        s["param"].copy_(w)
    top_m, top_r = (x.abs().amax(1, keepdim=True).clamp_(min=FLOOR) for x in (m, r))
    s["exp_avg"].copy_((m * (TOP / top_m)).to(torch.float8_e4m3fn).view(-1))
    # a second moment that is not zero does not become zero: the step divides by its root
    r = torch.where(r > 0, (r * (TOP / top_r)).clamp_(min=LEAST), 0.0)
    s["exp_avg_sq"].copy_(r.to(torch.float8_e4m3fn).view(-1))
    torch.mul(torch.cat([top_m, top_r], 1), 1.0 / TOP, out=s["scales"])
    return _adamw8_outputs(s)


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "adamw8":
        return _exact_adamw8(s)
    N, V = c["N"], c["V"]
    w = s["w"].double()
    t = s["targets"].long()
    counted = (t >= 0) & (t < V) & (s["weights"] != 0)
    losses, norm = (torch.zeros(N, dtype=torch.float64, device=DEV) for _ in range(2))
    grads = c["op"] != "head_fwd"
    if grads:
        dh = torch.zeros((N, c["D"]), dtype=torch.float64, device=DEV)
        dw = torch.zeros((V, c["D"]), dtype=torch.float64, device=DEV)
    for i in range(0, N, 1024):
        rows = torch.arange(i, min(N, i + 1024), device=DEV)
        rows = rows[counted[rows]]
        h, y = s["h"][rows].double(), t[rows]
        wt = s["weights"][rows].double()
        z = torch.einsum("nd,vd->nv", h, w)
        lse = s["lse"][rows].double() if c["op"] == "head_bwd" else torch.logsumexp(z, 1)
        one = torch.arange(len(rows), device=DEV)
        losses[rows] = -wt * torch.log_softmax(z, 1)[one, y]
        norm[rows] = lse
        if grads:
            if c["op"] == "head_bwd":
                wt = wt * s["grad"][rows].double()
            z.sub_(lse[:, None]).exp_()
            z[one, y] -= 1.0
            z.mul_(wt[:, None])
            dh[rows] = torch.einsum("nv,vd->nd", z, w)
            dw.addmm_(z.t(), h)
    if c["op"] == "head_fwd":
        return {"losses": losses, "lse": norm}
    return {"dh": dh, "dw": dw} if c["op"] == "head_bwd" else {"losses": losses, "lse": norm, "dh": dh, "dw": dw}


def _nearest_code(y):
    """The e4m3 value nearest to y (ties to the even one), from the format: 3 bits after the leading one, or multiples of
    2^-9 below 2^-6."""
    e = torch.frexp(y).exponent.sub_(4).clamp_(min=-9)
    return torch.ldexp(torch.round(torch.ldexp(y, -e)), e)


def _exact_adamw8(s):
    f = lambda k: float(np.float32(HP[k]))  # noqa: E731
    b1, b2, lr, wd = f("beta1"), f("beta2"), f("lr"), f("weight_decay")
    w = s["master"] if s["master"] is not None else s["param"]
    total = w.numel()
    out = {k: torch.empty(total, dtype=torch.float64, device=DEV) for k in ("param", "exp_avg", "exp_avg_sq")}
    out["scales"] = torch.empty((total // BLOCK, 2), dtype=torch.float64, device=DEV)
    for i in range(0, total, BLOCK << 16):
        at, bl = slice(i, i + (BLOCK << 16)), slice(i // BLOCK, i // BLOCK + (1 << 16))
        p, g = w[at].double(), s["grad"][at].double()
        if s["l2"]:
            g, keep = g + wd * p, 1.0
        else:
            keep = 1.0 - lr * wd
        sm, sr = (s["scales"][bl, k].double().repeat_interleave(BLOCK) for k in (0, 1))
        m = b1 * (s["exp_avg"][at].double() * sm) + (1.0 - b1) * g
        v = b2 * (s["exp_avg_sq"][at].double() * sr) ** 2 + (1.0 - b2) * g ** 2
        r = v ** 0.5
        mh, rh = m / (1.0 - b1 ** HP["step"]), r / (1.0 - b2 ** HP["step"]) ** 0.5
        out["param"][at] = keep * p - lr * mh / (rh + f("eps"))
        for k, name, x in ((0, "exp_avg", m), (1, "exp_avg_sq", r)):
            top = torch.clamp(x.view(-1, BLOCK).abs().max(1).values, min=FLOOR)
            out["scales"][bl, k] = top / TOP
            y = x / (top / TOP).repeat_interleave(BLOCK)
            if k == 1:
                y = torch.where(x > 0, torch.clamp(y, min=LEAST), y)
            out[name][at] = _nearest_code(y)
    if s["master"] is not None:
        out["master"] = out["param"]
    return out
