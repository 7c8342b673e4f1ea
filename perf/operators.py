"""Timed cases of the operators whose weights the AdamW half of the optimizer updates: the embedding lookup and its
gradient, layer norm and its gradients, and the distillation loss at the vocabulary head.

With ``own`` false, ``run`` computes a case in elementary torch operations in 32 bits; with ``own`` true it makes the
library's calls. Sizes come from the optimizer's workloads (width 768 with a vocabulary of 50304, width 4096 with
128256), beside odd ones.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-5
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZE = {"bf16": 2, "f32": 4, "i32": 4, "i64": 8}


def listed():
    return [
        # one new token for each of 32 sequences: latency alone
        dict(name="embed_fwd_few", op="embed_fwd", n=32, V=50304, D=768, tdt="bf16", odt="bf16", idt="i64", scale=1.0),
        # a training batch of 64 Ki tokens on the wide model's table
        dict(name="embed_fwd_long", op="embed_fwd", n=65536, V=128256, D=4096, tdt="bf16", odt="bf16", idt="i32",
             scale=64.0),
        # a small model's batch; fp32 gradient of the table
        dict(name="embed_bwd_768", op="embed_bwd", n=16384, V=50304, D=768, odt="bf16", gdt="f32", idt="i64",
             scale=1.0),
        # the wide model's batch; bf16 gradient of a 1 GB table, most of whose rows no token names
        dict(name="embed_bwd_4096", op="embed_bwd", n=32768, V=128256, D=4096, odt="bf16", gdt="bf16", idt="i32",
             scale=64.0),
        # the norm of a handful of tokens: latency alone
        dict(name="ln_fwd_few", op="ln_fwd", N=8, D=768, xdt="bf16", ydt="bf16", wdt="bf16"),
        # a training batch on the wide model
        dict(name="ln_fwd_long", op="ln_fwd", N=65536, D=4096, xdt="bf16", ydt="bf16", wdt="bf16"),
        # odd width in fp32: no row but the first is 16-byte aligned
        dict(name="ln_bwd_odd", op="ln_bwd", N=5001, D=1023, xdt="f32", ydt="f32", wdt="f32", gdt="f32"),
        # a training batch on the wide model
        dict(name="ln_bwd_long", op="ln_bwd", N=32768, D=4096, xdt="bf16", ydt="bf16", wdt="bf16", gdt="bf16"),
        # the loss of four positions under a large vocabulary (an evaluation of single tokens): few long rows
        dict(name="distill_fwd_few", op="distill_fwd", N=4, V=128256, K=64, zdt="f32", tdt="f32", idt="i32",
             T=2.0),
        # loss and gradient of a small model's batch in one call
        dict(name="distill_step_50304", op="distill_step", N=8192, V=50304, K=64, zdt="bf16", ddt="bf16", tdt="bf16",
             idt="i32", T=2.0),
        # odd vocabulary in fp32
        dict(name="distill_step_odd", op="distill_step", N=1001, V=32003, K=20, zdt="f32", ddt="f32", tdt="f32",
             idt="i64", T=1.0),
        # the gradient alone, from the statistics that the forward pass left, under a large vocabulary
        dict(name="distill_bwd_128256", op="distill_bwd", N=4096, V=128256, K=128, zdt="bf16", ddt="bf16", tdt="bf16",
             idt="i32", T=4.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_moved(c) for c in listed())
    while True:
        op = rng.choice(["embed_fwd", "embed_bwd", "ln_fwd", "ln_bwd", "distill_fwd", "distill_bwd", "distill_step"])
        f = lambda: rng.choice(["bf16", "bf16", "f32"])  # noqa: E731
        c = {"op": op}
        if op.startswith("embed"):
            D = rng.choice([768, 4096, 8 * _log(rng, 8, 1024), _log(rng, 33, 8192)])
            c.update(n=_log(rng, 1, 131072), V=rng.choice([50304, 128256, _log(rng, 500, 260000)]), D=D, odt=f(),
                     idt=rng.choice(["i32", "i64"]), scale=rng.choice([1.0, math.sqrt(D)]))
            c["tdt" if op == "embed_fwd" else "gdt"] = f()
        elif op.startswith("ln"):
            c.update(N=_log(rng, 1, 131072), D=rng.choice([768, 4096, 8 * _log(rng, 8, 2048), _log(rng, 33, 16384)]),
                     xdt=f(), ydt=f(), wdt=f())
            if op == "ln_bwd":
                c["gdt"] = f()
        else:
            c.update(N=_log(rng, 1, 16384), V=rng.choice([50304, 128256, _log(rng, 1000, 260000)]),
                     K=_log(rng, 1, 256), zdt=f(), tdt=f(), idt=rng.choice(["i32", "i64"]),
                     T=rng.choice([1.0, 2.0, 4.0]))
            if op != "distill_fwd":
                c["ddt"] = f()
        if _moved(c) <= most:
            return c


def _distinct(n, V):
    """Expected number of distinct ids among n draws of _ids."""
    v = np.arange(1, V + 1, dtype=np.float64)
    p = np.log1p(1.0 / v) / np.log(V + 1.0)
    return float(np.sum(-np.expm1(n * np.log1p(-p)))) if V > 1 else 1.0


def _moved(c):
    op = c["op"]
    if op.startswith("embed"):
        n, D = c["n"], c["D"]
        table = min(n, _distinct(n, c["V"])) * D * SIZE[c["tdt"]] if op == "embed_fwd" else c["V"] * D * SIZE[c["gdt"]]
        return n * SIZE[c["idt"]] + n * D * SIZE[c["odt"]] + table
    if op.startswith("ln"):
        N, D = c["N"], c["D"]
        x, y, w = SIZE[c["xdt"]], SIZE[c["ydt"]], SIZE[c["wdt"]]
        if op == "ln_fwd":
            return N * D * (x + y) + 2 * D * w + 8 * N
        return N * D * (2 * x + y) + D * w + 2 * D * SIZE[c["gdt"]] + 8 * N
    N, V = c["N"], c["V"]
    moved = N * V * SIZE[c["zdt"]] + N * c["K"] * (SIZE[c["tdt"]] + SIZE[c["idt"]]) + 16 * N
    return moved + (N * V * SIZE[c["ddt"]] if op != "distill_fwd" else 0)


def work(c):
    op = c["op"]
    if op.startswith("embed"):
        flops = c["n"] * c["D"] * (1 if op == "embed_fwd" else 2)
    elif op.startswith("ln"):
        flops = c["N"] * c["D"] * (8 if op == "ln_fwd" else 15)
    else:
        flops = c["N"] * c["V"] * {"distill_fwd": 4, "distill_bwd": 4, "distill_step": 8}[op]
    return {"bytes": _moved(c), "flops": flops}


def _ids(n, V, idt, g):
    """Token ids as text has them: the id of rank r with a probability of about 1 / r, ranks spread over the ids."""
    u = torch.rand(n, generator=g, device=DEV, dtype=torch.float64)
    rank = torch.clamp(torch.floor(torch.exp(u * math.log(V + 1.0))).to(torch.int64) - 1, 0, V - 1)
    step = 7919
    while math.gcd(step, V) != 1:
        step += 2
    return ((rank * step + 13) % V).to(torch.int32 if idt == "i32" else torch.int64)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    op = c["op"]
    s = dict(c)

    def normal(*shape, std=1.0, mean=0.0, dt="f32"):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(DT[dt])

    def empty(*shape, dt="f32"):
        return torch.empty(shape, dtype=DT[dt], device=DEV)

    if op.startswith("embed"):
        n, V, D = c["n"], c["V"], c["D"]
        s["ids"] = _ids(n, V, c["idt"], g)
        if op == "embed_fwd":
            s["table"] = normal(V, D, std=0.02, dt=c["tdt"])
            s["out"] = empty(n, D, dt=c["odt"])
        else:
            s["dout"] = normal(n, D, std=1e-3, dt=c["odt"])
            s["dtable"] = empty(V, D, dt=c["gdt"])
    elif op.startswith("ln"):
        N, D = c["N"], c["D"]
        x = torch.randn((N, D), generator=g, device=DEV) * 2.0
        x += torch.randn((N, 1), generator=g, device=DEV) * 0.5
        s["x"] = x.to(DT[c["xdt"]])
        s["w"] = normal(D, std=0.1, mean=1.0, dt=c["wdt"])
        s["b"] = normal(D, std=0.1, dt=c["wdt"])
        if op == "ln_fwd":
            s["y"], s["mean"], s["rstd"] = empty(N, D, dt=c["ydt"]), empty(N), empty(N)
        else:
            # what the forward pass left
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
            s["dy"] = normal(N, D, std=1e-2, dt=c["ydt"])
            s["dx"] = empty(N, D, dt=c["xdt"])
            s["dw"], s["db"] = empty(D, dt=c["gdt"]), empty(D, dt=c["gdt"])
    else:
        N, V, K = c["N"], c["V"], c["K"]
        it = torch.int32 if c["idt"] == "i32" else torch.int64
        # K distinct ids for each position (one from each of K strata), in an order of their own
        edge = (torch.arange(K + 1, device=DEV) * V) // K
        idx = edge[:-1] + (torch.rand((N, K), generator=g, device=DEV) * (edge[1:] - edge[:-1])).to(torch.int64)
        idx = torch.minimum(idx, edge[1:] - 1)
        idx = torch.gather(idx, 1, torch.argsort(torch.rand((N, K), generator=g, device=DEV), dim=1))
        # the teacher's logits fall from its best one; the student has learned part of them
        t = 12.0 - 2.0 * torch.log1p(torch.arange(K, device=DEV, dtype=torch.float32)) \
            + 0.3 * torch.randn((N, K), generator=g, device=DEV)
        z = torch.randn((N, V), generator=g, device=DEV) * 2.0
        z.scatter_add_(1, idx, 0.7 * t)
        s["logits"] = z.to(DT[c["zdt"]])
        # some positions have fewer than K teacher entries; one in twenty is padding, of weight zero
        short = torch.randint(0, max(1, K // 2), (N, 1), generator=g, device=DEV)
        some = torch.rand((N, 1), generator=g, device=DEV) < 0.1
        idx = torch.where(some & (torch.arange(K, device=DEV) >= K - short), torch.full_like(idx, -1), idx)
        s["t_idx"], s["t_val"] = idx.to(it), t.to(DT[c["tdt"]])
        keep = (torch.rand(N, generator=g, device=DEV) >= 0.05).float()
        s["weights"] = keep / N
        s["losses"], s["stats"] = empty(N), empty(N, 2)
        if op == "distill_bwd":
            zf = s["logits"]
            for i in range(0, N, 1024):   # what the forward pass left
                zi = zf[i:i + 1024].float()
                m = zi.max(1, keepdim=True).values
                s["stats"][i:i + 1024, 0] = m[:, 0]
                s["stats"][i:i + 1024, 1] = torch.exp((zi - m) / c["T"]).sum(1).log()
            s["grad"] = torch.rand(N, generator=g, device=DEV) + 0.5
        if op != "distill_fwd":
            s["dlogits"] = empty(N, V, dt=c["ddt"])
    return s


def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    from adamw_hybrid_optimizer_gb300 import libmuon as L
    op = s["op"]
    if op == "embed_fwd":
        L.embedding_forward(s["ids"], s["table"], s["out"], s["scale"])
        return {"out": s["out"]}
    if op == "embed_bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(L.embedding_workspace_bytes(s["n"], s["V"], s["D"]), dtype=torch.uint8, device=DEV)
        L.embedding_backward(s["ids"], s["dout"], s["dtable"], s["ws"], s["scale"])
        return {"dtable": s["dtable"]}
    if op == "ln_fwd":
        L.layernorm_forward(s["x"], s["w"], s["b"], s["y"], s["mean"], s["rstd"], EPS)
        return {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if op == "ln_bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(L.layernorm_workspace_bytes(s["N"], s["D"]), dtype=torch.uint8, device=DEV)
        L.layernorm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], s["dx"], s["dw"], s["db"], s["ws"])
        return {"dx": s["dx"], "dw": s["dw"], "db": s["db"]}
    if op == "distill_fwd":
        L.distill_forward(s["logits"], s["t_idx"], s["t_val"], s["T"], s["weights"], s["losses"], s["stats"])
        return {"losses": s["losses"], "stats": s["stats"]}
    if op == "distill_bwd":
        L.distill_backward(s["logits"], s["t_idx"], s["t_val"], s["T"], s["weights"], s["stats"], s["grad"],
                           s["dlogits"])
        return {"dlogits": s["dlogits"]}
    L.distill_forward_backward(s["logits"], s["t_idx"], s["t_val"], s["T"], s["weights"], 1.0, s["losses"],
                               s["stats"], s["dlogits"])
    return {"losses": s["losses"], "stats": s["stats"], "dlogits": s["dlogits"]}


def _plain(s):
    op = s["op"]
    if op == "embed_fwd":
        return {"out": (s["table"][s["ids"].long()].float() * s["scale"]).to(DT[s["odt"]])}
    if op == "embed_bwd":
        d = torch.zeros((s["V"], s["D"]), dtype=torch.float32, device=DEV)
        d.index_add_(0, s["ids"].long(), s["dout"].float())
        return {"dtable": (d * s["scale"]).to(DT[s["gdt"]])}
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        xc = x - mean[:, None]
        rstd = torch.rsqrt((xc * xc).mean(1) + EPS)
        y = xc * rstd[:, None] * s["w"].float() + s["b"].float()
        return {"y": y.to(DT[s["ydt"]]), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xh = (s["x"].float() - s["mean"][:, None]) * rstd
        gw = dy * s["w"].float()
        dx = rstd * (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True))
        gt = DT[s["gdt"]]
        return {"dx": dx.to(DT[s["xdt"]]), "dw": (dy * xh).sum(0).to(gt), "db": dy.sum(0).to(gt)}
    T, w = s["T"], s["weights"]
    z = s["logits"].float()
    idx = s["t_idx"].long()
    valid = (idx >= 0) & (idx < s["V"])
    at = torch.where(valid, idx, 0)
    t = torch.where(valid, s["t_val"].float() / T, -math.inf)
    tm = t.max(1, keepdim=True).values
    live = (w != 0) & (tm[:, 0] > -math.inf)
    e = torch.exp(t - torch.where(live[:, None], tm, 0.0))
    total = e.sum(1, keepdim=True)
    q = torch.where(live[:, None], e / total, 0.0)
    if op == "distill_bwd":
        m, l = s["stats"][:, :1], s["stats"][:, 1:]
        x = (z - m) / T
        p = torch.exp(x - l)
        scale = s["grad"] * w * T
    else:
        m = z.max(1, keepdim=True).values
        x = (z - m) / T
        ex = torch.exp(x)
        l = ex.sum(1, keepdim=True).log()
        # log q - log p at the teacher's entries
        diff = (t - tm - total.log()) - (x.gather(1, at) - l)
        losses = torch.where(live, w * T * T * torch.where(q > 0, q * diff, 0.0).sum(1), 0.0)
        stats = torch.where(live[:, None], torch.cat([m, l], 1), 0.0)
        if op == "distill_fwd":
            return {"losses": losses, "stats": stats}
        p = ex / ex.sum(1, keepdim=True)
        scale = w * T
    p.scatter_add_(1, at, -q)
    d = torch.where(live[:, None], p * scale[:, None], 0.0).to(DT[s["ddt"]])
    return {"dlogits": d} if op == "distill_bwd" else {"losses": losses, "stats": stats, "dlogits": d}


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "embed_fwd":
        # row by row of the output, from the definition
        return {"out": torch.index_select(s["table"], 0, s["ids"].long()).double().mul_(c["scale"])}
    if op == "embed_bwd":
        d = torch.zeros((c["V"], c["D"]), dtype=torch.float64, device=DEV)
        for i in range(0, c["n"], 8192):
            d.index_add_(0, s["ids"][i:i + 8192].long(), s["dout"][i:i + 8192].double(), alpha=c["scale"])
        return {"dtable": d}
    if op == "ln_fwd":
        y = torch.empty((c["N"], c["D"]), dtype=torch.float64, device=DEV)
        mean, rstd = (torch.empty(c["N"], dtype=torch.float64, device=DEV) for _ in range(2))
        w, b = s["w"].double(), s["b"].double()
        for i in range(0, c["N"], 4096):
            x = s["x"][i:i + 4096].double()
            var, mu = torch.var_mean(x, dim=1, correction=0)
            mean[i:i + 4096], rstd[i:i + 4096] = mu, (var + EPS) ** -0.5
            y[i:i + 4096] = (x - mu[:, None]) / (var[:, None] + EPS) ** 0.5 * w + b
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx = torch.empty((c["N"], c["D"]), dtype=torch.float64, device=DEV)
        dw, db = (torch.zeros(c["D"], dtype=torch.float64, device=DEV) for _ in range(2))
        w = s["w"].double()
        for i in range(0, c["N"], 4096):
            rows = slice(i, i + 4096)
            r = s["rstd"][rows].double()[:, None]
            n = (s["x"][rows].double() - s["mean"][rows].double()[:, None]) * r
            dy = s["dy"][rows].double()
            dw += torch.einsum("nd,nd->d", dy, n)
            db += torch.einsum("nd->d", dy)
            dn = dy * w
            # the gradient of the normalised row, less its parts along the constant and along the row itself
            dx[rows] = (dn - dn.sum(1, keepdim=True) / c["D"] - n * (dn * n).sum(1, keepdim=True) / c["D"]) * r
        return {"dx": dx, "dw": dw, "db": db}
    N, V, T = c["N"], c["V"], c["T"]
    losses = torch.zeros(N, dtype=torch.float64, device=DEV)
    stats = torch.zeros((N, 2), dtype=torch.float64, device=DEV)
    dl = torch.zeros((N, V), dtype=torch.float64, device=DEV) if op != "distill_fwd" else None
    for i in range(0, N, 1024):
        rows = slice(i, min(N, i + 1024))
        z = s["logits"][rows].double()
        idx, w = s["t_idx"][rows].long(), s["weights"][rows].double()
        ok = (idx >= 0) & (idx < V)
        tt = torch.where(ok, s["t_val"][rows].double() / T, torch.full_like(idx, -math.inf, dtype=torch.float64))
        live = (w != 0) & ok.any(1)
        lq = torch.where(live[:, None], tt - torch.logsumexp(tt, 1, keepdim=True), -math.inf)
        q = torch.exp(lq)
        top = z.amax(1)
        if op == "distill_bwd":
            norm = s["stats"][rows, 1].double() + s["stats"][rows, 0].double() / T
        else:
            norm = torch.logsumexp(z / T, 1)
        lp = z / T - norm[:, None]
        at = torch.where(ok, idx, 0)
        kl = torch.where(q > 0, q * (lq - torch.gather(lp, 1, at)), 0.0).sum(1)
        losses[rows] = torch.where(live, w * T ** 2 * kl, 0.0)
        stats[rows] = torch.where(live[:, None], torch.stack([top, norm - top / T], 1), 0.0)
        if dl is not None:
            up = s["grad"][rows].double() if op == "distill_bwd" else 1.0
            d = lp.exp_().scatter_add_(1, at, -q)
            dl[rows] = torch.where(live[:, None], d * (up * w * T)[:, None], 0.0)
    if op == "distill_fwd":
        return {"losses": losses, "stats": stats}
    return {"dlogits": dl} if op == "distill_bwd" else {"losses": losses, "stats": stats, "dlogits": dl}
