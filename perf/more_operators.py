"""The drafter's training operators: what is measured, and their plain form.

Two operators around the distillation of a drafter:

  head_loss      the cross entropy of given tokens under softmax(scale h W^T), from the
                 last hidden states h [N, D] and the head W [V, D], without the logits
                 [N, V] in memory; with the gradients by h and W, either in one call or
                 as a differentiable loss
  orthogonalize  an update G [m, n] (or a batch of them) with its singular values
                 drawn towards one by a few odd polynomials of Newton-Schulz kind,
                 X <- a X + (b S + c S^2) X with S = X X^T, from X = G / |G|_F:
                 the step that a drafter's weight matrices take

loss[i] = weights[i] (log sum_v exp(z_iv) - z_i,target); a target of -1 (a position that
is not trained on): loss 0 and no gradient.  Scoring returns log sum_v exp(z_iv) too.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
MOST_HEAD = 4096 * 4096 * 128256  # N D V of the largest case
MOST_ORTH = 446676598784  # multiplications of one step of the largest case


def listed():
    head = dict(op="head_loss", dtype="bf16")
    orth = dict(op="orthogonalize")
    return [
        # the log-probability of one drafted token under a small drafter: a latency case
        dict(head, name="score one token", N=1, D=2048, V=32000, form="score", ragged=False, pad=0),
        # the drafts of five requests, nine positions each, scored from the target's hidden states
        dict(head, name="score drafts", N=45, D=4096, V=128256, form="score", ragged=False, pad=0),
        # loss and gradients of a small micro-batch of a small drafter in one call
        dict(head, name="loss small", N=64, D=1024, V=32000, form="fused", ragged=False, pad=0),
        # odd sizes, positions that are not trained on, rows with gaps between them, the differentiable loss
        dict(head, name="loss odd rows", N=333, D=1000, V=50257, form="autograd", ragged=True, pad=8),
        # a micro-batch over a large vocabulary, the differentiable loss with an upstream gradient per row
        dict(head, name="loss micro-batch", N=2048, D=2048, V=152064, form="autograd", ragged=False, pad=0),
        # loss and gradients of a training batch in one call
        dict(head, name="loss batch", N=4096, D=4096, V=128256, form="fused", ragged=True, pad=0),
        # one small projection: a latency case
        dict(orth, name="orthogonalize one small", batch=1, m=128, n=512, dtype="bf16", decay=0.0, pad=0),
        # the square projections of every layer of a small drafter at once
        dict(orth, name="orthogonalize layers", batch=24, m=1024, n=1024, dtype="bf16", decay=0.5, pad=0),
        # odd sizes in fp32, rows with gaps between them
        dict(orth, name="orthogonalize odd", batch=1, m=1000, n=2333, dtype="fp32", decay=1.0, pad=3),
        # a tall projection (down from the feed-forward width) with an fp32 momentum
        dict(orth, name="orthogonalize tall", batch=1, m=8192, n=2048, dtype="fp32", decay=0.5, pad=0),
        # a square attention projection of a large drafter
        dict(orth, name="orthogonalize square", batch=1, m=4096, n=4096, dtype="bf16", decay=0.5, pad=0),
        # a wide projection (up to the feed-forward width) of a large drafter
        dict(orth, name="orthogonalize wide", batch=1, m=4096, n=16384, dtype="bf16", decay=0.0, pad=0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.55:
        V = _log_int(rng, 1000, 152064)
        D = _log_int(rng, 64, 8192)
        D = max(64, D // 8 * 8) if rng.random() < 0.8 else D
        N = _log_int(rng, 1, max(1, min(8192, MOST_HEAD // (V * D))))
        return dict(op="head_loss", dtype="bf16", N=N, D=D, V=V, form=rng.choice(["score", "fused", "autograd"]),
                    ragged=rng.random() < 0.5, pad=rng.choice([0, 0, 8, 3]))
    m, n = _log_int(rng, 32, 8192), _log_int(rng, 32, 16384)
    batch = _log_int(rng, 1, 32)
    while batch > 1 and batch * _step_macs(m, n) > MOST_ORTH:
        batch //= 2
    if _step_macs(m, n) > MOST_ORTH:
        n = m = 4096
    return dict(op="orthogonalize", batch=batch, m=m, n=n, dtype=rng.choice(["bf16", "fp32"]), decay=rng.choice([0.0, 0.5, 1.0]),
                pad=rng.choice([0, 0, 8, 3]))


def _step_macs(m, n):
    """Multiplications of one step: half of the symmetric S and S^2, all of the product with X."""
    s, t = min(m, n), max(m, n)
    return 1.5 * s * s * t + 0.5 * s ** 3


# ---- inputs

def _gaps(x, pad):
    """x with `pad` further values, never read, behind each row."""
    return torch.nn.functional.pad(x, (0, pad))[..., :x.shape[-1]] if pad else x


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    normal = lambda *shape: torch.empty(shape, dtype=torch.float32, device=DEV).normal_(generator=g)  # noqa: E731
    if c["op"] == "orthogonalize":
        # a gradient's spectrum: singular directions of a size that falls with their place, under a rotation
        x = normal(c["batch"], c["m"], c["n"])
        small = min(c["m"], c["n"])
        fall = (torch.arange(1, small + 1, dtype=torch.float32, device=DEV) ** -c["decay"])
        x = x * (fall[:, None] if c["m"] <= c["n"] else fall)
        x = x.flip(-2) + 0.3 * x  # rows that share directions
        x = (x * 1e-3).to(DT[c["dtype"]])
        x = x if c["batch"] > 1 else x[0]
        return dict(case=c, g=_gaps(x, c["pad"]))
    N, D, V = c["N"], c["D"], c["V"]
    W = normal(V, D) * (2.0 / math.sqrt(D))
    W += W.roll(1, 0) * 0.1
    W = W.to(DT[c["dtype"]])
    t = torch.randint(0, V, (N,), generator=g, device=DEV)
    # hidden states of unit scale that lean towards the target, from not at all to certainty
    lean = 3.0 * torch.rand((N, 1), generator=g, device=DEV)
    h = normal(N, D) + lean * W[t].float()
    h = h.to(DT[c["dtype"]])
    there = torch.rand(N, generator=g, device=DEV) < (0.7 if c["ragged"] else 2.0)
    weights = there.float() / there.sum().clamp_min(1) if c["form"] != "score" else None
    targets = torch.where(there, t, torch.full_like(t, -1)).to(torch.int32)
    up = torch.rand(N, generator=g, device=DEV) + 0.5
    return dict(case=c, h=_gaps(h, c["pad"]), W=_gaps(W, c["pad"]), t=targets, weights=weights, up=up)


# ---- one pass

def run(state):
    c = state["case"]
    if own:
        import speculative_decoding_verification_50_gb300 as sv
        if c["op"] == "orthogonalize":
            o = sv.specv_orthogonalize(state["g"], steps=5, coefficients=COEFFICIENTS)
            return {"orthogonal": o["orthogonal"], "norm": o["norm"]}
        h, W, t, w = state["h"], state["W"], state["t"], state["weights"]
        if c["form"] == "score":
            o = sv.specv_head_loss(h, W, t)
            return {"loss": o["loss"], "lse": o["stats"][:, 0]}
        if c["form"] == "fused":
            o = sv.specv_head_loss(h, W, t, weights=w, with_grad=True)
            return {"loss": o["loss"], "grad_hidden": o["grad_hidden"], "grad_head": o["grad_head"]}
        h, W = h.detach().requires_grad_(), W.detach().requires_grad_()
        loss = sv.head_loss(h, W, t, weights=w)
        gh, gW = torch.autograd.grad(loss, (h, W), state["up"])
        return {"loss": loss.detach(), "grad_hidden": gh, "grad_head": gW}
    return _plain_orthogonalize(state) if c["op"] == "orthogonalize" else _plain_head(state)


def _plain_orthogonalize(s):
    c = s["case"]
    x = s["g"].float().reshape(c["batch"], c["m"], c["n"])
    norm = x.square().sum((1, 2), keepdim=True).sqrt()
    x = x / norm
    if c["m"] > c["n"]:
        x = x.transpose(1, 2)
    a, b, k = COEFFICIENTS
    for _ in range(5):
        S = torch.bmm(x, x.transpose(1, 2))
        x = a * x + torch.bmm(b * S + k * torch.bmm(S, S), x)
    if c["m"] > c["n"]:
        x = x.transpose(1, 2)
    return {"orthogonal": x.reshape(s["g"].shape).to(torch.bfloat16).contiguous(), "norm": norm.reshape(s["g"].shape[:-2])}


def _plain_head(s):
    c = s["case"]
    h, W, t = s["h"].float(), s["W"].float(), s["t"].long()
    there = t >= 0
    at = t.clamp_min(0)[:, None]
    z = h @ W.t()
    z_t = z.gather(1, at)
    e = torch.exp(z - z_t)  # relative to the target: its own term is one exactly
    e.scatter_(1, at, 0.0)
    top = z.amax(1, keepdim=True)
    # far targets: the sum relative to the largest logit
    far = top - z_t > 40
    shifted = torch.exp(z - top).sum(1, keepdim=True)
    loss = torch.where(far, (top - z_t) + torch.log(shifted), torch.log1p(torch.where(far, 0.0, e.sum(1, keepdim=True))))
    w = there.float() if s["weights"] is None else torch.where(there, s["weights"], 0.0)
    out = {"loss": w * loss[:, 0]}
    if c["form"] == "score":
        return {**out, "lse": (z_t + loss)[:, 0]}
    d = torch.exp(z - z_t - loss)
    d.scatter_(1, at, torch.expm1(-loss))
    d *= (w * (s["up"] if c["form"] == "autograd" else 1.0))[:, None]
    out["grad_hidden"] = (d @ W).to(s["h"].dtype)
    out["grad_head"] = (d.t() @ h).to(s["W"].dtype)
    return out


# ---- what a pass cannot do without

def work(case):
    if case["op"] == "orthogonalize":
        n = case["batch"] * case["m"] * case["n"]
        return {"bytes": n * ((2 if case["dtype"] == "bf16" else 4) + 2), "flops": 5 * 2.0 * case["batch"] * _step_macs(case["m"], case["n"])}
    N, D, V = case["N"], case["D"], case["V"]
    once = 2 * (N * D + V * D)
    if case["form"] == "score":
        return {"bytes": once + 8 * N, "flops": 2.0 * N * D * V}
    return {"bytes": 2 * once + 12 * N, "flops": 6.0 * N * D * V}


# ---- the definition in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "orthogonalize":
        parts = [_exact_orthogonal(g) for g in s["g"].reshape(case["batch"], case["m"], case["n"])]
        shape = s["g"].shape
        return {"orthogonal": torch.stack([p[0] for p in parts]).reshape(shape), "norm": torch.stack([p[1] for p in parts]).reshape(shape[:-2])}
    W = s["W"].double()
    grads = case["form"] != "score"
    gW = torch.zeros_like(W) if grads else None
    loss, lse, gh = [], [], []
    step = max(1, 200_000_000 // case["V"])
    for first in range(0, case["N"], step):
        rows = slice(first, min(case["N"], first + step))
        h, t = s["h"][rows].double(), s["t"][rows].long()
        w = torch.ones(len(t), dtype=torch.float64, device=t.device) if s["weights"] is None else s["weights"][rows].double()
        w = torch.where(t < 0, 0.0, w)
        z = h @ W.t()
        lse.append(torch.logsumexp(z, 1))
        logp = torch.log_softmax(z, dim=1)
        loss.append(-w * logp.gather(1, t.clamp_min(0)[:, None])[:, 0])
        if grads:
            u = w * s["up"][rows].double() if case["form"] == "autograd" else w
            p = torch.exp(logp)
            p[torch.arange(len(t), device=t.device), t.clamp_min(0)] -= 1
            p *= u[:, None]
            gh.append(p @ W)
            gW += p.t() @ h
    out = {"loss": torch.cat(loss)}
    return {**out, "grad_hidden": torch.cat(gh), "grad_head": gW} if grads else {**out, "lse": torch.cat(lse)}


def _exact_orthogonal(g):
    g = g.double()
    norm = torch.linalg.matrix_norm(g)
    x = g / norm
    a, b, k = COEFFICIENTS
    for _ in range(5):
        if x.shape[0] <= x.shape[1]:
            S = x @ x.t()
            x = a * x + b * (S @ x) + k * (S @ (S @ x))
        else:
            S = x.t() @ x
            x = a * x + b * (x @ S) + k * ((x @ S) @ S)
    return x, norm
