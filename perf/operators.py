"""The sampling and distillation operators: what is measured, and their plain form.

Three operators over rows of logits [rows, V]:

  sample      one token per row from the logits under temperature, top-k, top-p
              and min-p, by inverse CDF (index order) of a given uniform; or
              the filtered logits themselves (kept logits, -inf elsewhere), as
              verification under the same rules reads them
  top_logits  the k largest logits of a row (value descending, index
              ascending), their ids and the row's log-sum-exp: what a teacher
              keeps of its distribution
  distill     the loss KL(teacher's top-k || student) per row, and its gradient
              with respect to the student's logits

Definition of the kept set of a row, with w_i = exp((z_i - max z) / T): tokens
of w_i < 2^-48 count as zero.  In the order (logit descending, index
ascending) the first n are kept, n = max(1, min(n_k, n_p, n_m)):
n_k = top_k (0: all), n_p = the smallest n whose weights reach top_p times
the weight of the first n_k (top_p >= 1: n_k), n_m = the number of w_i >= min_p.
T = 0 keeps the first maximum.
"""
import math

import numpy as np
import torch

own = False

FLOOR = 2.0 ** -48
DEV = "cuda" if torch.cuda.is_available() else "cpu"
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


def listed():
    return [
        # one request's next token from a small vocabulary: a latency case
        dict(name="sample one row", op="sample", rows=1, per=1, V=32000, dtype="bf16", mix="top_k", out="token", pad=0),
        # a decode batch whose requests each bring their own rules
        dict(name="sample decode batch", op="sample", rows=32, per=1, V=128256, dtype="bf16", mix="mixed", out="token", pad=0),
        # an odd vocabulary, rows that start at no 16-byte boundary
        dict(name="sample odd rows", op="sample", rows=37, per=1, V=50257, dtype="bf16", mix="mixed", out="token", pad=3),
        # every draft position of a large batch (256 requests x 9), nucleus sampling over the whole vocabulary
        dict(name="sample large batch", op="sample", rows=2304, per=9, V=152064, dtype="fp32", mix="top_p", out="token", pad=0),
        # the target's rows of a verification round (64 requests x 5), filtered
        dict(name="filter target rows", op="sample", rows=320, per=5, V=128256, dtype="bf16", mix="mixed", out="filtered", pad=0),
        # a few rows' top logits
        dict(name="top logits few rows", op="top_logits", rows=4, V=32000, dtype="fp32", k=32, T=1.0, pad=0),
        # a teacher's rows of a training batch
        dict(name="top logits teacher rows", op="top_logits", rows=2048, V=152064, dtype="bf16", k=256, T=1.0, pad=0),
        # odd sizes and a temperature
        dict(name="top logits odd", op="top_logits", rows=333, V=50257, dtype="fp32", k=100, T=2.0, pad=1),
        # loss and gradient of a small micro-batch in one call
        dict(name="distill small", op="distill", rows=16, V=32000, dtype="bf16", k=32, T=1.0, tail=False, form="fused", ragged=False, pad=0),
        # loss and gradient of a training batch in one call, the teacher's tail as one more outcome
        dict(name="distill fused", op="distill", rows=1024, V=128256, dtype="bf16", k=64, T=1.0, tail=True, form="fused", ragged=False, pad=0),
        # the differentiable loss: forward, then backward with a given gradient per row
        dict(name="distill autograd", op="distill", rows=1024, V=152064, dtype="fp32", k=256, T=2.0, tail=True, form="autograd", ragged=False, pad=0),
        # masked positions and ragged lists over an odd vocabulary
        dict(name="distill ragged", op="distill", rows=511, V=50257, dtype="bf16", k=100, T=1.5, tail=False, form="autograd", ragged=True, pad=5),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "top_logits", "distill"])
    V = _log_int(rng, 1000, 152064)
    V = V // 8 * 8 if rng.random() < 0.5 else V
    dtype = rng.choice(["bf16", "fp32"])
    pad = rng.choice([0, 0, 8 - V % 8, 1, 5])
    rows = _log_int(rng, 1, min(2304, 120_000_000 // V))
    if op == "sample":
        per = rng.choice([1, 1, 5, 9])
        return dict(op=op, rows=max(1, rows // per) * per, per=per, V=V, dtype=dtype, mix=rng.choice(["top_k", "mixed", "top_p", "plain"]),
                    out=rng.choice(["token", "token", "filtered"]), pad=pad)
    if op == "top_logits":
        return dict(op=op, rows=rows, V=V, dtype=dtype, k=_log_int(rng, 4, 512), T=rng.choice([1.0, 2.0, 0.7]), pad=pad)
    return dict(op=op, rows=min(rows, 60_000_000 // V), V=V, dtype=dtype, k=_log_int(rng, 4, 512), T=rng.choice([1.0, 2.0, 1.5]), tail=rng.random() < 0.5,
                form=rng.choice(["fused", "autograd"]), ragged=rng.random() < 0.5, pad=pad)


# ---- inputs

def _rows(g, rows, V, dtype, pad):
    """Logits of a row spread by its own width (1 to 3), with eight tokens well above the rest."""
    z = torch.empty((rows, V + pad), dtype=torch.float32, device=DEV).normal_(generator=g)
    z *= torch.rand((rows, 1), generator=g, device=DEV) * 2 + 1
    z.scatter_add_(1, torch.randint(0, V, (rows, 8), generator=g, device=DEV), torch.rand((rows, 8), generator=g, device=DEV) * 8)
    return z.to(DT[dtype])[:, :V]


def _choice(g, n, values, dtype):
    return torch.tensor(values, dtype=dtype, device=DEV)[torch.randint(0, len(values), (n,), generator=g, device=DEV)]


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    c = dict(case)
    z = _rows(g, c["rows"], c["V"], c["dtype"], c["pad"])
    if c["op"] == "sample":
        n, f, i = c["rows"] // c["per"], torch.float32, torch.int32
        T = {"top_k": [0.8], "top_p": [1.0], "plain": [0.7, 1.0], "mixed": [0.0, 0.6, 0.8, 1.0, 1.3]}[c["mix"]]
        k = {"top_k": [50], "mixed": [0, 0, 20, 50, 200]}.get(c["mix"])
        p = {"top_k": [0.95], "top_p": [0.8, 0.9, 0.95, 0.98], "mixed": [1.0, 0.8, 0.9, 0.95, 0.99]}.get(c["mix"])
        m = {"mixed": [0.0, 0.0, 0.02, 0.1]}.get(c["mix"])
        s = dict(z=z, T=_choice(g, n, T, f), top_k=_choice(g, n, k, i) if k else None, top_p=_choice(g, n, p, f) if p else None,
                 min_p=_choice(g, n, m, f) if m else None, u=torch.rand(c["rows"], generator=g, device=DEV))
    elif c["op"] == "top_logits":
        s = dict(z=z)
    else:
        t = z.float() + torch.empty((c["rows"], c["V"]), dtype=torch.float32, device=DEV).normal_(generator=g)
        k = min(c["k"], c["V"])
        val, ids = t.topk(k, dim=1)
        lse = torch.logsumexp(t / c["T"], dim=1)
        ids = ids.to(torch.int32)
        w = torch.ones(c["rows"], device=DEV)
        if c["ragged"]:
            length = torch.randint(0, k + 1, (c["rows"], 1), generator=g, device=DEV)
            ids = torch.where(torch.arange(k, device=DEV) < length, ids, torch.full_like(ids, -1))
            w = (torch.rand(c["rows"], generator=g, device=DEV) < 0.8).float()
        s = dict(z=z, ids=ids, val=val, lse=lse if c["tail"] else None, w=w, g=torch.rand(c["rows"], generator=g, device=DEV) + 0.5)
    s["case"] = c
    return s


# ---- one pass

def run(state):
    c = state["case"]
    if own:
        import speculative_decoding_verification_50_gb300 as sv
        z = state["z"]
        if c["op"] == "sample":
            z = z.unflatten(0, (-1, c["per"]))
            rules = dict(top_k=state["top_k"], top_p=state["top_p"], min_p=state["min_p"])
            if c["out"] == "filtered":
                o = sv.specv_filter_logits(z, state["T"], **rules)
                return {"filtered": o["filtered"].flatten(0, 1), "kept": o["kept"].flatten()}
            o = sv.specv_sample(z, state["T"], state["u"].view(-1, c["per"]), **rules)
            return {"tokens": o["tokens"].flatten(), "prob": o["prob"].flatten(), "kept": o["kept"].flatten()}
        if c["op"] == "top_logits":
            o = sv.specv_top_logits(z, min(c["k"], c["V"]), temperature=c["T"])
            return {"ids": o["ids"], "values": o["values"], "lse": o["lse"]}
        teacher = dict(teacher_lse=state["lse"], temperature=c["T"], weights=state["w"], tail=c["tail"])
        if c["form"] == "fused":
            o = sv.specv_distill(z, state["ids"], state["val"], with_grad=True, **teacher)
            return {"loss": o["loss"], "grad": o["grad"]}
        leaf = z.detach().requires_grad_()
        loss = sv.distill_loss(leaf, state["ids"], state["val"], **teacher)
        return {"loss": loss.detach(), "grad": torch.autograd.grad(loss, leaf, state["g"])[0]}
    return {"sample": _plain_sample, "top_logits": _plain_top, "distill": _plain_distill}[c["op"]](state)


def _plain_sample(s):
    """Weights and sums in 64 bits: cuts and draws fall next to borders."""
    c, z = s["case"], s["z"].float()
    rows, V = z.shape
    each = lambda x, off: (torch.full((rows,), off, device=z.device) if x is None else x.repeat_interleave(c["per"]))[:, None]  # noqa: E731
    T = each(s["T"], 1.0).double()
    top_k, top_p, min_p = each(s["top_k"], 0).long(), each(s["top_p"], 1.0).double(), each(s["min_p"], 0.0).double()
    greedy = T == 0
    T = torch.where(greedy, torch.ones_like(T), T)
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = zs[:, :1].double()
    live = zs >= top + T * math.log(FLOOR)
    w = torch.where(live, torch.exp((zs - top) / T), 0.0)
    cum = torch.cumsum(w, dim=1)
    n = live.sum(1, keepdim=True)
    n_k = torch.where(top_k > 0, torch.minimum(top_k, n), n)
    reach = top_p * cum.gather(1, n_k - 1)
    before = torch.cat([torch.zeros_like(cum[:, :1]), cum[:, :-1]], dim=1)
    n_p = torch.where(top_p >= 1, n_k, ((before < reach) & live).sum(1, keepdim=True))
    n_m = (zs >= top + T * torch.log(min_p.clamp_min(FLOOR))).sum(1, keepdim=True)
    n = torch.minimum(torch.minimum(n_k, n_p), n_m).clamp_min(1)
    n = torch.where(greedy, torch.ones_like(n), n)
    del cum, before, live
    first = torch.arange(V, device=z.device) < n
    keep = torch.zeros_like(first).scatter_(1, order, first)
    kept = n[:, 0].to(torch.int32)
    if c["out"] == "filtered":
        return {"filtered": torch.where(keep, s["z"], torch.full_like(s["z"], -math.inf)), "kept": kept}
    w = torch.where(keep, torch.exp((z - top) / T), 0.0)
    cum = torch.cumsum(w, dim=1)
    total = cum[:, -1:]
    token = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    last = (keep * torch.arange(V, device=z.device)).amax(1, keepdim=True)
    token = torch.minimum(token, last)
    return {"tokens": token[:, 0].to(torch.int32), "prob": (w.gather(1, token) / total)[:, 0].float(), "kept": kept}


def _plain_top(s):
    c, z = s["case"], s["z"].float()
    k = min(c["k"], c["V"])
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = zs[:, :1]
    lse = top[:, 0] / c["T"] + torch.log(torch.exp((z - top) / c["T"]).sum(1))
    return {"ids": order[:, :k].to(torch.int32), "values": zs[:, :k].contiguous(), "lse": lse}


def _plain_distill(s):
    c, z, T = s["case"], s["z"].float(), s["case"]["T"]
    ids, there = s["ids"].clamp_min(0).long(), s["ids"] >= 0
    t = torch.where(there, s["val"] / T, -math.inf)
    if s["lse"] is None:
        top = t.amax(1, keepdim=True).clamp_min(-1e30)
        log_p = t - top - torch.log(torch.exp(t - top).sum(1, keepdim=True).clamp_min(1e-30))
    else:
        log_p = t - s["lse"][:, None]
    p = torch.exp(log_p)
    m = p.sum(1, keepdim=True)
    top = z.amax(1, keepdim=True)
    y = (z - top) / T
    e = torch.exp(y)
    listed_ = torch.zeros_like(z).scatter_add_(1, ids, there.float())
    e_rest = torch.where(listed_ > 0, 0.0, e).sum(1, keepdim=True)
    e_listed = torch.where(there, e.gather(1, ids), 0.0).sum(1, keepdim=True)
    total = e_rest + e_listed
    log_q = y.gather(1, ids) - torch.log(total)
    loss = torch.where(there & (p > 0), p * (log_p - log_q), 0.0).sum(1, keepdim=True)
    alpha, beta = m, m
    if c["tail"]:
        r = (1 - m).clamp_min(0)
        r = torch.where(r < 2.0 ** -20, 0.0, r)
        rest = e_rest / total
        loss = loss + torch.where(r > 0, r * (torch.log(r.clamp_min(1e-30)) - torch.log(rest)), 0.0)
        over = torch.where(r > 0, r / rest, 0.0)
        alpha, beta = m - over * (e_listed / total), m - over * (e_listed / total) + over
    q = e / total
    w = s["w"][:, None] * (1.0 if c["form"] == "fused" else s["g"][:, None])
    grad = torch.where(listed_ > 0, beta, alpha) * q
    grad.scatter_add_(1, ids, torch.where(there, -p, 0.0))
    return {"loss": (s["w"] * loss[:, 0]), "grad": (grad * (w / T)).to(s["z"].dtype)}


# ---- what a pass cannot do without

def work(case):
    n = case["rows"] * case["V"]
    es = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "sample":
        return {"bytes": n * es * (2 if case["out"] == "filtered" else 1) + case["rows"] * 16, "flops": 4.0 * n}
    if case["op"] == "top_logits":
        return {"bytes": n * es + case["rows"] * (8 * case["k"] + 4), "flops": 4.0 * n}
    return {"bytes": 2 * n * es + case["rows"] * (8 * case["k"] + 16), "flops": 8.0 * n}


# ---- the definition in 64 bits, a block of rows at a time

def exact(case, seed):
    s = prepare(case, seed)
    parts = []
    step = max(1, 40_000_000 // case["V"])
    for a in range(0, case["rows"], step):
        sl = slice(a, min(case["rows"], a + step))
        parts.append({"sample": _exact_sample, "top_logits": _exact_top, "distill": _exact_distill}[case["op"]](case, s, sl))
    join = lambda k: None if parts[0][k] is None else np.concatenate([q[k] for q in parts])  # noqa: E731
    return {k: join(k) for k in parts[0]}


def _exact_sample(case, s, sl):
    z = s["z"][sl].double()
    row = torch.arange(sl.start, sl.stop, device=z.device) // case["per"]
    pick = lambda x, off: torch.full((len(row), 1), float(off), dtype=torch.float64, device=z.device) if x is None else x[row].double()[:, None]  # noqa: E731
    T, top_k, top_p, min_p = pick(s["T"], 1), pick(s["top_k"], 0), pick(s["top_p"], 1), pick(s["min_p"], 0)
    p = torch.softmax(torch.where(T > 0, z / T.clamp_min(1e-9), z), dim=1)
    p = torch.where(p < FLOOR * p.amax(1, keepdim=True), 0.0, p)
    # the threshold that each rule sets on the sorted probabilities
    ps, order = torch.sort(p, dim=1, descending=True, stable=True)
    place = torch.arange(case["V"], device=z.device, dtype=torch.float64)[None]
    ps = torch.where((top_k > 0) & (place >= top_k), 0.0, ps)
    ps = ps / ps.sum(1, keepdim=True)
    ahead = ps.cumsum(1) - ps
    ok = (ps > 0) & ((ahead < top_p) | (top_p >= 1)) & (ps >= min_p * ps[:, :1])
    ok[:, 0] = True
    ok &= (T > 0) | (place == 0)
    ps = torch.where(ok, ps, 0.0)
    ps = ps / ps.sum(1, keepdim=True)
    p = torch.zeros_like(ps).scatter_(1, order, ps)
    if case["out"] == "filtered":
        keep = torch.zeros_like(ok).scatter_(1, order, ok)
        return {"filtered": torch.where(keep, z, -math.inf).cpu().numpy(), "kept": None}
    below = p.cumsum(1)
    token = (below <= s["u"][sl].double()[:, None]).sum(1).clamp_max(case["V"] - 1)
    return {"tokens": None, "prob": p.gather(1, token[:, None])[:, 0].cpu().numpy(), "kept": None}


def _exact_top(case, s, sl):
    z = s["z"][sl].double()
    k = min(case["k"], case["V"])
    return {"ids": None, "values": z.topk(k, dim=1).values.cpu().numpy(), "lse": torch.logsumexp(z / case["T"], dim=1).cpu().numpy()}


def _exact_distill(case, s, sl):
    z = s["z"][sl].double() / case["T"]
    ids, val = s["ids"][sl].long(), s["val"][sl].double() / case["T"]
    rows, V = z.shape
    val = torch.where(ids >= 0, val, -math.inf)
    norm = torch.logsumexp(val, 1) if s["lse"] is None else s["lse"][sl].double()
    p = torch.zeros((rows, V + 1), dtype=torch.float64, device=z.device)
    p.scatter_(1, torch.where(ids >= 0, ids, V), torch.where(ids >= 0, torch.exp(val - norm[:, None]), 0.0))
    seen = torch.zeros((rows, V + 1), dtype=torch.bool, device=z.device).scatter_(1, torch.where(ids >= 0, ids, V), True)[:, :V]
    p = p[:, :V]
    log_q = torch.log_softmax(z, dim=1)
    loss = torch.where(p > 0, p * (torch.log(p) - log_q), 0.0).sum(1)
    dlog = p.clone()  # minus the derivative of the loss by log q
    if case["tail"]:
        r = (1 - p.sum(1)).clamp_min(0)
        r = torch.where(r < 2.0 ** -20, 0.0, r)
        log_rest = torch.logsumexp(torch.where(seen, -math.inf, log_q), dim=1)
        loss = loss + torch.where(r > 0, r * (torch.log(r) - log_rest), 0.0)
        share = torch.where(seen, 0.0, torch.exp(log_q - log_rest[:, None]))
        dlog += torch.where(r > 0, r, 0.0)[:, None] * share
    grad = (dlog.sum(1, keepdim=True) * torch.exp(log_q) - dlog) / case["T"]
    w = s["w"][sl].double()
    up = w if case["form"] == "fused" else w * s["g"][sl].double()
    return {"loss": torch.where(w > 0, w * loss, 0.0).cpu().numpy(), "grad": torch.where(up[:, None] > 0, grad * up[:, None], 0.0).cpu().numpy()}
