"""The row operators' definitions in 64 bits over whole batches (torch, on the
inputs' device), so that tests can hold every row against them."""
import math

import torch


def distill64(z, ids, t, lse=None, T=1.0, w=None, tail=False):
    """Loss [N], its gradient [N, V] (of the sum), the sum of the absolute terms
    of the loss [N], the mask of listed ids [N, V], and the sum of the absolute
    terms of the gradient [N, V]."""
    T = float(torch.tensor(T, dtype=torch.float32))
    N, V = z.shape
    y = z.double() / T
    there = ids >= 0
    at = torch.where(there, ids, V).long()
    t = torch.where(there, t.double() / T, -math.inf)
    L = lse.double()[:, None] if lse is not None else torch.logsumexp(t, 1, keepdim=True)
    L = torch.where(torch.isneginf(L), 0.0, L)
    lp = t - L
    p = torch.exp(lp)
    listed = torch.zeros((N, V + 1), dtype=torch.bool, device=z.device).scatter_(1, at, True)[:, :V]
    P = torch.zeros((N, V + 1), dtype=torch.float64, device=z.device).scatter_add_(1, at, p)[:, :V]
    m = p.sum(1, keepdim=True)
    lq = torch.log_softmax(y, dim=1)
    lqj = lq.gather(1, ids.clamp_min(0).long())
    loss = torch.where(p > 0, p * (lp - lqj), 0.0).sum(1)
    scale = torch.where(p > 0, p * (lp.abs() + lqj.abs()), 0.0).sum(1)
    grad, size = m * torch.exp(lq) - P, m * torch.exp(lq) + P
    if tail:
        r = 1 - m
        r = torch.where(r >= 2.0 ** -20, r, 0.0)
        rest = torch.logsumexp(torch.where(listed, -math.inf, lq), 1, keepdim=True)
        term = torch.where(r > 0, r * (torch.log(r.clamp_min(1e-300)) - rest), 0.0)[:, 0]
        loss = loss + term
        scale = scale + term.abs()
        share = torch.where(listed | torch.isneginf(rest), 0.0, torch.exp(lq - rest))
        r = torch.where(torch.isneginf(rest), 0.0, r)
        grad, size = grad + r * (torch.exp(lq) - share), size + r * (torch.exp(lq) + share)
    w = torch.ones(N, dtype=torch.float64, device=z.device) if w is None else w.double()
    none = w == 0
    each = lambda x: torch.where(none[:, None], 0.0, w[:, None] * x / T)  # noqa: E731
    return (torch.where(none, 0.0, w * loss), each(grad), torch.where(none, 0.0, w.abs() * scale), listed,
            each(size).abs())


def sample64(z, T, k, p, mp, u, near_by=1e-9):
    """Kept mask [B, V], token, prob and whether a cut or the draw lies within
    near_by of a border (equality to 1e-13 apart), of rows z under rules given as
    sequences; each kept token adds the 2^-44 to which its weight is held."""
    dev = z.device
    f = lambda x: torch.as_tensor(x, dtype=torch.float32).to(dev).double().view(-1, 1)  # noqa: E731
    T, p, mp, u = f(T), f(p), f(mp), f(u)
    k = torch.as_tensor(k, dtype=torch.int64).to(dev).view(-1, 1)
    greedy = T == 0
    T = torch.where(greedy, 1.0, T)
    z = z.double()
    V = z.shape[1]
    zs, order = torch.sort(z, dim=1, descending=True, stable=True)
    top = zs[:, :1]
    live = zs >= top - T * 48 * math.log(2.0)
    cum = torch.where(live, torch.exp((zs - top) / T), 0.0).cumsum(1)
    n = live.sum(1, keepdim=True)
    n_k = torch.where(k > 0, torch.minimum(k, n), n)
    inside = torch.arange(V, device=dev) < n_k
    goal = p * cum.gather(1, n_k - 1)
    n_p = torch.minimum((inside & (cum < goal * (1 - 1e-13))).sum(1, keepdim=True) + 1, n_k)
    n_p = torch.where(p < 1, n_p, n_k)
    gap = (cum - goal).abs()
    by = near_by * goal + n_k * 2.0 ** -44
    near = ((gap > 1e-13 * goal) & (gap < by) & inside & (p < 1)).any(1)
    n_m = (zs >= top + T * torch.log(mp.clamp_min(2.0 ** -48))).sum(1, keepdim=True)
    n = torch.where(greedy, 1, torch.minimum(n_p, n_m).clamp_min(1))
    keep = torch.zeros(z.shape, dtype=torch.bool, device=dev)
    keep.scatter_(1, order, torch.arange(V, device=dev) < n)
    w = torch.where(keep, torch.exp((z - top) / T), 0.0)
    run = w.cumsum(1)
    W = run[:, -1:]
    t = u * W
    last = torch.where(keep, torch.arange(V, device=dev), 0).amax(1, keepdim=True)
    token = torch.minimum((run <= t * (1 + 1e-13)).sum(1, keepdim=True), last)
    gap = (run - t).abs()
    near |= ((gap > 1e-13 * W) & (gap < near_by * W + n * 2.0 ** -44) & keep).any(1)
    near &= ~greedy[:, 0]
    return keep, token[:, 0].int(), (w.gather(1, token) / W)[:, 0], near
