"""The row operators' definitions in 64 bits over whole batches (torch, on the
inputs' device), so that tests can hold every row against them."""
import math

import torch


def distill64(z, ids, t, lse=None, T=1.0, w=None, tail=False):
    """Loss [N], its gradient [N, V] (of the sum), the sum of the absolute terms
    of the loss [N], and the mask of listed ids [N, V]."""
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
    grad = m * torch.exp(lq) - P
    if tail:
        r = 1 - m
        r = torch.where(r >= 2.0 ** -20, r, 0.0)
        rest = torch.logsumexp(torch.where(listed, -math.inf, lq), 1, keepdim=True)
        term = torch.where(r > 0, r * (torch.log(r.clamp_min(1e-300)) - rest), 0.0)[:, 0]
        loss = loss + term
        scale = scale + term.abs()
        share = torch.where(listed | torch.isneginf(rest), 0.0, torch.exp(lq - rest))
        grad = grad + torch.where(torch.isneginf(rest), 0.0, r) * (torch.exp(lq) - share)
    w = torch.ones(N, dtype=torch.float64, device=z.device) if w is None else w.double()
    none = w == 0
    return (torch.where(none, 0.0, w * loss), torch.where(none[:, None], 0.0, w[:, None] * grad / T),
            torch.where(none, 0.0, w.abs() * scale), listed)
