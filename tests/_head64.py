"""The cross entropy of given tokens from hidden states, and its gradients, in 64 bits, with
what fp32 sums and roundings to bf16 may make of them.

Bounds.  A logit is a sum of D exact products of bf16, taken 16 at a time in fp32: each of
the D / 16 additions is off by at most 2^-23 of the terms' absolute sum (twice half a step,
for sums that are cut off), and so are the additions within a group (two more are counted).
With dz that much, nll is off by 2 dz (its two logits) and 2^-21 (1 + nll) for the
exponentials (2^-22 each) and the sum.  A probability is off by 2 dz + 2^-20 of itself and
by its rounding to bf16, half a step: 2^-8.  Sums of those: the same shares of the absolute
sums; each gradient is rounded once more.
"""
import torch

HALF, HALF16 = torch.finfo(torch.bfloat16).eps / 2, torch.finfo(torch.float16).eps / 2


def head64(h, W, t, scale=1.0, weights=None, up=None):
    h, W, t = h.double(), W.double(), t.long()
    N, V = len(t), len(W)
    use = (t >= 0) & (t < V)
    w = torch.ones(N, dtype=torch.float64, device=h.device) if weights is None else weights.double()
    use &= w != 0
    h = torch.where(use[:, None], h, 0.0)
    z = scale * (h @ W.T)
    D = h.shape[1]
    size = scale * (h.abs() @ W.abs().T).amax(1, keepdim=True)  # of a row's products
    dz = (D / 16 + 2) * 2.0 ** -23 * size[:, 0] + 2.0 ** -23 * z.abs().amax(1)
    at = t.clamp(0, V - 1)[:, None]
    logp = torch.log_softmax(z, 1)
    rest = logp.exp().scatter(1, at, 0.0).sum(1)  # the other tokens' mass
    nll = torch.where(rest < 0.5, -torch.log1p(-rest), -logp.gather(1, at)[:, 0])
    lse = torch.logsumexp(z, 1)
    nll_off = 2 * dz + 2.0 ** -21 * (1 + nll.abs())
    # a row that is nearly certain: the loss keeps the digits of the other tokens' mass
    nll_off = torch.minimum(nll_off, (rest / (1 - rest).clamp_min(1e-300)) * (torch.expm1(2 * dz) + 2.0 ** -20))
    out = dict(loss=torch.where(use, w * nll, 0.0), loss_off=torch.where(use, w.abs() * nll_off, 0.0),
               nll=torch.where(use, nll, 0.0), nll_off=nll_off,
               lse=torch.where(use, lse, 0.0), lse_off=dz + 2.0 ** -21 * (1 + nll.abs()) + 2.0 ** -23 * lse.abs(), use=use)
    g = torch.where(use, w * (1.0 if up is None else up.double()), 0.0)
    d = torch.exp(logp)
    d.scatter_(1, at, -rest[:, None])
    d = torch.where(use[:, None], d * g[:, None], 0.0)
    share = HALF + HALF16 + 2 * dz[:, None] + 2.0 ** -20 + 2.0 ** -23 * lse.abs()[:, None]
    around = torch.nn.functional.pad(d.scatter(1, at, 0.0).abs(), (0, -V % 128)).view(N, -1, 128)
    around = around.amax(2, keepdim=True).expand_as(around).reshape(N, -1)[:, :V]
    doff = torch.where(use[:, None], d.abs() * share + 2.0 ** -40 * around, 0.0)
    gh, gW = scale * (d @ W), scale * (d.T @ h)
    # (sums in fp32: 2^-23 an addition of 16)
    gh_off = scale * ((doff + (V / 16 + 34) * 2.0 ** -23 * d.abs()) @ W.abs()) + HALF * gh.abs()
    gW_off = scale * ((doff + (N / 16 + 2) * 2.0 ** -23 * d.abs()).T @ h.abs()) + HALF * gW.abs()
    return {**out, "grad_hidden": gh, "grad_hidden_off": gh_off, "grad_head": gW, "grad_head_off": gW_off}


def hold(got, want, what, tiny=1e-37):
    """Every element within its bound."""
    off = (got.double() - want[what]).abs()
    most = want[what + "_off"] * 1.01 + tiny
    assert torch.isfinite(got).all(), what
    bad = off > most
    assert not bad.any(), (what, int(bad.sum()), bad.nonzero()[0].tolist(), got[bad][0].item(), want[what][bad][0].item(),
                           (off / most).max().item())


def inputs(N, D, V, seed=0, lean=3.0, pad=0, device="cuda", off=0):
    """hidden, head, targets: rows that lean towards their targets, from not at all to certainty."""
    g = torch.Generator(device=device).manual_seed(seed)
    W = torch.randn(V, D, generator=g, device=device) * (2.0 / D ** 0.5)
    t = torch.randint(0, V, (N,), generator=g, device=device)
    h = torch.randn(N, D, generator=g, device=device) + lean * torch.rand(N, 1, generator=g, device=device) * W[t]

    def place(x):
        x = x.bfloat16()
        if not pad and not off:
            return x
        room = torch.full((x.shape[0] * (D + pad) + off,), float("nan"), dtype=torch.bfloat16, device=device)
        y = room[off:].view(x.shape[0], D + pad)[:, :D]
        return y.copy_(x)

    return place(h), place(W), t.to(torch.int32)
