"""The distillation loss and its gradient against the formula in 64 bits, and
the gradient against differences of the loss.

Tolerances.  Each weight 2^x is taken at an argument rounded twice (2^-24 of
|x| each, |x| <= 64 where it carries weight in these inputs) by a function good
to 2^-22, and a row's sum adds one rounding per addend of one thread and its
tree (at most 2^-24 * 400 in all, in practice a few units): REL = 2^-17 of the
largest gradient in the row covers both; the rounding to the logits' type adds
eps / 2 of the value.  The loss is a sum of p (log p - log q), whose logarithms
are in 64 bits over such sums: REL again, of the sum of the absolute terms.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

REL = 2.0 ** -17


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    import speculative_decoding_verification_50_gb300 as m
    m.load_library()
    return m


def formula(z, ids, t, lse, T, w, tail):
    """(loss, gradient, scale of the loss) of one row, in 64 bits, entry by entry."""
    V = len(z)
    y = z / T
    log_q = y - y.max() - np.log(np.exp(y - y.max()).sum())
    at = [j for j in range(len(ids)) if ids[j] >= 0 and t[j] > -np.inf]
    listed = np.zeros(V, bool)
    listed[[i for i in ids if i >= 0]] = True
    grad, loss, scale = np.zeros(V), 0.0, 0.0
    if not listed.any() or (not at and lse is None):  # one outcome, or none: nothing to learn
        return 0.0, grad, 0.0
    L = lse if lse is not None else np.log(sum(np.exp(t[j] / T - max(t) / T) for j in at)) + max(t) / T
    m = 0.0
    for j in at:
        lp = t[j] / T - L
        p = np.exp(lp)
        m += p
        if p > 0:
            loss += p * (lp - log_q[ids[j]])
            scale += p * (abs(lp) + abs(log_q[ids[j]]))
            grad[ids[j]] -= p
    grad += m * np.exp(log_q)
    r = 1 - m
    if tail and r >= 2.0 ** -20:
        rest = np.exp(log_q[~listed]).sum() if (~listed).any() else 0.0
        if rest > 0:
            loss += r * (np.log(r) - np.log(rest))
            scale += abs(r * (np.log(r) - np.log(rest)))
            share = np.where(listed, 0.0, np.exp(log_q) / rest)
            grad += r * (np.exp(log_q) - share)
        else:
            loss = np.inf
    return w * loss, w * grad / T, w * scale


def make(seed, N, V, K, dtype, noise=1.0, scale=3.0):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(N, V, generator=g) * scale).to(dtype)
    teacher = z.float() + noise * torch.randn(N, V, generator=g)
    val, ids = teacher.topk(min(K, V), dim=1)
    return z.cuda(), ids.int().cuda(), val.contiguous().cuda(), teacher


def check(sv, z, ids, val, lse, T, w, tail, up=None):
    o = sv.specv_distill(z, ids, val, teacher_lse=lse, temperature=T, weights=w, tail=tail, with_grad=True)
    leaf = z.clone().requires_grad_()
    loss = sv.distill_loss(leaf, ids, val, teacher_lse=lse, temperature=T, weights=w, tail=tail)
    up = torch.ones_like(loss) if up is None else up
    (back,) = torch.autograd.grad(loss, leaf, up)
    torch.cuda.synchronize()
    assert (o["row_status"] == 0).all()
    assert torch.equal(loss.detach(), o["loss"])
    n64 = lambda x: None if x is None else x.detach().double().cpu().numpy()  # noqa: E731
    zn, idn, vn, ln, wn, un = n64(z), ids.cpu().numpy(), n64(val), n64(lse), n64(w), n64(up)
    eps = torch.finfo(z.dtype).eps / 2
    T = float(np.float32(T))
    for b in range(z.shape[0]):
        wb = 1.0 if wn is None else wn[b]
        if wb == 0:
            assert o["loss"][b] == 0 and (o["grad"][b] == 0).all() and (back[b] == 0).all()
            continue
        want, grad, scale = formula(zn[b], idn[b], vn[b], None if ln is None else ln[b], T, wb, tail)
        if np.isinf(want):
            assert float(o["loss"][b]) == want
        else:
            assert abs(float(o["loss"][b]) - want) <= REL * max(scale, 1e-3), b
        top = np.abs(grad).max()
        for got, s in ((o["grad"], 1.0), (back, un[b])):
            off = np.abs(n64(got[b]) - s * grad)
            assert (off <= s * (REL * top + eps * np.abs(grad)) + 1e-30).all(), (b, off.max(), top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,V,K,T", [(1, 2, 1, 1.0), (3, 9, 4, 2.0), (5, 37, 37, 1.0), (4, 4097, 64, 1.5),
                                     (3, 20001, 1024, 1.0), (2, 152064, 100, 0.5)])
@pytest.mark.parametrize("how", ["renorm", "lse", "tail"])
def test_random_rows(sv, N, V, K, T, how, dtype):
    z, ids, val, teacher = make(V + K, N, V, K, dtype)
    lse = None if how == "renorm" else torch.logsumexp(teacher.double() / T, 1).float().cuda()
    g = torch.Generator().manual_seed(1)
    w = torch.rand(N, generator=g).cuda() + 0.1
    check(sv, z, ids, val, lse, T, w, how == "tail", up=torch.rand(N, generator=g).cuda() + 0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tail", [False, True])
def test_ragged_lists_weights_and_repeats(sv, dtype, tail):
    z, ids, val, teacher = make(5, 8, 5000, 40, dtype)
    lse = torch.logsumexp(teacher, 1).cuda()
    for b, n in enumerate([0, 1, 5, 39, 40, 40, 40, 40]):
        ids[b, n:] = -1
    ids[2, 0] = -1                    # holes
    ids[5, 3] = ids[5, 7]             # an id listed twice, and three times
    ids[6, 10] = ids[6, 20] = ids[6, 30]
    val[7, 5:9] = -float("inf")       # entries without mass
    val[5] -= 1.0                     # (keeps the repeats' mass below one)
    val[6] -= 1.0
    w = torch.tensor([1, 1, 0, 2, 0.5, 1, 1, 1.0]).cuda()
    check(sv, z, ids, val, lse if tail else None, 1.0, w, tail)


def test_weightless_rows_are_not_read(sv):
    z, ids, val, _ = make(6, 4, 3000, 16, torch.float32)
    z[1] = float("nan")
    ids[1] = 1 << 30
    w = torch.tensor([1, 0, 1, 0.0]).cuda()
    check(sv, z, ids, val, None, 1.0, w, False)


def test_masked_student_logits(sv):
    """-inf and the lowest value among the student's logits, listed or not."""
    z, ids, val, teacher = make(7, 4, 2000, 16, torch.float32)
    lse = torch.logsumexp(teacher, 1).cuda()
    listed = torch.zeros(4, 2000, dtype=torch.bool).cuda().scatter_(1, ids.long(), True)
    z[0][~listed[0]] = -float("inf")          # no mass outside the list
    z[1][~listed[1] & (torch.arange(2000).cuda() % 2 == 0)] = -float("inf")
    z[2][~listed[2]] = torch.finfo(torch.float32).min
    check(sv, z, ids, val, lse, 1.0, None, True)
    z, ids, val, _ = make(8, 1, 2000, 16, torch.float32)
    z[0, ids[0, 3].long()] = -float("inf")    # the student rules out a listed token
    o = sv.specv_distill(z, ids, val, with_grad=True)
    assert float(o["loss"][0]) == float("inf") and torch.isfinite(o["grad"]).all()


def test_flagged_rows(sv):
    z, ids, val, teacher = make(9, 8, 1000, 8, torch.float32)
    lse = torch.logsumexp(teacher, 1).cuda()
    z[0, 4], z[1, 4] = float("nan"), float("inf")
    z[2] = -float("inf")
    ids[3, 2], ids[4, 2] = 1000, -2
    val[5, 1] = float("nan")
    lse[6] = float("inf")
    o = sv.specv_distill(z, ids, val, teacher_lse=lse, tail=True, with_grad=True)
    N, T = sv.ROW_NONFINITE, sv.ROW_BAD_TOKEN
    assert o["row_status"].tolist() == [N, N, N, T, T, N, N, 0]
    assert (o["loss"][:7] == 0).all() and (o["grad"][:7] == 0).all() and o["loss"][7] > 0
    back = sv.specv_distill_backward(z, ids, val, o["stats"], teacher_lse=lse, tail=True)
    assert (back[:7] == 0).all() and back[7].abs().max() > 0


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(sv, tail):
    """Central differences of the fp32 loss: a step of h = 2^-5 leaves h^2 of a
    third derivative below 1 (4e-4 of a gradient of order one, taken as 1e-3)
    and 2 * 2^-22 * 8 / 2h of rounding (6e-5)."""
    z, ids, val, teacher = make(10, 1, 50, 6, torch.float32, scale=1.0)
    lse = torch.logsumexp(teacher, 1).cuda()
    kw = dict(teacher_lse=lse, tail=tail)
    grad = sv.specv_distill(z, ids, val, with_grad=True, **kw)["grad"][0]
    h = 2.0 ** -5
    up, down = z.repeat(50, 1), z.repeat(50, 1)
    up.diagonal().add_(h)
    down.diagonal().sub_(h)
    many = lambda x: x.repeat(50, *[1] * (x.dim() - 1))  # noqa: E731
    f = lambda x: sv.specv_distill(x, many(ids), many(val), teacher_lse=many(lse), tail=tail)["loss"]  # noqa: E731
    diff = (f(up) - f(down)) / (2 * h)
    assert (diff - grad).abs().max() <= 1e-3 + 1e-4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 2), (8, 0)])
def test_layouts(sv, dtype, pad, off):
    z, ids, val, _ = make(11, 6, 4099, 32, dtype)
    buf = torch.zeros(6, 4099 + pad + off, dtype=dtype).cuda()
    view = buf[:, off:off + 4099]
    view.copy_(z)
    wide_i, wide_v = torch.full((6, 40), -7, dtype=torch.int32).cuda(), torch.zeros(6, 40).cuda()
    wide_i[:, :32], wide_v[:, :32] = ids, val
    out = torch.full((6, 4099 + pad + off), 9.0, dtype=dtype).cuda()
    a = sv.specv_distill(z, ids, val, with_grad=True)
    b = sv.specv_distill(view, wide_i[:, :32], wide_v[:, :32], grad=out[:, off:off + 4099])
    assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["grad"], out[:, off:off + 4099])
    assert (out[:, :off] == 9).all() and (out[:, off + 4099:] == 9).all()
    c = sv.specv_distill_backward(view, wide_i[:, :32], wide_v[:, :32], a["stats"])
    d = sv.specv_distill_backward(z, ids, val, a["stats"])
    assert torch.equal(c, d)


def test_graph_and_stream(sv):
    z, ids, val, _ = make(12, 16, 32000, 32, torch.bfloat16)
    want = sv.specv_distill(z, ids, val, with_grad=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = sv.specv_distill(z, ids, val, with_grad=True)
    s.synchronize()
    bufs = {n: torch.empty_like(want[n]) for n in ("loss", "stats", "grad", "row_status")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.specv_distill(z, ids, val, **bufs)
    graph.replay()
    torch.cuda.synchronize()
    for n in bufs:
        assert torch.equal(want[n], other[n]) and torch.equal(bufs[n], want[n]), n


def test_top_logits_feed_the_loss(sv):
    """A student equal to its teacher has no loss and no gradient but rounding."""
    g = torch.Generator().manual_seed(13)
    z = torch.randn(8, 6000, generator=g).mul(2).cuda()
    for T in (1.0, 2.0):
        top = sv.specv_top_logits(z, 64, temperature=T)
        o = sv.specv_distill(z, top["ids"], top["values"], teacher_lse=top["lse"], temperature=T, tail=True,
                             with_grad=True)
        assert o["loss"].abs().max() <= REL and o["grad"].abs().max() <= REL


@pytest.mark.parametrize("dtype,V", [(torch.float32, 30016), (torch.float32, 50255), (torch.bfloat16, 60032),
                                     (torch.bfloat16, 100001)])
@pytest.mark.parametrize("tail", [False, True])
def test_many_rows(sv, dtype, V, tail):
    """Rows enough to fill the GPU take another split than a few do."""
    g = torch.Generator(device="cuda").manual_seed(V)
    N, K = 400, 40
    z = (torch.randn(N, V, generator=g, device="cuda") * 3).to(dtype)
    teacher = z.float() + torch.randn(N, V, generator=g, device="cuda")
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(teacher, 1) if tail else None
    ids[::11, 3] = ids[::11, 9]        # repeats
    val[::11] -= 1.0
    ids[::13, 20:] = -1
    w = torch.rand(N, generator=g, device="cuda") + 0.1
    w[::17] = 0
    kw = lambda s: dict(teacher_lse=None if lse is None else lse[s], weights=w[s], tail=tail)  # noqa: E731
    whole = sv.specv_distill(z, ids, val, with_grad=True, **kw(slice(None)))
    alone = sv.specv_distill(z, ids, val, **kw(slice(None)))  # without the gradient: a third split
    assert (whole["loss"] - alone["loss"]).abs().max() <= REL * (1 + whole["loss"].abs().max())
    for a in range(0, N, 40):
        s = slice(a, a + 8)
        q = sv.specv_distill(z[s], ids[s], val[s], with_grad=True, **kw(s))
        assert (q["loss"] - whole["loss"][s]).abs().max() <= REL * (1 + q["loss"].abs().max())
        top = q["grad"].float().abs().amax(1, keepdim=True)
        off = (q["grad"].float() - whole["grad"][s].float()).abs()
        eps = torch.finfo(dtype).eps
        assert (off <= REL * top + eps * q["grad"].float().abs()).all()
    some = torch.arange(0, N, 23, device="cuda")
    check(sv, z[some].contiguous(), ids[some].contiguous(), val[some].contiguous(),
          None if lse is None else lse[some].contiguous(), 1.0, w[some].contiguous(), tail)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 769999), (torch.bfloat16, 1539999)])
def test_widest_rows(sv, dtype, V):
    z, ids, val, teacher = make(V, 2, V, 1024, dtype)
    lse = torch.logsumexp(teacher.double(), 1).float().cuda()
    check(sv, z, ids, val, lse, 1.0, None, True)
