"""Sampling under temperature, top-k, top-p and min-p, and filtered logits,
against a 64-bit restatement of the definition in numpy.

Whole numbers (the kept count, the kept set, the token) are equal unless the
restatement itself finds a cut or a draw within 1e-9 of a border, exact
equality apart.  prob is a quotient of sums good to about 1e-9, rounded once to
fp32: 2^-24 of its value and as much again for the sums.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

NEAR = 1e-9
PROB_RTOL = 2.0 ** -23
LOWEST = float(np.finfo(np.float32).min)


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    import speculative_decoding_verification_50_gb300 as m
    m.load_library()
    return m


def restate(z, T, k, p, mp, u):
    """(kept mask, token, prob, near a border) of one row z (float64)."""
    V = len(z)
    keep = np.zeros(V, bool)
    if T == 0:
        i = int(np.argmax(z))
        keep[i] = True
        return keep, i, 1.0, False
    T = float(np.float32(T))
    order = np.argsort(-z, kind="stable")
    w = np.exp((z[order] - z[order[0]]) / T)
    live = z[order] >= z[order[0]] + T * -48 * np.log(2.0)
    w = np.where(live, w, 0.0)
    n_k = int(live.sum()) if k == 0 else min(int(k), int(live.sum()))
    cum = np.cumsum(w)
    near = False
    n = n_k
    if p < 1:
        goal = float(np.float32(p)) * cum[n_k - 1]
        reached = cum[:n_k] >= goal * (1 - 1e-13)
        n = int(np.argmax(reached)) + 1 if reached.any() else n_k
        gap = np.abs(cum[:n_k] - goal)
        gap = gap[gap > 1e-12 * goal]
        near |= bool(gap.size and gap.min() < NEAR * goal)
    mp = float(np.float32(mp))
    n_m = int((z[order] >= z[order[0]] + T * np.log(max(mp, 2.0 ** -48))).sum())
    n = max(1, min(n, n_m))
    keep[order[:n]] = True
    wi = np.where(keep, np.exp((z - z[order[0]]) / T), 0.0)
    run = np.cumsum(wi)
    t = float(np.float32(u)) * run[-1]
    over = np.flatnonzero(run > t * (1 + 1e-13))
    tok = int(over[0]) if over.size else int(np.flatnonzero(keep)[-1])
    gap = np.abs(run[keep] - t)
    gap = gap[gap > 1e-12 * run[-1]]
    near |= bool(gap.size and gap.min() < NEAR * run[-1])
    return keep, tok, wi[tok] / run[-1], near


def check(sv, z, T, k, p, mp, u, dtype=torch.float32, max_near=0.05):
    """z float32 [B, V] (numpy), the rest per row; runs both entry points."""
    zt = torch.from_numpy(np.ascontiguousarray(z, np.float32)).to(dtype).cuda()
    dev = lambda x, t: torch.from_numpy(np.asarray(x, t)).cuda()  # noqa: E731
    rules = dict(top_k=dev(k, np.int32), top_p=dev(p, np.float32), min_p=dev(mp, np.float32))
    filt = torch.empty_like(zt)
    o = sv.specv_sample(zt, dev(T, np.float32), dev(u, np.float32), filtered=filt, **rules)
    f = sv.specv_filter_logits(zt, dev(T, np.float32), **rules)
    torch.cuda.synchronize()
    assert (o["row_status"] == 0).all()
    assert torch.equal(filt, f["filtered"]) and torch.equal(o["kept"], f["kept"])
    zd = zt.float().cpu().numpy().astype(np.float64)
    got = filt.float().cpu().numpy()
    tokens, prob, kept = (o[n].cpu().numpy() for n in ("tokens", "prob", "kept"))
    skipped = 0
    for b in range(z.shape[0]):
        keep, tok, pr, near = restate(zd[b], T[b], k[b], p[b], mp[b], u[b])
        if near:
            skipped += 1
            continue
        assert kept[b] == keep.sum(), (b, kept[b], keep.sum(), T[b], k[b], p[b], mp[b])
        assert np.array_equal(np.isfinite(got[b]) & (got[b] > -np.inf), keep), b
        assert np.array_equal(got[b][keep], zd[b][keep].astype(np.float32))
        assert tokens[b] == tok, (b, tokens[b], tok, T[b], k[b], p[b], mp[b], u[b])
        assert abs(prob[b] - pr) <= PROB_RTOL * pr
    assert skipped <= max(1, max_near * z.shape[0])


def rules_of(rng, B, V):
    return (rng.choice([0.0, 0.3, 0.7, 1.0, 1.7], B), rng.choice([0, 0, 1, 5, 50, max(1, V // 2), V, V + 3], B),
            rng.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.99], B), rng.choice([0.0, 0.0, 0.001, 0.1, 0.5, 1.0], B),
            np.where(rng.random(B) < 0.3, rng.choice([0.0, 0.25, 0.5, 1 - 2.0 ** -24, 2.0 ** -24], B),
                     rng.integers(0, 1 << 24, B) * 2.0 ** -24))  # fp32 in [0, 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 37, 511, 4097, 20001, 50257, 152064])
def test_random_rows(sv, V, dtype):
    rng = np.random.default_rng(V)
    B = 48 if V < 100000 else 24
    z = rng.normal(0, 1, (B, V)) * rng.uniform(0.5, 4, (B, 1)) + rng.normal(0, 20, (B, 1))
    z[:, rng.integers(0, V, 4)] += rng.uniform(0, 8, (B, 4))
    check(sv, z, *rules_of(rng, B, V), dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [64, 3000, 40000])
def test_equal_logits(sv, V, dtype):
    """Ties go to the lowest index, past what is sorted at once too."""
    rng = np.random.default_rng(3)
    B = 40
    z = np.zeros((B, V)) + rng.choice([0.0, -3.0, 700.0], (B, 1))
    z[10:] += np.where(rng.random((B - 10, V)) < 0.5, 0.0, -1.0)   # two levels
    z[25:] += np.where(rng.random((B - 25, V)) < 0.01, 2.0, 0.0)   # and a few above
    T, k, p, mp, u = rules_of(rng, B, V)
    k = rng.choice([0, 1, V // 3, V - 1, 2049, 2500], B)
    p = rng.choice([1.0, 0.5, 0.25, 0.9, 0.123], B)
    check(sv, z, np.where(T == 0, 1.0, T), k, p, mp, u, dtype=dtype)


def test_signed_zeros_are_equal(sv):
    z = np.tile(np.where(np.arange(300) % 2 == 0, -0.0, 0.0).astype(np.float32), (4, 1))
    check(sv, z, [1.0] * 4, [0, 7, 0, 100], [1.0, 1.0, 0.5, 0.5], [0.0, 0.0, 0.0, 1.0], [0.3, 0.99, 0.7, 0.2])


@pytest.mark.parametrize("T", [1e-6, 0.01, 100.0, 1e5])
@pytest.mark.parametrize("scale", [1e-3, 1.0, 1e4, 1e30])
def test_scales(sv, T, scale):
    """Logits and temperatures far from one: bins too full, or nearly empty."""
    rng = np.random.default_rng(int(abs(np.log10(T * scale)) * 7) + 1)
    B, V = 16, 9001
    z = rng.normal(0, 1, (B, V)).astype(np.float32) * np.float32(scale)
    _, k, p, mp, u = rules_of(rng, B, V)
    check(sv, z, np.full(B, T), k, p, mp, u)


def test_masked_logits(sv):
    """-inf and the lowest finite value in masked places; one token left; none."""
    rng = np.random.default_rng(5)
    B, V = 24, 3001
    z = rng.normal(0, 2, (B, V)).astype(np.float32)
    z[rng.random((B, V)) < 0.6] = -np.inf
    z[8:16][np.isinf(z[8:16])] = LOWEST
    z[16] = -np.inf
    z[16, 1234] = -5.0
    z[17] = LOWEST
    z[18, :] = LOWEST
    z[18, 3000] = 0.0
    z[19] = -np.inf
    z[19, 7] = LOWEST
    T, k, p, mp, u = rules_of(rng, B, V)
    T = np.where(T == 0, 0.8, T)
    check(sv, z, T, k, p, mp, u)
    check(sv, z, np.zeros(B), k, p, mp, u)


def test_flagged_rows(sv):
    V = 1000
    z = np.zeros((9, V), np.float32)
    z[0, 3] = np.nan
    z[1, 5] = np.inf
    z[2] = -np.inf
    zt = torch.from_numpy(z).cuda()
    T = torch.tensor([1, 1, 1, -1, float("nan"), float("inf"), 1, 1, 1.0]).cuda()
    k = torch.tensor([0, 0, 0, 0, 0, 0, -1, 0, 0], dtype=torch.int32).cuda()
    p = torch.tensor([1, 1, 1, 1, 1, 1, 1, float("nan"), 1.0]).cuda()
    mp = torch.tensor([0, 0, 0, 0, 0, 0, 0, 0, 1.5]).cuda()
    f = torch.empty_like(zt)
    o = sv.specv_sample(zt, T, torch.full((9,), 0.5).cuda(), top_k=k, top_p=p, min_p=mp, filtered=f)
    want = [sv.ROW_NONFINITE] * 3 + [sv.ROW_BAD_TEMP] * 3 + [sv.ROW_BAD_FILTER] * 3
    assert o["row_status"].tolist() == want
    assert o["tokens"].tolist() == [-1] * 9 and o["kept"].tolist() == [0] * 9
    assert o["prob"].tolist() == [0.0] * 9 and torch.isneginf(f).all()


def test_uniform_of_one_takes_the_last_kept_token(sv):
    z = torch.zeros(2, 100).cuda()
    z[:, 90:] = -100.0
    o = sv.specv_sample(z, torch.ones(2).cuda(), torch.tensor([1.0, float("nan")]).cuda(),
                        top_k=torch.tensor([80, 80], dtype=torch.int32).cuda())
    assert o["tokens"].tolist() == [79, 79]
    assert o["row_status"].tolist() == [sv.ROW_FALLBACK] * 2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("pad,off", [(0, 0), (5, 0), (8, 3), (7, 1)])
def test_layouts(sv, dtype, pad, off):
    """[B, R, V] views with any strides and base give what contiguous rows give;
    rules are shared by an entry's rows; filtering in place."""
    g = torch.Generator().manual_seed(7)
    B, R, V = 5, 3, 4099
    buf = torch.randn(B, R + 1, V + pad + off, generator=g).mul(3).to(dtype).cuda()
    view = buf[:, :R, off:off + V]
    T = torch.tensor([0.0, 0.7, 1.0, 1.0, 1.3]).cuda()
    k = torch.tensor([0, 20, 0, 300, 0], dtype=torch.int32).cuda()
    p = torch.tensor([1.0, 0.9, 0.95, 1.0, 0.5]).cuda()
    u = torch.rand(B, R, generator=g).cuda()
    rep = lambda x: x.repeat_interleave(R)  # noqa: E731
    flat = view.reshape(B * R, V).contiguous()
    a = sv.specv_sample(view, T, u, top_k=k, top_p=p)
    b = sv.specv_sample(flat, rep(T), u.flatten(), top_k=rep(k), top_p=rep(p))
    for n in ("tokens", "prob", "kept", "row_status"):
        assert torch.equal(a[n].flatten(), b[n]), n
    want = sv.specv_filter_logits(flat, rep(T), top_k=rep(k), top_p=rep(p))["filtered"]
    rest = buf.clone()
    sv.specv_filter_logits(view, T, top_k=k, top_p=p, filtered=view)
    assert torch.equal(view.reshape(B * R, V), want)
    rest[:, :R, off:off + V] = view
    assert torch.equal(buf, rest)  # nothing else was written


def test_large_vocabulary(sv):
    """A row that takes the largest cluster; beyond that the call is refused."""
    rng = np.random.default_rng(8)
    z = rng.normal(0, 3, (3, 700001)).astype(np.float32)
    check(sv, z, [1.0, 0.8, 1.0], [0, 1000, 0], [0.9, 0.9, 1.0], [0.0, 0.0, 0.001], [0.3, 0.6, 0.9])
    with pytest.raises(sv.SpecvError):
        sv.specv_filter_logits(torch.zeros(1, 1 << 20).cuda(), torch.ones(1).cuda())


def test_stream_and_graph(sv):
    g = torch.Generator().manual_seed(9)
    z = torch.randn(6, 32000, generator=g).mul(2.5).cuda()
    T, u = torch.full((6,), 0.9).cuda(), torch.rand(6, generator=g).cuda()
    p = torch.full((6,), 0.9).cuda()
    want = sv.specv_sample(z, T, u, top_p=p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = sv.specv_sample(z, T, u, top_p=p)
    s.synchronize()
    bufs = {n: torch.empty_like(want[n]) for n in ("tokens", "prob", "kept", "row_status")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.specv_sample(z, T, u, top_p=p, **bufs)
    z.copy_(z.roll(1, 0))
    u.copy_(u.roll(1, 0))
    graph.replay()
    torch.cuda.synchronize()
    for n in bufs:
        assert torch.equal(want[n], other[n]) and torch.equal(bufs[n], want[n].roll(1, 0))


def test_same_bits_every_time(sv):
    g = torch.Generator().manual_seed(10)
    z = torch.randn(64, 50257, generator=g).mul(2).to(torch.bfloat16).cuda()
    a = [sv.specv_sample(z, torch.ones(64).cuda(), torch.full((64,), 0.37).cuda(),
                         top_p=torch.full((64,), 0.95).cuda()) for _ in range(3)]
    for o in a[1:]:
        assert all(torch.equal(o[n], a[0][n]) for n in o)


def test_filtered_verification_keeps_the_rules(sv):
    """Draft tokens sampled under the rules, verified on filtered logits: every
    output token is one that the target's rules keep, and a draft equal to the
    target is accepted whole."""
    g = torch.Generator().manual_seed(11)
    B, K, V = 16, 4, 8000
    target = torch.randn(B, K + 1, V, generator=g).mul(3).cuda()
    draft = target[:, :K] + torch.randn(B, K, V, generator=g).cuda()
    T = torch.full((B,), 0.8).cuda()
    rules = dict(top_k=torch.full((B,), 40, dtype=torch.int32).cuda(), top_p=torch.full((B,), 0.9).cuda())
    u = torch.rand(B, 2 * K + 1, generator=g).cuda()
    fd = torch.empty_like(draft)
    x = sv.specv_sample(draft, T, u[:, :K].contiguous(), filtered=fd, **rules)["tokens"]
    ft = sv.specv_filter_logits(target, T, **rules)["filtered"]
    o = sv.specv_verify(ft, fd, x, T, u[:, K:].contiguous())
    for b in range(B):
        for i in range(int(o["accept_len"][b]) + 1):
            assert torch.isfinite(ft[b, i, o["out_tokens"][b, i]])
    x = sv.specv_sample(target[:, :K], T, u[:, :K].contiguous(), **rules)["tokens"]
    o = sv.specv_verify(ft, ft[:, :K], x, T, u[:, K:].contiguous())
    assert (o["accept_len"] == K).all()


@pytest.mark.parametrize("dtype,V", [(torch.float32, 30016), (torch.float32, 30011), (torch.bfloat16, 60032),
                                     (torch.bfloat16, 60005), (torch.float32, 152064)])
def test_many_rows(sv, dtype, V):
    """Rows enough to fill the GPU several times take another split than a few
    do: the same whole numbers, and the definition on some of them."""
    rng = np.random.default_rng(V)
    B = 1300
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(B, V, generator=g, device="cuda")
    z *= torch.rand(B, 1, generator=g, device="cuda") * 3 + 0.3
    z[:, 5:9] += 6
    z[::7] = (z[::7] * 4).round() / 4          # many ties
    z[3::50] = -1.25                           # nothing but ties
    z[11::50, 1:] = -float("inf")
    z = z.to(dtype)
    T, k, p, mp, u = rules_of(rng, B, V)
    k[40:80] = rng.choice([1500, V // 2, 3], 40)
    dev = lambda x, t: torch.from_numpy(np.asarray(x, t)).cuda()  # noqa: E731
    rules = [dev(k, np.int32), dev(p, np.float32), dev(mp, np.float32)]
    T32, u32 = dev(T, np.float32), dev(u, np.float32)
    f = torch.empty_like(z)
    o = sv.specv_sample(z, T32, u32, top_k=rules[0], top_p=rules[1], min_p=rules[2], filtered=f)
    fo = sv.specv_filter_logits(z, T32, top_k=rules[0], top_p=rules[1], min_p=rules[2])
    assert torch.equal(fo["filtered"], f) and torch.equal(fo["kept"], o["kept"])
    del fo
    for a in range(0, B, 20):
        s = slice(a, a + 20)
        few = torch.empty_like(z[s])
        q = sv.specv_sample(z[s], T32[s], u32[s], top_k=rules[0][s], top_p=rules[1][s], min_p=rules[2][s], filtered=few)
        assert torch.equal(few, f[s]), a
        for n in ("tokens", "kept", "row_status"):
            assert torch.equal(q[n], o[n][s]), (a, n)
        assert (q["prob"] - o["prob"][s]).abs().max() <= PROB_RTOL
    for b in range(0, B, 37):
        row = z[b].float().cpu().numpy().astype(np.float64)
        keep, tok, pr, near = restate(row, T[b], k[b], p[b], mp[b], u[b])
        if not near:
            assert int(o["kept"][b]) == keep.sum() and int(o["tokens"][b]) == tok
            assert abs(float(o["prob"][b]) - pr) <= PROB_RTOL * pr
            assert np.array_equal(f[b].float().cpu().numpy() > -np.inf, keep)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
def test_maximum_where_no_guess_finds_it(sv, dtype):
    """Many rows whose largest logits lie at the ends of the row: a little or far
    above all others, alone, infinite, or of a size that is shifted first."""
    V, B = 30016, 352
    rng = np.random.default_rng(5)
    g = torch.Generator(device="cuda").manual_seed(5)
    z = torch.randn(B, V, generator=g, device="cuda") * 2
    kind = torch.arange(B, device="cuda") % 11
    for i, up in enumerate((1.0, 4.0, 5.5, 6.0, 20.0, 300.0)):
        z[kind == i, -3] = 9.0 + up
    z[kind == 6, : V - 8] = -float("inf")
    z[kind == 7] = z[kind == 7] * 30000 - 4e5
    z[kind == 8, -5] = float("nan")
    z[kind == 9, -2] = float("inf")
    z = z.to(dtype)  # kind 10: as drawn
    T = rng.uniform(0.3, 1.5, B).astype(np.float32)
    p = rng.uniform(0.5, 1.0, B).astype(np.float32)
    p[::5] = 1.0
    mp = rng.choice([0.0, 1e-3], B).astype(np.float32)
    u = rng.uniform(0, 1, B).astype(np.float32)
    dev = lambda x: torch.from_numpy(x).cuda()  # noqa: E731
    f = torch.empty_like(z)
    o = sv.specv_sample(z, dev(T), dev(u), top_p=dev(p), min_p=dev(mp), filtered=f)
    for a in range(0, B, 16):
        s = slice(a, a + 16)
        few = torch.empty_like(z[s])
        q = sv.specv_sample(z[s], dev(T[s]), dev(u[s]), top_p=dev(p[s]), min_p=dev(mp[s]), filtered=few)
        assert torch.equal(few, f[s]), a
        for n in ("tokens", "kept", "row_status"):
            assert torch.equal(q[n], o[n][s]), (a, n)
        assert (q["prob"] - o["prob"][s]).abs().max() <= PROB_RTOL
    bad = ((kind == 8) | (kind == 9)).cpu().numpy()
    assert np.array_equal(o["row_status"].cpu().numpy() != 0, bad)
    for b in list(range(0, 33)) + list(range(33, B, 29)):
        if bad[b]:
            assert int(o["tokens"][b]) == -1 and int(o["kept"][b]) == 0
            continue
        row = z[b].float().cpu().numpy().astype(np.float64)
        keep, tok, pr, near = restate(row, T[b], 0, p[b], mp[b], u[b])
        if not near:
            assert int(o["kept"][b]) == keep.sum() and int(o["tokens"][b]) == tok, b
            assert abs(float(o["prob"][b]) - pr) <= PROB_RTOL * pr
            assert np.array_equal(f[b].float().cpu().numpy() > -np.inf, keep)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 769999), (torch.bfloat16, 1539999)], ids=["fp32", "bf16"])
def test_widest_rows(sv, dtype, V):
    """The widest rows that are taken, held by sixteen CTAs each."""
    rng = np.random.default_rng(12)
    z = rng.normal(0, 2, (3, V)).astype(np.float32)
    check(sv, z, [1.0, 0.7, 0.0], [0, 900, 0], [0.9, 0.95, 1.0], [0.0, 0.001, 0.0], [0.37, 0.62, 0.5], dtype=dtype)


def test_widest_rows_streamed(sv):
    """Wide rows enough to fill the GPU: more of them in flight than L2 holds."""
    V, B = 600001, 260
    g = torch.Generator(device="cuda").manual_seed(13)
    z = torch.randn(B, V, generator=g, device="cuda") * 2
    T = torch.full((B,), 0.9, device="cuda")
    u, p = torch.rand(B, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda") * 0.4 + 0.6
    o = sv.specv_sample(z, T, u, top_p=p)
    for a in range(0, B, 26):
        s = slice(a, a + 3)
        q = sv.specv_sample(z[s], T[s], u[s], top_p=p[s])
        for n in ("tokens", "kept", "row_status"):
            assert torch.equal(q[n], o[n][s]), (a, n)
        assert (q["prob"] - o["prob"][s]).abs().max() <= PROB_RTOL
