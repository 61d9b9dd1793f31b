"""Sampling over rows enough to be streamed, whose first pass adds up masses
below a guessed maximum: every row against the definition in 64 bits.

Whole numbers are equal unless the definition itself finds a cut or a draw
next to a border (1e-9 of the weight, and 2^-44 per kept token, to which the
kernel holds a weight).  prob: one rounding to fp32, 2^-24 of its value, and as
much again for the sums and weights.

The rows: V so that one CTA holds only a part of its row, and one and a half
times the 2 CTAs per SM that run at once.
"""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests._rows64 import sample64  # noqa: E402

PROB_RTOL = 2.0 ** -23
SIZES = [(torch.float32, 30016), (torch.float32, 30011), (torch.bfloat16, 60032), (torch.bfloat16, 60005)]


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    import speculative_decoding_verification_50_gb300 as m
    m.load_library()
    return m


def many():
    return 3 * torch.cuda.get_device_properties(0).multi_processor_count


def check(sv, z, T, k=None, p=None, mp=None, u=None, max_near=0.05, good=None):
    B = z.shape[0]
    dev = lambda x, t: None if x is None else torch.as_tensor(np.asarray(x), dtype=t).cuda()  # noqa: E731
    T, k, p, mp = dev(T, torch.float32), dev(k, torch.int32), dev(p, torch.float32), dev(mp, torch.float32)
    u = dev(u, torch.float32)
    rules = dict(top_k=k, top_p=p, min_p=mp)
    fill = dict(tokens=torch.full((B,), -7, dtype=torch.int32).cuda(), prob=torch.full((B,), -7.0).cuda())
    filt = torch.full_like(z, 5.0)
    o = sv.specv_sample(z, T, u, filtered=filt, **rules, **fill)
    f = sv.specv_filter_logits(z, T, **rules)
    alone = sv.specv_sample(z, T, u, **rules)
    assert torch.equal(f["filtered"], filt) and torch.equal(f["kept"], o["kept"])
    assert all(torch.equal(alone[n], o[n]) for n in ("tokens", "prob", "kept", "row_status"))
    good = torch.ones(B, dtype=torch.bool).cuda() if good is None else good
    bad = ~good
    assert torch.equal(o["row_status"] != 0, bad)
    assert (o["tokens"][bad] == -1).all() and (o["kept"][bad] == 0).all() and torch.isneginf(filt[bad]).all()
    zero = lambda x, off: torch.full((B,), off).cuda() if x is None else x  # noqa: E731
    keep, tok, pr, near = sample64(torch.where(bad[:, None], 0.0, z), T, zero(k, 0), zero(p, 1.0), zero(mp, 0.0), u)
    assert near[good].sum() <= max(1, max_near * B)
    ok = good & ~near
    assert torch.equal(o["kept"][ok].long(), keep[ok].sum(1))
    assert torch.equal(filt[ok], torch.where(keep, z, float("-inf"))[ok])
    assert torch.equal(o["tokens"][ok], tok[ok])
    assert ((o["prob"].double() - pr).abs() <= PROB_RTOL * pr)[ok].all()


@pytest.mark.parametrize("dtype,V", SIZES)
@pytest.mark.parametrize("how", ["top_p", "plain", "min_p", "both"])
def test_low_temperatures(sv, dtype, V, how):
    """The guess below the size from which logits are shifted before they are
    scaled, the maximum above it, below it, or both above; of either sign."""
    B = many()
    rng = np.random.default_rng(V)
    g = torch.Generator(device="cuda").manual_seed(V)
    T = rng.choice([1e-4, 3e-4, 1e-3, 3e-3, 1e-2, 0.1], B).astype(np.float32)
    scale = torch.from_numpy(rng.choice([0.001, 0.1, 2.0], B)).cuda()[:, None]
    shift = torch.from_numpy(rng.choice([-200.0, -9.0, -0.01, 0.0, 0.01, 8.0, 90.0], B)).cuda()[:, None]
    z = torch.randn(B, V, generator=g, device="cuda", dtype=torch.float64) * scale + shift
    # the largest logits, where no guess looks: as far apart as a few tens of T
    top = z.amax(1, keepdim=True) + torch.from_numpy(rng.choice([0.0, 1e-3, 0.03, 0.5, 3.0, 11.0, 150.0], B)).cuda()[:, None]
    room = torch.from_numpy(T.astype(np.float64)).cuda()[:, None]
    z[:, -200:-1] = top - room * 40 * torch.rand(B, 199, generator=g, device="cuda", dtype=torch.float64)
    z = z.to(dtype)
    p = rng.uniform(0.3, 0.999, B) if how in ("top_p", "both") else None
    mp = rng.choice([0.0, 1e-6, 0.01, 0.3], B) if how in ("min_p", "both") else None
    check(sv, z, T, None, p, mp, rng.uniform(0, 1, B))


@pytest.mark.parametrize("dtype,V", SIZES)
def test_maximum_where_no_guess_finds_it(sv, dtype, V):
    """The largest logits at the ends of rows: a little or far above all others,
    alone, infinite, not a number, or of a size that is shifted first."""
    B = many()
    rng = np.random.default_rng(V + 1)
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    z = torch.randn(B, V, generator=g, device="cuda") * 2
    kind = torch.arange(B, device="cuda") % 13
    for i, up in enumerate((0.5, 1.0, 4.0, 5.5, 6.0, 20.0, 300.0)):
        z[kind == i, -3] = 9.0 + up
    z[kind == 7, : V - 8] = -float("inf")
    z[kind == 8] = z[kind == 8] * 30000 - 4e5
    z[kind == 9, -5] = float("nan")
    z[kind == 10, -2] = float("inf")
    z[kind == 11, : V // 2] = torch.finfo(torch.float32).min
    z = z.to(dtype)  # kind 12: as drawn
    if dtype is torch.bfloat16:  # (the lowest value that bf16 has)
        z[kind == 11, : V // 2] = torch.finfo(torch.bfloat16).min
    T = rng.uniform(0.3, 1.5, B).astype(np.float32)
    T[::17] = 0.0
    p = rng.uniform(0.5, 1.0, B).astype(np.float32)
    p[::5] = 1.0
    check(sv, z, T, None, p, rng.choice([0.0, 1e-3], B), rng.uniform(0, 1, B), good=(kind != 9) & (kind != 10))


@pytest.mark.parametrize("dtype,V", SIZES)
def test_rules(sv, dtype, V):
    """Every rule of its row's own, ties among the logits."""
    B = many()
    rng = np.random.default_rng(V + 2)
    g = torch.Generator(device="cuda").manual_seed(V + 2)
    z = torch.randn(B, V, generator=g, device="cuda") * (torch.rand(B, 1, generator=g, device="cuda") * 3 + 0.3)
    z[::7] = (z[::7] * 4).round() / 4
    z[3::50] = -1.25
    z = z.to(dtype)
    check(sv, z, rng.choice([0.0, 0.3, 0.7, 1.0, 1.7], B), rng.choice([0, 0, 1, 5, 50, 1500, V // 2, V, V + 3], B),
          rng.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.99], B), rng.choice([0.0, 0.0, 0.001, 0.1, 0.5, 1.0], B),
          rng.integers(0, 1 << 24, B) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("how", ["list", "few", "streamed"])
def test_prob_of_light_tokens(sv, dtype, how):
    """A uniform of 0 draws the first kept token, of weight 2^0 to 2^-47.9: its
    share of the kept weight, to fp32's rounding."""
    B = many() if how == "streamed" else 64
    V = 60005 if how == "streamed" else 3001
    g = torch.Generator(device="cuda").manual_seed(V)
    T = 0.5 + torch.rand(B, generator=g, device="cuda")
    ln2 = float(np.log(2.0))
    z = torch.randn(B, V, generator=g, device="cuda") - 6
    if how == "list":
        z[:, 700:-1] = -float("inf")
    z[:, -1] = 2.0
    z[:, 0] = 2.0 - T * ln2 * torch.linspace(0.0, 47.9, B, device="cuda")
    z = z.to(dtype)
    k = torch.full((B,), 900, dtype=torch.int32, device="cuda") if how == "list" else None
    o = sv.specv_sample(z, T, torch.zeros(B, device="cuda"), top_k=k)
    y = z.double() / T.double()[:, None]
    w = torch.exp(y - y.amax(1, keepdim=True))
    kept = w >= 2.0 ** -48
    want = torch.where(kept, w, 0.0)[:, 0] / torch.where(kept, w, 0.0).sum(1)
    ok = kept[:, 0]
    assert ok.sum() >= B - B // 32 - 1 and want[ok].min() < 2.0 ** -46
    assert (o["tokens"][ok] == 0).all()
    assert ((o["prob"].double() - want).abs() <= PROB_RTOL * want)[ok].all()


@pytest.mark.parametrize("dtype,V", SIZES)
@pytest.mark.parametrize("end", ["first", "last"])
def test_parts_of_nothing_but_light_tokens(sv, dtype, V, end):
    """A first (last) quarter of tokens just above or below the floor of 2^-48, and
    the maximum where no guess finds it: a uniform of 0 (1) draws a kept token of that
    end."""
    B = many()
    z = torch.full((B, V), -float("inf"), device="cuda")
    light = 40.0 - float(np.log(2.0)) * torch.linspace(47.9, 48.6, B, device="cuda")[:, None]
    if end == "first":
        z[:, : V // 3] = light
        z[:, V // 2: V // 2 + 3000] = 38.0
        z[:, -3] = 40.0
    else:
        z[:, -V // 3:] = light
        z[:, :3000] = 38.0
        z[:, V // 2] = 40.0
    z = z.to(dtype)
    if dtype is torch.bfloat16:  # (steps of 2^-5 there: all rows' light tokens above the floor, or below)
        assert ((z > -float("inf")) & (z < 20)).any(1).all()
    T = torch.ones(B, device="cuda")
    fill = dict(tokens=torch.full((B,), -7, dtype=torch.int32).cuda())
    u = torch.full((B,), 0.0 if end == "first" else 1.0, device="cuda")
    o = sv.specv_sample(z, T, u, **fill)
    keep, tok, pr, _ = sample64(z, T, torch.zeros(B), torch.ones(B), torch.zeros(B), u)
    assert torch.equal(o["kept"].long(), keep.sum(1))
    assert (o["row_status"] == (sv.ROW_FALLBACK if end == "last" else 0)).all()
    # (The light tokens' sum is below the draw's resolution of 2^-44 for each kept
    # token: any of them may be drawn, or the first, last, that is heavier.)
    at = torch.arange(V, device="cuda")
    got = o["tokens"].long()
    assert ((got >= 0) & (got < V)).all() and keep.gather(1, got[:, None]).all()
    heavy = keep & (z > 30.0)
    if end == "first":
        assert (got <= torch.where(heavy, at, V).amin(1)).all()
    else:
        assert (got >= torch.where(heavy, at, -1).amax(1)).all()
        light = keep.any(1) & ((keep & ~heavy & (z.double() > 40.0 - 47.9 * np.log(2.0))).any(1))
        assert torch.equal(got[light], torch.where(keep, at, -1).amax(1)[light])


@pytest.mark.parametrize("dtype,V", [(torch.float32, 30016), (torch.bfloat16, 64000), (torch.bfloat16, 90001)])
def test_second_wave_nearly_empty(sv, dtype, V):
    """Rows a few more than the CTAs that run at once: streamed for tokens, held
    where filtered bf16 rows are wanted alone and fill their shared memory."""
    B = 2 * torch.cuda.get_device_properties(0).multi_processor_count + 16
    rng = np.random.default_rng(V + 3)
    g = torch.Generator(device="cuda").manual_seed(V + 3)
    z = (torch.randn(B, V, generator=g, device="cuda") * 2).to(dtype)
    check(sv, z, rng.choice([0.0, 0.5, 1.0], B), rng.choice([0, 0, 40, 2000], B), rng.choice([1.0, 0.8, 0.95], B),
          rng.choice([0.0, 0.01], B), rng.uniform(0, 1, B))


def test_widest_rows(sv):
    """More of them in flight than L2 holds."""
    V, B = 600001, 264
    g = torch.Generator(device="cuda").manual_seed(14)
    z = torch.randn(B, V, generator=g, device="cuda") * 2
    T = torch.full((B,), 0.9, device="cuda")
    u, p = torch.rand(B, generator=g, device="cuda"), torch.rand(B, generator=g, device="cuda") * 0.4 + 0.6
    f = torch.empty_like(z)
    o = sv.specv_sample(z, T, u, top_p=p, filtered=f)
    close = 0
    for a in range(0, B, 24):
        s = slice(a, a + 24)
        keep, tok, pr, near = sample64(z[s], T[s], torch.zeros(24), p[s], torch.zeros(24), u[s])
        ok = ~near
        close += int(near.sum())
        assert torch.equal(o["kept"][s][ok].long(), keep[ok].sum(1)) and torch.equal(o["tokens"][s][ok], tok[ok])
        assert torch.equal(f[s][ok], torch.where(keep, z[s], -float("inf"))[ok])
        assert ((o["prob"][s].double() - pr).abs() <= PROB_RTOL * pr)[ok].all()
    assert close <= B // 5  # (the borders here: 600001 units of 2^-42 beside 1e-9)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 20187), (torch.float32, 30016), (torch.bfloat16, 60005)])
def test_cuts_far_down_the_tail(sv, dtype, V):
    """top-p of 0.999 to 0.99999: the bins at the cut hold a few roundings of the
    row's sum."""
    g = torch.Generator(device="cuda").manual_seed(V + 4)
    for B in (150, 4 * many()):
        z = (torch.randn(B, V, generator=g, device="cuda") * (2 + 2 * torch.rand(B, 1, generator=g, device="cuda"))).to(dtype)
        u, p = torch.rand(B, generator=g, device="cuda"), 1 - 10 ** -(3 + 2 * torch.rand(B, generator=g, device="cuda"))
        check(sv, z, torch.ones(B), None, p.cpu(), None, u.cpu(), max_near=0.3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [5000, 24762, 60005])
@pytest.mark.parametrize("gap", [-50.0, 0.0, 30.0])
def test_a_few_levels(sv, dtype, V, gap):
    """Rows of a few values with thousands of tokens each, some far apart, and cuts
    just before, at and after the end of a level."""
    rng = np.random.default_rng(V)
    g = torch.Generator(device="cuda").manual_seed(V)
    for B in (60, many()):
        values = gap + torch.tensor([0.0, 0.01, 0.26, 0.5, 1.25, 7.0], device="cuda")
        values = values[torch.randint(0, 6, (B, 5), generator=g, device="cuda")]
        # shares of 0.5 to 0.97 for the first level, the rest of the row for the others
        share = 0.5 + 0.47 * torch.rand(B, 1, generator=g, device="cuda")
        which = torch.randint(1, 5, (B, V), generator=g, device="cuda")
        which[torch.rand(B, V, generator=g, device="cuda") < share] = 0
        z = values.gather(1, which).to(dtype)
        T = torch.from_numpy(rng.choice([0.5, 1.0, 3.0], B)).float()
        # p: the weight down to a level's end, a little more or less, or any
        y = z.double() / T.cuda().double()[:, None]
        w = torch.softmax(y, 1)
        level = z.double().gather(1, torch.randint(0, V, (B, 1), generator=g, device="cuda"))
        p = torch.where(z.double() >= level, w, 0.0).sum(1).float().cpu().numpy()
        p = p + rng.choice([0.0, 0.0, 1e-7, -1e-7, 1e-4, -1e-4, -0.2, 0.01], B).astype(np.float32)
        p[::7] = 0.9999
        check(sv, z, T, None, np.clip(p, 0, 1), rng.choice([0.0, 0.0, 1e-3], B), rng.uniform(0, 1, B), max_near=0.5)
