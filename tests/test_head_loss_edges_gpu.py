"""specv_head_loss and its backward pass where their range and their digits end, against the
definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._head64 import head64, hold, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def both(h, W, t, **how):
    """The gradients of one call, and of a backward pass from statistics."""
    one = sv.specv_head_loss(h, W, t, with_grad=True, **how)
    two = sv.specv_head_loss(h, W, t, targets_only=True, **how)
    two.update(sv.specv_head_loss_backward(h, W, t, two["stats"], **how))
    return one, two


@pytest.mark.parametrize("N", [6, 300])
def test_gradients_of_nearly_certain_rows(N):
    """The other tokens' probabilities are 2^-108 to 2^-122: the gradients are that small, and right.
    (bf16 numbers below 2^-126 are 2^-133 apart.)"""
    g = torch.Generator(device="cuda").manual_seed(N)
    W = torch.randn(9, 24, generator=g, device="cuda").bfloat16()
    W[:, 0] = 0
    W[4, 0] = 1
    h = torch.zeros(N, 24, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = torch.linspace(75, 84, N, device="cuda")
    t = torch.full((N,), 4, dtype=torch.int32, device="cuda")
    want = head64(h, W, t)
    assert (want["loss"] < 2.0 ** -104).all() and (want["loss"] > 2.0 ** -122).all()
    for o in both(h, W, t):
        for k in ("loss", "grad_hidden", "grad_head"):
            hold(o[k], want, k, tiny=2.0 ** -134)


FAR = [(6, 1, 1.0), (6, -1, 1.0), (12, 1, 1.0), (12, -1, 0.5), (17, 1, 1.0), (17, -1, 1.0), (20, 1, 1.0), (20, -1, 1.0),
       (1, 1, 2.0 ** 19), (5, -1, 2.0 ** 19), (24, 1, 1.0), (31, 1, 1.0), (33, -1, 1.0), (60, 1, 1.0), (60, -1, 1.0), (100, 1, 2.0 ** -8),
       (127, 1, 1.0), (127, -1, 1.0)]


@pytest.mark.parametrize("N", [3, 45, 200, 300])
@pytest.mark.parametrize("D", [16, 520])
@pytest.mark.parametrize("k,sign,scale", FAR)
def test_logits_far_from_zero(N, D, k, sign, scale):
    """Logits 2^k (+-1 + j 2^-18), which fp32 holds exactly, as it does their differences: losses
    and probabilities that are ordinary ones keep their digits.

    Bounds: exponentials and sums 2^-20, exponents of up to 128 rounded once 2^-18; dz in bf16
    2^-8, of weights in fp16 2^-11 and 2^-40 of the largest, its exponents (up to 2048, or what
    a probability above 2^-126 leaves of them) 2^-12.  A backward pass from statistics knows the
    smaller of nll and |lse| to 2^-24 of it, and takes it off in a step that is rounded as much."""
    V = 700
    g = torch.Generator(device="cuda").manual_seed(k + N)
    j = torch.randint(-6, 1, (V,), generator=g, device="cuda")
    j[5], j[300], j[699] = 1, 1, -6
    W = torch.zeros(V, D, dtype=torch.bfloat16, device="cuda")
    W[:, 0], W[:, 1] = 1, (j * 2.0 ** -18).bfloat16()
    W[:, 2] = torch.randn(V, generator=g, device="cuda").bfloat16()
    h = torch.zeros(N, D, dtype=torch.bfloat16, device="cuda")
    h[:, 0], h[:, 1] = sign * 2.0 ** k, 2.0 ** k
    t = torch.randint(0, V, (N,), generator=g, device="cuda").int()
    t[0], t[1], t[2] = 5, 699, 300
    z = scale * (h.double() @ W.double().T)
    assert torch.equal(z.float().double(), z)
    top = z.amax(1, keepdim=True)
    logp = (z - top) - (z - top).exp().sum(1, keepdim=True).log()
    at = t.long()[:, None]
    nll, lse = -logp.gather(1, at)[:, 0], top[:, 0] + (z - top).exp().sum(1).log()
    d = logp.exp()
    d.scatter_add_(1, at, -torch.ones_like(d[:, :1]))
    one, two = both(h, W, t, scale=scale)
    for o in (one, two):
        assert (o["row_status"] == 0).all()
        assert ((o["loss"].double() - nll).abs() <= (2.0 ** -18 + 2.0 ** -20) * (1 + nll)).all(), (o["loss"], nll)
        assert torch.equal(o["stats"][:, 1], o["loss"])
        assert ((o["stats"][:, 0].double() - lse).abs() <= 2.0 ** -18 + 2.0 ** -22 * lse.abs() + 2.0 ** -20 * nll).all()
    share = 2.0 ** -8 + 2.0 ** -11 + 2.0 ** -12
    most = d.abs().scatter(1, at, 0.0).amax(1, keepdim=True)
    for o, extra in ((one, torch.zeros_like(nll)), (two, 2.0 ** -21 * torch.minimum(nll, lse.abs()))):
        # (rows whose statistics do not hold their probabilities: no more than one each)
        known = extra < 2.0 ** -8
        off = torch.where(known[:, None], d.abs() * (share + extra[:, None]) + 2.0 ** -39 * most, 2.0)
        gh, gW = scale * (d @ W.double()), scale * (d.T @ h.double())
        # (-1 times a state as large as 2^127 scale may be more than bf16 holds)
        for got, exact, most_off in ((o["grad_hidden"], gh, scale * (off @ W.abs().double())),
                                     (o["grad_head"], gW, scale * (off.T @ h.abs().double()))):
            fits = exact.abs() + most_off < 3e38
            bad = (got.double() - exact).abs() > 1.01 * most_off + 2.0 ** -8 * exact.abs() + 1e-36
            assert not (bad & fits).any(), (bad & fits).nonzero()[0].tolist()
            assert not got.isnan().any()


@pytest.mark.parametrize("N", [5, 300])
def test_a_loss_past_the_range_of_its_logarithm(N):
    """A loss of 3.0e38, whose log2(e)-fold is not finite, beside rows that do not see it."""
    W = torch.zeros(300, 64, dtype=torch.bfloat16, device="cuda")
    h = torch.zeros(N, 64, dtype=torch.bfloat16, device="cuda")
    h[0, 0], W[1, 0] = 2e19, 1.5e19
    h[1:, 1] = 1
    W[:, 1] = torch.randn(300, device="cuda").bfloat16()
    t = torch.arange(N, device="cuda").int()
    exact = h[0, 0].double() * W[1, 0].double()
    one, two = both(h, W, t)
    for o in (one, two):
        assert (o["row_status"] == 0).all()
        assert abs(o["loss"][0].double() - exact) <= 2.0 ** -22 * exact
        want = head64(h[1:], W, t[1:])
        hold(o["loss"][1:], want, "loss")
        hold(o["grad_hidden"][1:], want, "grad_hidden")
    assert torch.equal(one["grad_hidden"][0], (W[1].double() - W[0].double()).bfloat16())
    assert two["grad_hidden"].isfinite().all()


@pytest.mark.parametrize("N", [6, 200, 300])
@pytest.mark.parametrize("D", [64, 520])
def test_rows_beside_one_far_from_zero(N, D):
    """A row's bits do not depend on the logits of its neighbours."""
    h, W, t = inputs(N, D, 777, seed=N)
    other = h.clone()
    other[1] *= 4096
    for scale in (1.0, 1.25):
        a, b = both(h, W, t, scale=scale), both(other, W, t, scale=scale)
        for x, y in zip(a, b):
            for k in ("loss", "stats", "grad_hidden"):
                same = (x[k] == y[k]).reshape(N, -1).all(1)
                same[1] = True
                assert same.all(), (k, same.nonzero()[:, 0].tolist())


@pytest.mark.parametrize("N", [64, 300])
@pytest.mark.parametrize("sign", [1, -1])
def test_statistics_that_do_not_hold_the_probabilities(N, sign):
    """A loss and a log-sum-exp of 10^9: a backward pass from them knows no probability, but takes
    none for more than one (the call that computes both knows them)."""
    g = torch.Generator(device="cuda").manual_seed(N)
    W = torch.zeros(300, 16, dtype=torch.bfloat16, device="cuda")
    W[:, 1] = torch.randn(300, generator=g, device="cuda").bfloat16()
    W[0, 0], W[7, 0] = (1, -2) if sign > 0 else (-1, -4)
    W[1:7, 0] = W[8:, 0] = -4 if sign > 0 else -8
    h = torch.zeros(N, 16, dtype=torch.bfloat16, device="cuda")
    h[:, 0] = (torch.rand(N, generator=g, device="cuda") + 0.5) * 2.0 ** 30
    t = torch.full((N,), 7, dtype=torch.int32, device="cuda")
    one, two = both(h, W, t)
    assert (one["row_status"] == 0).all() and (one["loss"] > 2e8).all()
    want = (W[0].double() - W[7].double()).bfloat16()
    assert torch.equal(one["grad_hidden"], want.expand(N, 16))
    most = 1.01 * (W[0].abs() + W[7].abs()).double()
    assert (two["grad_hidden"].double().abs() <= most).all(), (two["grad_hidden"].abs() / most).max()
