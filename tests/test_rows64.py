"""The batched 64-bit definitions against those of the operators' own tests,
row by row (CPU)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests._rows64 import distill64, sample64  # noqa: E402
from tests.test_distill_gpu import formula  # noqa: E402
from tests.test_filter_gpu import restate, rules_of  # noqa: E402


@pytest.mark.parametrize("how", ["renorm", "lse", "tail"])
@pytest.mark.parametrize("T", [1.0, 0.5, 2.0])
def test_distillation(how, T):
    g = torch.Generator().manual_seed(3)
    N, V, K = 12, 97, 11
    z = torch.randn(N, V, generator=g) * 3
    teacher = z + torch.randn(N, V, generator=g)
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    for b in range(N):
        ids[b, b:] = -1
    ids[5, 0], val[6, 2] = -1, -float("inf")
    ids[7, 3], val[7] = ids[7, 5], val[7] - 2
    z[8][torch.isin(torch.arange(V), ids[8].long(), invert=True)] = -float("inf")
    lse = None if how == "renorm" else torch.logsumexp(teacher / T, 1)
    w = torch.rand(N, generator=g)
    w[9] = 0
    loss, grad, scale, listed, size = distill64(z, ids, val, lse, T, w, how == "tail")
    for b in range(N):
        want, dz, s = formula(z[b].double().numpy(), ids[b].numpy(), val[b].double().numpy(),
                              None if lse is None else float(lse[b]), T, float(w[b]), how == "tail")
        # differently ordered sums of 64-bit terms
        assert loss[b] == want or abs(float(loss[b]) - want) <= 1e-12 * (1 + abs(want)), b
        assert np.abs(grad[b].numpy() - dz).max() <= 1e-12, b
        assert (size[b] >= grad[b].abs() * (1 - 1e-12)).all()
        assert scale[b] == s or np.isinf(want) or abs(float(scale[b]) - s) <= 1e-12 * (1 + s)
        assert set(np.flatnonzero(listed[b].numpy())) == {int(i) for i in ids[b] if i >= 0}


@pytest.mark.parametrize("V", [1, 9, 400])
def test_sampling(V):
    rng = np.random.default_rng(V)
    B = 200
    z = rng.normal(0, 3, (B, V)).astype(np.float32)
    z[::5] = np.round(z[::5])
    z[1::7, 1:] = -np.inf
    rules = rules_of(rng, B, V)
    keep, token, prob, near = sample64(torch.from_numpy(z), *rules)
    for b in range(B):
        mask, tok, pr, close = restate(z[b].astype(np.float64), *(x[b] for x in rules))
        assert close <= bool(near[b])  # (here a border is a little wider)
        if not near[b]:
            assert np.array_equal(keep[b].numpy(), mask) and int(token[b]) == tok
            assert abs(float(prob[b]) - pr) <= 1e-12 * pr
    assert near.sum() <= 4
