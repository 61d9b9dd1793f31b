"""The k largest logits and the log-sum-exp, against a sort in numpy and a
64-bit sum.  Ids and values are equal; lse is a sum of fp32 exponentials
(2^-22 each, their error in a sum of positive terms no larger) and one rounding:
2^-22 absolute and 2^-24 of its value."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    import speculative_decoding_verification_50_gb300 as m
    m.load_library()
    return m


def check(sv, zt, k, T=1.0):
    o = sv.specv_top_logits(zt, k, temperature=T)
    torch.cuda.synchronize()
    z = zt.float().cpu().numpy()
    ids, val, lse = (o[n].cpu().numpy() for n in ("ids", "values", "lse"))
    assert (o["row_status"] == 0).all()
    for b in range(z.shape[0]):
        order = np.argsort(-z[b], kind="stable")
        n = min(k, int((z[b] > -np.inf).sum()))
        assert np.array_equal(ids[b, :n], order[:n]), b
        assert np.array_equal(val[b, :n], z[b][order[:n]])
        assert (ids[b, n:] == -1).all() and np.isneginf(val[b, n:]).all()
        y = z[b].astype(np.float64) / float(np.float32(T))
        want = y.max() + np.log(np.exp(y - y.max()).sum())
        # the argument of each exponential is rounded too: (z - max) / T to two roundings
        spread = np.average(np.where(np.isfinite(y), y.max() - y, 0), weights=np.exp(y - y.max()))
        assert abs(lse[b] - want) <= 2.0 ** -22 * (1 + spread) + 2.0 ** -23 * abs(want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,k", [(1, 1), (5, 9), (37, 4), (1000, 1000), (4097, 32), (50257, 1024), (152064, 256)])
def test_random_rows(sv, V, k, dtype):
    g = torch.Generator().manual_seed(V + k)
    z = torch.randn(9, V, generator=g) * torch.tensor([0.01, 0.1, 1, 2, 3, 5, 20, 1e4, 1e20])[:, None]
    check(sv, z.to(dtype).cuda(), k)
    check(sv, z[:6].to(dtype).cuda(), k, T=2.5)


@pytest.mark.parametrize("V", [100, 5000, 30000])
def test_ties_and_masks(sv, V):
    g = torch.Generator().manual_seed(V)
    z = torch.zeros(6, V)
    z[1] = torch.randint(0, 3, (V,), generator=g).float()
    z[2] = torch.randint(-2, 1, (V,), generator=g).float() * 1e3
    z[3, V // 2:] = -float("inf")
    z[4] = -float("inf")
    z[4, V - 1] = 3.0
    z[5] = torch.finfo(torch.float32).min
    z[5, 17] = 0.0
    check(sv, z.cuda(), 60)
    check(sv, z.cuda(), 1024)


def test_flagged_rows_and_layout(sv):
    z = torch.zeros(4, 1000 + 3).cuda()[:, 3:]
    z[0, 1], z[1, 2] = float("nan"), float("inf")
    z[2] = -float("inf")
    z[3] = torch.arange(1000).cuda()
    o = sv.specv_top_logits(z, 8)
    assert o["row_status"].tolist() == [sv.ROW_NONFINITE] * 3 + [0]
    assert (o["ids"][:3] == -1).all() and torch.isneginf(o["values"][:3]).all() and o["lse"][:3].isnan().all()
    assert o["ids"][3].tolist() == list(range(999, 991, -1))


@pytest.mark.parametrize("dtype,V", [(torch.float32, 30016), (torch.float32, 50255), (torch.bfloat16, 152064)])
@pytest.mark.parametrize("k", [3, 300, 1000])
def test_many_rows(sv, dtype, V, k):
    """Rows enough to fill the GPU take another split than a few do."""
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn(400, V, generator=g, device="cuda") * 3
    z[::9] = (z[::9] * 2).round() / 2
    z[5] = 1.0
    z[6, 100:] = -float("inf")
    z = z.to(dtype)
    o = sv.specv_top_logits(z, k)
    for a in range(0, 400, 8):
        q = sv.specv_top_logits(z[a:a + 8], k)
        assert torch.equal(q["ids"], o["ids"][a:a + 8]) and torch.equal(q["values"], o["values"][a:a + 8]), a
        assert ((q["lse"] - o["lse"][a:a + 8]).abs() <= 2.0 ** -20 * (1 + q["lse"].abs())).all()
    check(sv, z[::40].contiguous(), k)


@pytest.mark.parametrize("dtype,V", [(torch.float32, 769999), (torch.bfloat16, 1539999)])
def test_widest_rows(sv, dtype, V):
    g = torch.Generator().manual_seed(V)
    check(sv, (torch.randn(2, V, generator=g) * 2).to(dtype).cuda(), 700)
