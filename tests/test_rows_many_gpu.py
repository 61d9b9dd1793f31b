"""Top logits and distillation over rows enough to fill the GPU, every row against
its definition.

Top logits: ids and values equal; the log-sum-exp as in the operator's own tests.
Distillation: as in test_distill_edges_gpu.py, every element to REL of the sum of
the absolute terms (TAIL where the tail counts, r at least 1/16), and eps / 2.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests._rows64 import distill64  # noqa: E402
from tests.test_distill_edges_gpu import REL, TAIL, both, close, sv  # noqa: E402,F401


def many():
    return 3 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("dtype,V", [(torch.float32, 30016), (torch.float32, 50255), (torch.bfloat16, 60032),
                                     (torch.bfloat16, 152064)])
@pytest.mark.parametrize("k", [5, 300, 1024])
def test_top_logits(sv, dtype, V, k):  # noqa: F811
    N = many()
    g = torch.Generator(device="cuda").manual_seed(V + k)
    z = torch.randn(N, V, generator=g, device="cuda") * 3
    z[::9] = (z[::9] * 2).round() / 2
    z[5] = 1.0
    z[6, 100:] = -float("inf")
    z[7, :V // 2] = torch.finfo(torch.float32).min
    z = z.to(dtype)
    o = sv.specv_top_logits(z, k)
    assert (o["row_status"] == 0).all()
    for a in range(0, N, 64):
        s = slice(a, a + 64)
        val, ids = torch.sort(z[s].float(), dim=1, descending=True, stable=True)
        val, ids = val[:, :k], ids[:, :k].int()
        none = torch.isneginf(val)
        assert torch.equal(o["ids"][s], torch.where(none, -1, ids)) and torch.equal(o["values"][s], val)
        y = z[s].double()
        want = torch.logsumexp(y, 1)
        w = torch.softmax(y, 1)
        spread = torch.where(w > 0, w * (y.amax(1, keepdim=True) - y), 0.0).sum(1)
        assert ((o["lse"][s].double() - want).abs() <= 2.0 ** -22 * (1 + spread) + 2.0 ** -23 * want.abs()).all()


@pytest.mark.parametrize("dtype,V", [(torch.float32, 30016), (torch.float32, 50255), (torch.bfloat16, 60032),
                                     (torch.bfloat16, 100001)])
@pytest.mark.parametrize("tail", [False, True])
def test_distillation(sv, dtype, V, tail):  # noqa: F811
    N, K = many(), 40
    g = torch.Generator(device="cuda").manual_seed(V + tail)
    z = (torch.randn(N, V, generator=g, device="cuda") * 2).to(dtype)
    teacher = z.float() + torch.randn(N, V, generator=g, device="cuda")
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(teacher, 1) if tail else None
    ids[::11, 3] = ids[::11, 9]        # repeats
    val[::11] -= 1.0
    ids[::13, 20:] = -1
    if tail:
        mass = torch.where(ids >= 0, torch.exp(val.double() - lse.double()[:, None]), 0.0).sum(1)
        assert mass.max() <= 15 / 16
    w = torch.rand(N, generator=g, device="cuda") + 0.1
    w[::17] = 0
    rel = TAIL if tail else REL
    got, fused, back = both(sv, z, ids, val, lse=lse, w=w, tail=tail)
    alone = sv.specv_distill(z, ids, val, teacher_lse=lse, weights=w, tail=tail)  # without the gradient: another split
    for a in range(0, N, 38):
        s = slice(a, a + 38)
        loss, want, scale, _, size = distill64(z[s], ids[s], val[s], None if lse is None else lse[s], 1.0, w[s], tail)
        for x in (got[s], alone["loss"][s]):
            assert ((x.double() - loss).abs() <= rel * scale).all(), a
        close(fused[s], want, size, rel)
        close(back[s], want, size, rel)
