"""The distillation loss where a row ends, begins or is all but empty: every
element of the gradients against the definition in 64 bits.

Tolerances.  A weight 2^x is taken at an argument rounded twice (2^-24 of |x|
each, |x| <= 64 in these inputs: 5.3e-6 of the weight) by a function good to
2^-22, in a quotient of sums good to a few 2^-24: REL = 2^-17 of the value, and
of a gradient of several terms REL of the sum of their absolute values (weights
below 2^-64: 2^-64 of the row's largest).  The
teacher's tail r is one less a sum whose addends are good to 2^-21 (log p to
2^-24 of up to 10, and its exponential): with r >= 1/16 a term in r is good to
REL + 2^-17 = TAIL.  Rounding to the logits' type adds eps / 2.
"""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from tests._rows64 import distill64  # noqa: E402

REL, TAIL = 2.0 ** -17, 2.0 ** -16


@pytest.fixture(scope="module")
def sv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    import speculative_decoding_verification_50_gb300 as m
    m.load_library()
    return m


def both(sv, z, ids, val, grads=(None, None), lse=None, T=1.0, w=None, tail=False):
    """Loss and the two gradients: of the one call, and from its statistics."""
    kw = dict(teacher_lse=lse, temperature=T, weights=w, tail=tail)
    o = sv.specv_distill(z, ids, val, with_grad=True, grad=grads[0], **kw)
    back = sv.specv_distill_backward(z, ids, val, o["stats"], grad=grads[1], **kw)
    assert (o["row_status"] == 0).all()
    return o["loss"], o["grad"], back


def close(got, want, size, rel=REL):
    """Every element; `want` fp64, `size` the sum of its absolute terms."""
    room = rel * size + 2.0 ** -64 * size.amax(1, keepdim=True) + torch.finfo(got.dtype).eps / 2 * want.abs() + torch.finfo(got.dtype).tiny
    off = (got.double() - want).abs()
    assert (off <= room).all(), (off - room).argmax()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V", [37, 4099, 50257, 65535])
@pytest.mark.parametrize("off", [0, 1, 3])
def test_absent_entries_of_unaligned_rows(sv, V, off, dtype):
    """Lists with absent entries, rows at no 16-byte boundary: nothing is written
    beside a row, and the rows' ends are their own."""
    g = torch.Generator(device="cuda").manual_seed(V + off)
    N, K = 24, 20
    wide = V + off + 2
    z = torch.zeros(N, wide, dtype=dtype, device="cuda")[:, off:off + V]
    z.copy_(torch.randn(N, V, generator=g, device="cuda") * 2)
    teacher = z.float() + torch.randn(N, V, generator=g, device="cuda")
    val, ids = teacher.topk(K, dim=1)
    length = torch.randint(0, K + 1, (N, 1), generator=g, device="cuda")
    length[0], length[1], length[2] = 0, 1, K
    gaps = torch.rand(N, K, generator=g, device="cuda") < 0.2
    ids = torch.where((torch.arange(K, device="cuda") < length) & ~gaps, ids, -1).int()
    ids[3, 0], ids[4, 1] = 0, V - 1  # the ends themselves
    ids[3, 1:], ids[4, 2:], ids[4, 0] = -1, -1, -1
    _, want, _, _, size = distill64(z, ids, val)
    bufs = [torch.full((N, wide), 9.0, dtype=dtype, device="cuda") for _ in range(2)]
    _, fused, back = both(sv, z, ids, val, [b[:, off:off + V] for b in bufs])
    for b, got in zip(bufs, (fused, back)):
        assert (b[:, :off] == 9).all() and (b[:, off + V:] == 9).all()
        close(got, want, size)
    # rows without a gap between them: the end of each is the next one's neighbour
    zc = z.contiguous()
    _, fused, back = both(sv, zc, ids, val)
    for got in (fused, back):
        close(got, want, size)
    again = sv.specv_distill_backward(zc, ids, val, sv.specv_distill(zc, ids, val)["stats"])
    assert torch.equal(again, back)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("V,K", [(2000, 16), (30011, 200)])
def test_confident_students(sv, V, K, dtype):
    """Students with 1e-2 to 1e-17 of their mass outside the teacher's list."""
    g = torch.Generator(device="cuda").manual_seed(V)
    N = 64
    teacher = torch.randn(N, V, generator=g, device="cuda") * 2
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(teacher, 1)
    z = torch.randn(N, V, generator=g, device="cuda") - 4
    gap = torch.linspace(8.0, 40.0, N, device="cuda")[:, None]
    z.scatter_add_(1, ids.long(), gap + 2 * torch.randn(N, K, generator=g, device="cuda"))
    z = z.to(dtype)
    loss, want, scale, listed, size = distill64(z, ids, val, lse, tail=True)
    r = 1 - torch.exp(val.double() - lse.double()[:, None]).sum(1)
    q = torch.where(listed, 0.0, torch.softmax(z.double(), 1)).sum(1)
    assert r.min() >= 1 / 16 and q.max() > 1e-4 and q.min() < 1e-14
    got, fused, back = both(sv, z, ids, val, lse=lse, tail=True)
    assert ((got.double() - loss).abs() <= TAIL * scale).all()
    close(fused, want, size, TAIL)
    close(back, want, size, TAIL)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1.0, 0.1, 0.01, 0.001])
@pytest.mark.parametrize("given", [False, True])
def test_low_temperatures(sv, T, given, dtype):
    """Logits of thousands of units (z / T), the gradient from saved statistics as
    good as that of the one call."""
    g = torch.Generator(device="cuda").manual_seed(int(1 / T))
    N, V, K = 32, 5003, 40
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    teacher = 20 * normal(N, 1) + 2 * T * normal(N, V)
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    ids[::5, 30:] = -1
    z = (20 * normal(N, 1) + 2 * T * normal(N, V)).to(dtype)
    z[::2] = teacher[::2].to(dtype)
    lse = torch.logsumexp(teacher.double() / float(torch.tensor(T)), 1).float() if given else None
    loss, want, scale, _, size = distill64(z, ids, val, lse, T)
    got, fused, back = both(sv, z, ids, val, lse=lse, T=T)
    assert ((got.double() - loss).abs() <= REL * scale).all()
    close(fused, want, size)
    close(back, want, size)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [1.0, 0.01])
@pytest.mark.parametrize("V", [2000, 30011])
def test_students_far_from_the_rest(sv, V, T, dtype):
    """Students with e^-60 to e^-2000 of their mass outside the list: the tail's
    term is finite, and its gradient goes to the tokens of the rest."""
    g = torch.Generator(device="cuda").manual_seed(V + 1)
    N, K = 48, 30
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    teacher = 2 * T * normal(N, V)
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(teacher.double() / float(torch.tensor(T)), 1).float()
    gap = torch.logspace(math.log10(60), math.log10(2000), N, device="cuda")[:, None]
    z = T * normal(N, V)
    z.scatter_add_(1, ids.long(), T * (gap + 2 * normal(N, K)))
    z = z.to(dtype)
    loss, want, scale, _, size = distill64(z, ids, val, lse, T, tail=True)
    assert torch.isfinite(loss).all()
    assert (1 - torch.exp(val.double() / float(torch.tensor(T)) - lse.double()[:, None]).sum(1)).min() >= 1 / 16
    got, fused, back = both(sv, z, ids, val, lse=lse, T=T, tail=True)
    assert ((got.double() - loss).abs() <= TAIL * scale).all()
    close(fused, want, size, TAIL)
    close(back, want, size, TAIL)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_masked_rest(sv, dtype):
    """Outside the list: -inf, the type's lowest value (a mask: no mass), -1e9 (a
    logit like others), and rows of nothing but the lowest value."""
    g = torch.Generator(device="cuda").manual_seed(4)
    N, V, K = 4, 3001, 12
    z = torch.randn(N, V, generator=g, device="cuda")
    val, ids = (z + 1).topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(z + 1, 1)
    rest = torch.ones(N, V, dtype=torch.bool, device="cuda").scatter_(1, ids.long(), False)
    z = z.to(dtype)
    for b, x in enumerate((-float("inf"), torch.finfo(dtype).min, -1e9)):
        z[b][rest[b]] = x
    z[3] = torch.finfo(dtype).min
    loss, want, scale, _, size = distill64(torch.where(rest & (z < -2e9), -float("inf"), z)[:3], ids[:3], val[:3], lse[:3],
                                           tail=True)
    got, fused, back = both(sv, z, ids, val, lse=lse, tail=True)
    assert got[:2].tolist() == [float("inf")] * 2
    assert abs(float(got[2]) - float(loss[2])) <= TAIL * float(scale[2])
    for grad in (fused, back):
        close(grad[:3], want, size, TAIL)
    _, want, _, _, size = distill64(torch.zeros(1, V).cuda(), ids[3:], val[3:], lse[3:], tail=True)  # equal logits
    for grad in (fused, back):
        close(grad[3:], want, size, TAIL)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("at", [0.0, 1e4, -1e30, "lowest"])
def test_equal_logits_of_any_size(sv, dtype, at):
    """A student of equal logits has the loss of one of zeros."""
    g = torch.Generator(device="cuda").manual_seed(6)
    N, V, K = 6, 2500, 20
    t = torch.randn(N, V, generator=g, device="cuda")
    val, ids = t.topk(K, dim=1)
    ids = ids.int()
    ids[1, 0] = ids[2, 3] = -1
    z = torch.full((N, V), torch.finfo(dtype).min if at == "lowest" else at, dtype=dtype, device="cuda")
    for lse, tail in ((None, False), (torch.logsumexp(t, 1), True)):
        loss, want, scale, _, size = distill64(torch.zeros(N, V).cuda(), ids, val, lse, tail=tail)
        got, fused, back = both(sv, z, ids, val, lse=lse, tail=tail)
        assert ((got.double() - loss).abs() <= TAIL * scale).all()
        close(fused, want, size, TAIL)
        close(back, want, size, TAIL)


def test_ruled_out_first_entry(sv):
    """-inf at the entry the loss is taken relative to, of mass and of none."""
    g = torch.Generator(device="cuda").manual_seed(8)
    z = torch.randn(2, 2000, generator=g, device="cuda")
    val, ids = (z + 1).topk(16, dim=1)
    ids = ids.int()
    z[0, ids[0, 0].long()] = -float("inf")
    val[1, 0] = -float("inf")
    got, fused, back = both(sv, z, ids, val)
    loss, want, scale, _, size = distill64(z[1:], ids[1:], val[1:])
    assert got[0] == float("inf") and torch.isfinite(fused).all() and torch.isfinite(back).all()
    assert abs(float(got[1]) - float(loss)) <= REL * float(scale)
    close(fused[1:], want, size)
    close(back[1:], want, size)


@pytest.mark.parametrize("V,K", [(50257, 100), (152064, 256)])
def test_small_losses(sv, V, K):
    """A student close to its teacher: a loss of about 0.01, the difference of
    logarithms of the size of one to ten.  In the mean over rows the error is that
    of a row's sum: addends' roundings (80 of 2^-25, averaged over 512 threads),
    scales of 16 warps good to 2^-23 and four additions of them, about 2^-25 each;
    taken together at most 2^-24.5, and nothing beside it from what follows."""
    g = torch.Generator(device="cuda").manual_seed(V)
    N, T = 128, 2.0
    z = torch.randn(N, V, generator=g, device="cuda") * (1 + 2 * torch.rand(N, 1, generator=g, device="cuda"))
    teacher = z + torch.randn(N, V, generator=g, device="cuda")
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(teacher / T, 1)
    loss, want, _, _, size = distill64(z, ids, val, lse, T, tail=True)
    got, fused, back = both(sv, z, ids, val, lse=lse, T=T, tail=True)
    off = got.double() - loss
    assert off.pow(2).mean().sqrt() <= 2.0 ** -24.5, off.pow(2).mean().sqrt()
    close(fused, want, size, TAIL)
    close(back, want, size, TAIL)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("tail", [False, True])
def test_logits_of_three_hundred_thousand_units(sv, dtype, tail):
    """z / T of 3e5, whose roundings to fp32 are 0.03 apart."""
    g = torch.Generator(device="cuda").manual_seed(9)
    N, V, K, T = 40, 1999, 25, 0.001
    normal = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    teacher = -300 + 2 * T * normal(N, V)
    val, ids = teacher.topk(K, dim=1)
    ids = ids.int()
    lse = torch.logsumexp(teacher.double() / float(torch.tensor(T)), 1).float()
    z = (-300 + 2 * T * normal(N, V)).to(dtype)
    assert (1 - torch.exp(val.double() / float(torch.tensor(T)) - lse.double()[:, None]).sum(1)).min() >= 1 / 16
    loss, want, scale, _, size = distill64(z, ids, val, lse, T, tail=tail)
    got, fused, back = both(sv, z, ids, val, lse=lse, T=T, tail=tail)
    assert ((got.double() - loss).abs() <= TAIL * scale).all()
    close(fused, want, size, TAIL)
    close(back, want, size, TAIL)
