"""specv_orthogonalize of matrices whose roundings agree, and of thin ones."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._orth64 import COEFFICIENTS, bound, hold, orth64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def same_way(size, steps=5):
    """How far a singular value `size` of G / |G| may be off after the steps, relative to where it
    ends, when every rounding to fp16 goes the same way (u = 2^-11 each: of the products' X, of S
    and of P): a step's error grows by the step's derivative, and the three roundings add
    u |3 b x^3 + 5 c x^5|, u |b x^3 + 2 c x^5| and u |b x^3 + c x^5|."""
    a, b, c = COEFFICIENTS
    x, e, u = size, 0.0, 2.0 ** -11
    for _ in range(steps):
        e = abs(a + 3 * b * x ** 2 + 5 * c * x ** 4) * e + u * (
            abs(3 * b * x ** 3 + 5 * c * x ** 5) + abs(b * x ** 3 + 2 * c * x ** 5) + abs(b * x ** 3 + c * x ** 5))
        x = a * x + b * x ** 3 + c * x ** 5
    return 1.05 * e / abs(x)  # (terms of second order)


def hadamard(n):
    H = torch.ones(1, 1)
    while H.shape[0] < n:
        H = torch.cat([torch.cat([H, H], 1), torch.cat([H, -H], 1)])
    return H


def matrices():
    for n in (300, 336, 428, 497):
        yield f"eye {n}", torch.eye(n), n
        yield f"ones {n}", torch.ones(n, n), 1
    yield "ones 700 x 300", torch.ones(700, 300), 1
    yield "hadamard 512", hadamard(512), 512
    one = torch.zeros(400, 900)
    one[3, 5] = -2.0
    yield "one entry", one, 1
    apart = torch.zeros(600, 1200)  # rows on columns of their own, of one size
    for r in range(5):
        apart[100 * r, 200 * r:200 * r + 200] = 1 - 2 * (torch.arange(200) % 2)
    yield "rows apart", apart, 5


@pytest.mark.parametrize("what,G,values", [pytest.param(*m, id=m[0]) for m in matrices()])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_roundings_that_agree(what, G, values, dtype):
    """`values` singular values of one size: all roundings of a step are the same one."""
    G = G.to("cuda", dtype)
    want, _ = orth64(G)
    o = sv.specv_orthogonalize(G)
    hold(o["orthogonal"], want, same_way(values ** -0.5) + 2.0 ** -8)


@pytest.mark.parametrize("shape", [(1, 5000), (3000, 1), (2, 4097), (2, 3000, 7), (5, 1, 2049), (3, 2300, 2)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_thin(shape, dtype):
    """Sides of one to seven entries, past what one kernel takes."""
    G = torch.randn(*shape, generator=torch.Generator(device="cuda").manual_seed(shape[-1]), device="cuda").to(dtype)
    want, norm = orth64(G)
    o = sv.specv_orthogonalize(G)
    hold(o["orthogonal"], want, bound(*shape[-2:]))
    assert ((o["norm"].double() - norm).abs() <= 2.0 ** -17 * norm).all() and (o["row_status"] == 0).all()


def test_matrices_that_overlap_are_refused():
    """Broadcast over the batch, or with each other's rows between their own."""
    G = torch.randn(40, 60, device="cuda")
    with pytest.raises(sv.SpecvError):
        sv.specv_orthogonalize(G.expand(2, 40, 60))
    with pytest.raises(sv.SpecvError):
        sv.specv_orthogonalize(torch.randn(40, 3, 60, device="cuda").transpose(0, 1))
