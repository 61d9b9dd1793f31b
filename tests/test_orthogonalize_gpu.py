"""specv_orthogonalize against its steps in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._orth64 import bound, hold, orth64  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def matrix(shape, kind="random", seed=0, dtype=torch.float32):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=g, device="cuda")
    small = min(shape[-2:])
    if kind == "falling":  # singular values that fall as 1 / k
        q, _ = torch.linalg.qr(torch.randn(shape[-2], shape[-2], generator=g, device="cuda", dtype=torch.float64))
        r, _ = torch.linalg.qr(torch.randn(shape[-1], shape[-1], generator=g, device="cuda", dtype=torch.float64))
        x = (q[:, :small] * (1.0 / torch.arange(1, small + 1, device="cuda"))) @ r[:small]
    if kind == "low rank":
        k = max(1, small // 16)
        x = torch.randn(*shape[:-1], k, generator=g, device="cuda") @ torch.randn(*shape[:-2], k, shape[-1], generator=g, device="cuda")
        x = x + 0.05 * torch.randn(*shape, generator=g, device="cuda")
    return x.to(dtype)


def check(G, **how):
    want, norm = orth64(G, **how)
    o = sv.specv_orthogonalize(G, **how)
    assert (o["row_status"] == 0).all()
    # squares of entries, sums of up to 2^24 of them in fp32 in several hundred parts
    assert ((o["norm"].double() - norm).abs() <= 2.0 ** -17 * norm).all()
    hold(o["orthogonal"], want, bound(*G.shape[-2:]))
    return o


SHAPES = [(1, 1), (1, 7), (2, 2), (3, 300), (64, 64), (65, 127), (128, 512), (255, 257), (256, 256), (300, 200), (512, 100),
          (700, 1111), (1030, 520), (2000, 64)]


@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_random(shape, dtype):
    check(matrix(shape, dtype=dtype, seed=shape[0]))


@pytest.mark.parametrize("shape", [(128, 512), (300, 200), (700, 1111)])
@pytest.mark.parametrize("kind", ["falling", "low rank"])
def test_spectra(shape, kind):
    check(matrix(shape, kind))


@pytest.mark.parametrize("shape", [(3, 64, 64), (5, 100, 333), (4, 333, 100), (24, 130, 130), (2, 1, 9)])
def test_batches(shape):
    G = matrix(shape, dtype=torch.bfloat16)
    G *= torch.logspace(-6, 6, shape[0], device="cuda").to(G.dtype)[:, None, None]
    o = check(G)
    for k in (0, shape[0] - 1):
        assert torch.equal(o["orthogonal"][k], sv.specv_orthogonalize(G[k])["orthogonal"])
