"""The 64-bit definitions that the GPU tests hold kernels to, against other routines and
against differences (CPU)."""
import pytest

torch = pytest.importorskip("torch")

from tests._head64 import head64, inputs  # noqa: E402
from tests._orth64 import orth64  # noqa: E402


def test_head_loss_and_gradients():
    h, W, t = (x for x in inputs(9, 24, 50, device="cpu"))
    t[2], t[5] = -1, 50
    w = torch.rand(9) + 0.5
    w[7] = 0.0
    up = torch.rand(9)
    got = head64(h, W, t, scale=0.6, weights=w, up=up)
    x, y = h.double().requires_grad_(), W.double().requires_grad_()
    use = (t >= 0) & (t < 50)
    nll = torch.nn.functional.cross_entropy(0.6 * x @ y.T, torch.where(use, t, 0).long(), reduction="none")
    loss = torch.where(use, w.double() * nll, 0.0)
    (loss * up.double()).sum().backward()
    assert torch.allclose(got["loss"], loss.detach(), rtol=1e-12, atol=1e-12)
    assert torch.allclose(got["grad_hidden"], x.grad, rtol=1e-10, atol=1e-12)
    assert torch.allclose(got["grad_head"], y.grad, rtol=1e-10, atol=1e-12)
    assert (got["grad_hidden"][~got["use"]] == 0).all() and got["use"].tolist() == [r not in (2, 5, 7) for r in range(9)]


def test_head_gradients_against_differences():
    h, W, t = (x.double() if x.is_floating_point() else x for x in inputs(4, 6, 11, device="cpu"))
    got = head64(h, W, t)
    step = 1e-5
    for x, k in ((h, "grad_hidden"), (W, "grad_head")):
        for i, j in ((0, 0), (1, 3), (3, 5)):
            at = []
            for s in (1, -1):
                x[i, j] += s * step
                at.append(head64(h, W, t)["loss"].sum())
                x[i, j] -= s * step
            assert abs((at[0] - at[1]) / (2 * step) - got[k][i, j]) < 1e-8


@pytest.mark.parametrize("shape", [(5, 9), (9, 5), (6, 6)])
def test_orthogonalized_singular_values(shape):
    """The polynomial of each singular value, the singular vectors as they are."""
    G = torch.randn(*shape, dtype=torch.float64, generator=torch.Generator().manual_seed(1))
    X, norm = orth64(G)
    u, s, v = torch.linalg.svd(G, full_matrices=False)
    s = s / G.norm()
    for _ in range(5):
        s = 3.4445 * s - 4.7750 * s ** 3 + 2.0315 * s ** 5
    assert torch.allclose(X, u @ torch.diag(s) @ v, atol=1e-12) and torch.allclose(norm, G.norm())
