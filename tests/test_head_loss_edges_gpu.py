"""specv_head_loss and its backward pass where their range and their digits end, against the
definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._head64 import head64, hold  # noqa: E402

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
