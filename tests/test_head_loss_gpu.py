"""specv_head_loss, its backward pass and head_loss against their definition in 64 bits."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests._head64 import head64, hold, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def check(h, W, t, **how):
    up = how.pop("up", None)
    want = head64(h, W, t, up=up, **how)
    if up is None:
        o = sv.specv_head_loss(h, W, t, with_grad=True, **how)
    else:
        o = sv.specv_head_loss(h, W, t, **how)
        o.update(sv.specv_head_loss_backward(h, W, t, o["stats"], grad_loss=up, **how))
    assert (o["row_status"] == 0).all()
    hold(o["loss"], want, "loss")
    hold(o["stats"][:, 0], want, "lse")
    hold(o["stats"][:, 1], want, "nll")
    hold(o["grad_hidden"], want, "grad_hidden")
    hold(o["grad_head"], want, "grad_head")
    return o, want


SIZES = [(1, 64, 256), (1, 8, 1), (2, 16, 2), (1, 200, 1000), (5, 64, 127), (33, 128, 129), (64, 264, 513), (128, 64, 1024),
         (255, 72, 300), (256, 512, 2000), (257, 96, 777), (600, 1024, 5000), (1100, 40, 3333)]


@pytest.mark.parametrize("N,D,V", SIZES)
def test_loss_and_gradients(N, D, V):
    check(*inputs(N, D, V, seed=N))


@pytest.mark.parametrize("N,D,V", SIZES[::2])
def test_backward_with_upstream(N, D, V):
    h, W, t = inputs(N, D, V, seed=N + 1)
    check(h, W, t, up=torch.rand(N, device="cuda") + 0.5, scale=0.7)


@pytest.mark.parametrize("N", [40, 400])
@pytest.mark.parametrize("D,pad,off", [(65, 0, 0), (64, 3, 0), (64, 8, 0), (64, 0, 1), (31, 2, 3), (7, 1, 0), (1, 0, 0)])
def test_strides_and_alignments(N, D, pad, off):
    h, W, t = inputs(N, D, 500, seed=D, pad=pad, off=off)
    o, want = check(h, W, t)
    # gradients into rows with gaps, which stay as they are
    room = [torch.full((x.shape[0], D + 5), 7.0, dtype=torch.bfloat16, device="cuda") for x in (h, W)]
    sv.specv_head_loss(h, W, t, grad_hidden=room[0][:, :D], grad_head=room[1][:, :D])
    assert torch.equal(room[0][:, :D], o["grad_hidden"]) and torch.equal(room[1][:, :D], o["grad_head"])
    assert all((x[:, D:] == 7).all() for x in room)
