"""Late copies in the gradients' products and in what an update's products add to, in a fresh process with SPECV_TEST_STALL set (the
library reads it once per process).  Run by tests/test_late_gpu.py as
`python -m tests._late_case <what> <rows>` (or, for an update, its smaller side).
"""
import sys
import time

import torch

import speculative_decoding_verification_50_gb300 as sv
from tests._head64 import head64, hold, inputs
from tests._orth64 import bound, orth64
from tests._orth64 import hold as hold_matrix


def late(o, N, given=("grad_hidden", "grad_head")):
    """Gradients of a call whose copy was late: zeros, and every row flagged."""
    torch.cuda.synchronize()
    assert all((o[k] == 0).all() for k in given), [(o[k] != 0).sum() for k in given]
    if "row_status" in o:
        assert (o["row_status"] & sv.ROW_DEVICE_TIMEOUT).all(), o["row_status"]
        assert len(o["row_status"]) == N


def head(what, N):
    """dz (the products of a backward pass alone), dW and dh."""
    h, W, t = inputs(N, 256, 20000)
    want = head64(h, W, t)
    stats = sv.specv_head_loss(h, W, t)["stats"]
    wide = lambda x: torch.full((x.shape[0], 263), 7.0, dtype=x.dtype, device="cuda")  # noqa: E731
    rooms = [wide(h), wide(W)]
    o = sv.specv_head_loss(h, W, t, grad_hidden=rooms[0][:, :256], grad_head=rooms[1][:, :256])
    hold(o["loss"], want, "loss")
    if what == "dz":  # (the logits' weights are kept)
        assert (o["row_status"] == 0).all()
        hold(o["grad_hidden"], want, "grad_hidden")
        hold(o["grad_head"], want, "grad_head")
    else:
        late(o, N)
    assert all((x[:, 256:] == 7).all() for x in rooms)
    status = torch.zeros(N, dtype=torch.int32, device="cuda")
    b = sv.specv_head_loss_backward(h, W, t, stats, row_status=status)
    late(dict(b, row_status=status), N)
    # the differentiable loss: no gradient in the place of an undefined one
    x, y = h.clone().requires_grad_(), W.clone().requires_grad_()
    sv.head_loss(x, y, t).sum().backward()
    late(dict(grad_hidden=x.grad, grad_head=y.grad), N)
    one = "grad_hidden" if what == "dh" else "grad_head"
    status.zero_()
    b = sv.specv_head_loss_backward(h, W, t, stats, row_status=status, **{one: rooms[one == "grad_head"][:, :256]})
    late(dict(b, row_status=status), N, (one,))
    return h, W, t, want


def update(N):
    """Every matrix flagged."""
    for shape in ((2, N, 700), (3, 700, N)):
        o = sv.specv_orthogonalize(torch.randn(*shape, device="cuda"))
        assert (o["row_status"] == sv.ROW_DEVICE_TIMEOUT).all(), o["row_status"]


def small(N):
    """All steps in one kernel, clusters of 1 to 16 CTAs: the second matrix alone is flagged."""
    for shape in ((3, N, 100), (3, 100, N)):
        G = torch.randn(*shape, device="cuda")
        o = sv.specv_orthogonalize(G)
        assert o["row_status"].tolist() == [0, sv.ROW_DEVICE_TIMEOUT, 0], o["row_status"]
        want, norm = orth64(G)
        hold_matrix(o["orthogonal"][::2], want[::2], bound(*shape[1:]))
        assert ((o["norm"].double() - norm).abs() <= 2.0 ** -17 * norm).all()


def main():
    what, N = sys.argv[1], int(sys.argv[2])
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    {"update": update, "small": small}.get(what, lambda n: head(what, n))(N)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    assert 0.3 < dt < 40, dt
    assert torch.arange(1000, device="cuda").sum().item() == 499500
    print(f"late case ok {dt:.2f}")


if __name__ == "__main__":
    main()
