"""Refusals of the head's loss and of orthogonalised updates, and the sizes of their
workspaces (CPU: no call gets to a launch)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402


@pytest.fixture(scope="module")
def lib():
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    return sv.load_library()


def head(**how):
    a = sv.HeadArgs(64, 1000, 128, sv.SPECV_BF16, 256, 128, 256, 128, 256, None, 1.0, 0, 256, 256, 256, None, 256, 128, 256, 128)
    for k, v in how.items():
        setattr(a, k, v)
    return a


def orth(**how):
    a = sv.OrthArgs(2, 200, 300, sv.SPECV_BF16, 256, 60000, 300, 5, 3.4445, -4.7750, 2.0315, 256, 60000, 300, 256, 256)
    for k, v in how.items():
        setattr(a, k, v)
    return a


HEAD_BAD = [dict(N=-1), dict(V=0), dict(D=0), dict(dtype=7), dict(scale=0.0), dict(scale=float("nan")), dict(scale=-1.0),
            dict(scale=1e7), dict(flags=2), dict(hidden=None), dict(head=None), dict(targets=None), dict(hidden=257), dict(targets=258),
            dict(weights=255), dict(stats=2), dict(row_status=3), dict(grad_head=11), dict(hidden_stride=127),
            dict(head_stride=100), dict(grad_hidden_stride=1), dict(grad_head_stride=127), dict(loss=None), dict(grad_loss=256)]


@pytest.mark.parametrize("how", HEAD_BAD, ids=str)
def test_head_loss_refusals(lib, how):
    assert lib.specv_head_loss(ctypes.byref(head(**how)), 256, 1 << 40, None) == sv.SPECV_ERR_INVALID_ARG
    assert lib.specv_last_error()


@pytest.mark.parametrize("how", [h for h in HEAD_BAD if "loss" not in h and "grad_loss" not in h] +
                         [dict(stats=None), dict(grad_hidden=None, grad_head=None), dict(grad_loss=2)], ids=str)
def test_head_loss_backward_refusals(lib, how):
    assert lib.specv_head_loss_backward(ctypes.byref(head(**how)), 256, 1 << 40, None) == sv.SPECV_ERR_INVALID_ARG


def test_head_loss_other_refusals(lib):
    call = lib.specv_head_loss
    assert call(None, 256, 1 << 40, None) == sv.SPECV_ERR_INVALID_ARG
    assert call(ctypes.byref(head(dtype=sv.SPECV_FP32)), 256, 1 << 40, None) == sv.SPECV_ERR_UNSUPPORTED
    big = head(N=2 ** 31 - 1, V=2 ** 31 - 1)
    assert call(ctypes.byref(big), 256, (1 << 63) - 1, None) == sv.SPECV_ERR_UNSUPPORTED
    need = lib.specv_head_workspace_bytes(ctypes.byref(head()))
    assert call(ctypes.byref(head()), 256, need - 1, None) == sv.SPECV_ERR_WORKSPACE
    assert call(ctypes.byref(head()), None, need, None) == sv.SPECV_ERR_WORKSPACE
    assert call(ctypes.byref(head()), 128, need, None) == sv.SPECV_ERR_INVALID_ARG
    # no rows and no gradient of the head: nothing to do
    assert call(ctypes.byref(head(N=0, grad_head=None)), None, 0, None) == sv.SPECV_OK
    assert lib.specv_last_launch_count() == 0
    assert lib.specv_head_workspace_bytes(None) == 0 and lib.specv_head_workspace_bytes(ctypes.byref(head(N=0))) == 0


def test_head_loss_workspace(lib):
    """Weights of the logits up to 1 GB; beyond that pieces of 256 MB."""
    size = lambda **how: lib.specv_head_workspace_bytes(ctypes.byref(head(**how)))  # noqa: E731
    kept, pieces = size(N=4096, V=131072, D=64), size(N=4097, V=131072, D=64)
    assert 1 << 30 < kept < (1 << 30) + (64 << 20) and 200 << 20 < pieces < 384 << 20
    assert size(N=64, grad_hidden=None, grad_head=None) < size(N=64)
    # rows that TMA cannot read in place are copied
    assert size(head=258) >= size() + 2 * 1000 * 128 and size(head_stride=129) >= size() + 2 * 1000 * 128


ORTH_BAD = [dict(B=-1), dict(m=0), dict(n=0), dict(dtype=9), dict(steps=0), dict(steps=33), dict(a=float("nan")),
            dict(c=float("inf")), dict(a=5.0), dict(b=0.0), dict(a=2.0, b=1.0, c=0.0, steps=32), dict(update=None), dict(out=None),
            dict(update=257), dict(out=1), dict(norm=2), dict(row_status=6), dict(row_stride=299), dict(out_row_stride=299),
            dict(batch_stride=59999), dict(out_batch_stride=59999)]


@pytest.mark.parametrize("how", ORTH_BAD, ids=str)
def test_orthogonalize_refusals(lib, how):
    assert lib.specv_orthogonalize(ctypes.byref(orth(**how)), 256, 1 << 40, None) == sv.SPECV_ERR_INVALID_ARG
    assert lib.specv_last_error()


def test_orthogonalize_other_refusals(lib):
    call = lib.specv_orthogonalize
    assert call(None, 256, 1 << 40, None) == sv.SPECV_ERR_INVALID_ARG
    need = lib.specv_orthogonalize_workspace_bytes(2, 200, 300)
    assert need > 0 and lib.specv_orthogonalize_workspace_bytes(0, 200, 300) == 0
    assert lib.specv_orthogonalize_workspace_bytes(9, 2048, 128) == 0 < lib.specv_orthogonalize_workspace_bytes(9, 2049, 128)
    assert call(ctypes.byref(orth()), 256, need - 1, None) == sv.SPECV_ERR_WORKSPACE
    assert call(ctypes.byref(orth()), None, need, None) == sv.SPECV_ERR_WORKSPACE
    assert call(ctypes.byref(orth()), 384, need, None) == sv.SPECV_ERR_INVALID_ARG
    assert call(ctypes.byref(orth(B=70000)), 256, 1 << 40, None) == sv.SPECV_ERR_UNSUPPORTED
    assert call(ctypes.byref(orth(B=0)), None, 0, None) == sv.SPECV_OK


@pytest.mark.parametrize("call", [
    lambda h, W, t: sv.specv_head_loss(h, W, t),  # not on a GPU
    lambda h, W, t: sv.specv_head_loss(h[:, :3], W, t),
    lambda h, W, t: sv.specv_head_loss(h[0], W, t),
    lambda h, W, t: sv.specv_head_loss(h, W.float(), t),
    lambda h, W, t: sv.specv_head_loss(h, W, t.long()),
    lambda h, W, t: sv.specv_head_loss(h, W, t[:-1]),
    lambda h, W, t: sv.specv_orthogonalize(W),
    lambda h, W, t: sv.specv_orthogonalize(W[0]),
    lambda h, W, t: sv.specv_orthogonalize(W.half()),
    lambda h, W, t: sv.specv_orthogonalize(W, out=W.float()),
])
def test_python_refusals(lib, call):
    h, W, t = torch.zeros(4, 8).bfloat16(), torch.zeros(10, 8).bfloat16(), torch.zeros(4, dtype=torch.int32)
    with pytest.raises((AssertionError, TypeError)):
        call(h, W, t)
