"""Sizes at the end of what 32 bits count, refused by the head's loss and by orthogonalised
updates (CPU: no call gets to a launch)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402
from tests.test_products_abi import head, lib, orth  # noqa: E402,F401

MOST = 2 ** 31 - 2 ** 11  # rows, tokens, and entries of a row or column


@pytest.mark.parametrize("what", ["N", "V", "D"])
@pytest.mark.parametrize("size", [MOST + 1, 2 ** 31 - 1])
def test_head_loss_sizes(lib, what, size):  # noqa: F811
    how = dict(N=4, V=4, D=4, hidden_stride=size, head_stride=size, grad_hidden_stride=size, grad_head_stride=size)
    how[what] = size
    for call in (lib.specv_head_loss, lib.specv_head_loss_backward):
        assert call(ctypes.byref(head(**how)), 256, (1 << 63) - 1, None) == sv.SPECV_ERR_UNSUPPORTED
    # the largest that are taken get as far as their workspace
    how[what] = MOST
    for call in (lib.specv_head_loss, lib.specv_head_loss_backward):
        assert call(ctypes.byref(head(**how)), None, 0, None) == sv.SPECV_ERR_WORKSPACE


@pytest.mark.parametrize("what", ["m", "n"])
@pytest.mark.parametrize("size", [MOST + 1, 2 ** 31 - 1])
def test_orthogonalize_sizes(lib, what, size):  # noqa: F811
    how = dict(B=1, m=4, n=4, row_stride=size, out_row_stride=size, batch_stride=1 << 40, out_batch_stride=1 << 40)
    how[what] = size
    assert lib.specv_orthogonalize(ctypes.byref(orth(**how)), 256, (1 << 63) - 1, None) == sv.SPECV_ERR_UNSUPPORTED
    how[what] = MOST
    assert lib.specv_orthogonalize(ctypes.byref(orth(**how)), None, 0, None) == sv.SPECV_ERR_WORKSPACE


def test_python_sizes(lib):  # noqa: F811
    """Sizes that 32 bits would cut off, to something that could be a size."""
    big = 2 ** 32 + 4
    of = lambda *shape, dtype=torch.bfloat16: torch.empty(shape, dtype=dtype, device="meta")  # noqa: E731
    for call in (lambda: sv.specv_head_loss(of(big, 8), of(9, 8), of(big, dtype=torch.int32)),
                 lambda: sv.specv_head_loss(of(4, 8), of(big, 8), of(4, dtype=torch.int32)),
                 lambda: sv.specv_head_loss(of(4, big), of(9, big), of(4, dtype=torch.int32)),
                 lambda: sv.specv_head_loss_backward(of(4, 8), of(big, 8), of(4, dtype=torch.int32), of(4, 2, dtype=torch.float32)),
                 lambda: sv.specv_orthogonalize(of(big, 8)), lambda: sv.specv_orthogonalize(of(3, 8, big)),
                 lambda: sv.specv_orthogonalize(of(big, 8, 9))):
        with pytest.raises(AssertionError, match="size"):
            call()
