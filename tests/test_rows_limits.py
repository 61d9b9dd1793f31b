"""The widest rows of the distillation kernels: both directions take and refuse
the same (CPU: refusals end before any CUDA call)."""
import ctypes

import pytest

import speculative_decoding_verification_50_gb300 as sv
from speculative_decoding_verification_50_gb300 import _build
from tests.test_rows_abi import distill_args


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load_library()


@pytest.mark.parametrize("dtype,V", [(sv.SPECV_FP32, 900_000), (sv.SPECV_FP32, 1 << 20), (sv.SPECV_BF16, 1_800_000),
                                     (sv.SPECV_BF16, 1 << 30), (sv.SPECV_FP32, (1 << 31) - 8),
                                     (sv.SPECV_BF16, (1 << 31) - 1), (sv.SPECV_FP32, (1 << 31) - 1)])
def test_rows_too_wide(lib, dtype, V):
    args = distill_args(dtype=dtype, V=V, row_stride=V, grad_row_stride=V)
    for fn in (lib.specv_distill, lib.specv_distill_backward):
        assert fn(ctypes.byref(args), None) == sv.SPECV_ERR_UNSUPPORTED
        assert b"V=" in lib.specv_last_error() and lib.specv_last_launch_count() == 0
