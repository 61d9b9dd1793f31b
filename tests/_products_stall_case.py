"""A head loss or an orthogonalised update in a fresh process with SPECV_TEST_STALL set (the
library reads it once per process): a wait for 16 bytes that no copy brings runs out, and the
call returns with every row (matrix) flagged and the CUDA context usable.  Run by
tests/test_products_stall_gpu.py as `python -m tests._products_stall_case <head|orth>`.
"""
import sys
import time

import torch

import speculative_decoding_verification_50_gb300 as sv
from tests._head64 import inputs


def main():
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    if sys.argv[1] == "head":
        o = sv.specv_head_loss(*inputs(300, 256, 40000), with_grad=True)
        torch.cuda.synchronize()
        assert (o["loss"] == 0).all() and o["stats"].isnan().all() and (o["grad_hidden"] == 0).all()
    else:
        o = sv.specv_orthogonalize(torch.randn(3, 600, 700, device="cuda"))
        torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    assert 0.3 < dt < 20, dt
    assert (o["row_status"] == sv.ROW_DEVICE_TIMEOUT).all(), o["row_status"]
    assert torch.arange(1000, device="cuda").sum().item() == 499500
    print(f"stall case ok {dt:.2f}")


if __name__ == "__main__":
    main()
