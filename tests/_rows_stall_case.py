"""One distillation call run in a fresh process with SPECV_TEST_STALL set (the
library reads it once per process): the wait for one copy of the given row runs
out, in the first or the second pass over it, and the call returns with that
row flagged, without loss, gradient or usable statistics, every other row right
and the CUDA context usable.  Run by tests/test_rows_stall_gpu.py as
`python -m tests._rows_stall_case <row> <rows> <V> <bf16|fp32>`.
"""
import sys
import time

import torch

import speculative_decoding_verification_50_gb300 as sv
from tests._rows64 import distill64


def main():
    row, N, V = (int(a) for a in sys.argv[1:4])
    dtype = {"bf16": torch.bfloat16, "fp32": torch.float32}[sys.argv[4]]
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn(N, V, generator=g, device="cuda").mul_(2).to(dtype)
    val, ids = (z[:, :4000].float() + 1).topk(16, dim=1)
    ids = ids.int()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    o = sv.specv_distill(z, ids, val, with_grad=True)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    assert 0.3 < dt < 20, dt
    status = o["row_status"].tolist()
    assert status[row] == sv.ROW_DEVICE_TIMEOUT and sum(s != 0 for s in status) == 1, status
    assert o["loss"][row] == 0 and (o["grad"][row] == 0).all()
    back = sv.specv_distill_backward(z, ids, val, o["stats"])
    assert (back[row] == 0).all()
    some = [b for b in range(max(0, row - 3), min(N, row + 4)) if b != row] + [N - 1]
    loss, want, scale, _, size = distill64(z[some], ids[some], val[some])
    assert ((o["loss"][some].double() - loss).abs() <= 2.0 ** -17 * scale).all()
    for grad in (o["grad"], back):
        off = (grad[some].double() - want).abs()
        assert (off <= 2.0 ** -17 * size + torch.finfo(dtype).eps / 2 * want.abs() + 1e-30).all()
    assert torch.arange(1000, device="cuda").sum().item() == 499500
    print(f"stall case ok {dt:.2f}")


if __name__ == "__main__":
    main()
