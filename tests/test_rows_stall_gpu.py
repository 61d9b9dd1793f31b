"""A copy that is late in either pass of the distillation kernel is reported
(SPECV_ROW_DEVICE_TIMEOUT, loss and gradient 0): without a fault, by a wait for
16 bytes that no copy brings (the hook SPECV_TEST_STALL, "C:<row>" in the first
pass, "D:<row>" in the second).  Each case in a fresh process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("stall", ["C", "D"])
@pytest.mark.parametrize("rows,V,dtype", [(456, 30016, "fp32"), (456, 60032, "bf16"), (200, 152064, "fp32")])
def test_late_copy_is_reported(stall, rows, V, dtype):
    """One CTA per row, and a cluster of two."""
    run(f"{stall}:{rows // 2}", rows // 2, rows, V, dtype)


def test_late_copy_of_a_held_row():
    run("C:3", 3, 8, 30016, "fp32")


def run(stall, row, rows, V, dtype):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    p = subprocess.run([sys.executable, "-m", "tests._rows_stall_case", str(row), str(rows), str(V), dtype], cwd=ROOT,
                       env=dict(os.environ, SPECV_TEST_STALL=stall), capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "stall case ok" in p.stdout, p.stdout[-2000:] + p.stderr[-3000:]
    print(p.stdout.strip())
