"""A copy that is late in a product is reported (SPECV_ROW_DEVICE_TIMEOUT), without a fault: by
a wait for 16 bytes that no copy brings (the hook SPECV_TEST_STALL, "E:<tile>" in the head's
loss, "F:<tile>" in an orthogonalised update).  Each case in a fresh process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("what,stall", [("head", "E:0"), ("head", "E:200"), ("orth", "F:0"), ("orth", "F:5")])
def test_late_copy_is_reported(what, stall):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    p = subprocess.run([sys.executable, "-m", "tests._products_stall_case", what], cwd=ROOT,
                       env=dict(os.environ, SPECV_TEST_STALL=stall), capture_output=True, text=True, timeout=120)
    assert p.returncode == 0 and "stall case ok" in p.stdout, p.stdout[-2000:] + p.stderr[-3000:]
    print(p.stdout.strip())
