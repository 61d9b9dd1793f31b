"""Copies and products that are late, in every kind of wait that the other stall tests do not
reach, end in zeros or in a status, without a fault: by a wait for bytes or an arrival that
nothing brings (the hook SPECV_TEST_STALL; "G:<t>" to "I:<t>": unit t of dz, dW and dh in the
head's loss; "J:<t>": what unit t's epilogues read in an update's first
step; "K:<n>": the end of matrix n's first products in the kernel of small updates).  Each case in a fresh process."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("what,stall,N", [("dz", "G:77", 45), ("dz", "G:0", 300), ("dW", "H:0", 45), ("dW", "H:33", 300),
                                          ("dh", "I:1", 45), ("dh", "I:0", 300), ("update", "J:0", 300), ("update", "J:2", 200),
                                          ("small", "K:1", 90), ("small", "K:1", 500), ("small", "K:1", 2048)])
def test_late_copies(what, stall, N):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    p = subprocess.run([sys.executable, "-m", "tests._late_case", what, str(N)], cwd=ROOT,
                       env=dict(os.environ, SPECV_TEST_STALL=stall), capture_output=True, text=True, timeout=180)
    assert p.returncode == 0 and "late case ok" in p.stdout, p.stdout[-2000:] + p.stderr[-3000:]
    print(p.stdout.strip())
