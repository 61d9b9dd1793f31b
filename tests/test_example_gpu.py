"""The example that runs filtered sampling, verification under the rules, top
logits and distillation together: the drafter learns, and more of its tokens
are accepted."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")

PATH = os.path.join(os.path.dirname(__file__), "..", "examples", "online_distillation.py")


def _load():
    spec = importlib.util.spec_from_file_location("online_distillation", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_imports():
    assert callable(_load().run)


@pytest.mark.gpu
def test_example_learns():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from speculative_decoding_verification_50_gb300 import _build
    _build.build()
    accepted, losses = _load().run(rounds=120, batch=64, vocab=1024)
    assert all(0.0 <= a <= 4.0 for a in accepted)
    assert sum(losses[-20:]) < 0.7 * sum(losses[:20])
    assert sum(accepted[-20:]) > sum(accepted[:20])
