"""smoke() runs on a GPU without what PyTorch loads when a GPU is asked for a factorisation:
a library of its own, which need not be there."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu


def test_smoke_needs_no_solver_library(monkeypatch):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    def on_host(name, fn):
        def call(*args, **kwargs):
            if any(torch.is_tensor(x) and x.is_cuda for x in (*args, *kwargs.values())):
                raise RuntimeError(f"torch.linalg.{name} of a CUDA tensor")
            return fn(*args, **kwargs)
        return call

    for name in dir(torch.linalg):
        fn = getattr(torch.linalg, name)
        if callable(fn) and not isinstance(fn, type) and not name.startswith("_"):
            monkeypatch.setattr(torch.linalg, name, on_host(name, fn))
    __graft_entry__.smoke()
