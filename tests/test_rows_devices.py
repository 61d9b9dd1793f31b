"""The row operators' operands lie on one device, and the call goes to it (CPU:
the checks that look for a GPU stand aside, the library's calls are recorded)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_50_gb300 as sv  # noqa: E402

B, V, K = 3, 64, 8


class Elsewhere(torch.Tensor):
    def get_device(self):
        return 1


class Library:
    """Takes every call, and notes the device that was current."""

    def __init__(self, now):
        self.now, self.calls = now, []

    def __getattr__(self, name):
        return lambda args, stream: self.calls.append((name, self.now[-1], stream)) or 0


@pytest.fixture
def lib(monkeypatch):
    now = [0]

    @contextlib.contextmanager
    def device(at):
        now.append(at)
        yield
        now.pop()

    lib = Library(now)
    monkeypatch.setattr(sv, "load_library", lambda: lib)
    monkeypatch.setattr(sv, "_on_gpu", lambda t: True)
    monkeypatch.setattr(sv, "_current_device", lambda: now[-1])
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


def calls(stream=None):
    """Entry points and their operands by name."""
    z, T, u = torch.zeros(B, V), torch.ones(B), torch.zeros(B)
    f = lambda *s: torch.zeros(*s)  # noqa: E731
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    rules = dict(top_k=i(B), top_p=f(B), min_p=f(B), kept=i(B), row_status=i(B), filtered=f(B, V))
    teacher = dict(teacher_ids=i(B, K), teacher_logits=f(B, K), teacher_lse=f(B), weights=f(B), grad=f(B, V), stats=f(B, 4))
    return [
        (sv.specv_sample, dict(logits=z, temperature=T, uniforms=u, tokens=i(B), prob=f(B), **rules)),
        (sv.specv_filter_logits, dict(logits=z, temperature=T, **rules)),
        (sv.specv_top_logits, dict(logits=z, k=K, ids=i(B, K), values=f(B, K), lse=f(B), row_status=i(B))),
        (sv.specv_distill, dict(logits=z, loss=f(B), row_status=i(B), **teacher)),
        (sv.specv_distill_backward, dict(logits=z, grad_loss=f(B), **teacher)),
    ]


def test_operands_of_another_device_are_refused(lib, monkeypatch):
    monkeypatch.setattr(sv, "_raw_stream", lambda *a: None)
    n = 0
    for fn, kw in calls():
        fn(**kw)
        for name in kw:
            if name in ("logits", "k"):
                continue
            with pytest.raises(AssertionError):
                fn(**{**kw, name: kw[name].as_subclass(Elsewhere)})
            n += 1
    assert n == 36 and len(lib.calls) == 5


def test_call_goes_to_the_logits_device(lib, monkeypatch):
    streams = []
    monkeypatch.setattr(sv, "_raw_stream", lambda stream, at: streams.append(at) or 5)
    fn = lib.specv_sample
    for at in (0, 1, -1):
        sv._launch(fn, sv.SampleArgs(), None, at)
    assert lib.calls == [("specv_sample", 0, 5), ("specv_sample", 1, 5), ("specv_sample", 0, 5)]
    assert streams == [0, 1, -1]


def test_stream_of_another_device_is_refused():
    class Stream:
        def __init__(self, index):
            self.device_index, self.cuda_stream = index, 7

    assert sv._raw_stream(Stream(1), 1) == 7
    with pytest.raises(AssertionError):
        sv._raw_stream(Stream(0), 1)
