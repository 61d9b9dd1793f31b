"""Host-side refusals of filtered sampling, top logits and distillation: every
call here ends in an argument check before any CUDA call (no GPU needed)."""
import ctypes

import pytest

import speculative_decoding_verification_50_gb300 as sv
from speculative_decoding_verification_50_gb300 import _build

PTR = 0x10000
INV, UNS = sv.SPECV_ERR_INVALID_ARG, sv.SPECV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return sv.load_library()


def sample_args(**kw):
    a = sv.SampleArgs()
    a.B, a.R, a.V, a.dtype = 2, 3, 100, sv.SPECV_FP32
    a.batch_stride, a.row_stride = 300, 100
    a.filtered_batch_stride, a.filtered_row_stride = 300, 100
    for f in ("logits", "temperature", "uniforms", "tokens", "prob", "kept", "filtered"):
        setattr(a, f, PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(R=0), INV), (dict(V=0), INV), (dict(dtype=2), INV),
    (dict(logits=None), INV), (dict(temperature=None), INV),
    (dict(uniforms=None), INV), (dict(tokens=None), INV),
    (dict(uniforms=None, tokens=None), INV),                      # prob without tokens
    (dict(uniforms=None, tokens=None, prob=None, filtered=None), INV),
    (dict(row_stride=99), INV), (dict(batch_stride=299), INV),
    (dict(filtered_row_stride=99), INV), (dict(filtered_batch_stride=299), INV),
    (dict(logits=PTR + 2), INV), (dict(top_k=PTR + 2), INV), (dict(top_p=PTR + 1), INV),
    (dict(V=1 << 20, row_stride=1 << 20, batch_stride=1 << 22, filtered=None), UNS),
])
def test_sample_refusals(lib, kw, code):
    assert lib.specv_sample(ctypes.byref(sample_args(**kw)), None) == code
    assert lib.specv_last_error() and lib.specv_last_launch_count() == 0


def test_empty_batches_launch_nothing(lib):
    assert lib.specv_sample(ctypes.byref(sample_args(B=0)), None) == sv.SPECV_OK
    assert lib.specv_top_logits(ctypes.byref(top_args(B=0)), None) == sv.SPECV_OK
    assert lib.specv_distill(ctypes.byref(distill_args(N=0)), None) == sv.SPECV_OK
    assert lib.specv_distill_backward(ctypes.byref(distill_args(N=0)), None) == sv.SPECV_OK
    assert lib.specv_last_launch_count() == 0


def top_args(**kw):
    a = sv.TopArgs()
    a.B, a.V, a.k, a.dtype, a.row_stride, a.temperature = 2, 100, 8, sv.SPECV_BF16, 100, 1.0
    for f in ("logits", "ids", "values", "lse"):
        setattr(a, f, PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), INV), (dict(V=0), INV), (dict(k=0), INV), (dict(k=sv.SPECV_MAX_TOP + 1), INV),
    (dict(dtype=5), INV), (dict(temperature=0.0), INV), (dict(temperature=float("nan")), INV),
    (dict(logits=None), INV), (dict(ids=None), INV), (dict(values=None), INV),
    (dict(row_stride=99), INV), (dict(logits=PTR + 1), INV), (dict(lse=PTR + 2), INV),
    (dict(V=1 << 21, row_stride=1 << 21), UNS),
])
def test_top_refusals(lib, kw, code):
    assert lib.specv_top_logits(ctypes.byref(top_args(**kw)), None) == code
    assert lib.specv_last_error()


def distill_args(**kw):
    a = sv.DistillArgs()
    a.N, a.V, a.K, a.dtype = 2, 100, 8, sv.SPECV_FP32
    a.row_stride, a.teacher_stride, a.grad_row_stride, a.temperature = 100, 8, 100, 1.0
    for f in ("logits", "teacher_ids", "teacher_logits", "teacher_lse", "weights", "loss", "stats", "grad"):
        setattr(a, f, PTR)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(N=-1), INV), (dict(V=0), INV), (dict(K=0), INV), (dict(K=sv.SPECV_MAX_TOP + 1), INV),
    (dict(dtype=-1), INV), (dict(temperature=-1.0), INV), (dict(temperature=1e9), INV), (dict(flags=2), INV),
    (dict(flags=sv.SPECV_DISTILL_TAIL, teacher_lse=None), INV),
    (dict(logits=None), INV), (dict(teacher_ids=None), INV), (dict(teacher_logits=None), INV),
    (dict(row_stride=99), INV), (dict(grad_row_stride=99), INV), (dict(teacher_stride=7), INV),
    (dict(logits=PTR + 1), INV), (dict(grad=PTR + 2), INV), (dict(stats=PTR + 8), INV), (dict(weights=PTR + 2), INV),
])
def test_distill_refusals(lib, kw, code):
    for fn in (lib.specv_distill, lib.specv_distill_backward):
        assert fn(ctypes.byref(distill_args(**kw)), None) == code
        assert lib.specv_last_error()


def test_distill_refusals_of_one_direction(lib):
    for kw in (dict(loss=None), dict(grad_loss=PTR)):
        assert lib.specv_distill(ctypes.byref(distill_args(**kw)), None) == INV
    big = dict(V=1 << 20, row_stride=1 << 20, grad_row_stride=1 << 20)
    assert lib.specv_distill(ctypes.byref(distill_args(**big)), None) == UNS
    for kw in (dict(stats=None), dict(grad=None)):
        assert lib.specv_distill_backward(ctypes.byref(distill_args(**kw)), None) == INV


def test_python_checks_of_types_and_shapes():
    torch = pytest.importorskip("torch")
    z = torch.zeros(2, 10)
    one = torch.ones(2)
    with pytest.raises(AssertionError):
        sv.specv_sample(z, torch.ones(3), one)
    with pytest.raises(AssertionError):
        sv.specv_sample(z, one.double(), one)
    with pytest.raises(AssertionError):
        sv.specv_sample(z, one, one, top_k=one)
    with pytest.raises(TypeError):
        sv.specv_filter_logits(z.half(), one)
    with pytest.raises(AssertionError):
        sv.specv_distill(z, torch.zeros(2, 3), torch.zeros(2, 3))


def test_rows_that_overlap_are_refused(lib, monkeypatch):
    """Broadcast and overlapping rows keep their strides, which are refused (no
    launch comes of any of these calls)."""
    torch = pytest.importorskip("torch")
    for name in ("_on_gpu", "_cuda"):
        if hasattr(sv, name):
            monkeypatch.setattr(sv, name, lambda *a: True)
    monkeypatch.setattr(sv, "_raw_stream", lambda *a: None)
    B, V, K = 3, 64, 8
    one, two = torch.zeros(1, V).expand(B, V), torch.zeros(B * V).as_strided((B, V), (V // 2, 1))
    good = torch.zeros(B, V)
    T, u = torch.ones(B), torch.full((B,), 0.5)
    ids, val = torch.zeros(B, K, dtype=torch.int32), torch.zeros(B, K)
    few = torch.zeros(1, K, dtype=torch.int32).expand(B, K), torch.zeros(1, K).expand(B, K)
    stats = torch.zeros(B, 4)
    calls = [lambda z=z, f=f: f(z) for z in (one, two) for f in (
        lambda z: sv.specv_sample(z, T, u),
        lambda z: sv.specv_sample(z[:, None], T, u[:, None]),
        lambda z: sv.specv_filter_logits(z, T),
        lambda z: sv.specv_filter_logits(good, T, filtered=z),
        lambda z: sv.specv_sample(z[None], T[:1], u[None]),
        lambda z: sv.specv_top_logits(z, 4),
        lambda z: sv.specv_distill(z, ids, val),
        lambda z: sv.specv_distill(good, ids, val, grad=z),
        lambda z: sv.specv_distill_backward(z, ids, val, stats))]
    calls.append(lambda: sv.specv_distill(good, *few))
    for i, call in enumerate(calls):
        with pytest.raises(sv.SpecvError) as e:
            call()
        assert e.value.status == INV, (i, str(e.value))
