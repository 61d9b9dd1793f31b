"""GB300 (sm_103a) speculative-sampling verification and SSD outcome prediction.

Thin Python binding over the C ABI of ``libspecv.so`` (declared in
``include/specv.h``): it marshals torch tensors into pointers, sizes and
strides and passes the current CUDA stream.  Every step of the computation
runs in the library's CUDA kernels; there is no Python or CPU fallback, and a
missing library raises.

Entry points (same names as the C ABI):
  specv_verify(target, draft, draft_tokens, temperature, uniforms, ...)
  specv_ssd_round(target, draft, draft_tokens, temperature, uniforms, F, ...)
  specv_predict_outcomes(draft, draft_tokens, F, ...)
  specv_check_hit(keys, accept_len, out_tokens, ...)
  specv_sample(logits, temperature, uniforms, top_k=, top_p=, min_p=, ...)
  specv_filter_logits(logits, temperature, top_k=, top_p=, min_p=, ...)
  specv_top_logits(logits, k, ...)
  specv_distill(logits, teacher_ids, teacher_logits, ...)
  specv_distill_backward(logits, teacher_ids, teacher_logits, stats, ...)
  distill_loss(logits, teacher_ids, teacher_logits, ...)  (differentiable)
  specv_head_loss(hidden, head, targets, ...)
  specv_head_loss_backward(hidden, head, targets, stats, ...)
  head_loss(hidden, head, targets, ...)  (differentiable)
  specv_orthogonalize(update, ...)
"""
from __future__ import annotations

import ctypes
import os

from . import workloads  # noqa: F401  (seeded inputs; no method arithmetic)

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libspecv.so")

SPECV_OK, SPECV_ERR_INVALID_ARG, SPECV_ERR_UNSUPPORTED, SPECV_ERR_CUDA, SPECV_ERR_WORKSPACE = range(5)
SPECV_BF16, SPECV_FP32 = 0, 1
ROW_BAD_TOKEN, ROW_NONFINITE, ROW_BAD_TEMP, ROW_FALLBACK, ROW_DEVICE_TIMEOUT = 1, 2, 4, 8, 16
ROW_BAD_COUNT = 32
ROW_BAD_FILTER = 64
SPECV_MAX_TOP = 1024
SPECV_DISTILL_TAIL = 1
SPECV_HEAD_TARGETS_ONLY = 1
SPECV_NO_DRAFT_PROBS = 1
SPECV_MSS_NAIVE = 1

_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64


class VerifyArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("K", _I32), ("V", _I32), ("dtype", _I32),
                ("target_logits", _P), ("target_batch_stride", _I64), ("target_row_stride", _I64),
                ("draft_logits", _P), ("draft_batch_stride", _I64), ("draft_row_stride", _I64),
                ("draft_tokens", _P), ("temperature", _P), ("uniforms", _P),
                ("accept_len", _P), ("out_tokens", _P), ("p_draft", _P), ("q_draft", _P),
                ("row_status", _P), ("cu_num_draft_tokens", _P), ("num_draft_tokens", _I32),
                ("flags", _I32)]


class SsdArgs(ctypes.Structure):
    _fields_ = [("verify", VerifyArgs), ("F", _I32), ("keys", _P), ("key_logits", _P),
                ("hit", _P), ("fanout", _P), ("saguaro_F", _I32), ("saguaro_C", ctypes.c_float)]


class SaguaroArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("V", _I32), ("dtype", _I32), ("logits", _P), ("row_stride", _I64),
                ("temperature", _P), ("F", _I32), ("C", ctypes.c_float), ("uniforms", _P),
                ("tokens", _P), ("q", _P), ("row_status", _P)]


class MssArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("M", _I32), ("V", _I32), ("dtype", _I32),
                ("target_logits", _P), ("target_row_stride", _I64),
                ("draft_logits", _P), ("draft_row_stride", _I64),
                ("candidates", _P), ("num_candidates", _P), ("temperature", _P), ("uniforms", _P),
                ("flags", _I32), ("accepted", _P), ("out_token", _P), ("accept_prob", _P),
                ("row_status", _P)]


class PredictArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("K", _I32), ("V", _I32), ("F", _I32), ("dtype", _I32),
                ("draft_logits", _P), ("draft_batch_stride", _I64), ("draft_row_stride", _I64),
                ("draft_tokens", _P), ("keys", _P), ("key_logits", _P), ("row_status", _P),
                ("fanout", _P)]


class SampleArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("R", _I32), ("V", _I32), ("dtype", _I32), ("logits", _P),
                ("batch_stride", _I64), ("row_stride", _I64), ("temperature", _P),
                ("top_k", _P), ("top_p", _P), ("min_p", _P), ("uniforms", _P), ("tokens", _P),
                ("prob", _P), ("kept", _P), ("filtered", _P), ("filtered_batch_stride", _I64),
                ("filtered_row_stride", _I64), ("row_status", _P)]


class TopArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("V", _I32), ("k", _I32), ("dtype", _I32), ("logits", _P),
                ("row_stride", _I64), ("temperature", ctypes.c_float), ("ids", _P),
                ("values", _P), ("lse", _P), ("row_status", _P)]


class DistillArgs(ctypes.Structure):
    _fields_ = [("N", _I32), ("V", _I32), ("K", _I32), ("dtype", _I32), ("logits", _P),
                ("row_stride", _I64), ("teacher_ids", _P), ("teacher_logits", _P),
                ("teacher_stride", _I64), ("teacher_lse", _P), ("weights", _P),
                ("temperature", ctypes.c_float), ("flags", _I32), ("loss", _P), ("stats", _P),
                ("grad_loss", _P), ("grad", _P), ("grad_row_stride", _I64), ("row_status", _P)]


class HeadArgs(ctypes.Structure):
    _fields_ = [("N", _I32), ("V", _I32), ("D", _I32), ("dtype", _I32),
                ("hidden", _P), ("hidden_stride", _I64), ("head", _P), ("head_stride", _I64),
                ("targets", _P), ("weights", _P), ("scale", ctypes.c_float), ("flags", _I32),
                ("loss", _P), ("stats", _P), ("row_status", _P), ("grad_loss", _P),
                ("grad_hidden", _P), ("grad_hidden_stride", _I64),
                ("grad_head", _P), ("grad_head_stride", _I64)]


class OrthArgs(ctypes.Structure):
    _fields_ = [("B", _I32), ("m", _I32), ("n", _I32), ("dtype", _I32),
                ("update", _P), ("batch_stride", _I64), ("row_stride", _I64), ("steps", _I32),
                ("a", ctypes.c_float), ("b", ctypes.c_float), ("c", ctypes.c_float),
                ("out", _P), ("out_batch_stride", _I64), ("out_row_stride", _I64), ("norm", _P), ("row_status", _P)]


class SpecvError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"specv status {status}: {msg}")
        self.status = status


_lib = None
_lib_path = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libspecv.so (built by __graft_entry__.build()); raise if absent."""
    global _lib, _lib_path
    if _lib is not None and path == _lib_path:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(path)
    lib.specv_verify_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_verify_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32]
    lib.specv_verify.restype = ctypes.c_int
    lib.specv_verify.argtypes = [ctypes.POINTER(VerifyArgs), _P, ctypes.c_size_t, _P]
    lib.specv_verify_noalloc.restype = ctypes.c_int
    lib.specv_verify_noalloc.argtypes = [ctypes.POINTER(VerifyArgs), _P]
    lib.specv_ssd_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_ssd_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32, _I32]
    lib.specv_ssd_round.restype = ctypes.c_int
    lib.specv_ssd_round.argtypes = [ctypes.POINTER(SsdArgs), _P, ctypes.c_size_t, _P]
    lib.specv_predict_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_predict_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32, _I32]
    lib.specv_predict_outcomes.restype = ctypes.c_int
    lib.specv_predict_outcomes.argtypes = [ctypes.POINTER(PredictArgs), _P, ctypes.c_size_t, _P]
    lib.specv_saguaro_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_saguaro_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32]
    lib.specv_saguaro_sample.restype = ctypes.c_int
    lib.specv_saguaro_sample.argtypes = [ctypes.POINTER(SaguaroArgs), _P, ctypes.c_size_t, _P]
    lib.specv_mss_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_mss_workspace_bytes.argtypes = [_I32, _I32, _I32, _I32]
    lib.specv_mss_verify.restype = ctypes.c_int
    lib.specv_mss_verify.argtypes = [ctypes.POINTER(MssArgs), _P, ctypes.c_size_t, _P]
    lib.specv_geometric_fanout.restype = ctypes.c_int
    lib.specv_geometric_fanout.argtypes = [_I32, ctypes.c_double, ctypes.c_double, _I32, _I32,
                                           _P, _P]
    lib.specv_check_hit.restype = ctypes.c_int
    lib.specv_check_hit.argtypes = [_I32, _I32, _I32, _P, _P, _P, _P, _P]
    for name, args in (("specv_sample", SampleArgs), ("specv_top_logits", TopArgs),
                       ("specv_distill", DistillArgs), ("specv_distill_backward", DistillArgs)):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.POINTER(args), _P]
    lib.specv_head_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_head_workspace_bytes.argtypes = [ctypes.POINTER(HeadArgs)]
    lib.specv_orthogonalize_workspace_bytes.restype = ctypes.c_size_t
    lib.specv_orthogonalize_workspace_bytes.argtypes = [_I32, _I32, _I32]
    for name, args in (("specv_head_loss", HeadArgs), ("specv_head_loss_backward", HeadArgs),
                       ("specv_orthogonalize", OrthArgs)):
        fn = getattr(lib, name)
        fn.restype = ctypes.c_int
        fn.argtypes = [ctypes.POINTER(args), _P, ctypes.c_size_t, _P]
    lib.specv_status_string.restype = ctypes.c_char_p
    lib.specv_status_string.argtypes = [ctypes.c_int]
    lib.specv_last_error.restype = ctypes.c_char_p
    lib.specv_last_error.argtypes = []
    lib.specv_last_launch_count.restype = _I32
    lib.specv_last_launch_count.argtypes = []
    lib.specv_set_split_event.restype = None
    lib.specv_set_split_event.argtypes = [_P]
    _lib, _lib_path = lib, path
    return lib


def _check(rc: int) -> None:
    if rc != SPECV_OK:
        lib = load_library()
        raise SpecvError(rc, lib.specv_last_error().decode() or lib.specv_status_string(rc).decode())


def _dtype_code(t) -> int:
    import torch
    if t.dtype == torch.bfloat16:
        return SPECV_BF16
    if t.dtype == torch.float32:
        return SPECV_FP32
    raise TypeError(f"logits must be bfloat16 or float32, got {t.dtype}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def specv_set_split_event(event) -> None:
    """Record `event` (a torch.cuda.Event, already recorded once so that it
    exists, or None) between the library's two kernels on later calls from
    this thread (measurement hook; see include/specv.h)."""
    handle = None if event is None else ctypes.c_void_p(event.cuda_event)
    load_library().specv_set_split_event(handle)


def last_launch_count() -> int:
    """Kernel launches enqueued by the most recent call on this thread."""
    return int(load_library().specv_last_launch_count())


def _verify_args(target, draft, draft_tokens, temperature, uniforms, draft_rows, accept_len,
                 out_tokens, p_draft, q_draft, row_status):
    import torch
    B, K = draft_tokens.shape
    V = target.shape[-1]
    assert target.dim() == 3 and target.shape[0] == B and target.shape[1] >= K + 1
    assert target.stride(-1) == 1
    if draft is not None:  # None: no draft probabilities (SPECV_NO_DRAFT_PROBS)
        assert draft.dim() == 3 and draft.shape[0] == B and draft.shape[1] >= draft_rows
        assert draft.shape[-1] == V and draft.stride(-1) == 1 and target.dtype == draft.dtype
    assert uniforms.shape == (B, K + 1) and temperature.shape == (B,)
    dev = target.device
    if accept_len is None:
        accept_len = torch.empty(B, dtype=torch.int32, device=dev)
    if out_tokens is None:
        out_tokens = torch.empty((B, K + 1), dtype=torch.int32, device=dev)
    if p_draft is None:
        p_draft = torch.empty((B, K), dtype=torch.float32, device=dev)
    if q_draft is None:
        q_draft = torch.empty((B, K), dtype=torch.float32, device=dev)
    if row_status is None:
        row_status = torch.empty(B, dtype=torch.int32, device=dev)
    args = VerifyArgs(B, K, V, _dtype_code(target),
                      target.data_ptr(), target.stride(0), target.stride(1),
                      None if draft is None else draft.data_ptr(),
                      0 if draft is None else draft.stride(0), 0 if draft is None else draft.stride(1),
                      draft_tokens.data_ptr(), temperature.data_ptr(), uniforms.data_ptr(),
                      accept_len.data_ptr(), out_tokens.data_ptr(),
                      p_draft.data_ptr(), q_draft.data_ptr(), row_status.data_ptr(),
                      None, 0, SPECV_NO_DRAFT_PROBS if draft is None else 0)
    outs = dict(accept_len=accept_len, out_tokens=out_tokens, p_draft=p_draft,
                q_draft=q_draft, row_status=row_status)
    return args, outs


def specv_verify(target, draft, draft_tokens, temperature, uniforms, *, accept_len=None,
                 out_tokens=None, p_draft=None, q_draft=None, row_status=None,
                 workspace=None, stream=None) -> dict:
    """Verify B batch rows on the GPU (see include/specv.h, specv_verify).

    target [B, >=K+1, V], draft [B, >=K, V] (bf16 or fp32, CUDA, last dim
    contiguous) or None for drafts without probabilities (SPECV_NO_DRAFT_PROBS);
    draft_tokens int32 [B, K]; temperature fp32 [B]; uniforms fp32 [B, K+1].
    Outputs are allocated when not given.  Returns a dict with accept_len,
    out_tokens, p_draft, q_draft, row_status.
    """
    import torch
    lib = load_library()
    B, K = draft_tokens.shape
    args, outs = _verify_args(target, draft, draft_tokens, temperature, uniforms, K, accept_len,
                              out_tokens, p_draft, q_draft, row_status)
    need = lib.specv_verify_workspace_bytes(B, K, target.shape[-1], args.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=target.device)
    _check(lib.specv_verify(ctypes.byref(args), _ptr(workspace), workspace.numel(), _stream(stream)))
    return outs


def specv_verify_ragged(target, draft, cu_num_draft_tokens, draft_tokens, temperature, uniforms,
                        K: int, *, num_draft_tokens: int | None = None, accept_len=None,
                        out_tokens=None, p_draft=None, q_draft=None, row_status=None,
                        workspace=None, stream=None) -> dict:
    """Verification with a per-row draft count (see include/specv.h,
    cu_num_draft_tokens): rows packed along one axis.

    target [N + B, V] (K_b + 1 rows per batch row, in order), draft [N, V] or
    None (no draft probabilities), cu_num_draft_tokens int32 [B] (inclusive
    prefix sums, on the device), draft_tokens int32 [N], temperature fp32 [B],
    uniforms fp32 [N + B]; K = the largest count allowed.  N defaults to
    draft_tokens.numel().  Returns accept_len [B], out_tokens [B, K+1],
    p_draft / q_draft [N], row_status [B].
    """
    import torch
    lib = load_library()
    B = cu_num_draft_tokens.shape[0]
    N = draft_tokens.numel() if num_draft_tokens is None else int(num_draft_tokens)
    V = target.shape[-1]
    assert target.dim() == 2 and target.stride(-1) == 1 and target.shape[0] >= N + B
    if draft is not None:
        assert draft.dim() == 2 and draft.stride(-1) == 1 and draft.shape[0] >= N
        assert draft.shape[-1] == V and draft.dtype == target.dtype
    assert draft_tokens.numel() >= N and uniforms.numel() >= N + B and temperature.shape == (B,)
    dev = target.device
    i32 = dict(dtype=torch.int32, device=dev)
    accept_len = torch.empty(B, **i32) if accept_len is None else accept_len
    out_tokens = torch.empty((B, K + 1), **i32) if out_tokens is None else out_tokens
    p_draft = torch.zeros(max(N, 1), dtype=torch.float32, device=dev) if p_draft is None else p_draft
    q_draft = torch.zeros(max(N, 1), dtype=torch.float32, device=dev) if q_draft is None else q_draft
    row_status = torch.empty(B, **i32) if row_status is None else row_status
    args = VerifyArgs(B, K, V, _dtype_code(target), target.data_ptr(), 0, target.stride(0),
                      None if draft is None else draft.data_ptr(), 0,
                      0 if draft is None else draft.stride(0),
                      draft_tokens.data_ptr(), temperature.data_ptr(), uniforms.data_ptr(),
                      accept_len.data_ptr(), out_tokens.data_ptr(), p_draft.data_ptr(),
                      q_draft.data_ptr(), row_status.data_ptr(), cu_num_draft_tokens.data_ptr(),
                      N, SPECV_NO_DRAFT_PROBS if draft is None else 0)
    need = lib.specv_verify_workspace_bytes(B, K, V, args.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    _check(lib.specv_verify(ctypes.byref(args), _ptr(workspace), workspace.numel(), _stream(stream)))
    return dict(accept_len=accept_len, out_tokens=out_tokens, p_draft=p_draft, q_draft=q_draft,
                row_status=row_status)


def specv_verify_noalloc(target, draft, draft_tokens, temperature, uniforms, *, accept_len=None,
                         out_tokens=None, p_draft=None, q_draft=None, row_status=None,
                         stream=None) -> dict:
    """specv_verify without a workspace: the library's built-in scratch is used
    (for callers that cannot allocate device memory where they call it; see
    include/specv.h).  Calls that may overlap on the GPU must be serialised."""
    lib = load_library()
    B, K = draft_tokens.shape
    args, outs = _verify_args(target, draft, draft_tokens, temperature, uniforms, K, accept_len,
                              out_tokens, p_draft, q_draft, row_status)
    _check(lib.specv_verify_noalloc(ctypes.byref(args), _stream(stream)))
    return outs


def _fanout_arg(fanout, K: int):
    """A host int32 array [K+1] kept alive by the caller, or None."""
    if fanout is None:
        return None, None
    vals = [int(x) for x in fanout]
    assert len(vals) == K + 1, "fanout needs K+1 entries"
    arr = (_I32 * (K + 1))(*vals)
    return arr, ctypes.cast(arr, _P)


def specv_ssd_round(target, draft, draft_tokens, temperature, uniforms, F: int, *,
                    accept_len=None, out_tokens=None, p_draft=None, q_draft=None,
                    row_status=None, keys=None, key_logits=None, hit=None, workspace=None,
                    fanout=None, saguaro=None, stream=None) -> dict:
    """One fused SSD round (see include/specv.h, specv_ssd_round): verification,
    top-F outcome keys at every lookahead and the hit flag, in one pass.

    draft must hold K+1 rows per batch row.  Returns the specv_verify outputs
    plus keys int32 [B, K+1, F], key_logits fp32 [B, K+1, F], hit uint8 [B].
    fanout (optional, K+1 ints in [0, F], e.g. from specv_geometric_fanout)
    keeps only the first fanout[k] keys at lookahead k.  saguaro=(F_s, C): the
    drafts were sampled from sigma_{F_s,C} (specv_saguaro_sample), so the
    accept test and the residual use it as q.
    """
    import torch
    lib = load_library()
    B, K = draft_tokens.shape
    args, outs = _verify_args(target, draft, draft_tokens, temperature, uniforms, K + 1,
                              accept_len, out_tokens, p_draft, q_draft, row_status)
    dev = target.device
    if keys is None:
        keys = torch.empty((B, K + 1, F), dtype=torch.int32, device=dev)
    if key_logits is None:
        key_logits = torch.empty((B, K + 1, F), dtype=torch.float32, device=dev)
    if hit is None:
        hit = torch.empty(B, dtype=torch.uint8, device=dev)
    need = lib.specv_ssd_workspace_bytes(B, K, target.shape[-1], F, args.dtype)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    fan_keep, fan_ptr = _fanout_arg(fanout, K)
    sg_F, sg_C = saguaro if saguaro else (0, 1.0)
    sargs = SsdArgs(args, F, keys.data_ptr(), key_logits.data_ptr(), hit.data_ptr(), fan_ptr,
                    int(sg_F), float(sg_C))
    _check(lib.specv_ssd_round(ctypes.byref(sargs), _ptr(workspace), workspace.numel(),
                               _stream(stream)))
    outs.update(keys=keys, key_logits=key_logits, hit=hit)
    return outs


def specv_predict_outcomes(draft, draft_tokens, F: int, *, keys=None, key_logits=None,
                           row_status=None, workspace=None, fanout=None, stream=None) -> dict:
    """Top-F outcome keys per lookahead (see include/specv.h).

    draft [B, >=K+1, V] (bf16 or fp32, CUDA); draft_tokens int32 [B, K].
    Returns keys int32 [B, K+1, F], key_logits fp32, row_status int32 [B].
    """
    import torch
    lib = load_library()
    B, K = draft_tokens.shape
    V = draft.shape[-1]
    assert draft.dim() == 3 and draft.shape[0] == B and draft.shape[1] >= K + 1
    assert draft.stride(-1) == 1
    dev = draft.device
    if keys is None:
        keys = torch.empty((B, K + 1, F), dtype=torch.int32, device=dev)
    if key_logits is None:
        key_logits = torch.empty((B, K + 1, F), dtype=torch.float32, device=dev)
    if row_status is None:
        row_status = torch.empty(B, dtype=torch.int32, device=dev)
    code = _dtype_code(draft)
    need = lib.specv_predict_workspace_bytes(B, K, V, F, code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    fan_keep, fan_ptr = _fanout_arg(fanout, K)
    args = PredictArgs(B, K, V, F, code, draft.data_ptr(), draft.stride(0), draft.stride(1),
                       draft_tokens.data_ptr(), keys.data_ptr(), key_logits.data_ptr(),
                       row_status.data_ptr(), fan_ptr)
    _check(lib.specv_predict_outcomes(ctypes.byref(args), _ptr(workspace), workspace.numel(),
                                      _stream(stream)))
    return dict(keys=keys, key_logits=key_logits, row_status=row_status)


def specv_saguaro_sample(logits, temperature, F: int, C: float, uniforms, *, tokens=None, q=None,
                         row_status=None, workspace=None, stream=None) -> dict:
    """Draft-side Saguaro sampling (see include/specv.h): one token per row of
    logits [B, V] (bf16 or fp32, CUDA) from sigma_{F,C}(z/T) by inverse CDF of
    uniforms [B].  Returns tokens int32 [B], q fp32 [B], row_status int32 [B]."""
    import torch
    lib = load_library()
    assert logits.dim() == 2 and logits.stride(-1) == 1
    B, V = logits.shape
    dev = logits.device
    tokens = torch.empty(B, dtype=torch.int32, device=dev) if tokens is None else tokens
    q = torch.empty(B, dtype=torch.float32, device=dev) if q is None else q
    row_status = torch.empty(B, dtype=torch.int32, device=dev) if row_status is None else row_status
    code = _dtype_code(logits)
    need = lib.specv_saguaro_workspace_bytes(B, V, int(F), code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    args = SaguaroArgs(B, V, code, logits.data_ptr(), logits.stride(0), temperature.data_ptr(),
                       int(F), float(C), uniforms.data_ptr(), tokens.data_ptr(), q.data_ptr(),
                       row_status.data_ptr())
    _check(lib.specv_saguaro_sample(ctypes.byref(args), _ptr(workspace), workspace.numel(),
                                    _stream(stream)))
    return dict(tokens=tokens, q=q, row_status=row_status)


def specv_mss_verify(target, draft, candidates, temperature, uniforms, *, num_candidates=None,
                     naive: bool = False, accepted=None, out_token=None, accept_prob=None,
                     row_status=None, workspace=None, stream=None) -> dict:
    """Multi-step speculative sampling at B token-tree nodes (see
    include/specv.h): target, draft [B, V] (bf16 or fp32, CUDA; rows may be
    strided), candidates int32 [B, M], num_candidates int32 [B] or None,
    temperature fp32 [B], uniforms fp32 [B, M+1].  naive=True: naive sampling.
    Returns accepted int32 [B], out_token int32 [B], accept_prob fp32 [B, M],
    row_status int32 [B]."""
    import torch
    lib = load_library()
    assert target.dim() == 2 and draft.dim() == 2 and target.shape == draft.shape
    assert target.stride(-1) == 1 and draft.stride(-1) == 1 and target.dtype == draft.dtype
    B, V = target.shape
    M = candidates.shape[1]
    dev = target.device
    i32 = dict(dtype=torch.int32, device=dev)
    accepted = torch.empty(B, **i32) if accepted is None else accepted
    out_token = torch.empty(B, **i32) if out_token is None else out_token
    accept_prob = (torch.empty((B, M), dtype=torch.float32, device=dev)
                   if accept_prob is None else accept_prob)
    row_status = torch.empty(B, **i32) if row_status is None else row_status
    code = _dtype_code(target)
    need = lib.specv_mss_workspace_bytes(B, M, V, code)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    args = MssArgs(B, M, V, code, target.data_ptr(), target.stride(0), draft.data_ptr(),
                   draft.stride(0), candidates.data_ptr(),
                   num_candidates.data_ptr() if num_candidates is not None else None,
                   temperature.data_ptr(), uniforms.data_ptr(),
                   SPECV_MSS_NAIVE if naive else 0, accepted.data_ptr(), out_token.data_ptr(),
                   accept_prob.data_ptr(), row_status.data_ptr())
    _check(lib.specv_mss_verify(ctypes.byref(args), _ptr(workspace), workspace.numel(),
                                _stream(stream)))
    return dict(accepted=accepted, out_token=out_token, accept_prob=accept_prob,
                row_status=row_status)


def specv_geometric_fanout(K: int, a: float, r: float, budget: int, max_f: int = 32) -> tuple:
    """Theorem 12 fan-out (see include/specv.h): (integer F_k list, real F_k list)."""
    lib = load_library()
    fk = (_I32 * (K + 1))()
    real = (ctypes.c_double * (K + 1))()
    _check(lib.specv_geometric_fanout(int(K), float(a), float(r), int(budget), int(max_f),
                                      ctypes.cast(fk, _P), ctypes.cast(real, _P)))
    return list(fk), list(real)


def specv_check_hit(keys, accept_len, out_tokens, *, hit=None, stream=None):
    """hit[b] = out_tokens[b, n_b] in keys[b, n_b, :] (uint8 [B])."""
    import torch
    lib = load_library()
    B, K1, F = keys.shape
    assert accept_len.shape == (B,) and out_tokens.shape == (B, K1)
    if hit is None:
        hit = torch.empty(B, dtype=torch.uint8, device=keys.device)
    _check(lib.specv_check_hit(B, K1 - 1, F, _ptr(keys), _ptr(accept_len), _ptr(out_tokens),
                               _ptr(hit), _stream(stream)))
    return hit


def _on_gpu(t) -> bool:
    return t.is_cuda


def _of(t, shape, dtype, what, at):
    """t's pointer after a check of its type, shape, layout and place: device `at`, the
    logits', which _cuda holds to be a GPU (None: optional)."""
    if t is None:
        return None
    assert t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == at, (
        f"{what}: {t.dtype} {tuple(t.shape)} on {t.device}, expected contiguous {dtype} {tuple(shape)} "
        f"on the logits' GPU ({at})")
    return t.data_ptr()


def _raw_stream(stream, at):
    """The stream's handle (the current stream of device `at` by default; asked for
    directly, since a decode step makes many small calls)."""
    import torch
    if stream is not None:
        its = getattr(stream, "device_index", at)
        assert its == at, f"a stream of GPU {its} for tensors on GPU {at}"
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(at)


def _current_device() -> int:
    import torch
    return torch._C._cuda_getDevice()


def _launch(fn, args, stream, at, *space):
    """The entry point fn on device `at`, where its operands lie: a kernel goes to
    the current device, whatever device its stream or its pointers are of."""
    if at < 0 or at == _current_device():
        _check(fn(ctypes.byref(args), *space, _raw_stream(stream, at)))
        return
    import torch
    with torch.cuda.device(at):
        _check(fn(ctypes.byref(args), *space, _raw_stream(stream, at)))


def _cuda(t, what, at=None):
    assert _on_gpu(t) and (t.stride(-1) == 1 or t.shape[-1] == 1), (
        f"{what} must be a CUDA tensor with a contiguous last dimension")
    assert at is None or t.get_device() == at, f"{what} on {t.device}, the logits on GPU {at}"


def _stride(t, dim, width):
    """t's stride along dim; `width`, the least that is taken, where dim has one
    entry (whose stride means nothing)."""
    return t.stride(dim) if t.shape[dim] > 1 else width


def _sample_call(logits, temperature, uniforms, top_k, top_p, min_p, tokens, prob, kept, filtered,
                 row_status, stream):
    import torch
    code = _dtype_code(logits)
    shape = logits.shape
    lead, V, flat = shape[:-1], shape[-1], len(shape) == 2
    assert flat or len(shape) == 3, "logits must be [B, V] or [B, R, V]"
    B, R = lead[0], 1 if flat else lead[1]
    f32, i32, dev = torch.float32, torch.int32, logits.device
    at = logits.get_device()
    per = (B,)
    T = _of(temperature, per, f32, "temperature", at)
    k, p = _of(top_k, per, i32, "top_k", at), _of(top_p, per, f32, "top_p", at)
    m, u = _of(min_p, per, f32, "min_p", at), _of(uniforms, lead, f32, "uniforms", at)
    out = {}
    if uniforms is not None:
        out["tokens"] = tokens = torch.empty(lead, dtype=i32, device=dev) if tokens is None else tokens
        out["prob"] = prob = torch.empty(lead, dtype=f32, device=dev) if prob is None else prob
    out["kept"] = kept = torch.empty(lead, dtype=i32, device=dev) if kept is None else kept
    out["row_status"] = row_status = (torch.empty(lead, dtype=i32, device=dev) if row_status is None
                                      else row_status)
    _cuda(logits, "logits")
    bs, rs = _stride(logits, 0, V), V if flat else _stride(logits, 1, V)
    fptr, fbs, frs = None, 0, 0
    if filtered is not None:
        assert filtered.shape == shape and filtered.dtype is logits.dtype, "filtered must be like logits"
        _cuda(filtered, "filtered", at)
        fptr = filtered.data_ptr()
        fbs, frs = _stride(filtered, 0, V), V if flat else _stride(filtered, 1, V)
        out["filtered"] = filtered
    args = SampleArgs(B, R, V, code, logits.data_ptr(), bs, rs, T, k, p, m, u,
                      _of(tokens, lead, i32, "tokens", at), _of(prob, lead, f32, "prob", at),
                      _of(kept, lead, i32, "kept", at), fptr, fbs, frs,
                      _of(row_status, lead, i32, "row_status", at))
    _launch(load_library().specv_sample, args, stream, at)
    return out


def specv_sample(logits, temperature, uniforms, *, top_k=None, top_p=None, min_p=None, tokens=None,
                 prob=None, kept=None, filtered=None, row_status=None, stream=None) -> dict:
    """One token per row under temperature, top-k, top-p and min-p, by inverse
    CDF of the given uniforms (see include/specv.h, specv_sample).

    logits [B, V] or [B, R, V] (bf16 or fp32, CUDA, last dim contiguous);
    temperature fp32 [B] (0: greedy), top_k int32 [B] (0: off), top_p fp32 [B]
    (1: off), min_p fp32 [B] (0: off), shared by an entry's R rows; uniforms
    fp32 [B] or [B, R].  Returns tokens int32, prob fp32, kept int32 and
    row_status int32, shaped as uniforms, and `filtered` if that was given (a
    tensor like logits, or logits itself) to be written.
    """
    assert uniforms is not None
    return _sample_call(logits, temperature, uniforms, top_k, top_p, min_p, tokens, prob, kept,
                        filtered, row_status, stream)


def specv_filter_logits(logits, temperature, *, top_k=None, top_p=None, min_p=None, filtered=None,
                        kept=None, row_status=None, stream=None) -> dict:
    """The logits that the rules of specv_sample keep, -inf elsewhere: filtered
    target and draft rows are verified (specv_verify) under those rules.

    Arguments as specv_sample; filtered may be logits itself.  Returns
    filtered, kept, row_status.
    """
    import torch
    if filtered is None:  # (not empty_like: that keeps gaps between strided rows)
        filtered = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    return _sample_call(logits, temperature, None, top_k, top_p, min_p, None, None, kept, filtered,
                        row_status, stream)


def specv_top_logits(logits, k: int, *, temperature: float = 1.0, ids=None, values=None, lse=None,
                     row_status=None, stream=None) -> dict:
    """The k largest logits per row of logits [B, V] (bf16 or fp32, CUDA), by
    (logit descending, index ascending), and log sum exp(logits / temperature)
    (see include/specv.h).  Returns ids int32 [B, k], values fp32 [B, k], lse
    fp32 [B], row_status int32 [B]."""
    import torch
    assert logits.dim() == 2
    code = _dtype_code(logits)
    B, V = logits.shape
    f32, i32, dev = torch.float32, torch.int32, logits.device
    at, rows = logits.get_device(), max(int(k), 0)
    ids = torch.empty((B, rows), dtype=i32, device=dev) if ids is None else ids
    values = torch.empty((B, rows), dtype=f32, device=dev) if values is None else values
    lse = torch.empty(B, dtype=f32, device=dev) if lse is None else lse
    row_status = torch.empty(B, dtype=i32, device=dev) if row_status is None else row_status
    _cuda(logits, "logits")
    args = TopArgs(B, V, int(k), code, logits.data_ptr(), _stride(logits, 0, V),
                   float(temperature), _of(ids, (B, rows), i32, "ids", at),
                   _of(values, (B, rows), f32, "values", at), _of(lse, (B,), f32, "lse", at),
                   _of(row_status, (B,), i32, "row_status", at))
    _launch(load_library().specv_top_logits, args, stream, at)
    return dict(ids=ids, values=values, lse=lse, row_status=row_status)


def _distill_args(logits, ids, values, teacher_lse, weights, temperature, tail, grad):
    import torch
    assert logits.dim() == 2
    code = _dtype_code(logits)
    N, V = logits.shape
    K = ids.shape[1]
    f32, at = torch.float32, logits.get_device()
    assert ids.shape == values.shape == (N, K) and ids.dtype == torch.int32 and values.dtype == f32
    _cuda(ids, "teacher_ids", at)
    _cuda(values, "teacher_logits", at)
    ts = _stride(ids, 0, K)
    assert N <= 1 or ids.stride(0) == values.stride(0), "teacher_ids and teacher_logits share one row stride"
    _cuda(logits, "logits")
    if grad is not None:
        assert grad.shape == logits.shape and grad.dtype == logits.dtype, "grad must be like logits"
        _cuda(grad, "grad", at)
    return DistillArgs(N, V, K, code, logits.data_ptr(), _stride(logits, 0, V),
                       ids.data_ptr(), values.data_ptr(), ts,
                       _of(teacher_lse, (N,), f32, "teacher_lse", at),
                       _of(weights, (N,), f32, "weights", at), float(temperature),
                       SPECV_DISTILL_TAIL if tail else 0, None, None, None,
                       None if grad is None else grad.data_ptr(),
                       0 if grad is None else _stride(grad, 0, V), None)


def specv_distill(logits, teacher_ids, teacher_logits, *, teacher_lse=None, temperature: float = 1.0,
                  weights=None, tail: bool = False, with_grad: bool = False, loss=None, stats=None,
                  grad=None, row_status=None, stream=None) -> dict:
    """Distillation loss of student rows against a teacher's top logits (see
    include/specv.h, specv_distill).

    logits [N, V] (bf16 or fp32, CUDA); teacher_ids int32 and teacher_logits
    fp32 [N, K], as specv_top_logits returns them (id -1: none); teacher_lse
    fp32 [N] at the same temperature (None: the listed entries alone are
    normalised; `tail` needs it); weights fp32 [N] or None.  Returns loss fp32
    [N], stats fp32 [N, 4] (for specv_distill_backward), row_status int32 [N],
    and grad (the gradient of loss.sum(), like logits) with with_grad or where
    a buffer is given.
    """
    import torch
    N, dev, at = logits.shape[0], logits.device, logits.get_device()
    if grad is None and with_grad:
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
    loss = torch.empty(N, dtype=torch.float32, device=dev) if loss is None else loss
    stats = torch.empty((N, 4), dtype=torch.float32, device=dev) if stats is None else stats
    row_status = torch.empty(N, dtype=torch.int32, device=dev) if row_status is None else row_status
    args = _distill_args(logits, teacher_ids, teacher_logits, teacher_lse, weights, temperature,
                         tail, grad)
    args.loss = _of(loss, (N,), torch.float32, "loss", at)
    args.stats = _of(stats, (N, 4), torch.float32, "stats", at)
    args.row_status = _of(row_status, (N,), torch.int32, "row_status", at)
    _launch(load_library().specv_distill, args, stream, at)
    out = dict(loss=loss, stats=stats, row_status=row_status)
    if grad is not None:
        out["grad"] = grad
    return out


def specv_distill_backward(logits, teacher_ids, teacher_logits, stats, *, grad_loss=None,
                           teacher_lse=None, temperature: float = 1.0, weights=None,
                           tail: bool = False, grad=None, stream=None):
    """The gradient of (grad_loss * loss).sum() with respect to logits, from
    the stats of specv_distill on the same inputs (see include/specv.h)."""
    import torch
    N, at = logits.shape[0], logits.get_device()
    if grad is None:
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
    args = _distill_args(logits, teacher_ids, teacher_logits, teacher_lse, weights, temperature,
                         tail, grad)
    args.stats = _of(stats, (N, 4), torch.float32, "stats", at)
    args.grad_loss = _of(grad_loss, (N,), torch.float32, "grad_loss", at)
    _launch(load_library().specv_distill_backward, args, stream, at)
    return grad


_DistillLoss = None


def distill_loss(logits, teacher_ids, teacher_logits, *, teacher_lse=None, temperature: float = 1.0,
                 weights=None, tail: bool = False):
    """specv_distill's loss per row [N], differentiable with respect to logits
    (once: the backward pass is specv_distill_backward).  To capture a training
    step in a CUDA graph, call specv_distill with a gradient buffer, or
    specv_distill_backward, in it: an autograd graph of the same leaves that was
    built outside the capture must not be alive while one is captured.
    """
    global _DistillLoss
    if _DistillLoss is None:
        import torch

        class DistillLoss(torch.autograd.Function):
            @staticmethod
            def forward(ctx, logits, ids, values, lse, temperature, weights, tail):
                out = specv_distill(logits, ids, values, teacher_lse=lse, temperature=temperature,
                                    weights=weights, tail=tail)
                ctx.save_for_backward(logits, ids, values, lse, weights, out["stats"])
                ctx.how = (temperature, tail)
                return out["loss"]

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, up):
                logits, ids, values, lse, weights, stats = ctx.saved_tensors
                temperature, tail = ctx.how
                grad = specv_distill_backward(logits, ids, values, stats, teacher_lse=lse,
                                              grad_loss=up.to(torch.float32).contiguous(),
                                              temperature=temperature, weights=weights, tail=tail)
                return grad, None, None, None, None, None, None

        _DistillLoss = DistillLoss
    return _DistillLoss.apply(logits, teacher_ids, teacher_logits, teacher_lse, temperature, weights,
                              tail)


def _work(need, workspace, device, stream):
    """The workspace's pointer, its size in bytes, and what keeps it.  Where none is given one
    is allocated, as the stream's own that the call goes to."""
    import torch
    if workspace is None:
        if stream is None or device.type != "cuda":
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    else:
        assert workspace.is_contiguous() and workspace.device == device, f"workspace must be contiguous, on {device}"
    return _ptr(workspace), workspace.numel() * workspace.element_size(), workspace


def _sizes(*tensors):
    """(ctypes cuts a size off that 32 bits do not hold.)"""
    for t in tensors:
        assert max(t.shape) < 2 ** 31, f"a size of {tuple(t.shape)} is 2^31 or more"


def _head_args(hidden, head, targets, scale, weights, grad_hidden, grad_head):
    import torch
    assert hidden.dim() == 2 and head.dim() == 2 and hidden.shape[1] == head.shape[1], (
        f"hidden [N, D] and head [V, D], got {tuple(hidden.shape)} and {tuple(head.shape)}")
    _sizes(hidden, head)
    code = _dtype_code(hidden)
    assert head.dtype == hidden.dtype, f"hidden is {hidden.dtype}, head {head.dtype}"
    (N, D), V, at = hidden.shape, head.shape[0], hidden.get_device()
    _cuda(hidden, "hidden")
    _cuda(head, "head", at)
    for grad, like, what in ((grad_hidden, hidden, "grad_hidden"), (grad_head, head, "grad_head")):
        if grad is not None:
            assert grad.shape == like.shape and grad.dtype == like.dtype, f"{what} must be like what it is the gradient of"
            _cuda(grad, what, at)
    of = lambda t: (None, 0) if t is None else (t.data_ptr(), _stride(t, 0, D))  # noqa: E731
    return HeadArgs(N, V, D, code, *of(hidden), *of(head), _of(targets, (N,), torch.int32, "targets", at),
                    _of(weights, (N,), torch.float32, "weights", at), float(scale), 0, None, None, None, None,
                    *of(grad_hidden), *of(grad_head))


def specv_head_loss(hidden, head, targets, *, scale: float = 1.0, weights=None, with_grad: bool = False,
                    targets_only: bool = False, loss=None, stats=None, row_status=None, grad_hidden=None, grad_head=None,
                    workspace=None, stream=None) -> dict:
    """Cross entropy of the tokens `targets` under softmax(scale * hidden @ head.T), without
    the logits as an input or an output (see include/specv.h, specv_head_loss).

    hidden [N, D] and head [V, D] (bf16, CUDA, last dim contiguous); targets int32 [N] (-1:
    none); weights fp32 [N] or None (0: a row that is left out).  Returns loss fp32 [N], stats
    fp32 [N, 2] (the row's log-sum-exp and minus the target's log-probability), row_status
    int32 [N], and with with_grad, or where a buffer is given, grad_hidden and grad_head (of
    loss.sum()).  Rows without a target are left out of a call with gradients, and of one with
    targets_only; in others they have their log-sum-exp.
    """
    import torch
    N, dev, at = hidden.shape[0], hidden.device, hidden.get_device()
    if with_grad:  # (not empty_like: that keeps gaps between strided rows)
        grad_hidden = torch.empty(hidden.shape, dtype=hidden.dtype, device=dev) if grad_hidden is None else grad_hidden
        grad_head = torch.empty(head.shape, dtype=head.dtype, device=dev) if grad_head is None else grad_head
    loss = torch.empty(N, dtype=torch.float32, device=dev) if loss is None else loss
    stats = torch.empty((N, 2), dtype=torch.float32, device=dev) if stats is None else stats
    row_status = torch.empty(N, dtype=torch.int32, device=dev) if row_status is None else row_status
    args = _head_args(hidden, head, targets, scale, weights, grad_hidden, grad_head)
    args.flags = SPECV_HEAD_TARGETS_ONLY if targets_only else 0
    args.loss = _of(loss, (N,), torch.float32, "loss", at)
    args.stats = _of(stats, (N, 2), torch.float32, "stats", at)
    args.row_status = _of(row_status, (N,), torch.int32, "row_status", at)
    lib = load_library()
    ptr, size, _keep = _work(lib.specv_head_workspace_bytes(ctypes.byref(args)), workspace, dev, stream)
    _launch(lib.specv_head_loss, args, stream, at, ptr, size)
    out = dict(loss=loss, stats=stats, row_status=row_status)
    if grad_hidden is not None:
        out["grad_hidden"] = grad_hidden
    if grad_head is not None:
        out["grad_head"] = grad_head
    return out


def specv_head_loss_backward(hidden, head, targets, stats, *, grad_loss=None, scale: float = 1.0, weights=None,
                             grad_hidden=None, grad_head=None, row_status=None, workspace=None, stream=None) -> dict:
    """The gradients of (grad_loss * loss).sum() by hidden and head, from the stats of
    specv_head_loss on the same inputs (see include/specv.h).  Where one of grad_hidden and
    grad_head is given, that one alone; else both.  Returns a dict of them."""
    import torch
    N, dev, at = hidden.shape[0], hidden.device, hidden.get_device()
    if grad_hidden is None and grad_head is None:
        grad_hidden = torch.empty(hidden.shape, dtype=hidden.dtype, device=dev)
        grad_head = torch.empty(head.shape, dtype=head.dtype, device=dev)
    args = _head_args(hidden, head, targets, scale, weights, grad_hidden, grad_head)
    args.stats = _of(stats, (N, 2), torch.float32, "stats", at)
    args.grad_loss = _of(grad_loss, (N,), torch.float32, "grad_loss", at)
    args.row_status = _of(row_status, (N,), torch.int32, "row_status", at)
    lib = load_library()
    ptr, size, _keep = _work(lib.specv_head_workspace_bytes(ctypes.byref(args)), workspace, dev, stream)
    _launch(lib.specv_head_loss_backward, args, stream, at, ptr, size)
    out = {}
    if grad_hidden is not None:
        out["grad_hidden"] = grad_hidden
    if grad_head is not None:
        out["grad_head"] = grad_head
    return out


_HeadLoss = None


def head_loss(hidden, head, targets, *, scale: float = 1.0, weights=None):
    """specv_head_loss's loss per row [N], differentiable with respect to hidden and head
    (once: the backward pass is specv_head_loss_backward, which computes the logits again;
    after a device wait that ran out its gradients are zeros).
    To capture a training step in a CUDA graph, call specv_head_loss with gradient buffers, or
    specv_head_loss_backward, in it, as for distill_loss."""
    global _HeadLoss
    if _HeadLoss is None:
        import torch

        class HeadLoss(torch.autograd.Function):
            @staticmethod
            def forward(ctx, hidden, head, targets, scale, weights):
                out = specv_head_loss(hidden, head, targets, scale=scale, weights=weights, targets_only=True)
                ctx.save_for_backward(hidden, head, targets, weights, out["stats"])
                ctx.scale = scale
                return out["loss"]

            @staticmethod
            @torch.autograd.function.once_differentiable
            def backward(ctx, up):
                hidden, head, targets, weights, stats = ctx.saved_tensors
                want = {}
                if ctx.needs_input_grad[0]:
                    want["grad_hidden"] = torch.empty(hidden.shape, dtype=hidden.dtype, device=hidden.device)
                if ctx.needs_input_grad[1]:
                    want["grad_head"] = torch.empty(head.shape, dtype=head.dtype, device=head.device)
                if want:
                    specv_head_loss_backward(hidden, head, targets, stats, scale=ctx.scale, weights=weights,
                                             grad_loss=up.to(torch.float32).contiguous(), **want)
                return want.get("grad_hidden"), want.get("grad_head"), None, None, None

        _HeadLoss = HeadLoss
    return _HeadLoss.apply(hidden, head, targets, scale, weights)


def specv_orthogonalize(update, *, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), out=None, norm=None,
                        row_status=None, workspace=None, stream=None) -> dict:
    """An update with its singular values drawn towards one, by `steps` of X <- a X + (b S +
    c S S) X with S = X X^T from X = update / |update|_F (see include/specv.h).

    update [m, n], or [B, m, n] for B matrices (bf16 or fp32, CUDA, last dim contiguous).
    Matrices of a batch that overlap (expand) or lie between each other's rows are refused.
    Returns orthogonal (bf16, shaped as update; `out`, which may be update itself), norm fp32
    and row_status int32 (scalars, or [B])."""
    import torch
    assert update.dim() in (2, 3), "update must be [m, n] or [B, m, n]"
    flat, dev, at = update.dim() == 2, update.device, update.get_device()
    lead = update.shape[:-2]
    _sizes(update)
    code = _dtype_code(update)
    if out is None:
        out = torch.empty(update.shape, dtype=torch.bfloat16, device=dev)
    norm = torch.empty(lead, dtype=torch.float32, device=dev) if norm is None else norm
    row_status = torch.empty(lead, dtype=torch.int32, device=dev) if row_status is None else row_status
    _cuda(update, "update")
    assert out.shape == update.shape and out.dtype == torch.bfloat16, "out must be bfloat16, shaped as update"
    _cuda(out, "out", at)
    B, (m, n) = 1 if flat else update.shape[0], update.shape[-2:]
    a, b, c = (float(x) for x in coefficients)
    strides = lambda t: (m * n if flat else _stride(t, 0, m * n), _stride(t, -2, n))  # noqa: E731
    args = OrthArgs(B, m, n, code, update.data_ptr(), *strides(update), int(steps), a, b, c, out.data_ptr(), *strides(out),
                    _of(norm, lead, torch.float32, "norm", at), _of(row_status, lead, torch.int32, "row_status", at))
    lib = load_library()
    ptr, size, _keep = _work(lib.specv_orthogonalize_workspace_bytes(B, m, n), workspace, dev, stream)
    _launch(lib.specv_orthogonalize, args, stream, at, ptr, size)
    return dict(orthogonal=out, norm=norm, row_status=row_status)
