"""Python binding of libstreamkl (ctypes).  Argument marshalling only: every
step of the computation runs in the library's CUDA kernels.  PyTorch supplies
device memory and the current stream.

Functions mirror the C ABI in ``include/streamkl.h``:

    kl_fwd(Q1, K1, Q2, K2, causal=False, scale=None) -> (KL, LSE1, LSE2)
    kl_bwd(setting, g, Q1, K1, Q2, K2, KL, LSE1, LSE2, causal=False) -> (dQ, dK)
    kl_bwd_joint(g, Q1, K1, Q2, K2, KL, LSE1, LSE2, causal=False) -> (dQ1, dK1, dQ2, dK2)

plus ``fwd_plan`` / ``bwd_plan`` (what a call launches) and ``AttentionKL``,
an autograd Function.  The divergence of attentions with capped or biased
scores and a key range per row:

    key_ranges(B, Nq, Nk, device, causal=True, ...) -> (begin, end, offset)
    kl_score_fwd(Scores(cap1=50.0, begin=begin, end=end), Q1, K1, Q2, K2) -> (KL, LSE1, LSE2)
    kl_score_bwd(setting, scores, g, Q1, K1, Q2, K2, KL, LSE1, LSE2) -> (dQ, dK)

and ``ScoredAttentionKL``, its autograd Function.  The step before the divergence, the norm of query and
key heads with their rotation:

    rope_table(rows, rot, device) -> table
    qk_norm_rope(q, k, wq, wk, table, positions=None) -> (q', k')
    qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, table, positions=None) -> (dq, dk, dwq, dwk)

and ``QKNormRope``, its autograd Function.  There is no fallback: without the compiled library
every call raises.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

from . import build as _build

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT = range(6)
PATH_TILE, PATH_DECODE, PATH_BWD_FUSED, PATH_BWD_SPLIT, PATH_BWD_KEYSPLIT, PATH_BWD_JOINT = range(6)
BWD_AUTO, BWD_FUSED, BWD_SPLIT, BWD_KEYSPLIT = 0, 1, 2, 3


class Shape(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int32), ("H", ctypes.c_int32), ("Nq", ctypes.c_int32), ("Nk", ctypes.c_int32),
                ("d", ctypes.c_int32), ("q_stride_b", ctypes.c_int64), ("q_stride_h", ctypes.c_int64),
                ("q_stride_n", ctypes.c_int64), ("k_stride_b", ctypes.c_int64), ("k_stride_h", ctypes.c_int64),
                ("k_stride_n", ctypes.c_int64), ("H_kv", ctypes.c_int32)]


class Options(ctypes.Structure):
    _fields_ = [("num_splits", ctypes.c_int32), ("bwd_mode", ctypes.c_int32), ("wait_limit_ns", ctypes.c_int64),
                ("debug_flags", ctypes.c_int32), ("grad_bf16", ctypes.c_int32)]


DEBUG_INJECT_STALL = 1


class Plan(ctypes.Structure):
    _fields_ = [("path", ctypes.c_int32), ("num_splits", ctypes.c_int32), ("num_ctas", ctypes.c_int32),
                ("launches", ctypes.c_int32), ("workspace_bytes", ctypes.c_size_t)]


class Strides(ctypes.Structure):
    _fields_ = [("b", ctypes.c_int64), ("h", ctypes.c_int64), ("n", ctypes.c_int64)]


class Score(ctypes.Structure):
    _fields_ = [("cap1", ctypes.c_float), ("cap2", ctypes.c_float)] + \
        [(n, ctypes.c_void_p) for n in ("slopes1", "slopes2", "begin", "end", "offset")]


class NormRope(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "Hq", "Hk", "N", "d", "rot", "interleaved", "weight_bf16",
                                              "grad_bf16", "pos_int64")] + \
        [("eps", ctypes.c_float), ("table_rows", ctypes.c_int64), ("start", ctypes.c_int64)] + \
        [(n, Strides) for n in ("q", "k", "yq", "yk", "dq", "dk")]


class StreamKLError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


EXPORTED = ("streamkl_fwd_plan", "streamkl_fwd", "streamkl_bwd_plan", "streamkl_bwd", "streamkl_workspace_status",
            "streamkl_status_string", "streamkl_version", "streamkl_fwd_noalloc", "streamkl_noalloc_status",
            "streamkl_fwd_workspace_bytes", "streamkl_bwd_workspace_bytes", "streamkl_bwd_joint_plan",
            "streamkl_bwd_joint", "streamkl_norm_rope_fwd", "streamkl_norm_rope_bwd",
            "streamkl_norm_rope_workspace_bytes", "streamkl_rope_table", "streamkl_score_fwd_plan", "streamkl_score_fwd",
            "streamkl_score_bwd_plan", "streamkl_score_bwd", "streamkl_key_ranges")

_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_stale: bool = True):
    """Load libstreamkl.so (building it first when sources are newer)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if build_if_stale and _build.is_stale():
            _build.build()
        if not os.path.exists(_build.LIB):
            raise RuntimeError(f"libstreamkl.so is missing ({_build.LIB}); run __graft_entry__.build()")
        lib = ctypes.CDLL(_build.LIB)
        P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        sp, op, pp = ctypes.POINTER(Shape), ctypes.POINTER(Options), ctypes.POINTER(Plan)
        lib.streamkl_fwd_plan.argtypes = [sp, I, op, pp]
        lib.streamkl_fwd.argtypes = [sp, P, P, P, P, F, I, P, P, P, P, Z, op, P]
        lib.streamkl_bwd_plan.argtypes = [sp, I, I, op, pp]
        lib.streamkl_bwd.argtypes = [sp, I, P, P, P, P, P, P, P, P, F, I, P, P, P, Z, op, P]
        lib.streamkl_workspace_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_uint32)]
        lib.streamkl_fwd_noalloc.argtypes = [sp, P, P, P, P, F, I, P, P, P, op, P]
        lib.streamkl_noalloc_status.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
        lib.streamkl_bwd_joint_plan.argtypes = [sp, I, op, pp]
        lib.streamkl_bwd_joint.argtypes = [sp, P, P, P, P, P, P, P, P, F, I, P, P, P, P, P, Z, op, P]
        lib.streamkl_fwd_workspace_bytes.argtypes = [sp, I]
        lib.streamkl_bwd_workspace_bytes.argtypes = [sp, I, I]
        lib.streamkl_fwd_workspace_bytes.restype = Z
        lib.streamkl_bwd_workspace_bytes.restype = Z
        sc = ctypes.POINTER(Score)
        i32 = ctypes.c_int32
        lib.streamkl_score_fwd_plan.argtypes = [sp, op, pp]
        lib.streamkl_score_fwd.argtypes = [sp, sc, P, P, P, P, F, I, P, P, P, P, Z, op, P]
        lib.streamkl_score_bwd_plan.argtypes = [sp, I, op, pp]
        lib.streamkl_score_bwd.argtypes = [sp, sc, I, P, P, P, P, P, P, P, P, F, I, P, P, P, Z, op, P]
        lib.streamkl_key_ranges.argtypes = [i32, i32, i32, I, i32, P, P, P, P, i32, i32, P, P, P, P]
        nr = ctypes.POINTER(NormRope)
        lib.streamkl_norm_rope_fwd.argtypes = [nr, *[P] * 9]
        lib.streamkl_norm_rope_bwd.argtypes = [nr, *[P] * 13, Z, P]
        lib.streamkl_norm_rope_workspace_bytes.argtypes = [nr]
        lib.streamkl_norm_rope_workspace_bytes.restype = Z
        lib.streamkl_rope_table.argtypes = [P, ctypes.c_int64, ctypes.c_int32, P, P]
        lib.streamkl_status_string.argtypes = [I]
        lib.streamkl_status_string.restype = ctypes.c_char_p
        for name in ("streamkl_fwd_plan", "streamkl_fwd", "streamkl_bwd_plan", "streamkl_bwd",
                     "streamkl_workspace_status", "streamkl_version", "streamkl_fwd_noalloc",
                     "streamkl_noalloc_status", "streamkl_bwd_joint_plan", "streamkl_bwd_joint",
                     "streamkl_norm_rope_fwd", "streamkl_norm_rope_bwd", "streamkl_rope_table",
                     "streamkl_score_fwd_plan", "streamkl_score_fwd", "streamkl_score_bwd_plan", "streamkl_score_bwd",
                     "streamkl_key_ranges"):
            getattr(lib, name).restype = ctypes.c_int
        _lib = lib
        return lib


def status_string(code: int) -> str:
    return load().streamkl_status_string(int(code)).decode()


def _raise(code, where):
    if code != OK:
        raise StreamKLError(code, where)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p(0)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def make_shape(Q1, K1) -> Shape:
    """Shape/strides struct of [B, H, N, d] tensors (d must be contiguous)."""
    B, H, Nq, d = Q1.shape
    Nk = K1.shape[2]
    qs, ks = Q1.stride(), K1.stride()
    return Shape(B, H, Nq, Nk, d, qs[0], qs[1], qs[2], ks[0], ks[1], ks[2], K1.shape[1])


def _check_qk(Q1, K1, Q2, K2):
    for name, t in (("Q1", Q1), ("K1", K1), ("Q2", Q2), ("K2", K2)):
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype != torch.bfloat16:
            raise ValueError(f"{name} must be bf16, got {t.dtype}")
        if t.dim() != 4 or t.stride(3) != 1:
            raise ValueError(f"{name} must be [B, H, N, d] with d contiguous")
    if Q1.shape != Q2.shape or K1.shape != K2.shape or Q1.stride() != Q2.stride() or K1.stride() != K2.stride():
        raise ValueError("teacher and student tensors must have equal shapes and strides")
    if Q1.shape[0] != K1.shape[0] or Q1.shape[3] != K1.shape[3]:
        raise ValueError("Q and K must share B and d")
    if Q1.shape[1] % K1.shape[1] != 0:
        raise ValueError("the key head count must divide the query head count")
    if any(t.device != Q1.device for t in (K1, Q2, K2)):
        raise ValueError("Q1, K1, Q2 and K2 must be on one device")


def _check_tensor(name, t, shape, dtype, device):
    """Outputs and per-row inputs are written or read as dense arrays of the
    given shape: anything else would send the kernels out of bounds."""
    if not isinstance(t, torch.Tensor) or t.device != device:
        raise ValueError(f"{name} must be a tensor on {device}")
    if t.dtype != dtype or not t.is_contiguous() or tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)}, got "
                         f"{t.dtype} {tuple(t.shape)}{'' if t.is_contiguous() else ' (not contiguous)'}")


def _check_workspace(workspace, nbytes, device):
    """None allocates one; a caller's workspace must be a large enough
    contiguous uint8 tensor on the inputs' device (it is never replaced)."""
    if workspace is None:
        return new_workspace(nbytes, device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    if workspace.numel() < nbytes:
        raise ValueError(f"workspace holds {workspace.numel()} bytes; this call needs {nbytes} (see fwd_plan / bwd_plan)")
    return workspace


def _opts(num_splits=0, bwd_mode=0, wait_limit_ns=0, debug_flags=0, grad_bf16=0):
    return Options(int(num_splits), int(bwd_mode), int(wait_limit_ns), int(debug_flags), int(grad_bf16))


def fwd_plan(Q1, K1, causal=False, num_splits=0) -> Plan:
    plan = Plan()
    _raise(load().streamkl_fwd_plan(ctypes.byref(make_shape(Q1, K1)), int(bool(causal)),
                                    ctypes.byref(_opts(num_splits)), ctypes.byref(plan)), "streamkl_fwd_plan")
    return plan


def bwd_plan(Q1, K1, setting, causal=False, mode=BWD_AUTO, grad_dtype=torch.float32, num_splits=0) -> Plan:
    plan = Plan()
    _raise(load().streamkl_bwd_plan(ctypes.byref(make_shape(Q1, K1)), int(setting), int(bool(causal)),
                                    ctypes.byref(_opts(num_splits, mode, grad_bf16=_grad_flag(grad_dtype))),
                                    ctypes.byref(plan)), "streamkl_bwd_plan")
    return plan


def fwd_workspace_bytes(Q1, K1, causal=False) -> int:
    """streamkl_fwd_workspace_bytes: the forward's workspace with default options (0 = invalid shape)."""
    return int(load().streamkl_fwd_workspace_bytes(ctypes.byref(make_shape(Q1, K1)), int(bool(causal))))


def bwd_workspace_bytes(Q1, K1, setting, causal=False) -> int:
    """streamkl_bwd_workspace_bytes: the backward's workspace with default options (0 = invalid)."""
    return int(load().streamkl_bwd_workspace_bytes(ctypes.byref(make_shape(Q1, K1)), int(setting),
                                                   int(bool(causal))))


def noalloc_status(device=None) -> int:
    """streamkl_noalloc_status: synchronise the current stream of ``device`` and
    return (and clear) the device error word of the allocation-free forward's
    built-in scratch (0 when no bounded wait gave up)."""
    word = ctypes.c_uint32(0)
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    rc = load().streamkl_noalloc_status(_stream(dev), ctypes.byref(word))
    if rc not in (OK, ERR_TIMEOUT):
        _raise(rc, "streamkl_noalloc_status")
    return int(word.value)


def _grad_flag(grad_dtype):
    if grad_dtype == torch.float32:
        return 0
    if grad_dtype == torch.bfloat16:
        return 1
    raise ValueError(f"gradients are float32 or bfloat16, not {grad_dtype}")


def new_workspace(nbytes, device) -> torch.Tensor:
    """A zeroed workspace (the first 256 bytes hold the device error word)."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def kl_fwd(Q1, K1, Q2, K2, causal=False, scale=None, num_splits=0, workspace=None, out=None,
           wait_limit_ns=0, debug_flags=0):
    """Per-row KL(P1 || P2), LSE1, LSE2 as float32 [B, H, Nq] tensors."""
    _check_qk(Q1, K1, Q2, K2)
    lib = load()
    shape = make_shape(Q1, K1)
    opts = _opts(num_splits, 0, wait_limit_ns, debug_flags)
    plan = Plan()
    _raise(lib.streamkl_fwd_plan(ctypes.byref(shape), int(bool(causal)), ctypes.byref(opts), ctypes.byref(plan)),
           "streamkl_fwd_plan")
    B, H, Nq, _ = Q1.shape
    if out is None:
        out = tuple(torch.empty((B, H, Nq), dtype=torch.float32, device=Q1.device) for _ in range(3))
    for name, t in zip(("KL", "LSE1", "LSE2"), out):
        _check_tensor(name, t, (B, H, Nq), torch.float32, Q1.device)
    workspace = _check_workspace(workspace, plan.workspace_bytes, Q1.device)
    KL, L1, L2 = out
    rc = lib.streamkl_fwd(ctypes.byref(shape), _ptr(Q1), _ptr(K1), _ptr(Q2), _ptr(K2),
                          ctypes.c_float(0.0 if scale is None else float(scale)), int(bool(causal)), _ptr(KL),
                          _ptr(L1), _ptr(L2), _ptr(workspace), workspace.numel(), ctypes.byref(opts),
                          _stream(Q1.device))
    _raise(rc, "streamkl_fwd")
    return KL, L1, L2


def kl_bwd(setting, g, Q1, K1, Q2, K2, KL, LSE1, LSE2, causal=False, scale=None, mode=BWD_AUTO, workspace=None,
           out=None, wait_limit_ns=0, debug_flags=0, grad_dtype=torch.float32, num_splits=0):
    """(dQ, dK) float32 of the trainable side: setting 1 -> (Q2, K2), 2 -> (Q1, K1).
    With keys shared by groups of query heads (K has fewer heads than Q), dK
    has K's head count and sums the gradients of each group.  num_splits sets
    the key-range splits of the key-split mode (0 = automatic)."""
    _check_qk(Q1, K1, Q2, K2)
    lib = load()
    shape = make_shape(Q1, K1)
    opts = _opts(num_splits, mode, wait_limit_ns, debug_flags, _grad_flag(grad_dtype))
    plan = Plan()
    _raise(lib.streamkl_bwd_plan(ctypes.byref(shape), int(setting), int(bool(causal)), ctypes.byref(opts),
                                 ctypes.byref(plan)), "streamkl_bwd_plan")
    B, H, Nq, d = Q1.shape
    Nk = K1.shape[2]
    for name, t in (("g", g), ("KL", KL), ("LSE1", LSE1), ("LSE2", LSE2)):
        _check_tensor(name, t, (B, H, Nq), torch.float32, Q1.device)
    if out is None:
        out = (torch.empty((B, H, Nq, d), dtype=grad_dtype, device=Q1.device),
               torch.empty((B, K1.shape[1], Nk, d), dtype=grad_dtype, device=Q1.device))
    _check_tensor("dQ", out[0], (B, H, Nq, d), grad_dtype, Q1.device)
    _check_tensor("dK", out[1], (B, K1.shape[1], Nk, d), grad_dtype, Q1.device)
    workspace = _check_workspace(workspace, plan.workspace_bytes, Q1.device)
    dQ, dK = out
    rc = lib.streamkl_bwd(ctypes.byref(shape), int(setting), _ptr(g), _ptr(Q1), _ptr(K1), _ptr(Q2), _ptr(K2),
                          _ptr(KL), _ptr(LSE1), _ptr(LSE2), ctypes.c_float(0.0 if scale is None else float(scale)),
                          int(bool(causal)), _ptr(dQ), _ptr(dK), _ptr(workspace), workspace.numel(),
                          ctypes.byref(opts), _stream(Q1.device))
    _raise(rc, "streamkl_bwd")
    return dQ, dK


def bwd_joint_plan(Q1, K1, causal=False, grad_dtype=torch.float32) -> Plan:
    plan = Plan()
    _raise(load().streamkl_bwd_joint_plan(ctypes.byref(make_shape(Q1, K1)), int(bool(causal)),
                                          ctypes.byref(_opts(grad_bf16=_grad_flag(grad_dtype))), ctypes.byref(plan)),
           "streamkl_bwd_joint_plan")
    return plan


def kl_bwd_joint(g, Q1, K1, Q2, K2, KL, LSE1, LSE2, causal=False, scale=None, workspace=None, out=None,
                 wait_limit_ns=0, debug_flags=0, grad_dtype=torch.float32):
    """(dQ1, dK1, dQ2, dK2): the gradients of both sides from one recompute of
    the scores per kernel -- the teacher's as in setting 2, the student's as
    in setting 1 (streamkl_bwd_joint)."""
    _check_qk(Q1, K1, Q2, K2)
    lib = load()
    shape = make_shape(Q1, K1)
    opts = _opts(0, 0, wait_limit_ns, debug_flags, _grad_flag(grad_dtype))
    plan = Plan()
    _raise(lib.streamkl_bwd_joint_plan(ctypes.byref(shape), int(bool(causal)), ctypes.byref(opts),
                                       ctypes.byref(plan)), "streamkl_bwd_joint_plan")
    B, H, Nq, d = Q1.shape
    Hk, Nk = K1.shape[1], K1.shape[2]
    for name, t in (("g", g), ("KL", KL), ("LSE1", LSE1), ("LSE2", LSE2)):
        _check_tensor(name, t, (B, H, Nq), torch.float32, Q1.device)
    if out is None:
        out = tuple(torch.empty(shp, dtype=grad_dtype, device=Q1.device)
                    for shp in ((B, H, Nq, d), (B, Hk, Nk, d), (B, H, Nq, d), (B, Hk, Nk, d)))
    for name, t, shp in zip(("dQ1", "dK1", "dQ2", "dK2"), out,
                            ((B, H, Nq, d), (B, Hk, Nk, d), (B, H, Nq, d), (B, Hk, Nk, d))):
        _check_tensor(name, t, shp, grad_dtype, Q1.device)
    workspace = _check_workspace(workspace, plan.workspace_bytes, Q1.device)
    dQ1, dK1, dQ2, dK2 = out
    rc = lib.streamkl_bwd_joint(ctypes.byref(shape), _ptr(g), _ptr(Q1), _ptr(K1), _ptr(Q2), _ptr(K2), _ptr(KL),
                                _ptr(LSE1), _ptr(LSE2), ctypes.c_float(0.0 if scale is None else float(scale)),
                                int(bool(causal)), _ptr(dQ1), _ptr(dK1), _ptr(dQ2), _ptr(dK2), _ptr(workspace),
                                workspace.numel(), ctypes.byref(opts), _stream(Q1.device))
    _raise(rc, "streamkl_bwd_joint")
    return dQ1, dK1, dQ2, dK2


def workspace_status(workspace) -> int:
    """Synchronise the current stream and return (and clear) the workspace's
    device error word; raises StreamKLError(ERR_TIMEOUT) when it was set."""
    word = ctypes.c_uint32(0)
    rc = load().streamkl_workspace_status(_ptr(workspace), _stream(workspace.device), ctypes.byref(word))
    if rc not in (OK, ERR_TIMEOUT):
        _raise(rc, "streamkl_workspace_status")
    return int(word.value)


class AttentionKL(torch.autograd.Function):
    """Per-row KL(softmax(Q1 K1^T s) || softmax(Q2 K2^T s)) with a recompute
    backward.  Gradients flow to the student (setting 1) or the teacher
    (setting 2), chosen by which inputs require grad; the other side gets
    None.  When both sides require grad, the joint backward forms the
    gradients of both from one recompute of the scores per kernel
    (streamkl_bwd_joint): measured on GB300 at 64K causal it takes as long as
    the two single-setting passes (145.7 vs 144.5 ms) and, adding no gradient
    through atomics, gives the same bits on every run.  For at most 16 query
    rows per key head (decode shapes) the two single-setting key-split passes
    run instead.  Together the two sides
    are the gradient of KL with respect to all four inputs: each setting
    differentiates through one side's distribution with the other side's held
    fixed.  Gradients come back in bf16, like the inputs."""

    @staticmethod
    def forward(ctx, Q1, K1, Q2, K2, causal=False, scale=None):
        _guard_capture(Q1, K1, Q2, K2)
        KL, L1, L2 = kl_fwd(Q1, K1, Q2, K2, causal=causal, scale=scale)
        ctx.save_for_backward(Q1, K1, Q2, K2, KL, L1, L2)
        ctx.causal, ctx.scale = causal, scale
        return KL

    @staticmethod
    def backward(ctx, gKL):
        Q1, K1, Q2, K2, KL, L1, L2 = ctx.saved_tensors
        student = ctx.needs_input_grad[2] or ctx.needs_input_grad[3]
        teacher = ctx.needs_input_grad[0] or ctx.needs_input_grad[1]
        if not (student or teacher):
            return (None,) * 6
        g = gKL.float().contiguous()
        # the joint pass where the single-setting backward is the fused kernel; for at most 16 query
        # rows per key head the two key-split passes stream the keys far faster
        if student and teacher and bwd_plan(Q1, K1, 1, causal=ctx.causal).path == PATH_BWD_FUSED:
            dQ1, dK1, dQ2, dK2 = kl_bwd_joint(g, Q1, K1, Q2, K2, KL, L1, L2, causal=ctx.causal, scale=ctx.scale,
                                              grad_dtype=torch.bfloat16)
            return dQ1, dK1, dQ2, dK2, None, None
        grads = [None] * 6
        for setting, want, slot in ((1, student, 2), (2, teacher, 0)):
            if want:
                dQ, dK = kl_bwd(setting, g, Q1, K1, Q2, K2, KL, L1, L2, causal=ctx.causal, scale=ctx.scale,
                                grad_dtype=torch.bfloat16)
                grads[slot], grads[slot + 1] = dQ, dK
        return tuple(grads)


# ---------------------------------------------------------------------------
# Divergence of attentions with modified scores
# ---------------------------------------------------------------------------
# Calls whose arguments passed every check, by what the checks look at (shapes,
# strides, types, devices, and options as plain numbers -- never the tensors, their
# values or addresses): the structs and sizes they led to.  Checking again and
# planning cost more host time than a small call's kernels.
_known = {}


def _tensors(*tensors):
    """What the checks look at of each tensor; None where something is no strided tensor, for them to refuse."""
    try:
        return tuple([None if t is None else (t.shape, t.stride(), t.dtype, t.device) for t in tensors])
    except (AttributeError, RuntimeError):
        return None


def _remember(key, entry):
    if key[1] is None:  # nothing to know the call by
        return entry
    with _lock:
        while len(_known) >= 512:
            del _known[next(iter(_known))]  # the oldest
        _known[key] = entry
    return entry


def _lookup(*key):
    try:
        return key, _known.get(key)
    except TypeError:  # an argument that is not hashable is none that passes the checks
        return key, None


# the current stream's handle without a Stream object (2 us on the GPU's host CPU)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _on(device, function, *args):
    """function(*args, current stream of device) with the device current."""
    if torch.cuda.current_device() == device.index:
        return function(*args, _raw_stream(device.index))
    with torch.cuda.device(device):
        return function(*args, torch.cuda.current_stream(device).cuda_stream)


def _guard_capture(*inputs):
    """Refuse to record a graph in a CUDA-graph capture on leaves (or views of leaves) that a still living graph made on
    the default stream uses: the leaves' gradient accumulators belong to that stream, which cannot be captured, and
    running them inside the capture breaks it (at worst the process ends).  An accumulator of any other stream, a
    warm-up's, joins the capture.  Calls mark the accumulators with the stream they found current; the marks die with
    the graphs."""
    for t in inputs:
        if isinstance(t, torch.Tensor) and t.is_cuda and t.requires_grad:
            leaf = t if t.grad_fn is None else t._base
            if leaf is None or leaf.grad_fn is not None or not leaf.requires_grad:
                continue
            made_on = torch.autograd.graph.get_gradient_edge(leaf).node.metadata.setdefault(
                "streamkl stream", _raw_stream(t.device.index))
            if made_on == 0 and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("an autograd graph of these leaves, made on the default stream, is still alive: drop it "
                                   "(or make it on a stream of its own) before the capture")


def _address(t):
    return None if t is None else t.data_ptr()


def _scratch(workspace, nbytes, device):
    """A caller's workspace, checked, or a new one.  A new one is not cleared: its error word is never read (the score
    kernels mark with NaN what a give-up leaves undone; the norm's wait for nothing)."""
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    return _check_workspace(workspace, nbytes, device)


class Scores:
    """How the raw products q.k of the teacher (1) and the student (2) become scores, and which keys each row sees:

        S_t = cap_t tanh(scale q.k / cap_t) - slopes_t[h] |i + offset[b] - j|,   begin[b, i] <= j < end[b, i]

    cap 0: no cap; slopes (float32 [H]), begin / end (int32 [B, Nq]) and offset (int32 [B], the key position of
    row 0) may be None: no bias, every key, Nk - Nq.  key_ranges makes begin, end and offset from masks."""

    __slots__ = ("cap1", "cap2", "slopes1", "slopes2", "begin", "end", "offset")

    def __init__(self, cap1=0.0, cap2=0.0, slopes1=None, slopes2=None, begin=None, end=None, offset=None):
        self.cap1, self.cap2 = float(cap1), float(cap2)
        self.slopes1, self.slopes2, self.begin, self.end, self.offset = slopes1, slopes2, begin, end, offset

    def tensors(self):
        return self.slopes1, self.slopes2, self.begin, self.end, self.offset

    def check(self, Q1):
        B, H, Nq, _ = Q1.shape
        for name, shape, dtype in (("slopes1", (H,), torch.float32), ("slopes2", (H,), torch.float32),
                                   ("begin", (B, Nq), torch.int32), ("end", (B, Nq), torch.int32),
                                   ("offset", (B,), torch.int32)):
            t = getattr(self, name)
            if t is not None:
                _check_tensor(name, t, shape, dtype, Q1.device)


def key_ranges(B, Nq, Nk, device, causal=True, window=0, prefix=None, docs=None, q_lengths=None, k_lengths=None):
    """(begin, end, offset) of Scores from masks.  Row i of batch b stands at key position p = i + offset[b], with
    offset = k_lengths - q_lengths (int32 [B]; None: Nk, Nq); rows behind q_lengths see nothing.  It sees the keys below
    k_lengths with j <= p (causal), p - window < j < p + window (window > 0), any j < prefix[b] (int32 [B], not with
    window or docs), and of p's document alone (docs: nondecreasing int32 bounds, [M] for every batch or [B, M]; document
    m is docs[m] <= j < docs[m + 1])."""
    B, Nq, Nk, window = int(B), int(Nq), int(Nk), int(window)
    for name, v in (("B", B), ("Nq", Nq), ("Nk", Nk), ("window", window)):
        if not -2 ** 31 <= v < 2 ** 31:
            raise ValueError(f"{name} must fit 32 bits, got {v}")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("device must be a CUDA device")
    with torch.cuda.device(device):
        device = torch.device("cuda", torch.cuda.current_device())
        for name, t in (("prefix", prefix), ("q_lengths", q_lengths), ("k_lengths", k_lengths)):
            if t is not None:
                _check_tensor(name, t, (B,), torch.int32, device)
        bounds = per_batch = 0
        if docs is not None:
            if not isinstance(docs, torch.Tensor) or docs.dim() not in (1, 2):
                raise ValueError("docs must be an int32 tensor [M] or [B, M]")
            bounds, per_batch = docs.shape[-1], int(docs.dim() == 2)
            _check_tensor("docs", docs, (B, bounds) if per_batch else (bounds,), torch.int32, device)
        begin, end = (torch.empty((B, Nq), dtype=torch.int32, device=device) for _ in range(2))
        offset = torch.empty((B,), dtype=torch.int32, device=device)
        _raise(load().streamkl_key_ranges(B, Nq, Nk, int(bool(causal)), window, _ptr(q_lengths), _ptr(k_lengths),
                                          _ptr(prefix), _ptr(docs), bounds, per_batch, _ptr(begin), _ptr(end),
                                          _ptr(offset), _stream(device)), "streamkl_key_ranges")
    return begin, end, offset


def _scores(scores):
    if not isinstance(scores, Scores):
        raise ValueError("scores must be a Scores")
    return scores


def score_fwd_plan(Q1, K1, num_splits=0) -> Plan:
    plan = Plan()
    with torch.cuda.device(Q1.device):
        _raise(load().streamkl_score_fwd_plan(ctypes.byref(make_shape(Q1, K1)), ctypes.byref(_opts(num_splits)),
                                              ctypes.byref(plan)), "streamkl_score_fwd_plan")
    return plan


def score_bwd_plan(Q1, K1, setting, grad_dtype=torch.float32, num_splits=0) -> Plan:
    plan = Plan()
    with torch.cuda.device(Q1.device):
        _raise(load().streamkl_score_bwd_plan(ctypes.byref(make_shape(Q1, K1)), int(setting),
                                              ctypes.byref(_opts(num_splits, grad_bf16=_grad_flag(grad_dtype))),
                                              ctypes.byref(plan)), "streamkl_score_bwd_plan")
    return plan


def kl_score_fwd(scores, Q1, K1, Q2, K2, causal=False, scale=None, num_splits=0, workspace=None, out=None,
                 wait_limit_ns=0, debug_flags=0):
    """Per-row KL(P1 || P2), LSE1, LSE2 as float32 [B, H, Nq] for the scores that ``scores`` describes.  A row that
    sees no key has KL = 0 and LSE = -inf; what a row does not see (NaN included) has no effect on it.  Rows that a
    give-up of a bounded wait left unfinished are NaN."""
    given = _scores(scores).tensors()
    num_splits, wait_limit_ns, debug_flags = int(num_splits), int(wait_limit_ns), int(debug_flags)
    key, known = _lookup("score_fwd", _tensors(Q1, K1, Q2, K2, *given), num_splits, wait_limit_ns, debug_flags)
    if known is None:
        _check_qk(Q1, K1, Q2, K2)
        scores.check(Q1)
        shape, opts, plan = make_shape(Q1, K1), _opts(num_splits, 0, wait_limit_ns, debug_flags), Plan()
        with torch.cuda.device(Q1.device):
            _raise(load().streamkl_score_fwd_plan(ctypes.byref(shape), ctypes.byref(opts), ctypes.byref(plan)),
                   "streamkl_score_fwd_plan")
        known = _remember(key, (shape, opts, plan.workspace_bytes, tuple(Q1.shape[:3]), Q1.device))
    shape, opts, nbytes, rows, device = known
    if out is None:
        out = tuple([torch.empty(rows, dtype=torch.float32, device=device) for _ in range(3)])
    else:
        for name, t in zip(("KL", "LSE1", "LSE2"), out):
            _check_tensor(name, t, rows, torch.float32, device)
    workspace = _scratch(workspace, nbytes, device)
    KL, L1, L2 = out
    score = Score(scores.cap1, scores.cap2, *[_address(t) for t in given])
    _raise(_on(device, load().streamkl_score_fwd, shape, score, Q1.data_ptr(), K1.data_ptr(), Q2.data_ptr(), K2.data_ptr(),
               0.0 if scale is None else float(scale), 1 if causal else 0, KL.data_ptr(), L1.data_ptr(), L2.data_ptr(),
               workspace.data_ptr(), workspace.numel(), opts), "streamkl_score_fwd")
    return KL, L1, L2


def kl_score_bwd(setting, scores, g, Q1, K1, Q2, K2, KL, LSE1, LSE2, causal=False, scale=None, workspace=None, out=None,
                 wait_limit_ns=0, debug_flags=0, grad_dtype=torch.float32, num_splits=0):
    """(dQ, dK) of the trainable side of kl_score_fwd: setting 1 -> (Q2, K2), 2 -> (Q1, K1), as kl_bwd.  dQ is added
    up in float32 in no fixed order (like kl_bwd's fused mode); dK is the same on every run.  bf16 gradients are the
    float32 ones, rounded once.  num_splits: CTAs that share a key tile's query rows (0 = automatic).  Rows of either
    gradient that a give-up of a bounded wait left without some of their terms are NaN."""
    given = _scores(scores).tensors()
    setting, num_splits, wait_limit_ns, debug_flags = int(setting), int(num_splits), int(wait_limit_ns), int(debug_flags)
    key, known = _lookup("score_bwd", _tensors(Q1, K1, Q2, K2, g, KL, LSE1, LSE2, *given), setting, grad_dtype, wait_limit_ns,
                         debug_flags, num_splits)
    if known is None:
        _check_qk(Q1, K1, Q2, K2)
        scores.check(Q1)
        shape, plan = make_shape(Q1, K1), Plan()
        opts = _opts(num_splits, 0, wait_limit_ns, debug_flags, _grad_flag(grad_dtype))
        with torch.cuda.device(Q1.device):
            _raise(load().streamkl_score_bwd_plan(ctypes.byref(shape), setting, ctypes.byref(opts), ctypes.byref(plan)),
                   "streamkl_score_bwd_plan")
        for name, t in (("g", g), ("KL", KL), ("LSE1", LSE1), ("LSE2", LSE2)):
            _check_tensor(name, t, Q1.shape[:3], torch.float32, Q1.device)
        known = _remember(key, (shape, opts, plan.workspace_bytes, tuple(Q1.shape), tuple(K1.shape), Q1.device))
    shape, opts, nbytes, q_shape, k_shape, device = known
    if out is None:
        out = (torch.empty(q_shape, dtype=grad_dtype, device=device), torch.empty(k_shape, dtype=grad_dtype, device=device))
    else:
        _check_tensor("dQ", out[0], q_shape, grad_dtype, device)
        _check_tensor("dK", out[1], k_shape, grad_dtype, device)
    workspace = _scratch(workspace, nbytes, device)
    dQ, dK = out
    score = Score(scores.cap1, scores.cap2, *[_address(t) for t in given])
    _raise(_on(device, load().streamkl_score_bwd, shape, score, setting, g.data_ptr(), Q1.data_ptr(), K1.data_ptr(),
               Q2.data_ptr(), K2.data_ptr(), KL.data_ptr(), LSE1.data_ptr(), LSE2.data_ptr(),
               0.0 if scale is None else float(scale), 1 if causal else 0, dQ.data_ptr(), dK.data_ptr(),
               workspace.data_ptr(), workspace.numel(), opts), "streamkl_score_bwd")
    return dQ, dK


class ScoredAttentionKL(torch.autograd.Function):
    """Per-row divergence of kl_score_fwd with gradients to whichever sides' Q and K require them (AttentionKL's
    settings), in bf16 like the inputs.  ``scores`` describes constants: slopes get no gradient."""

    @staticmethod
    def forward(ctx, Q1, K1, Q2, K2, scores, causal=False, scale=None):
        if any(t is not None and t.requires_grad for t in _scores(scores).tensors()):
            raise ValueError("the tensors of scores are constants: they get no gradient")
        _guard_capture(Q1, K1, Q2, K2)
        causal, scale = bool(causal), None if scale is None else float(scale)  # the backward's are the forward's
        KL, L1, L2 = kl_score_fwd(scores, Q1, K1, Q2, K2, causal=causal, scale=scale)
        ctx.save_for_backward(Q1, K1, Q2, K2, KL, L1, L2, *scores.tensors())
        ctx.caps, ctx.causal, ctx.scale = (scores.cap1, scores.cap2), causal, scale
        return KL

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, gKL):
        Q1, K1, Q2, K2, KL, L1, L2, *given = ctx.saved_tensors
        scores = Scores(*ctx.caps, *given)
        g = gKL.float().contiguous()
        grads = [None] * 7
        for setting, slot in ((1, 2), (2, 0)):
            if ctx.needs_input_grad[slot] or ctx.needs_input_grad[slot + 1]:
                grads[slot], grads[slot + 1] = kl_score_bwd(setting, scores, g, Q1, K1, Q2, K2, KL, L1, L2,
                                                            causal=ctx.causal, scale=ctx.scale,
                                                            grad_dtype=torch.bfloat16)
        return tuple(grads)


# ---------------------------------------------------------------------------
# Norm of query and key heads with the position rotation
# ---------------------------------------------------------------------------
def rope_table(rows, rot, device, base=10000.0, inv_freq=None) -> torch.Tensor:
    """Cosines and sines of the positions below ``rows`` as float32 [rows, rot/2, 2],
    from angles in float64.  inv_freq (rot/2 values) replaces base^(-2e/rot), for
    scaled frequencies.  Made once and kept.  Frequencies from the host (the default's
    too) are copied to the device first, which waits for the current stream and cannot
    be captured; a float64 tensor on the device is read as it is."""
    rot, rows = int(rot), int(rows)
    if rot < 8 or rot % 8 or rot > 128 or rows < 1:
        raise ValueError(f"rot must be a multiple of 8 up to 128 and rows at least 1, got {rot} and {rows}")
    if inv_freq is None:
        inv_freq = [float(base) ** (-2.0 * e / rot) for e in range(rot // 2)]
    freq = torch.as_tensor(inv_freq, dtype=torch.float64).to(device).contiguous()
    if freq.numel() != rot // 2 or not freq.is_cuda:
        raise ValueError(f"inv_freq must hold rot/2 = {rot // 2} values and device must be a CUDA device")
    with torch.cuda.device(freq.device):
        table = torch.empty((rows, rot // 2, 2), dtype=torch.float32, device=freq.device)
        _raise(load().streamkl_rope_table(_ptr(freq), rows, rot // 2, _ptr(table), _stream(freq.device)),
               "streamkl_rope_table")
    return table


def _heads(name, t, dtypes, device=None, shape=None):
    """A [B, H, N, d] tensor that the kernels read or write through its strides."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a CUDA tensor{'' if device is None else f' on {device}'}")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if t.dim() != 4 or (shape is not None and tuple(t.shape) != tuple(shape)):
        raise ValueError(f"{name} must be [B, H, N, d]{'' if shape is None else f' = {tuple(shape)}'}, got {tuple(t.shape)}")
    if t.stride(3) != 1 and t.shape[3] > 1:
        raise ValueError(f"{name} must have d contiguous")
    # the stride of an axis with one entry is never used
    return Strides(*[t.stride(k) if t.shape[k] > 1 else 0 for k in range(3)])


def _contiguous(shape) -> Strides:
    _, H, N, d = shape
    return Strides(H * max(N, 1) * d, max(N, 1) * d, d)


def _norm_rope_desc(q, k, wq, wk, table, positions, eps, interleaved):
    desc = NormRope()
    desc.q, desc.k = _heads("q", q, (torch.bfloat16,)), _heads("k", k, (torch.bfloat16,), q.device)
    B, Hq, N, d = q.shape
    if k.shape[0] != B or k.shape[2] != N or k.shape[3] != d:
        raise ValueError("q and k must share B, N and d")
    if d not in (64, 128):
        raise ValueError(f"d must be 64 or 128, got {d}")
    types = {w.dtype for w in (wq, wk) if w is not None}
    if len(types) > 1 or not types <= {torch.float32, torch.bfloat16}:
        raise ValueError("wq and wk must both be float32 or both bf16")
    for name, w in (("wq", wq), ("wk", wk)):
        if w is not None:
            _check_tensor(name, w, (d,), w.dtype, q.device)
    rot = 0
    if table is not None:
        if not isinstance(table, torch.Tensor) or table.dim() != 3:
            raise ValueError("table must be [rows, rot/2, 2] (see rope_table)")
        rot = 2 * table.shape[1]
        _check_tensor("table", table, (table.shape[0], rot // 2, 2), torch.float32, q.device)
        if rot > d or rot % 8 or rot == 0 or table.shape[0] == 0:
            raise ValueError(f"the table rotates {rot} values by {table.shape[0]} positions: rot must be a multiple of 8 up to d = {d}")
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or positions.dtype not in (torch.int32, torch.int64):
            raise ValueError("positions must be an int32 or int64 tensor")
        _check_tensor("positions", positions, (B, N), positions.dtype, q.device)
    desc.B, desc.Hq, desc.Hk, desc.N, desc.d, desc.rot = B, Hq, k.shape[1], N, d, rot
    desc.interleaved, desc.eps = int(interleaved), eps
    desc.weight_bf16 = int(torch.bfloat16 in types)
    desc.pos_int64 = int(positions is not None and positions.dtype == torch.int64)
    desc.table_rows = table.shape[0] if table is not None else 0
    return desc


def _plain(start, eps, interleaved):
    """Plain numbers, read now: a program may hand in a tensor or an array and change it in place."""
    start = int(start)
    if not -2 ** 63 <= start < 2 ** 63:
        raise ValueError(f"start must fit 64 bits, got {start}")
    return start, float(eps), bool(interleaved)


def _at(desc, start):
    """The description of a known call (whose start is 0: no check looks at it) from position ``start``."""
    if start:
        desc = NormRope.from_buffer_copy(desc)  # another thread may be using the known one
        desc.start = start
    return desc


def qk_norm_rope(q, k, wq=None, wk=None, table=None, positions=None, start=0, eps=1e-6, interleaved=False, out=None):
    """(q', k'): every head of q [B, Hq, N, d] and k [B, Hk, N, d] (bf16, any strides with d contiguous) divided by
    its root mean square, times wq / wk ([d], float32 or bf16; None: ones), its first 2 * table.shape[1] values turned
    by the angles of its position (positions [B, N], else start + n; table from rope_table; None: no rotation).  out: two
    bf16 tensors of the same shapes, any strides (rows of a cache, or q and k themselves); new contiguous ones otherwise."""
    start, eps, interleaved = _plain(start, eps, interleaved)
    key, known = _lookup("norm_rope", _tensors(q, k, wq, wk, table, positions, *(out or ())), eps, interleaved)
    if known is None:
        desc = _norm_rope_desc(q, k, wq, wk, table, positions, eps, interleaved)
        if out is not None:
            desc.yq = _heads("out[0]", out[0], (torch.bfloat16,), q.device, q.shape)
            desc.yk = _heads("out[1]", out[1], (torch.bfloat16,), q.device, k.shape)
        else:
            desc.yq, desc.yk = _contiguous(q.shape), _contiguous(k.shape)
        known = _remember(key, (desc, tuple(q.shape), tuple(k.shape), q.device))
    desc, q_shape, k_shape, device = known
    if out is None:
        out = (torch.empty(q_shape, dtype=torch.bfloat16, device=device),
               torch.empty(k_shape, dtype=torch.bfloat16, device=device))
    yq, yk = out
    _raise(_on(device, load().streamkl_norm_rope_fwd, _at(desc, start), q.data_ptr(), k.data_ptr(), _address(wq),
               _address(wk), _address(table), _address(positions), yq.data_ptr(), yk.data_ptr()), "streamkl_norm_rope_fwd")
    return yq, yk


def qk_norm_rope_bwd(dyq, dyk, q, k, wq=None, wk=None, table=None, positions=None, start=0, eps=1e-6,
                     interleaved=False, workspace=None, out=None):
    """(dq, dk, dwq, dwk) of sum(dyq q') + sum(dyk k') for qk_norm_rope's arguments; dyq, dyk are both bf16 or both
    float32 (kl_bwd's gradients as they come), any strides with d contiguous.  dq, dk are bf16, dwq, dwk of the weights'
    type (None without weights).  out: (dq, dk) to write into.  Equal inputs give equal bits."""
    start, eps, interleaved = _plain(start, eps, interleaved)
    key, known = _lookup("norm_rope_bwd", _tensors(dyq, dyk, q, k, wq, wk, table, positions, *(out or ())), eps, interleaved)
    if known is None:
        desc = _norm_rope_desc(q, k, wq, wk, table, positions, eps, interleaved)
        desc.yq = _heads("dyq", dyq, (torch.bfloat16, torch.float32), q.device, q.shape)
        desc.yk = _heads("dyk", dyk, (dyq.dtype,), q.device, k.shape)
        desc.grad_bf16 = int(dyq.dtype == torch.bfloat16)
        if out is not None:
            desc.dq = _heads("out[0]", out[0], (torch.bfloat16,), q.device, q.shape)
            desc.dk = _heads("out[1]", out[1], (torch.bfloat16,), q.device, k.shape)
        else:
            desc.dq, desc.dk = _contiguous(q.shape), _contiguous(k.shape)
        with torch.cuda.device(q.device):
            nbytes = max(int(load().streamkl_norm_rope_workspace_bytes(ctypes.byref(desc))), 256)
        known = _remember(key, (desc, nbytes, tuple(q.shape), tuple(k.shape), q.device))
    desc, nbytes, q_shape, k_shape, device = known
    if out is None:
        out = (torch.empty(q_shape, dtype=torch.bfloat16, device=device),
               torch.empty(k_shape, dtype=torch.bfloat16, device=device))
    dq, dk = out
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (wq, wk))
    workspace = _scratch(workspace, nbytes, device)
    _raise(_on(device, load().streamkl_norm_rope_bwd, _at(desc, start), dyq.data_ptr(), dyk.data_ptr(), q.data_ptr(),
               k.data_ptr(), _address(wq), _address(wk), _address(table), _address(positions), dq.data_ptr(), dk.data_ptr(),
               _address(dwq), _address(dwk), workspace.data_ptr(), workspace.numel()), "streamkl_norm_rope_bwd")
    return dq, dk, dwq, dwk


class QKNormRope(torch.autograd.Function):
    """(q', k') of qk_norm_rope with gradients to q, k, wq and wk.  Saves its
    inputs and recomputes the norms in the backward."""

    @staticmethod
    def forward(ctx, q, k, wq=None, wk=None, table=None, positions=None, start=0, eps=1e-6, interleaved=False):
        _guard_capture(q, k, wq, wk)
        ctx.save_for_backward(q, k, wq, wk, table, positions)
        ctx.how = dict(zip(("start", "eps", "interleaved"), _plain(start, eps, interleaved)))
        return qk_norm_rope(q, k, wq, wk, table, positions, **ctx.how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, table, positions = ctx.saved_tensors
        dyq, dyk = (torch.zeros_like(x, memory_format=torch.contiguous_format) if g is None else g.contiguous()
                    for g, x in ((dyq, q), (dyk, k)))
        grads = qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, table, positions, **ctx.how)
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None, None, None, None)
