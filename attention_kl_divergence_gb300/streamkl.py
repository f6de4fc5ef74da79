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

and ``QKNormRope``, its autograd Function; with positions on several axes (time, height, width) and
``axes=rope_axes(sections)`` each pair turns by the position on an axis of its own.  The attention itself, over
whole prompts and with gradients:

    attn_fwd(Q, K, V, ranges=key_ranges(...)) -> (O, LSE)
    attn_fwd(Q, K, V, ranges, rest=True) -> (O, LSE, rest)
    attn_bwd(dO, Q, K, V, O, LSE, rest=rest, ranges=ranges) -> (dQ, dK, dV)

and ``Attention``, its autograd Function.  For serving, a paged cache of keys and values in 8 bits and the attention of a
few new tokens over it:

    cache = Cache8.empty(pages, heads, tokens, d, device)
    cache8_append(cache, table, lengths, k, v, counts=None)
    attn_cache8(Q, cache, table, lengths) -> (O, LSE)
    cache8_read(cache, table, lengths) -> (K, V)

There is no fallback: without the compiled library
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


class RopeAxes(ctypes.Structure):
    _fields_ = [("axes", ctypes.c_int32), ("axis_of", ctypes.c_uint8 * 64)]


class Attn(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "H", "H_kv", "Nq", "Nk", "d")] + \
        [(n, Strides) for n in ("q", "k", "v", "o", "d_o")]


class CacheDesc(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("pages", "H_kv", "T", "d", "B", "M", "H", "N")] + \
        [(n, Strides) for n in ("x", "y")]


class StreamKLError(RuntimeError):
    def __init__(self, code, where):
        self.code = code
        super().__init__(f"{where}: {status_string(code)} (status {code})")


EXPORTED = ("streamkl_fwd_plan", "streamkl_fwd", "streamkl_bwd_plan", "streamkl_bwd", "streamkl_workspace_status",
            "streamkl_status_string", "streamkl_version", "streamkl_fwd_noalloc", "streamkl_noalloc_status",
            "streamkl_fwd_workspace_bytes", "streamkl_bwd_workspace_bytes", "streamkl_bwd_joint_plan",
            "streamkl_bwd_joint", "streamkl_norm_rope_fwd", "streamkl_norm_rope_bwd",
            "streamkl_norm_rope_workspace_bytes", "streamkl_rope_table", "streamkl_score_fwd_plan", "streamkl_score_fwd",
            "streamkl_score_bwd_plan", "streamkl_score_bwd", "streamkl_key_ranges", "streamkl_attn_fwd_plan",
            "streamkl_attn_fwd", "streamkl_attn_bwd_plan", "streamkl_attn_bwd",
            "streamkl_norm_rope_axes_fwd", "streamkl_norm_rope_axes_bwd", "streamkl_cache8_append", "streamkl_cache8_read",
            "streamkl_attn_cache8_plan", "streamkl_attn_cache8")

_lock = threading.Lock()
_lib = None


def library_path() -> str:
    return _build.LIB


def load(build_if_stale: bool = True):
    """Load libstreamkl.so (building it first when sources are newer)."""
    global _lib
    if _lib is not None:  # set once, complete
        return _lib
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
        ra = ctypes.POINTER(RopeAxes)
        lib.streamkl_norm_rope_axes_fwd.argtypes = [nr, ra, *[P] * 9]
        lib.streamkl_norm_rope_axes_bwd.argtypes = [nr, ra, *[P] * 13, Z, P]
        at = ctypes.POINTER(Attn)
        lib.streamkl_attn_fwd_plan.argtypes = [at, op, pp]
        lib.streamkl_attn_fwd.argtypes = [at, *[P] * 6, F, I, P, P, P, P, Z, op, P]
        lib.streamkl_attn_bwd_plan.argtypes = [at, op, pp]
        lib.streamkl_attn_bwd.argtypes = [at, *[P] * 10, F, I, P, P, P, P, Z, op, P]
        cd = ctypes.POINTER(CacheDesc)
        lib.streamkl_cache8_append.argtypes = [cd, *[P] * 10]
        lib.streamkl_cache8_read.argtypes = [cd, *[P] * 9]
        lib.streamkl_attn_cache8_plan.argtypes = [cd, op, pp]
        lib.streamkl_attn_cache8.argtypes = [cd, *[P] * 7, F, P, P, P, Z, op, P]
        lib.streamkl_status_string.argtypes = [I]
        lib.streamkl_status_string.restype = ctypes.c_char_p
        for name in ("streamkl_fwd_plan", "streamkl_fwd", "streamkl_bwd_plan", "streamkl_bwd",
                     "streamkl_workspace_status", "streamkl_version", "streamkl_fwd_noalloc",
                     "streamkl_noalloc_status", "streamkl_bwd_joint_plan", "streamkl_bwd_joint",
                     "streamkl_norm_rope_fwd", "streamkl_norm_rope_bwd", "streamkl_rope_table",
                     "streamkl_score_fwd_plan", "streamkl_score_fwd", "streamkl_score_bwd_plan", "streamkl_score_bwd",
                     "streamkl_key_ranges", "streamkl_attn_fwd_plan", "streamkl_attn_fwd", "streamkl_attn_bwd_plan", "streamkl_attn_bwd",
                     "streamkl_norm_rope_axes_fwd", "streamkl_norm_rope_axes_bwd", "streamkl_cache8_append",
                     "streamkl_cache8_read", "streamkl_attn_cache8_plan", "streamkl_attn_cache8"):
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


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _on(device, function, *args):
    """function(*args, current stream of device) with the device current."""
    if _current_device() == device.index:
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


def _own_scratch(workspace, nbytes, device):
    """(address, bytes, tensor to keep until the call returns) for calls that need none where nothing but the error word
    would stand there."""
    if workspace is None and nbytes <= 256:
        return None, 0, None
    workspace = _scratch(workspace, nbytes, device)
    return workspace.data_ptr(), workspace.numel(), workspace


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


def rope_axes(sections, spread=False) -> tuple:
    """The axis that turns each pair, for qk_norm_rope's axes: sections[a] pairs of axis a, one axis after the other, or
    (spread) the axes in turn, each as long as it has pairs left."""
    left = [int(n) for n in sections]
    if not left or any(n < 0 for n in left):
        raise ValueError(f"sections must be numbers of pairs, got {tuple(sections)}")
    if not spread:
        return tuple([a for a, n in enumerate(left) for _ in range(n)])
    return tuple([a for k in range(max(left)) for a, n in enumerate(left) if k < n])


def _axes(axes, table, positions):
    """None or (struct, number of axes); axes is a tuple of whole numbers."""
    if axes is None:
        return None
    if not isinstance(positions, torch.Tensor) or positions.dim() != 3 or not 1 <= positions.shape[0] <= 4:
        raise ValueError("positions on several axes must be [axes, B, N], up to 4 axes")
    if not isinstance(table, torch.Tensor) or table.dim() != 3 or len(axes) != table.shape[1]:
        raise ValueError("axes must name the axis of each of the table's pairs (see rope_axes)")
    if any(not 0 <= a < positions.shape[0] for a in axes):
        raise ValueError(f"axes must be below {positions.shape[0]}, the axes of positions")
    out = RopeAxes(positions.shape[0])
    for e, a in enumerate(axes):
        out.axis_of[e] = a
    return out


def _norm_rope_desc(q, k, wq, wk, table, positions, eps, interleaved, axes=None):
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
        _check_tensor("positions", positions, (B, N) if axes is None else (positions.shape[0], B, N), positions.dtype, q.device)
    desc.B, desc.Hq, desc.Hk, desc.N, desc.d, desc.rot = B, Hq, k.shape[1], N, d, rot
    desc.interleaved, desc.eps = int(interleaved), eps
    desc.weight_bf16 = int(torch.bfloat16 in types)
    desc.pos_int64 = int(positions is not None and positions.dtype == torch.int64)
    desc.table_rows = table.shape[0] if table is not None else 0
    return desc


def _plain_axes(axes):
    """A tuple of whole numbers that no program can change."""
    if axes is None or (type(axes) is tuple and set(map(type, axes)) <= {int}):
        return axes
    return tuple([int(a) for a in axes])


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


def qk_norm_rope(q, k, wq=None, wk=None, table=None, positions=None, start=0, eps=1e-6, interleaved=False, out=None,
                 axes=None):
    """(q', k'): every head of q [B, Hq, N, d] and k [B, Hk, N, d] (bf16, any strides with d contiguous) divided by
    its root mean square, times wq / wk ([d], float32 or bf16; None: ones), its first 2 * table.shape[1] values turned
    by the angles of its position (positions [B, N], else start + n; table from rope_table; None: no rotation).  out: two
    bf16 tensors of the same shapes, any strides (rows of a cache, or q and k themselves); new contiguous ones otherwise.
    axes: several positions per token, positions [A, B, N] (time, height and width of a patch, say): pair e is turned by
    the position on axis axes[e] (see rope_axes)."""
    start, eps, interleaved = _plain(start, eps, interleaved)
    axes = _plain_axes(axes)
    key, known = _lookup("norm_rope", _tensors(q, k, wq, wk, table, positions, *(out or ())), eps, interleaved, axes)
    if known is None:
        more = _axes(axes, table, positions)
        desc = _norm_rope_desc(q, k, wq, wk, table, positions, eps, interleaved, axes)
        if out is not None:
            desc.yq = _heads("out[0]", out[0], (torch.bfloat16,), q.device, q.shape)
            desc.yk = _heads("out[1]", out[1], (torch.bfloat16,), q.device, k.shape)
        else:
            desc.yq, desc.yk = _contiguous(q.shape), _contiguous(k.shape)
        known = _remember(key, (desc, tuple(q.shape), tuple(k.shape), q.device, more))
    desc, q_shape, k_shape, device, more = known
    if out is None:
        out = (torch.empty(q_shape, dtype=torch.bfloat16, device=device),
               torch.empty(k_shape, dtype=torch.bfloat16, device=device))
    yq, yk = out
    args = (q.data_ptr(), k.data_ptr(), _address(wq), _address(wk), _address(table), _address(positions), yq.data_ptr(),
            yk.data_ptr())
    if more is None:
        _raise(_on(device, load().streamkl_norm_rope_fwd, _at(desc, start), *args), "streamkl_norm_rope_fwd")
    else:
        _raise(_on(device, load().streamkl_norm_rope_axes_fwd, desc, more, *args), "streamkl_norm_rope_axes_fwd")
    return yq, yk


def qk_norm_rope_bwd(dyq, dyk, q, k, wq=None, wk=None, table=None, positions=None, start=0, eps=1e-6,
                     interleaved=False, workspace=None, out=None, axes=None):
    """(dq, dk, dwq, dwk) of sum(dyq q') + sum(dyk k') for qk_norm_rope's arguments; dyq, dyk are both bf16 or both
    float32 (kl_bwd's gradients as they come), any strides with d contiguous.  dq, dk are bf16, dwq, dwk of the weights'
    type (None without weights).  out: (dq, dk) to write into.  Equal inputs give equal bits."""
    start, eps, interleaved = _plain(start, eps, interleaved)
    axes = _plain_axes(axes)
    key, known = _lookup("norm_rope_bwd", _tensors(dyq, dyk, q, k, wq, wk, table, positions, *(out or ())), eps, interleaved,
                         axes)
    if known is None:
        more = _axes(axes, table, positions)
        desc = _norm_rope_desc(q, k, wq, wk, table, positions, eps, interleaved, axes)
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
        known = _remember(key, (desc, nbytes, tuple(q.shape), tuple(k.shape), q.device, more))
    desc, nbytes, q_shape, k_shape, device, more = known
    if out is None:
        out = (torch.empty(q_shape, dtype=torch.bfloat16, device=device),
               torch.empty(k_shape, dtype=torch.bfloat16, device=device))
    dq, dk = out
    dwq, dwk = (None if w is None else torch.empty_like(w) for w in (wq, wk))
    workspace = _scratch(workspace, nbytes, device)
    args = (dyq.data_ptr(), dyk.data_ptr(), q.data_ptr(), k.data_ptr(), _address(wq), _address(wk), _address(table),
            _address(positions), dq.data_ptr(), dk.data_ptr(), _address(dwq), _address(dwk), workspace.data_ptr(),
            workspace.numel())
    if more is None:
        _raise(_on(device, load().streamkl_norm_rope_bwd, _at(desc, start), *args), "streamkl_norm_rope_bwd")
    else:
        _raise(_on(device, load().streamkl_norm_rope_axes_bwd, desc, more, *args), "streamkl_norm_rope_axes_bwd")
    return dq, dk, dwq, dwk


class QKNormRope(torch.autograd.Function):
    """(q', k') of qk_norm_rope with gradients to q, k, wq and wk.  Saves its
    inputs and recomputes the norms in the backward."""

    @staticmethod
    def forward(ctx, q, k, wq=None, wk=None, table=None, positions=None, start=0, eps=1e-6, interleaved=False, axes=None):
        _guard_capture(q, k, wq, wk)
        ctx.save_for_backward(q, k, wq, wk, table, positions)
        ctx.how = dict(zip(("start", "eps", "interleaved"), _plain(start, eps, interleaved)), axes=_plain_axes(axes))
        return qk_norm_rope(q, k, wq, wk, table, positions, **ctx.how)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dyq, dyk):
        q, k, wq, wk, table, positions = ctx.saved_tensors
        dyq, dyk = (torch.zeros_like(x, memory_format=torch.contiguous_format) if g is None else g.contiguous()
                    for g, x in ((dyq, q), (dyk, k)))
        grads = qk_norm_rope_bwd(dyq, dyk, q, k, wq, wk, table, positions, **ctx.how)
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None, None, None, None, None)


# ---------------------------------------------------------------------------
# Attention over whole prompts
# ---------------------------------------------------------------------------
def _attn_desc(Q, K, V):
    desc = Attn()
    desc.q = _heads("Q", Q, (torch.bfloat16,))
    desc.k, desc.v = _heads("K", K, (torch.bfloat16,), Q.device), _heads("V", V, (torch.bfloat16,), Q.device)
    B, H, Nq, d = Q.shape
    if K.shape != V.shape or K.shape[0] != B or K.shape[3] != d:
        raise ValueError("K and V must have one shape, and share B and d with Q")
    if K.shape[1] < 1 or H % K.shape[1] != 0:
        raise ValueError("the key head count must divide the query head count")
    desc.B, desc.H, desc.H_kv, desc.Nq, desc.Nk, desc.d = B, H, K.shape[1], Nq, K.shape[2], d
    return desc


def _ranges(ranges, Q):
    """(begin, end, offset) of key_ranges, checked; None: every key."""
    if ranges is None:
        return None, None, None
    if not isinstance(ranges, (tuple, list)) or len(ranges) != 3:
        raise ValueError("ranges must be (begin, end, offset) (see key_ranges)")
    B, _, Nq, _ = Q.shape
    for name, t, shape in zip(("begin", "end", "offset"), ranges, ((B, Nq), (B, Nq), (B,))):
        if t is not None:
            _check_tensor(name, t, shape, torch.int32, Q.device)
    return tuple(ranges)


def _given_ranges(ranges):
    if ranges is None:
        return None, None, None
    return tuple(ranges) if isinstance(ranges, (tuple, list)) else (ranges,)


def attn_fwd_plan(Q, K, V, num_splits=0) -> Plan:
    plan, desc = Plan(), _attn_desc(Q, K, V)
    desc.o = _contiguous(Q.shape)
    with torch.cuda.device(Q.device):
        _raise(load().streamkl_attn_fwd_plan(ctypes.byref(desc), ctypes.byref(_opts(num_splits)), ctypes.byref(plan)),
               "streamkl_attn_fwd_plan")
    return plan


def attn_fwd(Q, K, V, ranges=None, causal=False, scale=None, rest=False, out=None, num_splits=0, workspace=None,
             wait_limit_ns=0, debug_flags=0):
    """(O, LSE): softmax attention of Q [B, H, Nq, d] over K, V [B, Hk, Nk, d] (bf16, any strides with d contiguous; Hk
    divides H), O bf16 like Q, LSE float32 [B, H, Nq].  ranges: (begin, end, offset) of key_ranges (None: every key);
    causal: row i also sees no key behind i + offset (None: Nk - Nq).  A row that sees no key has O = 0 and LSE = -inf;
    what a row does not see (NaN included) has no effect on it.  out: a bf16 tensor for O, any strides; a new contiguous
    one otherwise.  rest=True returns (O, LSE, rest): rest, contiguous, is what O's rounding left; attn_bwd takes it."""
    given = _given_ranges(ranges)
    num_splits, wait_limit_ns, debug_flags, rest = int(num_splits), int(wait_limit_ns), int(debug_flags), bool(rest)
    key, known = _lookup("attn_fwd", _tensors(Q, K, V, *given, *(() if out is None else (out,))), num_splits, wait_limit_ns,
                         debug_flags, out is None)
    if known is None:
        desc = _attn_desc(Q, K, V)
        _ranges(ranges, Q)
        desc.o = _contiguous(Q.shape) if out is None else _heads("out", out, (torch.bfloat16,), Q.device, Q.shape)
        opts, plan = _opts(num_splits, 0, wait_limit_ns, debug_flags), Plan()
        with torch.cuda.device(Q.device):
            _raise(load().streamkl_attn_fwd_plan(ctypes.byref(desc), ctypes.byref(opts), ctypes.byref(plan)),
                   "streamkl_attn_fwd_plan")
        known = _remember(key, (desc, opts, plan.workspace_bytes, tuple(Q.shape), Q.device))
    desc, opts, nbytes, shape, device = known
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=device)
    left = torch.empty(shape, dtype=torch.bfloat16, device=device) if rest else None
    LSE = torch.empty(shape[:3], dtype=torch.float32, device=device)
    at, size, _keep = _own_scratch(workspace, nbytes, device)
    begin, end, offset = given
    _raise(_on(device, load().streamkl_attn_fwd, desc, Q.data_ptr(), K.data_ptr(), V.data_ptr(), _address(begin),
               _address(end), _address(offset), 0.0 if scale is None else float(scale), 1 if causal else 0, out.data_ptr(),
               _address(left), LSE.data_ptr(), at, size, opts), "streamkl_attn_fwd")
    return (out, LSE, left) if rest else (out, LSE)


def attn_bwd_plan(Q, K, V, num_splits=0) -> Plan:
    plan, desc = Plan(), _attn_desc(Q, K, V)
    desc.o = desc.d_o = _contiguous(Q.shape)
    with torch.cuda.device(Q.device):
        _raise(load().streamkl_attn_bwd_plan(ctypes.byref(desc), ctypes.byref(_opts(num_splits)), ctypes.byref(plan)),
               "streamkl_attn_bwd_plan")
    return plan


def attn_bwd(dO, Q, K, V, O, LSE, rest=None, ranges=None, causal=False, scale=None, out=None, num_splits=0,
             workspace=None, wait_limit_ns=0, debug_flags=0):
    """(dQ, dK, dV), bf16 and contiguous, of sum(dO O) for attn_fwd's arguments and outputs; dO and O are bf16 with any
    strides with d contiguous.  rest: attn_fwd's third output; without it the row sums of dO O carry O's rounding, which
    shows in dQ where a row's keys have much in common.  dK and dV sum over the query heads of a key head and are the
    same on every run; dQ is added up in float32 in no fixed order.  out: (dQ, dK, dV) to write into.  num_splits: CTAs
    that share a key tile's query rows (0 = automatic)."""
    given = _given_ranges(ranges)
    num_splits, wait_limit_ns, debug_flags = int(num_splits), int(wait_limit_ns), int(debug_flags)
    key, known = _lookup("attn_bwd", _tensors(dO, Q, K, V, O, LSE, rest, *given), num_splits, wait_limit_ns, debug_flags)
    if known is None:
        desc = _attn_desc(Q, K, V)
        _ranges(ranges, Q)
        desc.d_o = _heads("dO", dO, (torch.bfloat16,), Q.device, Q.shape)
        desc.o = _heads("O", O, (torch.bfloat16,), Q.device, Q.shape)
        _check_tensor("LSE", LSE, Q.shape[:3], torch.float32, Q.device)
        if rest is not None:
            _check_tensor("rest", rest, Q.shape, torch.bfloat16, Q.device)
        opts, plan = _opts(num_splits, 0, wait_limit_ns, debug_flags), Plan()
        with torch.cuda.device(Q.device):
            _raise(load().streamkl_attn_bwd_plan(ctypes.byref(desc), ctypes.byref(opts), ctypes.byref(plan)),
                   "streamkl_attn_bwd_plan")
        known = _remember(key, (desc, opts, plan.workspace_bytes, tuple(Q.shape), tuple(K.shape), Q.device))
    desc, opts, nbytes, q_shape, k_shape, device = known
    if out is None:
        out = tuple([torch.empty(s, dtype=torch.bfloat16, device=device) for s in (q_shape, k_shape, k_shape)])
    else:
        for name, t, s in zip(("dQ", "dK", "dV"), out, (q_shape, k_shape, k_shape)):
            _check_tensor(name, t, s, torch.bfloat16, device)
    dQ, dK, dV = out
    workspace = _scratch(workspace, nbytes, device)
    begin, end, offset = given
    _raise(_on(device, load().streamkl_attn_bwd, desc, dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
               _address(rest), LSE.data_ptr(), _address(begin), _address(end), _address(offset),
               0.0 if scale is None else float(scale), 1 if causal else 0, dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(),
               workspace.data_ptr(), workspace.numel(), opts), "streamkl_attn_bwd")
    return dQ, dK, dV


class Attention(torch.autograd.Function):
    """O of attn_fwd with gradients to Q, K and V, in bf16 like the inputs.  Saves its inputs, O, what O's rounding left
    and LSE, and recomputes the probabilities in the backward.  Where no input requires a gradient it is attn_fwd without
    rest, and saves nothing."""

    @staticmethod
    def forward(ctx, Q, K, V, ranges=None, causal=False, scale=None):
        _guard_capture(Q, K, V)
        causal, scale = bool(causal), None if scale is None else float(scale)  # the backward's are the forward's
        if not any(ctx.needs_input_grad[:3]):
            return attn_fwd(Q, K, V, ranges, causal, scale)[0]
        O, LSE, rest = attn_fwd(Q, K, V, ranges, causal, scale, rest=True)
        ctx.save_for_backward(Q, K, V, O, LSE, rest, *(ranges if ranges is not None else ()))
        ctx.how = dict(causal=causal, scale=scale)
        return O

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dO):
        Q, K, V, O, LSE, rest, *ranges = ctx.saved_tensors
        if dO.dtype != torch.bfloat16 or dO.stride(3) != 1 or any(s % 8 or s < dO.shape[3] for s in dO.stride()[:3]) or dO.data_ptr() % 16:
            dO = dO.to(torch.bfloat16).contiguous()  # a broadcast or oddly strided gradient
            dO = dO.clone() if dO.data_ptr() % 16 else dO
        grads = attn_bwd(dO, Q, K, V, O, LSE, rest, tuple(ranges) if ranges else None, **ctx.how)
        return (*(g if need else None for g, need in zip(grads, ctx.needs_input_grad)), None, None, None)


# ---------------------------------------------------------------------------
# A paged cache of keys and values in 8 bits, and attention over it
# ---------------------------------------------------------------------------
class Cache8:
    """k, v [pages, Hk, T, d] in float8_e4m3fn (or uint8, the same bytes) and k_scale, v_scale float32 [pages, Hk]: a
    stored value stands for itself times the scale of its page and head.  T is 16, 32, 64 or 128, d is 64 or 128.  Token
    j of sequence b stands in row j % T of page table[b, j // T], table int32 [B, M] being an argument of each call;
    a page may be listed by several sequences as long as none of them appends to it."""

    __slots__ = ("k", "v", "k_scale", "v_scale")

    def __init__(self, k, v, k_scale, v_scale):
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale

    @classmethod
    def empty(cls, pages, heads, tokens, d, device):
        """A cache of ``pages`` pages of ``tokens`` tokens, all zeros."""
        new = lambda: torch.zeros((int(pages), int(heads), int(tokens), int(d)), dtype=torch.uint8, device=device)  # noqa: E731
        one = lambda: torch.ones((int(pages), int(heads)), dtype=torch.float32, device=device)  # noqa: E731
        return cls(new().view(torch.float8_e4m3fn), new().view(torch.float8_e4m3fn), one(), one())

    def tensors(self):
        return self.k, self.v, self.k_scale, self.v_scale


def _cache(cache):
    if not isinstance(cache, Cache8):
        raise ValueError("cache must be a Cache8")
    return cache.tensors()


def _cache_desc(cache, table, lengths) -> CacheDesc:
    k, v, k_scale, v_scale = cache
    if not isinstance(k, torch.Tensor) or not k.is_cuda or k.dim() != 4:
        raise ValueError("the cache's k must be a CUDA tensor [pages, Hk, T, d]")
    if k.dtype not in (torch.float8_e4m3fn, torch.uint8):
        raise ValueError(f"the cache's k must be float8_e4m3fn or uint8, got {k.dtype}")
    _check_tensor("k", k, k.shape, k.dtype, k.device)
    _check_tensor("v", v, k.shape, k.dtype, k.device)
    _check_tensor("k_scale", k_scale, k.shape[:2], torch.float32, k.device)
    _check_tensor("v_scale", v_scale, k.shape[:2], torch.float32, k.device)
    if not isinstance(table, torch.Tensor) or table.dim() != 2:
        raise ValueError("table must be an int32 tensor [B, M]")
    _check_tensor("table", table, table.shape, torch.int32, k.device)
    _check_tensor("lengths", lengths, table.shape[:1], torch.int32, k.device)
    desc = CacheDesc()
    desc.pages, desc.H_kv, desc.T, desc.d = k.shape
    desc.B, desc.M = table.shape
    if desc.T not in (16, 32, 64, 128) or desc.d not in (64, 128):
        raise ValueError(f"pages hold 16, 32, 64 or 128 tokens of d = 64 or 128, not {desc.T} of {desc.d}")
    return desc


def cache8_append(cache, table, lengths, k, v, counts=None) -> None:
    """Write new tokens k, v [B, Hk, N, d] (bf16, any strides with d contiguous) into the cache behind the lengths (int32
    [B]) tokens that each sequence holds: counts[b] of them (int32 [B], clamped to N; None: N).  A page's scale is the
    smallest power of two 2^e, e >= -100, that brings every finite value within 448, and never shrinks while the page is
    being filled: tokens that it holds are rounded again where it grows.  NaN and infinities are stored as NaN.  Tokens
    behind the table, or of a page outside the cache, are not written.  lengths stay as they are (lengths + counts is for
    the caller to keep).  A page that a call appends to must be listed once, by one sequence."""
    held = _cache(cache)
    key, known = _lookup("cache8_append", _tensors(*held, table, lengths, k, v, counts))
    if known is None:
        desc = _cache_desc(held, table, lengths)
        desc.x, desc.y = _heads("k", k, (torch.bfloat16,), held[0].device), _heads("v", v, (torch.bfloat16,), held[0].device, k.shape)
        if tuple(k.shape[:2]) + (k.shape[3],) != (desc.B, desc.H_kv, desc.d):
            raise ValueError(f"k and v must be [B, Hk, N, d] = ({desc.B}, {desc.H_kv}, N, {desc.d}), got {tuple(k.shape)}")
        if counts is not None:
            _check_tensor("counts", counts, (desc.B,), torch.int32, held[0].device)
        desc.N = k.shape[2]
        known = _remember(key, (desc, held[0].device))
    desc, device = known
    _raise(_on(device, load().streamkl_cache8_append, desc, *[t.data_ptr() for t in held], table.data_ptr(),
               lengths.data_ptr(), k.data_ptr(), v.data_ptr(), _address(counts)), "streamkl_cache8_append")


def cache8_read(cache, table, lengths, tokens=None, out=None):
    """(K, V): the first ``tokens`` tokens (None: as many as the table's pages hold) of each sequence as bf16 [B, Hk, tokens,
    d], for attn_fwd over what a cache holds: zeros behind lengths[b], NaN for pages outside the cache.  Exact for scales
    that are powers of two.  out: two bf16 tensors of that shape, any strides; new contiguous ones otherwise."""
    held = _cache(cache)
    tokens = None if tokens is None else int(tokens)
    key, known = _lookup("cache8_read", _tensors(*held, table, lengths, *(out or ())), tokens)
    if known is None:
        desc = _cache_desc(held, table, lengths)
        desc.N = desc.M * desc.T if tokens is None else tokens
        if desc.N < 0:
            raise ValueError(f"tokens must not be negative, got {tokens}")
        shape, device = (desc.B, desc.H_kv, desc.N, desc.d), held[0].device
        if out is None:
            desc.x = desc.y = _contiguous(shape)
        else:
            desc.x = _heads("out[0]", out[0], (torch.bfloat16,), device, shape)
            desc.y = _heads("out[1]", out[1], (torch.bfloat16,), device, shape)
        known = _remember(key, (desc, shape, device))
    desc, shape, device = known
    if out is None:
        out = tuple([torch.empty(shape, dtype=torch.bfloat16, device=device) for _ in range(2)])
    _raise(_on(device, load().streamkl_cache8_read, desc, *[t.data_ptr() for t in held], table.data_ptr(),
               lengths.data_ptr(), out[0].data_ptr(), out[1].data_ptr()), "streamkl_cache8_read")
    return out


def _attn_cache8_desc(Q, held, table, lengths) -> CacheDesc:
    desc = _cache_desc(held, table, lengths)
    desc.x = _heads("Q", Q, (torch.bfloat16,), held[0].device)
    B, desc.H, desc.N, d = Q.shape
    if (B, d) != (desc.B, desc.d):
        raise ValueError(f"Q must be [B, H, Nq, d] with B = {desc.B} and d = {desc.d}, got {tuple(Q.shape)}")
    if desc.H_kv < 1 or desc.H % desc.H_kv != 0:
        raise ValueError("the cache's head count must divide the query head count")
    return desc


def attn_cache8_plan(Q, cache, table, lengths, num_splits=0) -> Plan:
    plan, desc = Plan(), _attn_cache8_desc(Q, _cache(cache), table, lengths)
    desc.y = _contiguous(Q.shape)
    with torch.cuda.device(Q.device):
        _raise(load().streamkl_attn_cache8_plan(ctypes.byref(desc), ctypes.byref(_opts(num_splits)), ctypes.byref(plan)),
               "streamkl_attn_cache8_plan")
    return plan


def attn_cache8(Q, cache, table, lengths, scale=None, out=None, num_splits=0, workspace=None, wait_limit_ns=0,
                debug_flags=0):
    """(O, LSE): softmax attention of the last Nq tokens (1 to 16) of each sequence, Q [B, H, Nq, d] (bf16, any strides with
    d contiguous), over the lengths[b] tokens that it holds in the cache, its own among them: row i sees the keys before
    lengths[b] - Nq + 1 + i.  Hk divides H.  A row that sees no key has O = 0 and LSE = -inf; a row that sees a page
    outside the cache, and a sequence longer than its table, is NaN.  Longer chunks: attn_fwd over cache8_read."""
    held = _cache(cache)
    num_splits, wait_limit_ns, debug_flags = int(num_splits), int(wait_limit_ns), int(debug_flags)
    key, known = _lookup("attn_cache8", _tensors(Q, *held, table, lengths, *(() if out is None else (out,))), num_splits,
                         wait_limit_ns, debug_flags)
    if known is None:
        desc = _attn_cache8_desc(Q, held, table, lengths)
        desc.y = _contiguous(Q.shape) if out is None else _heads("out", out, (torch.bfloat16,), Q.device, Q.shape)
        opts, plan = _opts(num_splits, 0, wait_limit_ns, debug_flags), Plan()
        with torch.cuda.device(Q.device):
            _raise(load().streamkl_attn_cache8_plan(ctypes.byref(desc), ctypes.byref(opts), ctypes.byref(plan)),
                   "streamkl_attn_cache8_plan")
        known = _remember(key, (desc, opts, plan.workspace_bytes, tuple(Q.shape), Q.device))
    desc, opts, nbytes, shape, device = known
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=device)
    LSE = torch.empty(shape[:3], dtype=torch.float32, device=device)
    at, size, _keep = _own_scratch(workspace, nbytes, device)
    _raise(_on(device, load().streamkl_attn_cache8, desc, Q.data_ptr(), *[t.data_ptr() for t in held], table.data_ptr(),
               lengths.data_ptr(), 0.0 if scale is None else float(scale), out.data_ptr(), LSE.data_ptr(), at, size, opts),
           "streamkl_attn_cache8")
    return out, LSE
