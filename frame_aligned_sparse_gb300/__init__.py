"""Frame-aligned sparse attention for GB300 (sm_103a): Python binding.

A thin ctypes layer over the C ABI in ``include/fas.h`` (``libfas.so``).  It
only marshals arguments: every step of the computation runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  If the library is
not built, every call raises: there is no CPU fallback.

The operation ("HeyGen x Google Cloud: Avatar IV on TPU", sections "Deleting
the Mask" and "Unchaining the Softmax"): queries of each video frame attend
to a window of neighbouring frames plus the global reference frame(s), in one
pass over frame-aligned full key blocks; eligible heads use a precomputed
Cauchy-Schwarz row bound instead of a running maximum.
"""
from __future__ import annotations

import ctypes
import dataclasses
import functools
import os
from typing import NamedTuple, Optional, Tuple

import numpy as np

__all__ = [
    "FasError", "PlanInfo", "MODES", "library_path", "load",
    "fas_plan", "fas_plan_describe", "fas_prepass", "fas_forward", "fas_free",
    "fas_status", "fas_prepass_readback", "fas_selftest_wait_timeout", "fas_selftest_row_wait_timeout",
    "fas_last_launch_count",
    "fas_prepass_noalloc", "fas_forward_host", "fas_set_layout", "LAYOUTS", "fas_forward_ablation",
    "fas_prologue", "fas_prologue_fold_weights", "PROLOGUE_LAYOUTS",
    "fas_prologue_with_key_sums", "fas_prepass_with_key_sums", "key_sums_shape",
    "fas_backward", "fas_residual_norm", "fas_residual_norm_backward", "Checkpoint", "fas_checkpoint_pack",
    "fas_checkpoint_unpack",
]

FAS_OK, FAS_ERR_ARG, FAS_ERR_STATE, FAS_ERR_ALIGN, FAS_ERR_CUDA, FAS_ERR_TIMEOUT, FAS_ERR_UNSUPPORTED = 0, -1, -2, -3, -4, -5, -6
FAS_ERR_SCRATCH = -7
FAS_ERR_BOUND = -8
FAS_NOALLOC_SCRATCH_BYTES = 4 << 20
MODES = {"auto": 0, "online": 1, "bounded": 2}
LAYOUTS = {"hnd": 0, "nhd": 1}  # q, k, v, out as [H, N, d] or [N, H, d]
PROLOGUE_LAYOUTS = {"hnd": 0, "nhd": 1, "a2a": 2}  # fas_prologue's outputs (a2a: [G, P, n, H/(G*P), d])
RMS_EPS = 1e-6
CHECKPOINT_BLOCK = 32  # elements of a checkpoint that share one scale
BACKWARD_WORKSPACE = 32  # FAS_BACKWARD_WORKSPACE: bytes a row and head

_HERE = os.path.dirname(os.path.abspath(__file__))


def library_path() -> str:
    return os.path.join(_HERE, "libfas.so")


class FasError(RuntimeError):
    def __init__(self, call: str, code: int, message: str):
        super().__init__(f"{call} failed: {message} (status {code})")
        self.code = code


class _PlanInfoC(ctypes.Structure):
    _fields_ = [
        ("block_k", ctypes.c_int32),
        ("q_tile", ctypes.c_int32),
        ("n_work", ctypes.c_int32),
        ("total_frames", ctypes.c_int32),
        ("tokens", ctypes.c_int64),
        ("key_blocks", ctypes.c_int64),
        ("visible_flops", ctypes.c_double),
        ("host_table", ctypes.POINTER(ctypes.c_int32)),
    ]


@dataclasses.dataclass
class PlanInfo:
    block_k: int
    q_tile: int
    n_work: int
    total_frames: int
    tokens: int
    key_blocks: int
    visible_flops: float
    table: np.ndarray  # [Nf, 4] int32: start0, len0, start1, len1


_LIB: Optional[ctypes.CDLL] = None

_SIGS = {
    "fas_plan": (ctypes.c_int, [ctypes.c_int] * 6 + [ctypes.POINTER(_PlanInfoC)]),
    "fas_plan_ex": (ctypes.c_int, [ctypes.c_int] * 7 + [ctypes.POINTER(_PlanInfoC)]),
    "fas_plan_describe": (ctypes.c_int, [ctypes.c_int] * 7 + [ctypes.POINTER(_PlanInfoC), ctypes.c_void_p,
                                                              ctypes.c_void_p]),
    "fas_plan_ragged": (ctypes.c_int, [ctypes.c_void_p] + [ctypes.c_int] * 6 + [ctypes.POINTER(_PlanInfoC)]),
    "fas_plan_describe_ragged": (ctypes.c_int, [ctypes.c_void_p] + [ctypes.c_int] * 6 +
                                 [ctypes.POINTER(_PlanInfoC), ctypes.c_void_p, ctypes.c_void_p]),
    "fas_prepass": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]),
    "fas_prepass_with_key_sums": (ctypes.c_int, [ctypes.c_void_p] * 5),
    "fas_forward": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int, ctypes.c_void_p]),
    "fas_forward_host": (ctypes.c_int, [ctypes.c_void_p] * 5 + [ctypes.c_int, ctypes.c_int, ctypes.c_void_p]),
    "fas_forward_ablation": (ctypes.c_int, [ctypes.c_void_p] * 6),
    "fas_prologue": (ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_int] * 4 + [ctypes.c_float] +
                     [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 + [ctypes.c_void_p]),
    "fas_prologue_with_key_sums": (ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_int] * 4 + [ctypes.c_float] +
                                   [ctypes.c_void_p] * 3 + [ctypes.c_int] * 3 + [ctypes.c_void_p] * 2),
    "fas_prologue_fold_weights": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int] * 2 + [ctypes.c_void_p]),
    "fas_free": (ctypes.c_int, []),
    "fas_status": (ctypes.c_int, [ctypes.c_void_p]),
    "fas_prepass_readback": (ctypes.c_int, [ctypes.c_void_p] * 6),
    "fas_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p]),
    "fas_selftest_row_wait_timeout": (ctypes.c_int, [ctypes.c_int, ctypes.c_void_p]),
    "fas_last_launch_count": (ctypes.c_int, []),
    "fas_prepass_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p] + [ctypes.c_int] * 6 +
                            [ctypes.c_void_p] * 4),
    "fas_backward": (ctypes.c_int, [ctypes.c_void_p] * 11),
    "fas_residual_norm": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int] + [ctypes.c_void_p] * 3 +
                          [ctypes.c_float, ctypes.c_float, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                           ctypes.c_int] + [ctypes.c_void_p] * 8),
    "fas_residual_norm_backward": (ctypes.c_int, [ctypes.c_void_p] * 4 + [ctypes.c_int] + [ctypes.c_void_p] * 8 +
                                   [ctypes.c_float, ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_int] +
                                   [ctypes.c_void_p] * 6 + [ctypes.c_int64, ctypes.c_void_p]),
    "fas_residual_norm_backward_workspace": (ctypes.c_int, [ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                                            ctypes.c_int, ctypes.POINTER(ctypes.c_int64)]),
    "fas_checkpoint_pack": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                                           ctypes.c_int64, ctypes.c_void_p]),
    "fas_checkpoint_unpack": (ctypes.c_int, [ctypes.c_void_p] * 3 + [ctypes.c_int, ctypes.c_int64, ctypes.c_void_p]),
    "fas_error_string": (ctypes.c_char_p, [ctypes.c_int]),
    "fas_set_layout": (ctypes.c_int, [ctypes.c_int]),
}


def load() -> ctypes.CDLL:
    """Loads libfas.so (raises if it has not been built)."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(
                f"{path} is missing: build it with `python -m frame_aligned_sparse_gb300.build` "
                "(nvcc, sm_103a). There is no CPU fallback.")
        lib = ctypes.CDLL(path)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = lib
    return _LIB


_HOST = None  # False: there is none


def _host():
    """The operators' calls on torch tensors in native code (csrc/host), bound
    to the loaded library; False, with a warning, if it was not built or does
    not load (the calls below then do the same, only slower)."""
    global _HOST
    if _HOST is None:
        import importlib.machinery
        import importlib.util
        import torch  # its libraries, which the module uses  # noqa: F401
        lib = load()
        path = os.path.join(os.path.dirname(library_path()), "_host.so")
        try:
            if not os.path.exists(path):
                raise ImportError(f"{path} is missing")
            loader = importlib.machinery.ExtensionFileLoader("_host", path)
            host = importlib.util.module_from_spec(importlib.util.spec_from_loader("_host", loader))
            loader.exec_module(host)
        except ImportError as e:
            import warnings
            warnings.warn(f"small calls take longer without the native binding ({e}): build it with "
                          "`python -m frame_aligned_sparse_gb300.build --force`", RuntimeWarning, stacklevel=4)
            _HOST = False
            return _HOST
        host.bind(*(ctypes.cast(getattr(lib, f"fas_{name}"), ctypes.c_void_p).value for name in (
            "backward", "residual_norm", "residual_norm_backward", "residual_norm_backward_workspace",
            "checkpoint_pack", "checkpoint_unpack")))
        _HOST = host
    return _HOST


def _native(call: str, first, *args):
    """The call's results from native code, or None if it is not a plain one
    (see csrc/host/calls.cpp) and the caller has to go on by itself."""
    if not getattr(first, "is_cuda", False):
        return None
    host = _host() if _HOST is None else _HOST
    got = getattr(host, call)(*args) if host else None
    if type(got) is int:
        _check(f"fas_{call}", got)
    return got


def _check(call: str, rc: int) -> None:
    if rc != FAS_OK:
        msg = load().fas_error_string(rc).decode()
        raise FasError(call, rc, msg)


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        return _current_device_stream()[1]
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream_object(stream):
    """A torch stream for a stream argument (a stream or a handle)."""
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return stream
    handle = _stream_handle(stream)
    # (Handle 0 is the default stream; an ExternalStream of 0 would be a new one.)
    return torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()


def _empty(stream, shape, dtype, device):
    """A tensor that a call on ``stream`` (None: the current one) writes.

    Its memory is that stream's own: a block of the current stream may have
    been freed with work on it still queued there, which the call would not
    wait for.  The current stream, where the caller goes on, is a user too."""
    import torch
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(_stream_object(stream)):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(torch.cuda.current_stream())
    return t


def _info(c: _PlanInfoC, table: Optional[np.ndarray] = None) -> PlanInfo:
    if table is None:
        table = np.ctypeslib.as_array(c.host_table, shape=(c.total_frames * 4,)).reshape(-1, 4).copy()
    return PlanInfo(c.block_k, c.q_tile, c.n_work, c.total_frames, c.tokens, c.key_blocks, c.visible_flops, table)


_PLAN: dict = {}


def _spans_arg(frame_tokens, n_frames: int, ref_frames: int):
    """(int32 array of per-frame spans, or None for uniform frames)."""
    if np.ndim(frame_tokens) == 0:
        return None
    spans = np.ascontiguousarray(frame_tokens, dtype=np.int32)
    if spans.ndim != 1 or len(spans) != ref_frames + n_frames:
        raise ValueError(f"frame_tokens must hold ref_frames + n_frames = {ref_frames + n_frames} spans")
    return spans


def fas_plan(frame_tokens, n_frames: int, ref_frames: int, window_radius: int, heads: int, head_dim: int,
             block_k: int = 0) -> PlanInfo:
    """Builds (or reuses) the library's plan; see ``fas_plan`` in fas.h.
    ``frame_tokens``: one span for every frame, or a sequence of
    ref_frames + n_frames per-frame spans (``fas_plan_ragged``)."""
    c = _PlanInfoC()
    spans = _spans_arg(frame_tokens, n_frames, ref_frames)
    if spans is None:
        rc = load().fas_plan_ex(frame_tokens, n_frames, ref_frames, window_radius, heads, head_dim, block_k,
                                ctypes.byref(c))
    else:
        rc = load().fas_plan_ragged(spans.ctypes.data, n_frames, ref_frames, window_radius, heads, head_dim,
                                    block_k, ctypes.byref(c))
    _check("fas_plan", rc)
    info = _info(c)
    geometry = (tuple(spans.tolist()) if spans is not None else frame_tokens, n_frames, ref_frames, window_radius,
                heads, head_dim, info.block_k)
    if _PLAN.get("geometry") != geometry:
        _PLAN["layout"] = "hnd"  # a new plan starts head-major (the library resets it too)
    _PLAN.update(heads=heads, head_dim=head_dim, tokens=info.tokens, info=info, geometry=geometry)
    return info


def fas_set_layout(layout: str) -> None:
    """Layout of q, k, v and out for the following calls: "hnd" ([H, N, d])
    or "nhd" ([N, H, d]); lse stays [H, N].  See ``fas_set_layout`` in fas.h."""
    _check("fas_set_layout", load().fas_set_layout(LAYOUTS[layout]))
    _PLAN["layout"] = layout


def fas_plan_describe(frame_tokens, n_frames: int, ref_frames: int, window_radius: int, heads: int,
                      head_dim: int, block_k: int = 0) -> Tuple[PlanInfo, np.ndarray, np.ndarray]:
    """Host-only plan: (info, table [Nf, 4], work [n_work, 4]).  frame_tokens
    as in ``fas_plan``."""
    lib = load()
    spans = _spans_arg(frame_tokens, n_frames, ref_frames)

    def call(c, table, work):
        if spans is None:
            return lib.fas_plan_describe(frame_tokens, n_frames, ref_frames, window_radius, heads, head_dim,
                                         block_k, ctypes.byref(c), table, work)
        return lib.fas_plan_describe_ragged(spans.ctypes.data, n_frames, ref_frames, window_radius, heads,
                                            head_dim, block_k, ctypes.byref(c), table, work)

    c = _PlanInfoC()
    _check("fas_plan_describe", call(c, None, None))
    table = np.zeros((c.total_frames, 4), dtype=np.int32)
    work = np.zeros((c.n_work, 4), dtype=np.int32)
    _check("fas_plan_describe", call(c, table.ctypes.data, work.ctypes.data))
    return _info(c, table), table, work


def _check_tensor(name, t, shape, dtype):
    import torch
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return  # the usual case, in one expression
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the plan needs {tuple(shape)}")


def _qkv_shape():
    """Shape of q, k, v and out in the current layout."""
    if not _PLAN:
        raise FasError("fas_plan", FAS_ERR_STATE, "no plan")
    if _PLAN.get("layout", "hnd") == "nhd":
        return (_PLAN["tokens"], _PLAN["heads"], _PLAN["head_dim"])
    return (_PLAN["heads"], _PLAN["tokens"], _PLAN["head_dim"])


def _lse_shape():
    return (_PLAN["heads"], _PLAN["tokens"])


def fas_prepass(q, k, stream=None, want_elig: bool = False) -> Optional[np.ndarray]:
    """Mean-centred key norms, row bounds and head eligibility (bf16 q, k [H, N, d])."""
    import torch
    shape = _qkv_shape()
    _check_tensor("q", q, shape, torch.bfloat16)
    _check_tensor("k", k, shape, torch.bfloat16)
    elig = np.zeros(_PLAN["heads"], dtype=np.uint8) if want_elig else None
    rc = load().fas_prepass(q.data_ptr(), k.data_ptr(), _stream_handle(stream),
                            elig.ctypes.data if want_elig else None)
    _check("fas_prepass", rc)
    return elig


def key_sums_shape(heads: int, tokens: int, head_dim: int) -> tuple:
    """Shape of the 16-token key column sums: [H, N/16, d] (fp32)."""
    if tokens % 16:
        raise ValueError(f"tokens ({tokens}) must be a multiple of 16 for key sums")
    return (heads, tokens // 16, head_dim)


def fas_prepass_with_key_sums(q, k, key_sums, stream=None, want_elig: bool = False) -> Optional[np.ndarray]:
    """fas_prepass with the key column sums per 16 tokens given (fp32
    [H, N/16, d], e.g. from fas_prologue_with_key_sums): k is read once."""
    import torch
    shape = _qkv_shape()
    _check_tensor("q", q, shape, torch.bfloat16)
    _check_tensor("k", k, shape, torch.bfloat16)
    _check_tensor("key_sums", key_sums, key_sums_shape(_PLAN["heads"], _PLAN["tokens"], _PLAN["head_dim"]),
                  torch.float32)
    elig = np.zeros(_PLAN["heads"], dtype=np.uint8) if want_elig else None
    rc = load().fas_prepass_with_key_sums(q.data_ptr(), k.data_ptr(), key_sums.data_ptr(), _stream_handle(stream),
                                          elig.ctypes.data if want_elig else None)
    _check("fas_prepass_with_key_sums", rc)
    return elig


def fas_forward(q, k, v, out=None, lse=None, mode: str = "auto", stream=None):
    """Attention; returns (out bf16 [H, N, d], lse fp32 [H, N])."""
    import torch
    shape = _qkv_shape()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, shape, torch.bfloat16)
    if out is None:
        out = _empty(stream, shape, torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(stream, _lse_shape(), torch.float32, q.device)
    _check_tensor("out", out, shape, torch.bfloat16)
    _check_tensor("lse", lse, _lse_shape(), torch.float32)
    rc = load().fas_forward(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                            MODES[mode], _stream_handle(stream))
    _check("fas_forward", rc)
    return out, lse


def fas_forward_ablation(q, k, v, out=None, lse=None, stream=None):
    """The splash-style ablation (128-multiple tiles, padding, mask
    predicates, two passes and a merge; see ``fas_forward_ablation`` in
    fas.h); head-major [H, N, d] only.  Returns (out, lse)."""
    import torch
    shape = _qkv_shape()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_tensor(name, t, shape, torch.bfloat16)
    if out is None:
        out = _empty(stream, shape, torch.bfloat16, q.device)
    if lse is None:
        lse = _empty(stream, _lse_shape(), torch.float32, q.device)
    _check_tensor("out", out, shape, torch.bfloat16)
    _check_tensor("lse", lse, _lse_shape(), torch.float32)
    rc = load().fas_forward_ablation(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                     _stream_handle(stream))
    _check("fas_forward_ablation", rc)
    return out, lse


def fas_prologue_fold_weights(w, gamma, out=None, stream=None):
    """W' = bf16(W * gamma) per input feature (see fas.h): w bf16
    [3*H*d, C], gamma fp32 [C] (CUDA tensors)."""
    import torch
    O, C = w.shape
    _check_tensor("w", w, (O, C), torch.bfloat16)
    _check_tensor("gamma", gamma, (C,), torch.float32)
    if out is None:
        out = _empty(stream, w.shape, w.dtype, w.device)
    _check_tensor("out", out, (O, C), torch.bfloat16)
    _check("fas_prologue_fold_weights",
           load().fas_prologue_fold_weights(w.data_ptr(), gamma.data_ptr(), out.data_ptr(), C, O,
                                            _stream_handle(stream)))
    return out


def fas_prologue(x, w_folded, cos, sin, heads: int, head_dim: int, layout: str = "hnd", groups: int = 1,
                 ranks: int = 1, q=None, k=None, v=None, eps: float = RMS_EPS, stream=None):
    """RMSNorm -> QKV projection -> rotary -> head packing in one kernel
    (see ``fas_prologue`` in fas.h).  x bf16 [N, C]; w_folded bf16
    [3*H*d, C]; cos, sin fp32 [N, d/2].  Returns (q, k, v) bf16 in
    ``layout``: "hnd" [H, N, d], "nhd" [N, H, d] or "a2a" [G, P, N, H/(G*P), d]."""
    return _prologue(x, w_folded, cos, sin, heads, head_dim, layout, groups, ranks, q, k, v, False, None, eps,
                     stream)


def fas_prologue_with_key_sums(x, w_folded, cos, sin, heads: int, head_dim: int, layout: str = "hnd",
                               groups: int = 1, ranks: int = 1, q=None, k=None, v=None, key_sums=None,
                               eps: float = RMS_EPS, stream=None):
    """fas_prologue that also writes the column sums of the written k over
    each 16 tokens (fp32 [H, N/16, d], the input of
    fas_prepass_with_key_sums).  Returns (q, k, v, key_sums)."""
    return _prologue(x, w_folded, cos, sin, heads, head_dim, layout, groups, ranks, q, k, v, True, key_sums, eps,
                     stream)


def _prologue(x, w_folded, cos, sin, heads, head_dim, layout, groups, ranks, q, k, v, sums, key_sums, eps, stream):
    import torch
    N, C = x.shape
    _check_tensor("x", x, (N, C), torch.bfloat16)
    _check_tensor("w_folded", w_folded, (3 * heads * head_dim, C), torch.bfloat16)
    _check_tensor("cos", cos, (N, head_dim // 2), torch.float32)
    _check_tensor("sin", sin, (N, head_dim // 2), torch.float32)
    if layout == "hnd":
        shape = (heads, N, head_dim)
    elif layout == "nhd":
        shape = (N, heads, head_dim)
    elif layout == "a2a":
        if heads % (groups * ranks):
            raise ValueError(f"heads ({heads}) must divide into {groups} groups x {ranks} ranks")
        shape = (groups, ranks, N, heads // (groups * ranks), head_dim)
    else:
        raise ValueError(layout)
    outs = []
    for name, t in (("q", q), ("k", k), ("v", v)):
        if t is None:
            t = _empty(stream, shape, torch.bfloat16, x.device)
        _check_tensor(name, t, shape, torch.bfloat16)
        outs.append(t)
    if not sums:
        rc = load().fas_prologue(x.data_ptr(), w_folded.data_ptr(), cos.data_ptr(), sin.data_ptr(), N, C, heads,
                                 head_dim, float(eps), outs[0].data_ptr(), outs[1].data_ptr(), outs[2].data_ptr(),
                                 PROLOGUE_LAYOUTS[layout], groups, ranks, _stream_handle(stream))
        _check("fas_prologue", rc)
        return tuple(outs)
    ks_shape = key_sums_shape(heads, N, head_dim)
    if key_sums is None:
        key_sums = _empty(stream, ks_shape, torch.float32, x.device)
    _check_tensor("key_sums", key_sums, ks_shape, torch.float32)
    rc = load().fas_prologue_with_key_sums(x.data_ptr(), w_folded.data_ptr(), cos.data_ptr(), sin.data_ptr(), N, C,
                                           heads, head_dim, float(eps), outs[0].data_ptr(), outs[1].data_ptr(),
                                           outs[2].data_ptr(), PROLOGUE_LAYOUTS[layout], groups, ranks,
                                           key_sums.data_ptr(), _stream_handle(stream))
    _check("fas_prologue_with_key_sums", rc)
    return (*outs, key_sums)


# A small call's time is the host's: the checks below read each property once,
# and the current stream's raw handle replaces its Stream object, which costs
# more than a launch to build.

def _check_here(name, t, shape, dtype, device: int) -> int:
    """_check_tensor, and that the tensor is on the current device (the
    kernels launch there).  Returns its address."""
    try:
        if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass  # not a tensor: told below
    _check_tensor(name, t, shape, dtype)
    raise ValueError(f"{name} is on {t.device}, the current device is cuda:{device}")


def _current(name, t) -> Tuple[int, int]:
    """The current device and its current stream's handle, for a call on t."""
    if not getattr(t, "is_cuda", False):
        raise TypeError(f"{name} must be a CUDA tensor")
    return _current_device_stream()


def _current_device_stream() -> Tuple[int, int]:
    import torch
    device = torch.cuda.current_device()
    return device, torch._C._cuda_getCurrentRawStream(device)


def _output(name, t, like, device: int, stream):
    """An output with like's type and shape, and its address."""
    if t is None:
        t = _empty(stream, like.shape, like.dtype, like.device)
        return t, t.data_ptr()
    return t, _check_here(name, t, like.shape, like.dtype, device)


def _on(stream, current: int) -> int:
    return current if stream is None else stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _own_until_run(stream, *outputs):
    """Keeps the memory of a caller's outputs until the stream of a call has
    written them."""
    import torch
    stream = _stream_object(stream)
    if stream != torch.cuda.current_stream():
        for t in outputs:
            t.record_stream(stream)


def fas_backward(q, k, v, out, lse, dout, dq=None, dk=None, dv=None, stream=None):
    """The attention's backward pass (see ``fas_backward`` in fas.h): q, k, v,
    out, lse as fas_forward took and returned them, dout the gradient of out
    (bf16, the plan's layout).  Returns (dq, dk, dv)."""
    import torch
    shape, lse_shape, bf16 = _qkv_shape(), _lse_shape(), torch.bfloat16
    if dq is None and dk is None and dv is None and stream is None:
        got = _native("backward", q, q, k, v, out, lse, dout, shape, lse_shape, BACKWARD_WORKSPACE)
        if got is not None:
            return got
    device, current = _current("q", q)
    ptrs = [_check_here("q", q, shape, bf16, device), _check_here("k", k, shape, bf16, device),
            _check_here("v", v, shape, bf16, device), _check_here("out", out, shape, bf16, device),
            _check_here("lse", lse, lse_shape, torch.float32, device),
            _check_here("dout", dout, shape, bf16, device)]
    dq, p = _output("dq", dq, q, device, stream)
    ptrs.append(p)
    dk, p = _output("dk", dk, q, device, stream)
    ptrs.append(p)
    dv, p = _output("dv", dv, q, device, stream)
    ptrs.append(p)
    workspace = _empty(stream, (BACKWARD_WORKSPACE, *lse_shape), torch.uint8, q.device)
    rc = load().fas_backward(*ptrs, workspace.data_ptr(), _on(stream, current))
    _check("fas_backward", rc)
    if stream is not None:
        _own_until_run(stream, dq, dk, dv)
    return dq, dk, dv


class Checkpoint(NamedTuple):
    """A tensor held in 8 bits: e4m3 codes in the tensor's shape and one
    exponent byte per 32 elements of the last axis (value = code *
    2^(scale - 127); see ``fas_checkpoint_pack`` in fas.h)."""
    codes: "torch.Tensor"
    scales: "torch.Tensor"


def _dtype_code(name, t) -> int:
    import torch
    if isinstance(t, torch.Tensor):
        if t.dtype is torch.bfloat16:
            return 0
        if t.dtype is torch.float32:
            return 1
    raise TypeError(f"{name} must be a bfloat16 or float32 tensor")


def _checkpoint_empty(shape, device, stream):
    import torch
    if not shape or shape[-1] % CHECKPOINT_BLOCK or 0 in shape:
        raise ValueError(f"a checkpointed tensor's last axis must be a positive multiple of {CHECKPOINT_BLOCK} "
                         f"and its shape not empty, got {tuple(shape)}")
    return Checkpoint(_empty(stream, shape, torch.float8_e4m3fn, device),
                      _empty(stream, (*shape[:-1], shape[-1] // CHECKPOINT_BLOCK), torch.uint8, device))


def _check_checkpoint(name, c, device: int, shape=None):
    """The checkpoint and the addresses of its codes and scales."""
    import torch
    if not isinstance(c, tuple) or len(c) != 2:
        raise TypeError(f"{name} must be a Checkpoint (codes, scales)")
    c = Checkpoint(*c)
    shape = tuple(c.codes.shape) if shape is None else tuple(shape)
    if not shape or shape[-1] % CHECKPOINT_BLOCK:
        raise ValueError(f"{name}: the last axis must be a multiple of {CHECKPOINT_BLOCK}, got {shape}")
    return c, [_check_here(f"{name}.codes", c.codes, shape, torch.float8_e4m3fn, device),
               _check_here(f"{name}.scales", c.scales, (*shape[:-1], shape[-1] // CHECKPOINT_BLOCK), torch.uint8,
                           device)]


def fas_checkpoint_pack(x, out: Optional[Checkpoint] = None, stream=None) -> Checkpoint:
    """Holds x (bf16 or fp32, contiguous, last axis a multiple of 32) in 8
    bits: see ``fas_checkpoint_pack`` in fas.h."""
    if out is None and stream is None:
        got = _native("checkpoint_pack", x, x)
        if got is not None:
            return Checkpoint(*got)
    dtype = _dtype_code("x", x)
    device, current = _current("x", x)
    ptr = _check_here("x", x, x.shape, x.dtype, device)
    c = _checkpoint_empty(tuple(x.shape), x.device, stream) if out is None else out
    c, ptrs = _check_checkpoint("out", c, device, x.shape)
    _check("fas_checkpoint_pack", load().fas_checkpoint_pack(ptr, dtype, *ptrs, x.numel(), _on(stream, current)))
    if stream is not None:
        _own_until_run(stream, *c)
    return c


def fas_checkpoint_unpack(c: Checkpoint, dtype=None, out=None, stream=None):
    """The tensor a checkpoint stands for, as bf16 (the default) or fp32."""
    import torch
    if not isinstance(c, tuple) or len(c) != 2:
        raise TypeError("c must be a Checkpoint (codes, scales)")
    if out is None and stream is None:
        got = _native("checkpoint_unpack", c[0], c, dtype)
        if got is not None:
            return got[0]
    device, current = _current("c.codes", c[0])
    c, ptrs = _check_checkpoint("c", c, device)
    shape = c.codes.shape
    if out is None:
        out = _empty(stream, shape, dtype or torch.bfloat16, c.codes.device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError(f"out must be {dtype}, got {out.dtype}")
    code = _dtype_code("out", out)
    ptr = _check_here("out", out, shape, out.dtype, device)
    _check("fas_checkpoint_unpack",
           load().fas_checkpoint_unpack(*ptrs, ptr, code, out.numel(), _on(stream, current)))
    if stream is not None:
        _own_until_run(stream, out)
    return out


def _whole(frame_tokens):
    """Tokens of the frames as Python ints: a list, or one number for all."""
    given = np.asarray(frame_tokens)
    with np.errstate(invalid="ignore"):
        spans = given.astype(np.int64)
    if (spans != given).any():
        raise ValueError(f"frame_tokens must be whole numbers, got {frame_tokens}")
    return spans.tolist()


def _norm_frames(tokens: int, width: int, gate, frame_tokens, device: int):
    """(gate's address, host spans or None, number of frames)."""
    import torch
    if gate is None:
        return None, None, 1
    n = gate.shape[0] if getattr(gate, "ndim", 0) == 2 else 0
    ptr = _check_here("gate", gate, (n, width), torch.float32, device)
    if frame_tokens is None:
        if n == 0 or tokens % n:
            raise ValueError(f"{tokens} tokens are not {n} equal frames (one per row of gate)")
        return ptr, None, n
    if not (isinstance(frame_tokens, (list, tuple)) and all(type(t) is int for t in frame_tokens)):
        frame_tokens = _whole(frame_tokens)
    if isinstance(frame_tokens, int):
        if n * frame_tokens != tokens:
            raise ValueError(f"gate has {n} frames of {frame_tokens} tokens; x has {tokens} tokens")
        return ptr, None, n
    if frame_tokens and isinstance(frame_tokens[0], list):
        raise ValueError("frame_tokens must be one number or a sequence of numbers")
    if len(frame_tokens) != n or sum(frame_tokens) != tokens or min(frame_tokens) < 0:
        raise ValueError(f"frame_tokens must hold {n} spans (one per row of gate) that add up to {tokens} tokens")
    return ptr, (ctypes.c_int32 * n)(*frame_tokens), n


@functools.lru_cache(maxsize=256)
def _norm_workspace(tokens: int, width: int, spans: Optional[bytes], frames: int, device: int) -> int:
    """Workspace bytes of the backward norm for a shape on a device."""
    need = ctypes.c_int64()
    _check("fas_residual_norm_backward",
           load().fas_residual_norm_backward_workspace(tokens, width, spans, frames, ctypes.byref(need)))
    return need.value


def fas_residual_norm(y, x, gamma_post, gamma_pre, gate=None, frame_tokens=None, alpha: float = 1.0,
                      eps: float = RMS_EPS, checkpoint: bool = False, x_out=None, h=None, stream=None):
    """The norm after a block, its gate and residual, and the norm before the
    next one, in one kernel (see ``fas_residual_norm`` in fas.h):
    x' = x + alpha * gate * rmsnorm(y) * gamma_post, h = rmsnorm(x') * gamma_pre.
    y bf16 [N, C]; x bf16 or fp32 [N, C]; gammas fp32 [C]; gate fp32
    [frames, C] or None; frame_tokens: tokens of each frame (one number, a
    sequence, or None for equal frames).  x_out may be x and h may be y.
    Returns (x', h, rstd [2, N]), and with ``checkpoint`` also the 8-bit
    Checkpoints of y and of x'."""
    import torch
    if x_out is None and h is None and stream is None:
        got = _native("residual_norm", x, y, x, gamma_post, gamma_pre, gate, frame_tokens, alpha, eps, checkpoint)
        if got is not None:
            return (*got[:3], Checkpoint(*got[3:5]), Checkpoint(*got[5:])) if checkpoint else got
    residual = _dtype_code("x", x)
    if x.ndim != 2:
        raise ValueError(f"x must be [tokens, width], got {tuple(x.shape)}")
    shape = N, C = x.shape
    bf16, f32 = torch.bfloat16, torch.float32
    device, current = _current("x", x)
    py, px = _check_here("y", y, shape, bf16, device), _check_here("x", x, shape, x.dtype, device)
    ppost = _check_here("gamma_post", gamma_post, (C,), f32, device)
    ppre = _check_here("gamma_pre", gamma_pre, (C,), f32, device)
    pgate, spans, frames = _norm_frames(N, C, gate, frame_tokens, device)
    x_out, px_out = _output("x_out", x_out, x, device, stream)
    h, ph = _output("h", h, y, device, stream)
    rstd = _empty(stream, (2, N), f32, x.device)
    held, ptrs = (), (None, None, None, None)
    if checkpoint:
        held = _checkpoint_empty((N, C), x.device, stream), _checkpoint_empty((N, C), x.device, stream)
        ptrs = [t.data_ptr() for t in (*held[0], *held[1])]
    rc = load().fas_residual_norm(py, px, residual, pgate, ppost, ppre, alpha, eps, N, C,
                                  spans, frames, px_out, ph, rstd.data_ptr(),
                                  *ptrs, _on(stream, current))
    if rc:
        _check("fas_residual_norm", rc)
    if stream is not None:
        _own_until_run(stream, x_out, h)
    return (x_out, h, rstd, *held)


def fas_residual_norm_backward(dx_out, dh, y, x_out, rstd, gamma_post, gamma_pre, gate=None, frame_tokens=None,
                               alpha: float = 1.0, dx=None, dy=None, stream=None):
    """Backward pass of fas_residual_norm (see fas.h): dx_out the gradient of
    x' (x's type), dh that of h; y and x_out as tensors or both as the
    forward's Checkpoints; rstd as the forward returned it.  dx may be dx_out
    and dy may be dh.  Returns (dx, dy, dgamma_post, dgamma_pre, dgate), dgate
    None without a gate."""
    import torch
    if dx is None and dy is None and stream is None:
        got = _native("residual_norm_backward", dx_out, dx_out, dh, y, x_out, rstd, gamma_post, gamma_pre, gate,
                      frame_tokens, alpha)
        if got is not None:
            return got
    residual = _dtype_code("dx_out", dx_out)
    if dx_out.ndim != 2:
        raise ValueError(f"dx_out must be [tokens, width], got {tuple(dx_out.shape)}")
    shape = N, C = dx_out.shape
    bf16, f32 = torch.bfloat16, torch.float32
    device, current = _current("dx_out", dx_out)
    args = [_check_here("dx_out", dx_out, shape, dx_out.dtype, device), _check_here("dh", dh, shape, bf16, device)]
    if isinstance(y, torch.Tensor) != isinstance(x_out, torch.Tensor):
        raise TypeError("y and x_out must both be tensors or both be Checkpoints")
    if isinstance(y, torch.Tensor):
        args += [_check_here("y", y, shape, bf16, device), _check_here("x_out", x_out, shape, dx_out.dtype, device),
                 residual, None, None, None, None]
    else:
        args += [None, None, residual, *_check_checkpoint("y", y, device, shape)[1],
                 *_check_checkpoint("x_out", x_out, device, shape)[1]]
    args += [_check_here("rstd", rstd, (2, N), f32, device), None,
             _check_here("gamma_post", gamma_post, (C,), f32, device),
             _check_here("gamma_pre", gamma_pre, (C,), f32, device)]
    args[-3], spans, frames = _norm_frames(N, C, gate, frame_tokens, device)
    dx, pdx = _output("dx", dx, dx_out, device, stream)
    dy, pdy = _output("dy", dy, dh, device, stream)
    need = _norm_workspace(N, C, None if spans is None else bytes(spans), frames, device)
    workspace = _empty(stream, need, torch.uint8, dx_out.device)
    dpost, dpre = (_empty(stream, (C,), f32, dx_out.device) for _ in range(2))
    dgate = None if gate is None else _empty(stream, gate.shape, f32, dx_out.device)
    rc = load().fas_residual_norm_backward(
        *args, alpha, N, C, spans, frames,
        pdx, pdy,
        None if dgate is None else dgate.data_ptr(), dpost.data_ptr(), dpre.data_ptr(), workspace.data_ptr(), need,
        _on(stream, current))
    _check("fas_residual_norm_backward", rc)
    if stream is not None:
        _own_until_run(stream, dx, dy)
    return dx, dy, dpost, dpre, dgate


def _check_host_tensor(name, t, shape, dtype):
    import torch
    if not isinstance(t, torch.Tensor) or t.is_cuda:
        raise TypeError(f"{name} must be a host (CPU) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, the plan needs {tuple(shape)}")


def fas_forward_host(q, k, v, out=None, lse=None, mode: str = "auto", heads_per_group: int = 0, stream=None):
    """Prepass + attention on HOST tensors (bf16 [H, N, d]; page-locked for
    copy/compute overlap), pipelined over head groups on the library's own
    streams; see ``fas_forward_host`` in fas.h.  Returns (out, lse) host
    tensors, complete once ``stream`` (default: the current CUDA stream) has
    reached this point."""
    import torch
    shape = _qkv_shape()
    for name, t in (("q", q), ("k", k), ("v", v)):
        _check_host_tensor(name, t, shape, torch.bfloat16)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, pin_memory=True)
    if lse is None:
        lse = torch.empty(_lse_shape(), dtype=torch.float32, pin_memory=True)
    _check_host_tensor("out", out, shape, torch.bfloat16)
    _check_host_tensor("lse", lse, _lse_shape(), torch.float32)
    rc = load().fas_forward_host(q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                 MODES[mode], int(heads_per_group), _stream_handle(stream))
    _check("fas_forward_host", rc)
    return out, lse


def fas_free() -> None:
    _PLAN.clear()
    _check("fas_free", load().fas_free())


def fas_status(stream=None) -> int:
    """Synchronises the stream; returns FAS_OK, FAS_ERR_TIMEOUT (a device wait
    gave up) or FAS_ERR_BOUND (a bounded row's softmax sum left its safe
    range: q or k changed since the prepass); raises on other errors."""
    rc = load().fas_status(_stream_handle(stream))
    if rc not in (FAS_OK, FAS_ERR_TIMEOUT, FAS_ERR_BOUND):
        _check("fas_status", rc)
    return rc


def fas_prepass_readback(stream=None, row_bound: bool = False) -> dict:
    H, N, d = _PLAN["heads"], _PLAN["tokens"], _PLAN["head_dim"]
    nf = _PLAN["info"].total_frames
    res = {"mu": np.zeros((H, d), np.float32), "frame_max": np.zeros((H, nf), np.float32),
           "stat": np.zeros(H, np.float32), "elig": np.zeros(H, np.uint8)}
    rb = np.zeros((H, N), np.float32) if row_bound else None
    rc = load().fas_prepass_readback(res["mu"].ctypes.data, res["frame_max"].ctypes.data, res["stat"].ctypes.data,
                                     res["elig"].ctypes.data, rb.ctypes.data if row_bound else None,
                                     _stream_handle(stream))
    _check("fas_prepass_readback", rc)
    if row_bound:
        res["row_bound"] = rb
    return res


def fas_selftest_wait_timeout(limit_us: int, stream=None) -> int:
    return load().fas_selftest_wait_timeout(limit_us, _stream_handle(stream))


def fas_selftest_row_wait_timeout(limit_us: int, stream=None) -> int:
    return load().fas_selftest_row_wait_timeout(limit_us, _stream_handle(stream))


def fas_prepass_noalloc(q, k, frame_tokens: int, n_frames: int, ref_frames: int, window_radius: int,
                        row_bound, stat, elig, stream=None) -> None:
    """The prepass without any allocation (see ``fas_prepass_noalloc`` in
    fas.h): the caller provides every output buffer; the library uses a fixed
    device array as scratch.  q, k: bf16 [H, N, d]; row_bound: fp32 [H, N];
    stat: fp32 [H]; elig: uint8 [H] (all CUDA tensors)."""
    import torch
    H, N, d = q.shape
    if N != (ref_frames + n_frames) * frame_tokens:
        # The C call has no plan to check the buffers against: a geometry
        # that does not match q would read past the ends of q and k.
        raise ValueError(f"q has {N} rows per head; the geometry needs (ref_frames + n_frames) * frame_tokens = "
                         f"{(ref_frames + n_frames) * frame_tokens}")
    _check_tensor("q", q, (H, N, d), torch.bfloat16)
    _check_tensor("k", k, (H, N, d), torch.bfloat16)
    _check_tensor("row_bound", row_bound, (H, N), torch.float32)
    _check_tensor("stat", stat, (H,), torch.float32)
    _check_tensor("elig", elig, (H,), torch.uint8)
    rc = load().fas_prepass_noalloc(q.data_ptr(), k.data_ptr(), frame_tokens, n_frames, ref_frames, window_radius,
                                    H, d, row_bound.data_ptr(), stat.data_ptr(), elig.data_ptr(),
                                    _stream_handle(stream))
    _check("fas_prepass_noalloc", rc)


def fas_last_launch_count() -> int:
    return load().fas_last_launch_count()
