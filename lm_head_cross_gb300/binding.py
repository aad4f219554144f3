"""ctypes binding over ``libflce.so`` (C-ABI declared in ``include/flce.h``).

Argument marshalling only: shapes, dtypes and device pointers are checked and
passed through; every step of the computation runs in the library's kernels.
PyTorch is used for device memory and the current stream.  There is no CPU
fallback: if the library is missing or fails to load, every call raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple

HERE = os.path.dirname(os.path.abspath(__file__))
_LIB = None

FLCE_OK = 0
FLCE_ERR_LABEL_OUT_OF_RANGE = 5
FLCE_ERR_TIMEOUT = 6
REDUCTIONS = {"mean": 0, "sum": 1, "none": 2}

EXPORTED = ("flce_workspace_bytes", "flce_workspace_bytes_rowchunk", "flce_forward", "flce_backward", "flce_fwd_bwd",
            "flce_fwd_bwd_rowchunk", "flce_read_device_status", "flce_selftest_timeout", "flce_profile_enable",
            "flce_profile_read", "flce_forward_noalloc", "flce_scale_grads", "flce_topk_workspace_bytes", "flce_topk",
            "flce_soft_fwd_bwd", "flce_soft_fwd_bwd_rowchunk", "flce_host_buffer_bytes", "flce_fwd_bwd_host", "flce_shard_workspace_bytes",
            "flce_shard_forward", "flce_shard_combine", "flce_shard_backward", "flce_valid_count",
            "flce_f32_to_bf16", "flce_layernorm_forward", "flce_layernorm_workspace_bytes", "flce_layernorm_backward",
            "flce_embedding_forward", "flce_embedding_workspace_bytes", "flce_embedding_backward",
            "flce_adamw_step", "flce_orthogonalize_workspace_bytes", "flce_orthogonalize", "flce_muon_workspace_bytes",
            "flce_muon_step", "flce_token_logprobs", "flce_token_logprobs_workspace_bytes",
            "flce_token_logprobs_backward", "flce_token_logprobs_backward_workspace_bytes",
            "flce_debug_checks", "flce_selftest_bounds", "flce_status_string")
_NO_CONTEXT = contextlib.nullcontext()
KERNEL_KINDS = ("forward", "grad", "dxdw", "small")


class FlceError(RuntimeError):
    def __init__(self, code: int, where: str = ""):
        self.code = int(code)
        msg = status_string(code) if _LIB is not None else f"status {code}"
        super().__init__(f"{where}: {msg} (status {code})" if where else f"{msg} (status {code})")


class Problem(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("v", ctypes.c_int64),
                ("ignore_index", ctypes.c_int32), ("reduction", ctypes.c_int32),
                ("shift", ctypes.c_int32), ("seq_len", ctypes.c_int32)]


class VocabShard(ctypes.Structure):
    _fields_ = [("v_offset", ctypes.c_int64), ("v_rows", ctypes.c_int64)]


class Norm(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("x_pitch", ctypes.c_int64), ("eps", ctypes.c_float),
                ("x_dtype", ctypes.c_int32), ("w_dtype", ctypes.c_int32)]


class Embedding(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("h", ctypes.c_int64), ("v", ctypes.c_int64), ("scale", ctypes.c_float),
                ("padding_idx", ctypes.c_int32), ("w_dtype", ctypes.c_int32), ("y_dtype", ctypes.c_int32)]


class AdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p), ("exp_avg_scale", ctypes.c_void_p),
                ("exp_avg_sq_scale", ctypes.c_void_p), ("count", ctypes.c_int64), ("lr", ctypes.c_float),
                ("weight_decay", ctypes.c_float), ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class AdamwOptions(ctypes.Structure):
    _fields_ = [("beta1", ctypes.c_double), ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("step", ctypes.c_int64), ("state_bits", ctypes.c_int32)]


class Matrix(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("x_dtype", ctypes.c_int32)]


class MuonTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p), ("master", ctypes.c_void_p),
                ("momentum", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("lr", ctypes.c_float), ("weight_decay", ctypes.c_float), ("scale", ctypes.c_float),
                ("param_dtype", ctypes.c_int32), ("grad_dtype", ctypes.c_int32)]


class MuonOptions(ctypes.Structure):
    _fields_ = [("momentum", ctypes.c_double), ("eps", ctypes.c_double),
                ("coefficients", ctypes.POINTER(ctypes.c_double)), ("steps", ctypes.c_int32),
                ("nesterov", ctypes.c_int32)]


def lib_path() -> str:
    return os.environ.get("FLCE_LIB", os.path.join(HERE, "libflce.so"))


def lib():
    """Load the C-ABI library (once).  Raises if it is not built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = lib_path()
    if not os.path.exists(path):
        raise FlceError(-1, f"{path} is not built; run __graft_entry__.build() or "
                            "python -m lm_head_cross_gb300.build")
    L = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    P = ctypes.POINTER(Problem)
    L.flce_workspace_bytes.argtypes = [P]
    L.flce_workspace_bytes.restype = sz
    L.flce_workspace_bytes_rowchunk.argtypes = [P]
    L.flce_workspace_bytes_rowchunk.restype = sz
    S = ctypes.POINTER(VocabShard)
    L.flce_shard_workspace_bytes.argtypes = [P, S]
    L.flce_shard_workspace_bytes.restype = sz
    L.flce_shard_forward.argtypes = [P, S, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_shard_forward.restype = ctypes.c_int
    L.flce_shard_combine.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_shard_combine.restype = ctypes.c_int
    L.flce_shard_backward.argtypes = [P, S, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_shard_backward.restype = ctypes.c_int
    L.flce_valid_count.argtypes = [P, vp, vp, vp, sz, vp]
    L.flce_valid_count.restype = ctypes.c_int
    L.flce_f32_to_bf16.argtypes = [vp, vp, ctypes.c_int64, vp]
    L.flce_f32_to_bf16.restype = ctypes.c_int
    Q = ctypes.POINTER(Norm)
    L.flce_layernorm_forward.argtypes = [Q, vp, vp, vp, vp, vp, vp, vp]
    L.flce_layernorm_forward.restype = ctypes.c_int
    L.flce_layernorm_workspace_bytes.argtypes = [Q]
    L.flce_layernorm_workspace_bytes.restype = sz
    L.flce_layernorm_backward.argtypes = [Q, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_layernorm_backward.restype = ctypes.c_int
    E = ctypes.POINTER(Embedding)
    L.flce_embedding_forward.argtypes = [E, vp, vp, vp, vp, sz, vp]
    L.flce_embedding_forward.restype = ctypes.c_int
    L.flce_embedding_workspace_bytes.argtypes = [E]
    L.flce_embedding_workspace_bytes.restype = sz
    L.flce_embedding_backward.argtypes = [E, vp, vp, vp, ctypes.c_int32, vp, sz, vp]
    L.flce_embedding_backward.restype = ctypes.c_int
    L.flce_adamw_step.argtypes = [ctypes.POINTER(AdamwTensor), ctypes.c_int32, ctypes.POINTER(AdamwOptions), vp, vp]
    L.flce_adamw_step.restype = ctypes.c_int
    for name, entry in (("orthogonalize", Matrix), ("muon", MuonTensor)):
        size = getattr(L, f"flce_{name}_workspace_bytes")
        size.argtypes, size.restype = [ctypes.POINTER(entry), ctypes.c_int32], sz
    O = ctypes.POINTER(MuonOptions)
    L.flce_orthogonalize.argtypes = [ctypes.POINTER(Matrix), ctypes.c_int32, O, vp, sz, vp]
    L.flce_orthogonalize.restype = ctypes.c_int
    L.flce_muon_step.argtypes = [ctypes.POINTER(MuonTensor), ctypes.c_int32, O, vp, vp, sz, vp]
    L.flce_muon_step.restype = ctypes.c_int
    L.flce_token_logprobs_workspace_bytes.argtypes = [P, ctypes.c_int32]
    L.flce_token_logprobs_workspace_bytes.restype = sz
    L.flce_token_logprobs.argtypes = [P, ctypes.c_int32, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_token_logprobs.restype = ctypes.c_int
    L.flce_token_logprobs_backward_workspace_bytes.argtypes = [P]
    L.flce_token_logprobs_backward_workspace_bytes.restype = sz
    L.flce_token_logprobs_backward.argtypes = [P, ctypes.c_float, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_token_logprobs_backward.restype = ctypes.c_int
    L.flce_forward_noalloc.argtypes = [P, vp, vp, vp, vp, vp, vp]
    L.flce_forward_noalloc.restype = ctypes.c_int
    L.flce_forward.argtypes = [P, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_forward.restype = ctypes.c_int
    L.flce_backward.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_backward.restype = ctypes.c_int
    L.flce_fwd_bwd.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_fwd_bwd.restype = ctypes.c_int
    L.flce_fwd_bwd_rowchunk.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_fwd_bwd_rowchunk.restype = ctypes.c_int
    L.flce_topk_workspace_bytes.argtypes = [P, ctypes.c_int32]
    L.flce_topk_workspace_bytes.restype = sz
    L.flce_topk.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_topk.restype = ctypes.c_int
    L.flce_soft_fwd_bwd.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_soft_fwd_bwd.restype = ctypes.c_int
    L.flce_soft_fwd_bwd_rowchunk.argtypes = [P, ctypes.c_int32, vp, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    L.flce_soft_fwd_bwd_rowchunk.restype = ctypes.c_int
    L.flce_host_buffer_bytes.argtypes = [P]
    L.flce_host_buffer_bytes.restype = sz
    L.flce_fwd_bwd_host.argtypes = [P, vp, vp, vp, vp, vp, vp, vp, vp, sz, vp, vp, vp]
    L.flce_fwd_bwd_host.restype = ctypes.c_int
    L.flce_scale_grads.argtypes = [P, vp, vp, vp, vp]
    L.flce_scale_grads.restype = ctypes.c_int
    L.flce_read_device_status.argtypes = [vp, vp]
    L.flce_read_device_status.restype = ctypes.c_int
    L.flce_selftest_timeout.argtypes = [vp, sz, ctypes.c_uint64, vp]
    L.flce_selftest_timeout.restype = ctypes.c_int
    L.flce_profile_enable.argtypes = [ctypes.c_int]
    L.flce_profile_enable.restype = ctypes.c_int
    L.flce_profile_read.argtypes = [ctypes.c_int, ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_double),
                                    ctypes.POINTER(ctypes.c_double)]
    L.flce_profile_read.restype = ctypes.c_int
    L.flce_debug_checks.argtypes = []
    L.flce_debug_checks.restype = ctypes.c_int
    L.flce_selftest_bounds.argtypes = [vp, sz, vp]
    L.flce_selftest_bounds.restype = ctypes.c_int
    L.flce_status_string.argtypes = [ctypes.c_int]
    L.flce_status_string.restype = ctypes.c_char_p
    _LIB = L
    return L


def status_string(code: int) -> str:
    return lib().flce_status_string(int(code)).decode()


def logits_footprint_bytes(n_rows: int, v: int, elem_bytes: int) -> int:
    """Bytes of a materialised [N, V] logits tensor (what the fused path never allocates)."""
    return int(n_rows) * int(v) * int(elem_bytes)


def _problem(n, h, v, ignore_index, reduction, shift=0, seq_len=0) -> Problem:
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be 'mean', 'sum' or 'none', got {reduction!r}")
    if shift not in (0, 1):
        raise ValueError("shift must be 0 or 1")
    if shift and (seq_len < 1 or n % seq_len):
        raise ValueError("shift=1 needs seq_len dividing the number of rows")
    return Problem(int(n), int(h), int(v), int(ignore_index), REDUCTIONS[reduction], int(shift),
                   int(seq_len) if shift else 0)


def workspace_bytes(n, h, v, ignore_index=-100, reduction="mean") -> int:
    """Workspace of forward, backward and fwd_bwd: bounded, independent of V."""
    p = _problem(n, h, v, ignore_index, reduction)
    return int(lib().flce_workspace_bytes(ctypes.byref(p)))


def workspace_bytes_rowchunk(n, h, v, ignore_index=-100, reduction="mean") -> int:
    """Workspace of the row-chunk calls (fwd_bwd(rowchunk=True), soft_fwd_bwd); grows with V."""
    p = _problem(n, h, v, ignore_index, reduction)
    return int(lib().flce_workspace_bytes_rowchunk(ctypes.byref(p)))


_TORCH = None


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        _TORCH = torch
    return _TORCH


def _stream_ptr(stream, device=None):
    """The cudaStream_t of a torch stream, or of the current one (asked for without building
    a torch.cuda.Stream object, which takes 3 us) of the current device, whose index a caller
    may know."""
    if stream is not None:
        return stream.cuda_stream
    return _torch()._C._cuda_getCurrentRawStream(_current_device() if device is None else device)


def _current_device():
    return _torch()._C._cuda_getDevice()


def _check_device(x, stream, *tensors):
    """Kernels start on the current device and read every pointer there: it must be the one that
    holds x, the call's other tensors (None: not given) and the stream, if one is given.  Returns
    its index (by number: comparing torch.device objects took 3 us a call)."""
    device = x.get_device()
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"all tensors must be on one device, got {x.device} and {t.device}")
    if device != _current_device() or (stream is not None and stream.device.index != device):
        raise ValueError(f"the tensors are on {x.device}, which is not the current device, or not the stream's")
    return device


def _check_inputs(x, w, labels):
    torch = _torch()
    if x.dim() != 2 or w.dim() != 2 or labels.dim() != 1:
        raise ValueError("x must be [N, H], w [V, H], labels [N]")
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16:
        raise TypeError("x and w must be bfloat16")
    if labels.dtype != torch.int32:
        raise TypeError("labels must be int32")
    if not (x.is_cuda and w.is_cuda and labels.is_cuda):
        raise ValueError("x, w and labels must be CUDA tensors")
    if not (x.is_contiguous() and w.is_contiguous() and labels.is_contiguous()):
        raise ValueError("x, w and labels must be contiguous")
    if x.shape[1] != w.shape[1] or labels.shape[0] != x.shape[0]:
        raise ValueError(f"shape mismatch: x {tuple(x.shape)}, w {tuple(w.shape)}, labels {tuple(labels.shape)}")


def _alloc_ws(n, h, v, ignore_index, reduction, device, rowchunk=False):
    torch = _torch()
    nbytes = (workspace_bytes_rowchunk if rowchunk else workspace_bytes)(n, h, v, ignore_index, reduction)
    if nbytes == 0:
        raise FlceError(1, "workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _call(name, code):
    if code != FLCE_OK:
        raise FlceError(code, name)


def forward(x, w, labels, ignore_index=-100, reduction="mean", ws=None, stream=None, check=False, shift=0,
            seq_len=0):
    """Returns (loss fp32 ([1], or [N] per row for reduction 'none'), lse [N] fp32, ws)."""
    torch = _torch()
    _check_inputs(x, w, labels)
    n, h = x.shape
    v = w.shape[0]
    p = _problem(n, h, v, ignore_index, reduction, shift, seq_len)
    if ws is None:
        ws = _alloc_ws(n, h, v, ignore_index, reduction, x.device)
    loss = torch.empty(n if reduction == "none" else 1, dtype=torch.float32, device=x.device)
    lse = torch.empty(n, dtype=torch.float32, device=x.device)
    s = _stream_ptr(stream)
    _call("flce_forward", lib().flce_forward(ctypes.byref(p), x.data_ptr(), w.data_ptr(), labels.data_ptr(),
                                             loss.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), s))
    if check:
        _call("device", read_device_status(ws, stream))
    return loss, lse, ws


def backward(x, w, labels, lse, grad_loss=None, ignore_index=-100, reduction="mean", ws=None, stream=None,
             check=False, shift=0, seq_len=0):
    """Returns (dX [N,H] bf16, dW [V,H] bf16, ws).  grad_loss: None or a 1-element fp32 CUDA
    tensor; for reduction 'none', an [N] fp32 CUDA tensor of per-row gradients (required)."""
    torch = _torch()
    _check_inputs(x, w, labels)
    n, h = x.shape
    v = w.shape[0]
    if lse.dtype != torch.float32 or lse.shape != (n,) or not lse.is_contiguous():
        raise ValueError("lse must be contiguous fp32 [N]")
    want = n if reduction == "none" else 1
    if reduction == "none" and grad_loss is None:
        raise ValueError("reduction 'none' needs per-row gradients")
    if grad_loss is not None and (grad_loss.dtype != torch.float32 or grad_loss.numel() != want or not grad_loss.is_cuda
                                  or not grad_loss.is_contiguous()):
        raise ValueError(f"grad_loss must be a contiguous {want}-element fp32 CUDA tensor")
    p = _problem(n, h, v, ignore_index, reduction, shift, seq_len)
    if ws is None:
        ws = _alloc_ws(n, h, v, ignore_index, reduction, x.device)
    dX = torch.empty_like(x)
    dW = torch.empty_like(w)
    s = _stream_ptr(stream)
    g = None if grad_loss is None else grad_loss.data_ptr()
    _call("flce_backward", lib().flce_backward(ctypes.byref(p), x.data_ptr(), w.data_ptr(), labels.data_ptr(),
                                               lse.data_ptr(), g, dX.data_ptr(), dW.data_ptr(), ws.data_ptr(),
                                               ws.numel(), s))
    if check:
        _call("device", read_device_status(ws, stream))
    return dX, dW, ws


def fwd_bwd(x, w, labels, ignore_index=-100, reduction="mean", ws=None, stream=None, out=None, check=False,
            rowchunk=False, shift=0, seq_len=0):
    """Returns (loss, lse, dX, dW, ws).  ``out`` may pass preallocated (loss, lse, dX, dW).
    Default: flce_fwd_bwd on the bounded, V-independent workspace (logits recomputed in
    the backward pass).  ``rowchunk=True``: flce_fwd_bwd_rowchunk (logits computed once,
    a row chunk of the vocabulary gradient kept in a workspace that grows with V).  For
    reduction 'none' the loss is per row and the gradients are those of its sum."""
    torch = _torch()
    _check_inputs(x, w, labels)
    n, h = x.shape
    v = w.shape[0]
    p = _problem(n, h, v, ignore_index, reduction, shift, seq_len)
    if ws is None:
        ws = _alloc_ws(n, h, v, ignore_index, reduction, x.device, rowchunk=rowchunk)
    if out is None:
        out = (torch.empty(n if reduction == "none" else 1, dtype=torch.float32, device=x.device),
               torch.empty(n, dtype=torch.float32, device=x.device), torch.empty_like(x), torch.empty_like(w))
    loss, lse, dX, dW = out
    s = _stream_ptr(stream)
    name = "flce_fwd_bwd_rowchunk" if rowchunk else "flce_fwd_bwd"
    _call(name, getattr(lib(), name)(ctypes.byref(p), x.data_ptr(), w.data_ptr(), labels.data_ptr(),
                                     loss.data_ptr(), lse.data_ptr(), dX.data_ptr(), dW.data_ptr(),
                                     ws.data_ptr(), ws.numel(), s))
    if check:
        _call("device", read_device_status(ws, stream))
    return loss, lse, dX, dW, ws


def host_buffer_bytes(n, h, v, ignore_index=-100, reduction="mean") -> int:
    """Device buffer of fwd_bwd_host: the workspace, then device copies of inputs and results."""
    p = _problem(n, h, v, ignore_index, reduction)
    return int(lib().flce_host_buffer_bytes(ctypes.byref(p)))


def fwd_bwd_host(x, w, labels, out, dev, ignore_index=-100, reduction="mean", stream=None, shift=0, seq_len=0,
                 in_stream=None, out_stream=None):
    """flce_fwd_bwd_host: x, w, labels and out = (loss, lse, dX, dW) are CPU tensors (pinned for
    asynchronous copies), dev a CUDA uint8 tensor of host_buffer_bytes.  Input copies on
    `in_stream`, the pass on `stream`, result copies on `out_stream` (each defaults to `stream`);
    synchronise before reading `out`.  Device status: read_device_status(dev)."""
    torch = _torch()
    if x.is_cuda or w.is_cuda or labels.is_cuda or any(t.is_cuda for t in out):
        raise ValueError("fwd_bwd_host takes host tensors")
    if x.dtype != torch.bfloat16 or w.dtype != torch.bfloat16 or labels.dtype != torch.int32:
        raise TypeError("x and w must be bfloat16, labels int32")
    if not (x.is_contiguous() and w.is_contiguous() and labels.is_contiguous()):
        raise ValueError("inputs must be contiguous")
    n, h = x.shape
    v = w.shape[0]
    p = _problem(n, h, v, ignore_index, reduction, shift, seq_len)
    loss, lse, dX, dW = out
    s = _stream_ptr(stream)
    si = _stream_ptr(in_stream) if in_stream is not None else s
    so = _stream_ptr(out_stream) if out_stream is not None else s
    _call("flce_fwd_bwd_host", lib().flce_fwd_bwd_host(ctypes.byref(p), x.data_ptr(), w.data_ptr(), labels.data_ptr(),
                                                       loss.data_ptr(), lse.data_ptr(), dX.data_ptr(), dW.data_ptr(),
                                                       dev.data_ptr(), dev.numel(), s, si, so))
    return out


def topk_workspace_bytes(n, h, v, k) -> int:
    p = _problem(n, h, v, -100, "mean")
    return int(lib().flce_topk_workspace_bytes(ctypes.byref(p), int(k)))


def topk(x, w, k, ws=None, stream=None):
    """Per row, the k largest logits of x @ w.T (high to low), their ids and the row's lse.
    Returns (idx [N,k] int32, logit [N,k] fp32, lse [N] fp32, ws)."""
    torch = _torch()
    n, h = x.shape
    v = w.shape[0]
    dummy = torch.empty(n, dtype=torch.int32, device=x.device)
    _check_inputs(x, w, dummy)
    p = _problem(n, h, v, -100, "mean")
    if ws is None:
        nbytes = int(lib().flce_topk_workspace_bytes(ctypes.byref(p), int(k)))
        if nbytes == 0:
            raise FlceError(1, "flce_topk_workspace_bytes")
        ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    idx = torch.empty(n, k, dtype=torch.int32, device=x.device)
    val = torch.empty(n, k, dtype=torch.float32, device=x.device)
    lse = torch.empty(n, dtype=torch.float32, device=x.device)
    _call("flce_topk", lib().flce_topk(ctypes.byref(p), int(k), x.data_ptr(), w.data_ptr(), idx.data_ptr(),
                                       val.data_ptr(), lse.data_ptr(), ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
    return idx, val, lse, ws


def soft_fwd_bwd(x, w, tgt_idx, tgt_prob, reduction="mean", ws=None, stream=None, rowchunk=False):
    """KL of sparse soft targets (k ids and probabilities per row) against softmax(x @ w.T),
    forward and backward.  Returns (loss, lse, dX, dW, ws).  Bounded workspace by default;
    ``rowchunk=True``: flce_soft_fwd_bwd_rowchunk."""
    torch = _torch()
    n, h = x.shape
    v = w.shape[0]
    k = int(tgt_idx.shape[1])
    if tgt_idx.shape != (n, k) or tgt_prob.shape != (n, k) or tgt_idx.dtype != torch.int32 or \
            tgt_prob.dtype != torch.float32 or not (tgt_idx.is_contiguous() and tgt_prob.is_contiguous()):
        raise ValueError("targets must be contiguous [N, k] int32 ids and fp32 probabilities")
    _check_inputs(x, w, torch.empty(n, dtype=torch.int32, device=x.device))
    p = _problem(n, h, v, -100, reduction)
    if ws is None:
        ws = _alloc_ws(n, h, v, -100, reduction, x.device, rowchunk=rowchunk)
    loss = torch.empty(n if reduction == "none" else 1, dtype=torch.float32, device=x.device)
    lse = torch.empty(n, dtype=torch.float32, device=x.device)
    dX = torch.empty_like(x)
    dW = torch.empty_like(w)
    name = "flce_soft_fwd_bwd_rowchunk" if rowchunk else "flce_soft_fwd_bwd"
    _call(name, getattr(lib(), name)(ctypes.byref(p), k, x.data_ptr(), w.data_ptr(), tgt_idx.data_ptr(),
                                     tgt_prob.data_ptr(), loss.data_ptr(), lse.data_ptr(), dX.data_ptr(),
                                     dW.data_ptr(), ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
    return loss, lse, dX, dW, ws


def read_device_status(ws, stream=None) -> int:
    """Synchronises the stream and returns (and clears) the workspace's status word."""
    return int(lib().flce_read_device_status(ctypes.c_void_p(ws.data_ptr()), _stream_ptr(stream)))


def profile_enable(on: bool = True, kinds=None) -> None:
    """Time the launches of the given kernel kinds (names from KERNEL_KINDS; all when None)."""
    mask = 0
    if on:
        mask = -1 if kinds is None else sum(1 << KERNEL_KINDS.index(k) for k in kinds)
    _call("flce_profile_enable", lib().flce_profile_enable(mask))


def profile_read() -> dict:
    """{kind: (launches, total_ms, flops)} for the launches recorded since profile_enable."""
    out = {}
    for k, name in enumerate(KERNEL_KINDS):
        n, ms, fl = ctypes.c_int64(), ctypes.c_double(), ctypes.c_double()
        _call("flce_profile_read", lib().flce_profile_read(k, ctypes.byref(n), ctypes.byref(ms), ctypes.byref(fl)))
        out[name] = (int(n.value), float(ms.value), float(fl.value))
    return out


def scale_grads(dX, dW, grad_loss, stream=None):
    """dX *= g, dW *= g in place (g: one-element fp32 CUDA tensor)."""
    n, h = dX.shape
    v = dW.shape[0]
    p = _problem(n, h, v, -100, "mean")
    _call("flce_scale_grads", lib().flce_scale_grads(ctypes.byref(p), grad_loss.data_ptr(), dX.data_ptr(),
                                                     dW.data_ptr(), _stream_ptr(stream)))


def _f32(t, shape, name):
    torch = _torch()
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous fp32 CUDA tensor of shape {tuple(shape)}")


def shard_workspace_bytes(n, h, v_total, v_offset, v_rows, ignore_index=-100, reduction="mean") -> int:
    p = _problem(n, h, v_total, ignore_index, reduction)
    sh = VocabShard(int(v_offset), int(v_rows))
    return int(lib().flce_shard_workspace_bytes(ctypes.byref(p), ctypes.byref(sh)))


def _shard_ws(x, w_shard, v_total, v_offset, ignore_index, reduction, shift, seq_len, ws):
    torch = _torch()
    n, h = x.shape
    if ws is not None:
        return ws
    p = _problem(n, h, v_total, ignore_index, reduction, shift, seq_len)
    sh = VocabShard(int(v_offset), int(w_shard.shape[0]))
    nbytes = int(lib().flce_shard_workspace_bytes(ctypes.byref(p), ctypes.byref(sh)))
    if nbytes == 0:
        raise FlceError(1, "flce_shard_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=x.device)


def shard_forward(x, w_shard, labels, v_offset, v_total, ignore_index=-100, shift=0, seq_len=0, ws=None,
                  stream=None):
    """Vocabulary shard [v_offset, v_offset + w_shard.shape[0]) of a v_total-row LM head:
    (lse_part [N], tgt_part [N], ws) — the shard's per-row lse and the target logit
    where the shard holds the label (else 0)."""
    torch = _torch()
    _check_inputs(x, w_shard, labels)
    n, h = x.shape
    p = _problem(n, h, v_total, ignore_index, "mean", shift, seq_len)
    sh = VocabShard(int(v_offset), int(w_shard.shape[0]))
    ws = _shard_ws(x, w_shard, v_total, v_offset, ignore_index, "mean", shift, seq_len, ws)
    lse_p = torch.empty(n, dtype=torch.float32, device=x.device)
    tgt_p = torch.empty(n, dtype=torch.float32, device=x.device)
    _call("flce_shard_forward", lib().flce_shard_forward(ctypes.byref(p), ctypes.byref(sh), x.data_ptr(),
                                                         w_shard.data_ptr(), labels.data_ptr(), lse_p.data_ptr(),
                                                         tgt_p.data_ptr(), ws.data_ptr(), ws.numel(),
                                                         _stream_ptr(stream)))
    return lse_p, tgt_p, ws


def shard_combine(lse_parts, tgt_parts, labels, v_total, h, ignore_index=-100, reduction="mean", shift=0,
                  seq_len=0, ws=None, stream=None):
    """lse_parts, tgt_parts: [P, N] fp32 (shard r in row r).  Returns (loss, lse [N], ws).
    ``ws``: any workspace of a shard call (or of fwd_bwd) on the same rows serves."""
    torch = _torch()
    P, n = lse_parts.shape
    _f32(lse_parts, (P, n), "lse_parts")
    _f32(tgt_parts, (P, n), "tgt_parts")
    if labels.dtype != torch.int32 or labels.shape != (n,) or not labels.is_contiguous():
        raise ValueError("labels must be contiguous int32 [N]")
    p = _problem(n, h, v_total, ignore_index, reduction, shift, seq_len)
    if ws is None:
        nbytes = int(lib().flce_workspace_bytes(ctypes.byref(p)))
        ws = torch.empty(nbytes, dtype=torch.uint8, device=lse_parts.device)
    loss = torch.empty(n if reduction == "none" else 1, dtype=torch.float32, device=lse_parts.device)
    lse = torch.empty(n, dtype=torch.float32, device=lse_parts.device)
    _call("flce_shard_combine", lib().flce_shard_combine(ctypes.byref(p), int(P), lse_parts.data_ptr(),
                                                         tgt_parts.data_ptr(), labels.data_ptr(), loss.data_ptr(),
                                                         lse.data_ptr(), ws.data_ptr(), ws.numel(),
                                                         _stream_ptr(stream)))
    return loss, lse, ws


def shard_backward(x, w_shard, labels, lse, v_offset, v_total, grad_loss=None, ignore_index=-100,
                   reduction="mean", shift=0, seq_len=0, ws=None, stream=None):
    """Given the global lse: (dX_part [N, H] fp32, dW_shard [rows, H] bf16, ws)."""
    torch = _torch()
    _check_inputs(x, w_shard, labels)
    n, h = x.shape
    _f32(lse, (n,), "lse")
    p = _problem(n, h, v_total, ignore_index, reduction, shift, seq_len)
    sh = VocabShard(int(v_offset), int(w_shard.shape[0]))
    ws = _shard_ws(x, w_shard, v_total, v_offset, ignore_index, reduction, shift, seq_len, ws)
    dXp = torch.empty(n, h, dtype=torch.float32, device=x.device)
    dWs = torch.empty_like(w_shard)
    g = None if grad_loss is None else grad_loss.data_ptr()
    _call("flce_shard_backward", lib().flce_shard_backward(ctypes.byref(p), ctypes.byref(sh), x.data_ptr(),
                                                           w_shard.data_ptr(), labels.data_ptr(), lse.data_ptr(), g,
                                                           dXp.data_ptr(), dWs.data_ptr(), ws.data_ptr(), ws.numel(),
                                                           _stream_ptr(stream)))
    return dXp, dWs, ws


def valid_count(labels, v, h=8, ignore_index=-100, shift=0, seq_len=0, ws=None, stream=None):
    """Rows whose label is not ignore_index, as a one-element int32 CUDA tensor.
    ``ws``: any workspace of another call on the same rows serves."""
    torch = _torch()
    n = labels.shape[0]
    p = _problem(n, h, v, ignore_index, "sum", shift, seq_len)
    if ws is None:
        ws = torch.empty(max(256, int(lib().flce_workspace_bytes(ctypes.byref(p)))), dtype=torch.uint8,
                         device=labels.device)
    out = torch.empty(1, dtype=torch.int32, device=labels.device)
    _call("flce_valid_count", lib().flce_valid_count(ctypes.byref(p), labels.data_ptr(), out.data_ptr(),
                                                     ws.data_ptr(), ws.numel(), _stream_ptr(stream)))
    return out, ws


def f32_to_bf16(src, out=None, stream=None):
    """bf16 copy of a contiguous fp32 CUDA tensor (round to nearest even)."""
    torch = _torch()
    if src.dtype != torch.float32 or not src.is_contiguous() or not src.is_cuda:
        raise ValueError("src must be a contiguous fp32 CUDA tensor")
    if out is None:
        out = torch.empty(src.shape, dtype=torch.bfloat16, device=src.device)
    _call("flce_f32_to_bf16", lib().flce_f32_to_bf16(src.data_ptr(), out.data_ptr(), src.numel(),
                                                     _stream_ptr(stream)))
    return out


class _LinearCrossEntropy:
    """torch.autograd.Function wrapper, built lazily so importing needs no torch.

    When a gradient is needed, the forward runs the fused forward + backward
    (flce_fwd_bwd, upstream gradient 1) and keeps dX and dW; the backward then
    only multiplies them by the upstream gradient.  Otherwise the forward runs
    the forward pass alone."""
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class Fn(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x2, w, labels, ignore_index, reduction, shift, seq_len, rowchunk):
                    ctx.reduction = reduction
                    kw = dict(shift=shift, seq_len=seq_len)
                    needs = ctx.needs_input_grad[0] or ctx.needs_input_grad[1]
                    if needs and reduction != "none":
                        loss, _, dX, dW, _ = fwd_bwd(x2, w, labels, ignore_index, reduction, rowchunk=rowchunk, **kw)
                        ctx.save_for_backward(dX, dW)
                        return loss.reshape(())
                    loss, lse, _ = forward(x2, w, labels, ignore_index, reduction, **kw)
                    if needs:  # per-row upstream gradients are only known in backward: recompute there
                        ctx.save_for_backward(x2, w, labels, lse)
                        ctx.args = (ignore_index, kw)
                    return loss if reduction == "none" else loss.reshape(())

                @staticmethod
                def backward(ctx, grad):
                    if ctx.reduction == "none":
                        x2, w, labels, lse = ctx.saved_tensors
                        ignore_index, kw = ctx.args
                        g = grad.detach().to(torch.float32).reshape(-1).contiguous()
                        dX, dW, _ = backward(x2, w, labels, lse, g, ignore_index, "none", **kw)
                        return dX, dW, None, None, None, None, None, None
                    dX, dW = ctx.saved_tensors
                    g = grad.detach().to(torch.float32).reshape(1).contiguous()
                    scale_grads(dX, dW, g)
                    return dX, dW, None, None, None, None, None, None

            cls.fn = Fn
        return cls.fn


def linear_cross_entropy(x, w, labels, ignore_index: int = -100, reduction: str = "mean", shift: int = 0,
                         rowchunk: bool = False):
    """Cross-entropy of ``x @ w.T`` against ``labels`` without materialising the logits.

    x: [..., H] bf16 CUDA, w: [V, H] bf16, labels: [...] integer (same leading
    shape as x).  reduction: 'mean' (over non-ignored rows), 'sum' or 'none'
    (per-row losses, shaped like labels).  shift=1 scores position t of each
    sequence against the label at t + 1 (x and labels [B, S, ...]; the last
    position of each sequence is ignored).  Autograd flows to x and w.
    The extra device memory is bounded and independent of V (logits recomputed
    in the backward pass); ``rowchunk=True`` computes the logits once and keeps a
    row chunk of the vocabulary gradient instead (memory grows with V).
    """
    torch = _torch()
    h = x.shape[-1]
    seq_len = 0
    if shift:
        if x.dim() < 3:
            raise ValueError("shift=1 needs x shaped [B, S, H]")
        seq_len = int(x.shape[-2])
    x2 = x.reshape(-1, h).contiguous()
    lab = labels.reshape(-1).to(torch.int32).contiguous()
    loss = _LinearCrossEntropy.get().apply(x2, w.contiguous(), lab, int(ignore_index), reduction, int(shift),
                                           seq_len, bool(rowchunk))
    return loss.reshape(labels.shape) if reduction == "none" else loss


class _SparseKL:
    """torch.autograd.Function for the soft-target KL: the forward runs the fused
    forward + backward (flce_soft_fwd_bwd, upstream gradient 1) and keeps dX and
    dW; the backward multiplies them by the upstream gradient."""
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class Fn(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x2, w, tgt_idx, tgt_prob, reduction, rowchunk):
                    loss, _, dX, dW, _ = soft_fwd_bwd(x2, w, tgt_idx, tgt_prob, reduction, rowchunk=rowchunk)
                    ctx.save_for_backward(dX, dW)
                    return loss.reshape(())

                @staticmethod
                def backward(ctx, grad):
                    dX, dW = ctx.saved_tensors
                    g = grad.detach().to(torch.float32).reshape(1).contiguous()
                    scale_grads(dX, dW, g)
                    return dX, dW, None, None, None, None

            cls.fn = Fn
        return cls.fn


def sparse_kl_divergence(x, w, tgt_idx, tgt_prob, reduction: str = "mean", rowchunk: bool = False):
    """KL(q || softmax(x @ w.T)) against sparse soft targets (a teacher's top-k ids
    and probabilities per row), without materialising the logits.

    x: [..., H] bf16 CUDA, w: [V, H] bf16, tgt_idx / tgt_prob: [..., k] (k <= 16)
    integer ids and fp32 probabilities; a row whose probabilities are all 0 is
    ignored.  reduction: 'mean' (over rows with targets) or 'sum'.  Autograd flows
    to x and w.  Bounded, V-independent extra memory by default; ``rowchunk=True``
    computes the logits once and keeps a row chunk of the vocabulary gradient.
    """
    torch = _torch()
    if reduction not in ("mean", "sum"):
        raise ValueError("sparse_kl_divergence takes reduction 'mean' or 'sum'")
    h = x.shape[-1]
    k = tgt_idx.shape[-1]
    x2 = x.reshape(-1, h).contiguous()
    idx = tgt_idx.reshape(-1, k).to(torch.int32).contiguous()
    q = tgt_prob.reshape(-1, k).to(torch.float32).contiguous()
    return _SparseKL.get().apply(x2, w.contiguous(), idx, q, reduction, bool(rowchunk))


def _dtype(t, name):
    """flce_dtype_t of a tensor: 0 bf16, 1 fp32."""
    torch, kind = _torch(), t.dtype
    if kind is torch.bfloat16:
        return 0
    if kind is torch.float32:
        return 1
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _allocating(stream):
    """Allocations inside belong to ``stream`` (the current one when None): the caching
    allocator then reuses them only after that stream's work."""
    return _NO_CONTEXT if stream is None else _torch().cuda.stream(stream)


def _record(stream, *tensors):
    """What is freed after the call is reused only once ``stream`` is done with it."""
    if stream is not None:
        for t in tensors:
            if t is not None:
                t.record_stream(stream)


def _norm(x, weight, bias, eps):
    if x.dim() != 2 or weight.dim() != 1:
        raise ValueError(f"x must be [N, H] and weight [H], got {tuple(x.shape)} and {tuple(weight.shape)}")
    n, h = x.shape
    if h < 1 or weight.numel() != h:
        raise ValueError(f"x must be [N, H] and weight [H], H >= 1, got {tuple(x.shape)} and {tuple(weight.shape)}")
    if not (x.is_cuda and weight.is_cuda and weight.is_contiguous()):
        raise ValueError("x and weight must be CUDA tensors, weight contiguous")
    if bias is not None and (bias.shape != weight.shape or bias.dtype != weight.dtype or not bias.is_cuda
                             or not bias.is_contiguous()):
        raise ValueError("bias must be a contiguous CUDA tensor of weight's shape and dtype")
    pitch, along = x.stride()
    if (h > 1 and along != 1) or (n > 1 and pitch < h):
        raise ValueError("the rows of x must be contiguous and must not overlap")
    return Norm(n, h, pitch if n > 1 else h, eps, _dtype(x, "x"), _dtype(weight, "weight"))


def layernorm_forward(x, weight, bias=None, eps=1e-5, stream=None):
    """Layer norm of the rows of x [N, H] (bf16 or fp32; the rows may be those of a larger
    tensor).  weight, bias: [H], bf16 or fp32.  Returns (y [N, H] of x's type, mean [N],
    rstd [N] fp32)."""
    torch = _torch()
    q = _norm(x, weight, bias, eps)
    device = _check_device(x, stream, weight, bias)
    with _allocating(stream):
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        mean = torch.empty(q.n, dtype=torch.float32, device=x.device)
        rstd = torch.empty_like(mean)
    _call("flce_layernorm_forward", lib().flce_layernorm_forward(
        ctypes.byref(q), x.data_ptr(), weight.data_ptr(), None if bias is None else bias.data_ptr(), y.data_ptr(),
        mean.data_ptr(), rstd.data_ptr(), _stream_ptr(stream, device)))
    return y, mean, rstd


@functools.lru_cache(maxsize=256)
def layernorm_workspace_bytes(n, h) -> int:
    return int(lib().flce_layernorm_workspace_bytes(ctypes.byref(Norm(int(n), int(h), int(h), 0.0, 0, 0))))


def layernorm_backward(dy, x, weight, mean, rstd, bias=True, ws=None, stream=None):
    """Gradients of layernorm_forward.  Returns (dx of x's type, dweight, dbias of weight's
    type, ws); ``bias=False``: dbias is None."""
    torch = _torch()
    q = _norm(x, weight, None, 0.0)
    if dy.shape != x.shape or dy.dtype != x.dtype or not dy.is_contiguous() or not dy.is_cuda:
        raise ValueError("dy must be a contiguous CUDA tensor of x's shape and dtype")
    _f32(mean, (q.n,), "mean")
    _f32(rstd, (q.n,), "rstd")
    device = _check_device(x, stream, dy, weight, mean, rstd, ws)
    with _allocating(stream):
        if ws is None:
            ws = torch.empty(layernorm_workspace_bytes(q.n, q.h), dtype=torch.uint8, device=x.device)
        dx = torch.empty_like(dy)
        dweight = torch.empty_like(weight)
        dbias = torch.empty_like(weight) if bias else None
    _call("flce_layernorm_backward", lib().flce_layernorm_backward(
        ctypes.byref(q), dy.data_ptr(), x.data_ptr(), weight.data_ptr(), mean.data_ptr(), rstd.data_ptr(),
        dx.data_ptr(), dweight.data_ptr(), dbias.data_ptr() if bias else None, ws.data_ptr(), ws.numel(),
        _stream_ptr(stream, device)))
    return dx, dweight, dbias, ws


class _LayerNorm:
    """torch.autograd.Function over layernorm_forward / layernorm_backward."""
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class Fn(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x2, weight, bias, eps):
                    y, mean, rstd = layernorm_forward(x2, weight, bias, eps)
                    ctx.save_for_backward(x2, weight, mean, rstd)
                    ctx.has_bias = bias is not None
                    return y

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dy):
                    x2, weight, mean, rstd = ctx.saved_tensors
                    dx, dweight, dbias, _ = layernorm_backward(dy.contiguous(), x2, weight, mean, rstd,
                                                               bias=ctx.has_bias)
                    return dx, dweight, dbias, None

            cls.fn = Fn
        return cls.fn


def layer_norm(x, weight, bias=None, eps: float = 1e-5):
    """Layer norm over the last dimension of x [..., H] (bf16 or fp32 CUDA); weight and bias
    [H], bf16 or fp32.  Autograd flows to x, weight and bias."""
    h = x.shape[-1]
    x2 = x.reshape(-1, h)
    if h > 1 and x2.stride(1) != 1 or (x2.shape[0] > 1 and x2.stride(0) < h):
        x2 = x2.contiguous()
    y = _LayerNorm.get().apply(x2, weight.contiguous(), None if bias is None else bias.contiguous(), float(eps))
    return y.reshape(x.shape)


def _check_ids(ids):
    if ids.dtype is not _torch().int32:
        raise TypeError("ids must be int32")
    if ids.dim() != 1 or not ids.is_cuda or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous CUDA tensor [N]")


def embedding_forward(ids, weight, scale=1.0, ws=None, stream=None, check=False):
    """scale * weight[ids] for ids [N] int32 and weight [V, H], bf16 or fp32.  Returns (y [N, H] of
    weight's type, ws).  ws: 256 bytes or more, for the device status."""
    torch = _torch()
    _check_ids(ids)
    if weight.dim() != 2 or not weight.is_cuda or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous CUDA tensor [V, H]")
    code = _dtype(weight, "weight")
    device = _check_device(weight, stream, ids, ws)
    (v, h), n = weight.shape, ids.numel()
    q = Embedding(n, h, v, scale, -1, code, code)
    with _allocating(stream):
        if ws is None:
            ws = torch.empty(256, dtype=torch.uint8, device=weight.device)
        y = torch.empty(n, h, dtype=weight.dtype, device=weight.device)
    _call("flce_embedding_forward", lib().flce_embedding_forward(
        ctypes.byref(q), ids.data_ptr(), weight.data_ptr(), y.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream_ptr(stream, device)))
    _record(stream, ids, weight, ws)
    if check:
        _call("device", read_device_status(ws, stream))
    return y, ws


@functools.lru_cache(maxsize=256)
def embedding_workspace_bytes(n, h, v) -> int:
    return int(lib().flce_embedding_workspace_bytes(ctypes.byref(Embedding(int(n), int(h), int(v), 1.0, -1, 0, 0))))


def embedding_backward(dy, ids, v, scale=1.0, padding_idx=None, add_to=None, dtype=None, ws=None, stream=None,
                       check=False):
    """The gradient of embedding_forward's weight [v, H] for dy [N, H]: a new tensor (of type dtype,
    else dy's), or added in place to ``add_to``, the gradient that the head's backward pass left
    for a matrix that both share.  Tokens equal to padding_idx add nothing.  Returns (dweight, ws)."""
    torch = _torch()
    _check_ids(ids)
    n, v = ids.numel(), int(v)
    if padding_idx is not None and padding_idx < 0:
        raise ValueError(f"padding_idx must be None or in [0, {v}), got {padding_idx}")
    if dy.dim() != 2 or dy.shape[0] != n or not dy.is_cuda or not dy.is_contiguous():
        raise ValueError(f"dy must be a contiguous CUDA tensor [N, H] for ids [N], got {tuple(dy.shape)}")
    h = dy.shape[1]
    if add_to is not None:
        if add_to.shape != (v, h) or not add_to.is_cuda or not add_to.is_contiguous():
            raise ValueError(f"add_to must be a contiguous CUDA tensor {(v, h)}")
        if dtype is not None and dtype != add_to.dtype:
            raise TypeError("dtype is add_to's where it is given")
    device = _check_device(dy, stream, ids, add_to, ws)
    with _allocating(stream):
        dw = torch.empty(v, h, dtype=dtype or dy.dtype, device=dy.device) if add_to is None else add_to
        q = Embedding(n, h, v, scale, -1 if padding_idx is None else int(padding_idx), _dtype(dw, "dweight"),
                      _dtype(dy, "dy"))
        if ws is None:
            nbytes = embedding_workspace_bytes(n, h, v)
            if nbytes == 0:
                raise FlceError(1, "flce_embedding_workspace_bytes")
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dy.device)
    _call("flce_embedding_backward", lib().flce_embedding_backward(
        ctypes.byref(q), dy.data_ptr(), ids.data_ptr(), dw.data_ptr(), int(add_to is not None), ws.data_ptr(),
        ws.numel(), _stream_ptr(stream, device)))
    _record(stream, dy, ids, add_to, ws)
    if add_to is not None:  # autograd learns of the write
        torch.autograd.graph.increment_version([add_to])
    if check:
        _call("device", read_device_status(ws, stream))
    return dw, ws


class _Embedding:
    """torch.autograd.Function over embedding_forward / embedding_backward."""
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class Fn(torch.autograd.Function):
                @staticmethod
                def forward(ctx, ids, weight, scale, padding_idx):
                    y, _ = embedding_forward(ids, weight, scale)
                    ctx.save_for_backward(ids)
                    ctx.args = (weight.shape[0], scale, padding_idx)
                    return y

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, dy):
                    ids, = ctx.saved_tensors
                    dw, _ = embedding_backward(dy.contiguous(), ids, *ctx.args)
                    return None, dw, None, None

            cls.fn = Fn
        return cls.fn


def embedding(ids, weight, scale: float = 1.0, padding_idx=None):
    """scale * weight[ids] for ids [...] (integer CUDA) and weight [V, H] (bf16 or fp32): [..., H].
    Autograd flows to weight, except from tokens equal to padding_idx.  An id outside [0, V) gives a
    row of zeros and passes no gradient (embedding_forward reports it)."""
    torch = _torch()
    v = weight.shape[0]
    if padding_idx is not None and not 0 <= padding_idx < v:
        raise ValueError(f"padding_idx must be in [0, {v}), got {padding_idx}")
    if ids.dtype not in (torch.int32, torch.int64, torch.int16, torch.int8, torch.uint8):
        raise TypeError(f"ids must be integers, got {ids.dtype}")
    flat = ids.reshape(-1)
    if flat.dtype is torch.int64:  # those beyond 32 bits stay outside
        flat = flat.clamp(-1, v)
    flat = flat.to(torch.int32).contiguous()
    y = _Embedding.get().apply(flat, weight.contiguous(), float(scale), padding_idx)
    return y.reshape(*ids.shape, weight.shape[1])


class TokenLogprobs(NamedTuple):
    """What logprobs_forward and token_logprobs return for each row: the given token's log
    probability (None without tokens), the entropy, the log-sum-exp, and the top alternatives'
    ids and log probabilities (None when top = 0)."""
    logprob: object
    entropy: object
    lse: object
    top_ids: object
    top_logprobs: object


def _check_head(x, w, tokens):
    torch = _torch()
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError(f"x must be [N, H] and w [V, H], got {tuple(x.shape)} and {tuple(w.shape)}")
    if x.dtype is not torch.bfloat16 or w.dtype is not torch.bfloat16:
        raise TypeError("x and w must be bfloat16")
    if not (x.is_cuda and w.is_cuda and x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous CUDA tensors")
    if tokens is not None:
        if tokens.dtype is not torch.int32:
            raise TypeError("tokens must be int32")
        if tokens.dim() != 1 or tokens.numel() != x.shape[0] or not tokens.is_cuda or not tokens.is_contiguous():
            raise ValueError("tokens must be a contiguous CUDA tensor [N]")


@functools.lru_cache(maxsize=256)
def token_logprobs_workspace_bytes(n, h, v, top=0) -> int:
    return int(lib().flce_token_logprobs_workspace_bytes(ctypes.byref(_problem(n, h, v, -100, "none")), int(top)))


def logprobs_forward(x, w, tokens=None, top=0, temperature=1.0, ignore_index=-100, shift=0, seq_len=0, ws=None,
                     stream=None, check=False):
    """Log probabilities of ``tokens`` [N] int32 under softmax(x @ w.T / temperature), with each
    row's entropy, log-sum-exp and ``top`` (at most 16) alternatives.  Returns (TokenLogprobs, ws)."""
    torch = _torch()
    _check_head(x, w, tokens)
    device = _check_device(x, stream, w, tokens, ws)
    n, h = x.shape
    p = _problem(n, h, w.shape[0], ignore_index, "none", shift, seq_len)
    top, dev, f32 = int(top), x.device, torch.float32
    with _allocating(stream):
        if ws is None:
            nbytes = token_logprobs_workspace_bytes(n, h, w.shape[0], top)
            if nbytes == 0:
                raise FlceError(1, "flce_token_logprobs_workspace_bytes")
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        lse = torch.empty(n, dtype=f32, device=dev)
        entropy = torch.empty_like(lse)
        lp = None if tokens is None else torch.empty_like(lse)
        ids = torch.empty(n, top, dtype=torch.int32, device=dev) if top > 0 else None
        tlp = torch.empty(n, top, dtype=f32, device=dev) if top > 0 else None
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call("flce_token_logprobs", lib().flce_token_logprobs(
        ctypes.byref(p), top, float(temperature), x.data_ptr(), w.data_ptr(), ptr(tokens), ptr(lp), entropy.data_ptr(),
        lse.data_ptr(), ptr(ids), ptr(tlp), ws.data_ptr(), ws.numel(), _stream_ptr(stream, device)))
    if check:
        _call("device", read_device_status(ws, stream))
    return TokenLogprobs(lp, entropy, lse, ids, tlp), ws


@functools.lru_cache(maxsize=256)
def logprobs_backward_workspace_bytes(n, h, v) -> int:
    p = _problem(n, h, v, -100, "none")
    return int(lib().flce_token_logprobs_backward_workspace_bytes(ctypes.byref(p)))


def logprobs_backward(x, w, tokens, lse, entropy, grad_logprob=None, grad_entropy=None, temperature=1.0,
                      ignore_index=-100, shift=0, seq_len=0, ws=None, stream=None, check=False):
    """Gradients of sum(grad_logprob * logprob + grad_entropy * entropy) given logprobs_forward's
    lse and entropy.  grad_logprob, grad_entropy: fp32 [N], or None.  Returns (dX, dW, ws)."""
    torch = _torch()
    _check_head(x, w, tokens)
    n, h = x.shape
    _f32(lse, (n,), "lse")
    if grad_logprob is not None:
        _f32(grad_logprob, (n,), "grad_logprob")
        if tokens is None:
            raise ValueError("grad_logprob needs tokens")
    if grad_entropy is not None:
        _f32(grad_entropy, (n,), "grad_entropy")
        if entropy is None:
            raise ValueError("grad_entropy needs entropy")
    if entropy is not None:
        _f32(entropy, (n,), "entropy")
    device = _check_device(x, stream, w, tokens, lse, entropy, grad_logprob, grad_entropy, ws)
    p = _problem(n, h, w.shape[0], ignore_index, "none", shift, seq_len)
    with _allocating(stream):
        if ws is None:
            nbytes = logprobs_backward_workspace_bytes(n, h, w.shape[0])
            if nbytes == 0:
                raise FlceError(1, "flce_token_logprobs_backward_workspace_bytes")
            ws = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        dX, dW = torch.empty_like(x), torch.empty_like(w)
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    _call("flce_token_logprobs_backward", lib().flce_token_logprobs_backward(
        ctypes.byref(p), float(temperature), x.data_ptr(), w.data_ptr(), ptr(tokens), lse.data_ptr(), ptr(entropy),
        ptr(grad_logprob), ptr(grad_entropy), dX.data_ptr(), dW.data_ptr(), ws.data_ptr(), ws.numel(),
        _stream_ptr(stream, device)))
    if check:
        _call("device", read_device_status(ws, stream))
    return dX, dW, ws


class _TokenLogprobs:
    """torch.autograd.Function over logprobs_forward / logprobs_backward; gradients flow through
    the log probabilities and the entropies."""
    fn = None

    @classmethod
    def get(cls):
        if cls.fn is None:
            torch = _torch()

            class Fn(torch.autograd.Function):
                @staticmethod
                def forward(ctx, x2, w, tokens, top, kw):
                    r, _ = logprobs_forward(x2, w, tokens, top=top, **kw)
                    ctx.save_for_backward(x2, w, r.lse, r.entropy, *(() if tokens is None else (tokens,)))
                    ctx.kw = kw
                    ctx.mark_non_differentiable(*(t for t in (r.lse, r.top_ids, r.top_logprobs) if t is not None))
                    ctx.set_materialize_grads(False)
                    return tuple(r)

                @staticmethod
                @torch.autograd.function.once_differentiable
                def backward(ctx, g_logprob, g_entropy, *_):
                    x2, w, lse, entropy, *rest = ctx.saved_tensors
                    if g_logprob is None and g_entropy is None:
                        return None, None, None, None, None
                    g = [None if t is None else t.to(torch.float32).contiguous() for t in (g_logprob, g_entropy)]
                    dX, dW, _ = logprobs_backward(x2, w, rest[0] if rest else None, lse, entropy, *g, **ctx.kw)
                    return dX, dW, None, None, None

            cls.fn = Fn
        return cls.fn


def token_logprobs(x, w, tokens=None, top: int = 0, temperature: float = 1.0, ignore_index: int = -100,
                   shift: int = 0):
    """Log probabilities of given tokens under softmax(x @ w.T / temperature), with entropies and
    top alternatives, without materialising the logits.

    x: [..., H] bf16 CUDA, w: [V, H] bf16, tokens: [...] integer (same leading shape as x), or
    None.  Rows whose token is ignore_index have log probability 0 and pass no gradient through
    it; their entropy and alternatives are those of any row.  top: alternatives per row (at most
    16), by logit, the lower id first among equals (so too among banned tokens, logits of minus
    infinity, where fewer others are left); -1 only past the vocabulary's end.  shift=1 scores position t of each sequence
    against the token at t + 1.  Returns TokenLogprobs shaped like x's leading dimensions;
    autograd flows from logprob and entropy to x and w.
    """
    torch = _torch()
    h, lead = x.shape[-1], x.shape[:-1]
    seq_len = 0
    if shift:
        if x.dim() < 3:
            raise ValueError("shift=1 needs x shaped [B, S, H]")
        seq_len = int(x.shape[-2])
    tok = None if tokens is None else tokens.reshape(-1).to(torch.int32).contiguous()
    kw = dict(temperature=float(temperature), ignore_index=int(ignore_index), shift=int(shift), seq_len=seq_len)
    r = _TokenLogprobs.get().apply(x.reshape(-1, h).contiguous(), w.contiguous(), tok, int(top), kw)
    return TokenLogprobs(*(None if t is None else t.reshape(lead + t.shape[1:]) for t in r))
