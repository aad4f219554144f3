"""Muon: updates orthogonalised by Newton-Schulz products (flce_orthogonalize, flce_muon_step).

``orthogonalize`` takes matrices as they are; ``muon_plan`` describes a model's matrices
once (parameters, momenta, optional fp32 master weights) and ``muon_step`` takes one step
with the current gradients.  ``Muon`` is the optimizer object on top of both.  It is for
the matrices of a model's hidden layers; ``AdamW`` takes its embedding, head and vectors.
"""
from __future__ import annotations

import ctypes
import math

from .binding import (FlceError, Matrix, MuonOptions, MuonTensor, _allocating, _call, _check_device, _dtype,
                      _record, _stream_ptr, _torch, lib, read_device_status)
from .optim import _check, _contiguous

#: Newton-Schulz coefficients (a, b, c) of X <- a X + (b X X^T + c (X X^T)^2) X, for every step
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
MAX_STEPS = 16


def _apart(written, read=()):
    """What a call writes must not overlap anything else that it writes or reads: (name, tensor)
    pairs, those of tensors that are None left out.  (The library looks at every call's addresses;
    here they have names.)"""
    spans = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size(), writes, name)
                   for writes, named in ((True, written), (False, read)) for name, t in named
                   if t is not None and t.numel())
    any_end = written_end = (0, "")
    for begin, end, writes, name in spans:
        before = any_end if writes else written_end
        if begin < before[0]:
            raise ValueError(f"{name} and {before[1]} are the same memory, or overlap")
        any_end = max(any_end, (end, name))
        if writes:
            written_end = max(written_end, (end, name))


def _options(momentum, nesterov, steps, coefficients, eps):
    """MuonOptions, which keeps its coefficients alive."""
    steps = int(steps)
    if not 1 <= steps <= MAX_STEPS:
        raise ValueError(f"steps must be 1 to {MAX_STEPS}, got {steps}")
    rows = list(coefficients)
    if len(rows) == 3 and all(isinstance(x, (int, float)) for x in rows):
        rows = [tuple(rows)] * steps
    if len(rows) != steps or any(len(r) != 3 for r in rows):
        raise ValueError("coefficients are three numbers, or three for each step")
    flat = (ctypes.c_double * (3 * steps))(*(float(x) for r in rows for x in r))
    return MuonOptions(float(momentum), float(eps), flat, steps, int(bool(nesterov)))


def orthogonalize(x, steps=5, coefficients=COEFFICIENTS, eps=1e-7, out=None, ws=None, stream=None, check=False):
    """Each matrix of x, u / (|u|_F + eps), taken through `steps` Newton-Schulz products; bf16.

    x: [..., R, C], or a list of matrices [R, C] of any shapes; bf16 or fp32, contiguous CUDA.
    out: where to write (bf16, shaped like x; may be x itself, but overlap nothing else), else it is allocated.
    coefficients: (a, b, c), or a list of them for the steps, which keep singular values within 2.1.
    Products take fp16 operands, pairs of them up to 128 rows or columns (the header says what their
    rounding leaves).  Returns out, without a gradient.  stream: the torch stream to run on, else the current one."""
    torch = _torch()
    listed = isinstance(x, (list, tuple))
    xs = list(x) if listed else [x]
    if not xs:
        return []
    for i, t in enumerate(xs):
        if t.dim() < 2 or (listed and t.dim() != 2):
            raise ValueError("x is a tensor [..., R, C] or a list of matrices [R, C]")
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("x must be contiguous CUDA tensors")
    outs = [None] * len(xs) if out is None else list(out) if listed else [out]
    if len(outs) != len(xs):
        raise ValueError("out must have one tensor for each of x")
    for t, o in zip(xs, outs):
        if o is not None and (o.shape != t.shape or o.dtype is not torch.bfloat16 or not o.is_contiguous()
                              or not o.is_cuda):
            raise ValueError("out must be contiguous bf16 CUDA tensors shaped like x")
    if out is not None:
        # (an output may be its own input)
        _apart([(f"out[{i}]", o) for i, o in enumerate(outs)],
               [(f"x[{i}]", t) for i, (t, o) in enumerate(zip(xs, outs))
                if o is None or t.data_ptr() != o.data_ptr() or t.dtype is not torch.bfloat16])
    device = _check_device(xs[0], stream, *xs[1:], *outs, ws)
    options = _options(0.0, False, steps, coefficients, eps)
    with _allocating(stream):
        outs = [torch.empty(t.shape, dtype=torch.bfloat16, device=t.device) if o is None else o
                for t, o in zip(xs, outs)]
        rows = []
        for t, o in zip(xs, outs):
            r, c = t.shape[-2:]
            code, size = _dtype(t, "x"), r * c
            at, to, step = t.data_ptr(), o.data_ptr(), size * t.element_size()
            rows += [(at + k * step, to + 2 * k * size, r, c, code) for k in range(t.numel() // size if size else 0)]
        table = (Matrix * max(len(rows), 1))(*rows)
        if ws is None:
            nbytes = int(lib().flce_orthogonalize_workspace_bytes(table, len(rows)))
            if nbytes == 0:
                raise FlceError(2, "flce_orthogonalize_workspace_bytes")
            ws = torch.empty(nbytes, dtype=torch.uint8, device=xs[0].device)
    _call("flce_orthogonalize", lib().flce_orthogonalize(table, len(rows), ctypes.byref(options), ws.data_ptr(),
                                                         ws.numel(), _stream_ptr(stream, device)))
    _record(stream, *xs, *outs, ws)
    given = [o for o in (out if listed else [out]) if o is not None] if out is not None else []
    if given:  # autograd learns of the writes
        torch.autograd.graph.increment_version(given)
    if check:
        _call("device", read_device_status(ws, stream))
    return outs if listed else outs[0]


def shape_factor(rows, cols, adjust):
    """The factor on lr for a matrix's shape: 'original', sqrt(max(1, rows / cols)), or
    'match_rms_adamw', 0.2 sqrt(max(rows, cols)), with which AdamW's lr and weight decay serve."""
    if adjust == "original":
        return math.sqrt(max(1.0, rows / max(cols, 1)))
    if adjust == "match_rms_adamw":
        return 0.2 * math.sqrt(max(rows, cols))
    raise ValueError(f"adjust must be 'original' or 'match_rms_adamw', got {adjust!r}")


class MuonPlan:
    """The matrices of a Muon step and its hyperparameters (see ``muon_plan``)."""

    def __init__(self, params, momenta, masters, lr, weight_decay, momentum, nesterov, steps, coefficients, eps,
                 adjust):
        torch = _torch()
        n = len(params)
        masters = [None] * n if masters is None else list(masters)
        if len(momenta) != n or len(masters) != n:
            raise ValueError("one entry per parameter is needed in every list")
        if not 0.0 <= momentum < 1.0:
            raise ValueError(f"momentum must be in [0, 1), got {momentum}")
        self.options = _options(momentum, nesterov, steps, coefficients, eps)
        self.table = (MuonTensor * max(n, 1))()
        self.shapes = []
        self.device = params[0].device if n else None
        for i, p in enumerate(params):
            if p.dim() != 2:
                raise ValueError(f"params[{i}] must be a matrix [rows, cols], got {tuple(p.shape)}")
            _check(p, f"params[{i}]", p)
            _check(momenta[i], f"momenta[{i}]", p, torch.float32)
            if masters[i] is not None:
                _check(masters[i], f"masters[{i}]", p, torch.float32)
            for t in (p, momenta[i], masters[i]):
                if t is not None and t.device != self.device:
                    raise ValueError("all tensors of a plan must be on one device")
            rows, cols = p.shape
            self.shapes.append((rows, cols))
            self.table[i] = MuonTensor(p.data_ptr(), None, None if masters[i] is None else masters[i].data_ptr(),
                                       momenta[i].data_ptr(), rows, cols, 0.0, 0.0, shape_factor(rows, cols, adjust),
                                       _dtype(p, f"params[{i}]"), 0)
        _apart([(f"{name}[{i}]", t) for name, held in (("params", params), ("momenta", momenta), ("masters", masters))
                for i, t in enumerate(held)])
        self._held = (list(params), list(momenta), list(masters))  # the table holds their addresses
        self._recorded = set()  # streams that _held's memory is known to be used on
        self._bytes = {}        # workspace size by which parameters have a gradient
        self.set_lr(lr)
        self.set_weight_decay(weight_decay)

    def __len__(self):
        return len(self.shapes)

    def set_param(self, i, p):
        """Parameter i now lives in ``p`` (same dtype and shape)."""
        old = self._held[0][i]
        _check(p, f"params[{i}]", old, old.dtype)
        if p.shape != old.shape or p.device != self.device:
            raise ValueError("the parameter must keep its shape, on the plan's device")
        self._held[0][i] = p
        self.table[i].param = p.data_ptr()
        self._recorded.clear()

    def set_lr(self, lr):
        """A number for every matrix, or one number per matrix, used from the next step on."""
        self._set("lr", lr)

    def set_weight_decay(self, weight_decay):
        """A number for every matrix, or one number per matrix, used from the next step on."""
        self._set("weight_decay", weight_decay)

    def _set(self, name, value):
        values = list(value) if isinstance(value, (list, tuple)) else [value] * len(self)
        if len(values) != len(self):
            raise ValueError(f"{name} is a number, or one number per parameter")
        for i, v in enumerate(values):
            setattr(self.table[i], name, v)

    def workspace_bytes(self, live=None):
        """Workspace of a step in which the parameters that ``live`` (truth values; None: all) names
        have a gradient, or any of them."""
        key = None if live is None or all(live) else tuple(live)
        if key not in self._bytes:
            table = (MuonTensor * max(len(self), 1))()
            for i, (rows, cols) in enumerate(self.shapes):
                table[i].rows, table[i].cols = (rows, cols) if key is None or key[i] else (0, 0)
            nbytes = int(lib().flce_muon_workspace_bytes(table, len(self)))
            if nbytes == 0:
                raise FlceError(2, "flce_muon_workspace_bytes")
            if len(self._bytes) >= 64:  # (experts that come and go)
                self._bytes.clear()
            self._bytes[key] = nbytes
        return self._bytes[key]


def muon_plan(params, momenta, masters=None, lr=0.02, weight_decay=0.0, momentum=0.95, nesterov=True, steps=5,
              coefficients=COEFFICIENTS, eps=1e-7, adjust="original"):
    """Describes the matrices of a Muon step.  Lists of contiguous CUDA tensors, one entry per
    parameter: params (bf16 or fp32, [rows, cols]), momenta (fp32), masters (fp32 master weights; an
    entry, or the list, may be None).  lr and weight_decay: a number, or a list of one number per
    parameter.  adjust: see ``shape_factor``."""
    return MuonPlan(params, momenta, masters, lr, weight_decay, momentum, nesterov, steps, coefficients, eps, adjust)


def muon_step(plan, grads, grad_scale=None, ws=None, stream=None, check=False):
    """One step in place.  grads: one contiguous bf16 or fp32 CUDA tensor per parameter, or None for
    a parameter that is left alone.  grad_scale: a one-element fp32 CUDA tensor that multiplies every
    gradient.  ws: at least plan.workspace_bytes(), else it is allocated.  Returns ws."""
    torch = _torch()
    if len(grads) != len(plan):
        raise ValueError(f"{len(plan)} gradients are needed, got {len(grads)}")
    table, f32, b16 = plan.table, torch.float32, torch.bfloat16
    for i, g in enumerate(grads):
        row = table[i]
        if g is None:
            row.rows = row.cols = 0
            continue
        if g.dtype is not f32 and g.dtype is not b16:
            raise TypeError(f"grads[{i}] must be bfloat16 or float32, got {g.dtype}")
        if tuple(g.shape) != plan.shapes[i] or not g.is_contiguous() or g.device != plan.device:
            raise ValueError(f"grads[{i}] must be contiguous, on the plan's device, with the parameter's shape")
        row.grad = g.data_ptr()
        row.grad_dtype = 1 if g.dtype is f32 else 0
        row.rows, row.cols = plan.shapes[i]
    if grad_scale is not None and (grad_scale.dtype != f32 or grad_scale.numel() != 1 or not grad_scale.is_cuda):
        raise ValueError("grad_scale must be a one-element fp32 CUDA tensor")
    if all(g is None for g in grads):
        return ws
    device = _check_device(plan._held[0][0], stream, grad_scale, ws)
    if ws is None:
        with _allocating(stream):
            ws = torch.empty(plan.workspace_bytes([g is not None for g in grads]), dtype=torch.uint8,
                             device=plan.device)
    _call("flce_muon_step", lib().flce_muon_step(
        table, len(plan), ctypes.byref(plan.options), None if grad_scale is None else grad_scale.data_ptr(),
        ws.data_ptr(), ws.numel(), _stream_ptr(stream, device)))
    if stream is not None:
        _record(stream, *grads, grad_scale, ws)
        if stream.cuda_stream not in plan._recorded:
            _record(stream, *(t for held in plan._held for t in held))
            plan._recorded.add(stream.cuda_stream)
    # autograd learns of the writes: a graph that saved the old weights refuses its backward pass
    params, _, masters = plan._held
    torch.autograd.graph.increment_version(
        [t for i, g in enumerate(grads) if g is not None for t in (params[i], masters[i]) if t is not None])
    if check:
        _call("device", read_device_status(ws, stream))
    return ws


class Muon:
    """Muon over the matrices of a model's hidden layers.

    params: matrices, or groups {"params": [...], "lr": ..., "weight_decay": ...}.  momentum,
    nesterov, steps, coefficients, eps, adjust: see ``muon_plan``.  master_weights: keep fp32 master
    weights for bf16 parameters; the next step overwrites what was written to such a parameter from
    outside.  Gradients are read from ``.grad`` (copied first where they are not contiguous); a
    parameter without one is left alone.
    """

    def __init__(self, params, lr=0.02, weight_decay=0.0, momentum=0.95, nesterov=True, steps=5,
                 coefficients=COEFFICIENTS, eps=1e-7, adjust="original", master_weights=True):
        torch = _torch()
        params = list(params)
        groups = params if params and isinstance(params[0], dict) else [{"params": params}]
        for g in groups:
            if not {"params"} <= set(g) <= {"params", "lr", "weight_decay"}:
                raise ValueError(f"a group is params, lr and weight_decay, got {sorted(g)}")
        self.groups = [{"lr": lr, "weight_decay": weight_decay, **g, "params": list(g["params"])} for g in groups]
        self.params = [p for g in self.groups for p in g["params"]]
        if len({id(p) for p in self.params}) != len(self.params):
            raise ValueError("a parameter appears twice")
        self.state = {"momentum": [torch.zeros(p.shape, dtype=torch.float32, device=p.device) for p in self.params],
                      "master": [p.detach().float().contiguous()
                                 if master_weights and p.dtype == torch.bfloat16 else None for p in self.params]}
        self.plan = muon_plan([p.detach() for p in self.params], self.state["momentum"], self.state["master"],
                              lr=self._per_param("lr"), weight_decay=self._per_param("weight_decay"),
                              momentum=momentum, nesterov=nesterov, steps=steps, coefficients=coefficients, eps=eps,
                              adjust=adjust)

    def _per_param(self, key):
        return [g[key] for g in self.groups for _ in g["params"]]

    def step(self, grad_scale=None, stream=None):
        """One step from the parameters' .grad (see muon_step), at the groups' present lr and
        weight_decay; without any gradient, none."""
        self.plan.set_lr(self._per_param("lr"))
        self.plan.set_weight_decay(self._per_param("weight_decay"))
        for i, p in enumerate(self.params):  # a parameter may have been given new storage
            if p.data_ptr() != self.plan.table[i].param:
                self.plan.set_param(i, p.detach())
        muon_step(self.plan, _contiguous([p.grad for p in self.params], stream), grad_scale, stream=stream)

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def state_dict(self):
        """The momenta and master weights; tensors are the optimizer's own."""
        return {"state": {k: list(v) for k, v in self.state.items()}}

    def load_state_dict(self, d):
        """Copies a state_dict of the same parameters and master weights in."""
        for k, mine in self.state.items():
            theirs = d["state"][k]
            if len(theirs) != len(mine) or any((a is None) != (b is None) or (a is not None and a.shape != b.shape)
                                               for a, b in zip(mine, theirs)):
                raise ValueError(f"{k} does not match this optimizer's parameters")
        for k, mine in self.state.items():
            for a, b in zip(mine, d["state"][k]):
                if a is not None:
                    a.copy_(b)
