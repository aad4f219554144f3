"""AdamW over many tensors, one launch for each 400 of them (flce_adamw_step).

``adamw_plan`` describes the tensors once (parameters, moments, optional fp32 master
weights); ``adamw_step`` takes one step with the current gradients.  ``AdamW`` is the
optimizer object on top of both: it owns the moments and the step count.
"""
from __future__ import annotations

import ctypes

from .binding import AdamwOptions, AdamwTensor, _allocating, _call, _check_device, _record, _stream_ptr, _torch, lib

BLOCK = 256  # elements that share one scale of an 8-bit moment


def _dtype_code(t, name):
    torch = _torch()
    if t.dtype is torch.float32:
        return 1
    if t.dtype is torch.bfloat16:
        return 0
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _check(t, name, like=None, dtype=None, count=None):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    want = like.numel() if count is None else count
    if t.numel() != want:
        raise ValueError(f"{name} must have {want} elements, got {t.numel()}")


def _contiguous(grads, stream):
    """The gradients, those of other layouts copied on the step's stream.  That stream reads what it
    copies, so they are recorded on it too."""
    if all(g is None or g.is_contiguous() for g in grads):
        return grads
    with _allocating(stream):
        copies = [None if g is None else g.contiguous() for g in grads]
    _record(stream, *(g for g, c in zip(grads, copies) if c is not g))
    return copies


class AdamWPlan:
    """The tensors of an AdamW step and its hyperparameters (see ``adamw_plan``)."""

    def __init__(self, params, exp_avgs, exp_avg_sqs, masters, scales, lr, betas, eps, weight_decay):
        torch = _torch()
        n = len(params)
        self.state_bits = 32 if scales is None else 8
        masters = [None] * n if masters is None else list(masters)
        m_scales, v_scales = ([None] * n, [None] * n) if scales is None else (list(scales[0]), list(scales[1]))
        lists = (exp_avgs, exp_avg_sqs, masters, m_scales, v_scales)
        if any(len(x) != n for x in lists):
            raise ValueError("one entry per parameter is needed in every list")
        lrs = list(lr) if isinstance(lr, (list, tuple)) else [lr] * n
        wds = list(weight_decay) if isinstance(weight_decay, (list, tuple)) else [weight_decay] * n
        if len(lrs) != n or len(wds) != n:
            raise ValueError("lr and weight_decay are numbers, or one number per parameter")
        state = torch.float32 if scales is None else torch.float8_e4m3fn
        self.table = (AdamwTensor * max(n, 1))()
        self.numels = [p.numel() for p in params]
        self.device = params[0].device if n else None
        for i, p in enumerate(params):
            _check(p, f"params[{i}]", p)
            code = _dtype_code(p, f"params[{i}]")
            _check(exp_avgs[i], f"exp_avgs[{i}]", p, state)
            _check(exp_avg_sqs[i], f"exp_avg_sqs[{i}]", p, state)
            if masters[i] is not None:
                _check(masters[i], f"masters[{i}]", p, torch.float32)
            if scales is not None:
                blocks = (p.numel() + BLOCK - 1) // BLOCK
                _check(m_scales[i], f"scales[0][{i}]", dtype=torch.float32, count=blocks)
                _check(v_scales[i], f"scales[1][{i}]", dtype=torch.float32, count=blocks)
            for t in (p, exp_avgs[i], exp_avg_sqs[i], masters[i], m_scales[i], v_scales[i]):
                if t is not None and t.device != self.device:
                    raise ValueError("all tensors of a plan must be on one device")
            ptr = [None if t is None else t.data_ptr()
                   for t in (p, None, masters[i], exp_avgs[i], exp_avg_sqs[i], m_scales[i], v_scales[i])]
            self.table[i] = AdamwTensor(*ptr, p.numel(), lrs[i], wds[i], code, 0)
        self.options = AdamwOptions(betas[0], betas[1], eps, 1, self.state_bits)
        self._held = (list(params), *(list(x) for x in lists))  # the table holds their addresses
        self._recorded = set()  # streams that _held's memory is known to be used on

    def __len__(self):
        return len(self.numels)

    def set_param(self, i, p):
        """Parameter i now lives in ``p`` (same dtype and size)."""
        old = self._held[0][i]
        _check(p, f"params[{i}]", old, old.dtype)
        if p.device != self.device:
            raise ValueError("all tensors of a plan must be on one device")
        self._held[0][i] = p
        self.table[i].param = p.data_ptr()
        self._recorded.clear()

    def set_lr(self, lr):
        """A number for every tensor, or one number per tensor, used from the next step on."""
        self._set("lr", lr)

    def set_weight_decay(self, weight_decay):
        """A number for every tensor, or one number per tensor, used from the next step on."""
        self._set("weight_decay", weight_decay)

    def _set(self, name, value):
        values = list(value) if isinstance(value, (list, tuple)) else [value] * len(self)
        if len(values) != len(self):
            raise ValueError(f"{name} is a number, or one number per parameter")
        for i, v in enumerate(values):
            setattr(self.table[i], name, v)


def adamw_plan(params, exp_avgs, exp_avg_sqs, masters=None, scales=None, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
               weight_decay=1e-2):
    """Describes the tensors of an AdamW step.  Lists of contiguous CUDA tensors, one entry per
    parameter: params (bf16 or fp32), moments (fp32; or float8_e4m3fn with ``scales`` = (lists of
    fp32 scales of the first, of the second moment), one scale per 256 elements, the second moment
    as its square root), masters (fp32 master weights; an entry, or the list, may be None).  lr and
    weight_decay: a number, or a list of one number per parameter."""
    return AdamWPlan(params, exp_avgs, exp_avg_sqs, masters, scales, lr, betas, eps, weight_decay)


def adamw_step(plan, grads, step, grad_scale=None, stream=None):
    """One step (number ``step``, from 1) in place.  grads: one contiguous bf16 or fp32 CUDA tensor
    per parameter, or None for a parameter that is left alone.  grad_scale: a one-element fp32 CUDA
    tensor that multiplies every gradient (clipping, loss scaling).  stream: the torch stream to
    run on, else the current one; the tensors may be freed once the call has returned."""
    torch = _torch()
    if len(grads) != len(plan):
        raise ValueError(f"{len(plan)} gradients are needed, got {len(grads)}")
    table, f32, b16 = plan.table, torch.float32, torch.bfloat16
    for i, g in enumerate(grads):
        row = table[i]
        if g is None:
            row.count = 0
            continue
        if g.dtype is not f32 and g.dtype is not b16:
            raise TypeError(f"grads[{i}] must be bfloat16 or float32, got {g.dtype}")
        if g.numel() != plan.numels[i] or not g.is_contiguous() or g.device != plan.device:
            raise ValueError(f"grads[{i}] must be contiguous, on the plan's device, with the parameter's elements")
        row.grad = g.data_ptr()
        row.grad_dtype = 1 if g.dtype is f32 else 0
        row.count = plan.numels[i]
    if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1
                                   or not grad_scale.is_cuda):
        raise ValueError("grad_scale must be a one-element fp32 CUDA tensor")
    device = _check_device(plan._held[0][0], stream, grad_scale) if len(plan) else None
    plan.options.step = int(step)
    _call("flce_adamw_step", lib().flce_adamw_step(
        table, len(plan), ctypes.byref(plan.options), None if grad_scale is None else grad_scale.data_ptr(),
        _stream_ptr(stream, device)))
    if stream is not None:  # what is freed after the call is reused only once the stream is done with it
        used = [*grads, grad_scale]
        if stream.cuda_stream not in plan._recorded:
            used += [t for held in plan._held for t in held]
            plan._recorded.add(stream.cuda_stream)
        for t in used:
            if t is not None:
                t.record_stream(stream)
    # autograd learns of the writes: a graph that saved the old weights refuses its backward pass
    params, masters = plan._held[0], plan._held[3]
    torch.autograd.graph.increment_version(
        [t for i, g in enumerate(grads) if g is not None for t in (params[i], masters[i]) if t is not None])


class AdamW:
    """AdamW with moments in 32 or 8 bits, one launch for each 400 parameters.

    params: tensors, or groups {"params": [...], "lr": ..., "weight_decay": ...}.  state_bits 32
    or 8.  master_weights: keep fp32 master weights for bf16 parameters (their own rounding
    would swallow updates smaller than 2^-9 of a weight); the next step overwrites what was
    written to such a parameter from outside.  Gradients are read from ``.grad`` (copied first
    where they are not contiguous); a parameter without one is left alone.
    """

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=1e-2, state_bits=32,
                 master_weights=True):
        torch = _torch()
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32")
        params = list(params)
        groups = params if params and isinstance(params[0], dict) else [{"params": params}]
        self.groups = [{"lr": lr, "weight_decay": weight_decay, **g, "params": list(g["params"])} for g in groups]
        self.params = [p for g in self.groups for p in g["params"]]
        if len({id(p) for p in self.params}) != len(self.params):
            raise ValueError("a parameter appears twice")
        self.betas, self.eps, self.state_bits, self.steps = tuple(betas), eps, state_bits, 0
        self.state = {"exp_avg": [], "exp_avg_sq": [], "exp_avg_scale": [], "exp_avg_sq_scale": [], "master": []}
        kind = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        for p in self.params:
            blocks = (p.numel() + BLOCK - 1) // BLOCK
            for name in ("exp_avg", "exp_avg_sq"):
                self.state[name].append(torch.zeros(p.numel(), dtype=torch.float32 if state_bits == 32 else torch.uint8,
                                                    device=p.device).view(kind))
                if state_bits == 8:
                    self.state[name + "_scale"].append(torch.zeros(blocks, dtype=torch.float32, device=p.device))
            keep = master_weights and p.dtype == torch.bfloat16
            self.state["master"].append(p.detach().float().contiguous() if keep else None)
        s = self.state
        self.plan = adamw_plan([p.detach() for p in self.params], s["exp_avg"], s["exp_avg_sq"], s["master"],
                               None if state_bits == 32 else (s["exp_avg_scale"], s["exp_avg_sq_scale"]),
                               lr=self._per_param("lr"), betas=self.betas, eps=eps,
                               weight_decay=self._per_param("weight_decay"))

    def _per_param(self, key):
        return [g[key] for g in self.groups for _ in g["params"]]

    def step(self, grad_scale=None, stream=None):
        """One step from the parameters' .grad (see adamw_step), at the groups' present lr and
        weight_decay; without any gradient, none."""
        self.plan.set_lr(self._per_param("lr"))
        self.plan.set_weight_decay(self._per_param("weight_decay"))
        for i, p in enumerate(self.params):  # a parameter may have been given new storage
            if p.data_ptr() != self.plan.table[i].param:
                self.plan.set_param(i, p.detach())
        grads = [p.grad for p in self.params]
        if all(g is None for g in grads):
            return
        adamw_step(self.plan, _contiguous(grads, stream), self.steps + 1, grad_scale, stream)
        self.steps += 1

    def zero_grad(self):
        for p in self.params:
            p.grad = None

    def state_dict(self):
        """The moments, master weights and step count; tensors are the optimizer's own."""
        return {"steps": self.steps, "state_bits": self.state_bits, "state": {k: list(v) for k, v in self.state.items()}}

    def load_state_dict(self, d):
        """Copies a state_dict of the same parameters, state_bits and master weights in."""
        torch = _torch()
        if d["state_bits"] != self.state_bits:
            raise ValueError(f"state of {d['state_bits']} bits for an optimizer of {self.state_bits}")
        for k, mine in self.state.items():
            theirs = d["state"][k]
            if len(theirs) != len(mine) or any((a is None) != (b is None) or (a is not None and a.shape != b.shape)
                                               for a, b in zip(mine, theirs)):
                raise ValueError(f"{k} does not match this optimizer's parameters")
        for k, mine in self.state.items():
            for a, b in zip(mine, d["state"][k]):
                if a is not None:
                    (a.view(torch.uint8) if a.dtype == torch.float8_e4m3fn else a).copy_(
                        b.view(torch.uint8) if b.dtype == torch.float8_e4m3fn else b)
        self.steps = int(d["steps"])
