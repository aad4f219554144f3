"""What the optimizers' steps do with memory that is not theirs (stand-ins as in test_ops_devices)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding, muon, optim  # noqa: E402
from test_ops_devices import Stream  # noqa: E402
from test_update_devices import Recorded  # noqa: E402


class Copied(Recorded):
    """One whose copies are stand-ins too."""

    def contiguous(self):
        return self if self.is_contiguous() else stand_in(*self.shape)


def stand_in(*shape):
    t = torch.zeros(*shape).as_subclass(Copied)
    t.index = 0
    return t


def optimizer(kind):
    """One over two matrices (its constructor allocates on their device)."""
    params = [stand_in(6, 4), stand_in(3, 5)]
    states = [[stand_in(*p.shape) for p in params] for _ in range(2)]
    opt = kind.__new__(kind)
    opt.groups = [{"params": params, "lr": 0.1, "weight_decay": 0.0}]
    opt.params, opt.steps = params, 0
    opt.plan = flce.muon_plan(params, states[0]) if kind is flce.Muon else flce.adamw_plan(params, *states)
    return opt


class Library:
    """One whose calls succeed and whose workspaces are 256 bytes."""

    def __getattr__(self, name):
        return lambda *a: 256 if name.endswith("bytes") else 0


@pytest.fixture
def fake(monkeypatch):
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    for mod in (binding, muon, optim):
        monkeypatch.setattr(mod, "lib", Library)
        monkeypatch.setattr(mod, "_stream_ptr", lambda *a: None)
        monkeypatch.setattr(mod, "_allocating", lambda s: contextlib.nullcontext())
    real = torch.empty

    def empty(*a, device=None, **k):
        t = real(*a, **k).as_subclass(Copied)
        t.index = 0
        return t
    monkeypatch.setattr(torch, "empty", empty)


@pytest.mark.parametrize("stream", [None, Stream(0)], ids=["current", "given"])
@pytest.mark.parametrize("kind", [flce.Muon, flce.AdamW], ids=lambda k: k.__name__)
def test_gradients_that_a_step_copies_are_recorded(fake, kind, stream):
    """The copy is made on the step's stream: what it reads may be freed after the call as well."""
    opt = optimizer(kind)
    opt.params[0].grad = stand_in(4, 6).t().as_subclass(Copied)
    opt.params[0].grad.index = 0
    opt.params[1].grad = stand_in(3, 5)
    grads = [p.grad for p in opt.params]
    assert not grads[0].is_contiguous()
    opt.step(stream=stream)
    for g in grads:
        assert getattr(g, "streams", []) == ([] if stream is None else [stream])
