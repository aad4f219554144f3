"""What the optimizers' steps do with memory that is not theirs (stand-ins as in test_ops_devices)."""
import contextlib
import ctypes
import os
import random
import subprocess
import sys

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


def step_bytes(shapes):
    table = (binding.MuonTensor * max(len(shapes), 1))()
    for row, (r, c) in zip(table, shapes):
        row.rows, row.cols = r, c
    return binding.lib().flce_muon_workspace_bytes(table, len(shapes))


def call_bytes(shapes):
    """What exactly these need: orthogonalize's rounds are the same."""
    table = (binding.Matrix * max(len(shapes), 1))(*((1, 1, r, c, 0) for r, c in shapes))
    return binding.lib().flce_orthogonalize_workspace_bytes(table, len(shapes))


def test_a_workspace_is_enough_where_gradients_are_missing():
    """Rounds are cut anew: without the first 200 the others share one, which all of them do not."""
    shapes = [(300, 310)] * 200 + [(299, 8000)] * 200
    assert call_bytes(shapes[200:]) > call_bytes(shapes)
    assert step_bytes(shapes) >= call_bytes(shapes[200:])
    rng = random.Random(0)
    for _ in range(40):
        kinds = [(rng.randint(1, 900), rng.choice([rng.randint(1, 900), rng.randint(1, 90000)])) for _ in range(rng.randint(1, 30))]
        shapes = [rng.choice(kinds) for _ in range(rng.randint(1, 700))]
        most = step_bytes(shapes)
        assert most >= call_bytes(shapes)
        for _ in range(30):
            some = set(rng.sample(kinds, rng.randint(1, len(kinds))))
            part = rng.random()
            live = [s for s in shapes if s in some or rng.random() < part]
            assert call_bytes(live) <= most
            assert step_bytes([s if s in some else (0, 0) for s in shapes]) <= most


def test_a_workspace_of_one_round_is_what_it_takes():
    for shapes in ([(300, 310)] * 200, [(64, 64), (4096, 4096), (5, 9000)], [(3, 0)], []):
        assert step_bytes(shapes) == call_bytes(shapes)


@pytest.mark.gpu
def test_a_step_without_some_gradients_in_the_plans_workspace():
    """18 shapes, 12 of a round: the last 12 share one only where the first have no gradient."""
    shapes = [(300 + i, 310) for i in range(6)] + [(200, 1000 + 8 * i) for i in range(12)]
    assert call_bytes(shapes[6:]) > call_bytes(shapes)
    g = torch.Generator().manual_seed(0)
    gs = [None if i < 6 else torch.randn(s, generator=g).cuda() for i, s in enumerate(shapes)]
    results = []
    for given in (True, False):
        ps, ms = ([torch.zeros(s, device="cuda") for s in shapes] for _ in range(2))
        plan = flce.muon_plan(ps, ms)
        ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda") if given else None
        flce.muon_step(plan, gs, ws=ws, check=True)
        results.append(ps + ms)
    assert all(torch.equal(a, b) for a, b in zip(*results))


def cut(base, at, *shape, dtype=None):
    """A view of base's memory from element `at` on."""
    n = shape[0] * shape[1]
    t = base.view(-1)[at:at + n].view(shape)
    t = (t if dtype is None else t.view(dtype)).as_subclass(Copied)
    t.index = 0
    return t


def test_overlapping_memory_is_refused_by_name():
    base = torch.zeros(64)
    p, m = cut(base, 0, 4, 6), cut(base, 24, 4, 6)
    flce.muon_plan([p], [m])
    for first, second in ((cut(base, 23, 4, 6), p), (p, cut(base, 23, 4, 6))):
        with pytest.raises(ValueError, match="overlap"):
            flce.muon_plan([first], [second])
    with pytest.raises(ValueError, match="overlap"):
        flce.muon_plan([p, cut(base, 8, 2, 3)], [m, cut(base, 50, 2, 3)])


def test_outputs_over_other_inputs_are_refused(fake):
    base = torch.zeros(256, dtype=torch.bfloat16)
    a, b, c = (cut(base, 32 * i, 4, 6) for i in range(3))
    for x, out in (([a, b], [b, a]), ([a, b], [c, cut(base, 8, 4, 6)]), ([a, b], [a, cut(base, 33, 4, 6)]),
                   ([a], [cut(base, 1, 4, 6)]), ([a, a], [a, c])):
        with pytest.raises(ValueError, match="overlap"):
            flce.orthogonalize(x, out=out)
    for x, out in (([a, b], [a, b]), ([a, b], [a, c]), ([a, a], [b, c])):
        flce.orthogonalize(x, out=out)


@pytest.mark.skipif(torch.cuda.is_available(), reason="addresses of nothing")
def test_the_library_refuses_overlapping_memory():
    """A call that is not refused gets as far as the device, which is missing (7)."""
    L, o = binding.lib(), ctypes.byref(muon._options(0.9, True, 5, muon.COEFFICIENTS, 1e-7))
    size = 8 * 8

    def ortho(*rows, ws=0x1000000, nbytes=1 << 20):  # (x, out, dtype)
        table = (binding.Matrix * len(rows))(*((x, out, 8, 8, code) for x, out, code in rows))
        return L.flce_orthogonalize(table, len(rows), o, ws, nbytes, None)
    x, y = 0x10000, 0x20000
    assert ortho((x, y, 0)) == ortho((x, x, 0)) == ortho((x, x + 2 * size, 0)) == ortho((x, y, 0), (x, y + 2 * size, 0)) == 7
    for rows in ([(x, x + 2, 0)], [(x, x + 2 * size - 2, 0)], [(x, x, 1)], [(x, y, 0), (y, x, 0)], [(x, y, 0), (x + 512, y + 2, 0)],
                 [(x, x, 0), (x, y, 0)], [(x, 0x1000100, 0)], [(0x1000100, y, 0)]):
        assert ortho(*rows) == 1, rows
    # addresses past what a call needs of a larger workspace are nobody's
    assert ortho((x, 0x1000000 + (1 << 19), 0)) == 7

    def step(gs=None, **over):
        row = dict(param=0x10000, grad=0x20000, master=0x30000, momentum=0x40000, rows=8, cols=8, lr=0.1, weight_decay=0.0,
                   scale=1.0, param_dtype=0, grad_dtype=0)
        table = (binding.MuonTensor * 1)(tuple({**row, **over}.values()))
        return L.flce_muon_step(table, 1, o, gs, 0x1000000, 1 << 20, None)
    assert step() == step(master=None) == step(grad=0x10080) == step(gs=0x20000) == step(gs=0x10080) == 7
    for over in (dict(grad=0x10000), dict(grad=0x1007e), dict(momentum=0x10040), dict(master=0x400fc), dict(master=0x10000),
                 dict(grad=0x40080), dict(momentum=0x1000000), dict(gs=0x1007c), dict(gs=0x40000)):
        assert step(**over) == 1, over


CHILD = """
import ctypes, resource
import lm_head_cross_gb300 as flce
from lm_head_cross_gb300 import binding, muon
L, o, n = binding.lib(), muon._options(0.9, True, 5, muon.COEFFICIENTS, 1e-7), 1 << 20
matrices, tensors = (binding.Matrix * n)(), (binding.MuonTensor * n)()
size = int(open("/proc/self/statm").read().split()[0]) * resource.getpagesize()
resource.setrlimit(resource.RLIMIT_AS, (size + (32 << 20), resource.getrlimit(resource.RLIMIT_AS)[1]))
print(L.flce_orthogonalize(matrices, n, ctypes.byref(o), 0x1000000, 256, None),
      L.flce_muon_step(tensors, n, ctypes.byref(o), None, 0x1000000, 256, None),
      L.flce_muon_workspace_bytes(tensors, n), binding.status_string(11))
"""


@pytest.mark.skipif(torch.cuda.is_available(), reason="where an allocation does not fail the call ends at the missing device")
def test_host_memory_that_is_missing_is_a_status():
    r = subprocess.run([sys.executable, "-c", CHILD], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr
    assert r.stdout.startswith("11 11 0 host memory"), r.stdout


@pytest.mark.skipif(torch.cuda.is_available(), reason="memory of the host")
def test_parameters_that_came_to_share_memory_are_refused(monkeypatch):
    """New storage is looked at by the step: two parameters that were tied after the plan was made."""
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(muon, "_stream_ptr", lambda *a: None)
    base = torch.zeros(96)
    plan = flce.muon_plan([cut(base, 0, 4, 6), cut(base, 24, 4, 6)], [stand_in(4, 6), stand_in(4, 6)])
    room = torch.zeros(plan.workspace_bytes() + 256, dtype=torch.uint8)
    ws = room[-room.data_ptr() % 256:].as_subclass(Copied)
    ws.index = 0
    for second, code in ((cut(base, 48, 4, 6), 7), (cut(base, 12, 4, 6), 1), (cut(base, 0, 4, 6), 1)):
        plan.set_param(1, second)
        with pytest.raises(flce.FlceError) as e:
            flce.muon_step(plan, [stand_in(4, 6), stand_in(4, 6)], ws=ws)
        assert e.value.code == code
