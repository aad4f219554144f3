"""The embedding's and Muon's calls run on the current device alone, like the others around the
head: tensors or a stream of another one are refused on the host (stand-ins as in
test_ops_devices)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding, muon  # noqa: E402
from test_ops_devices import BF16, F32, I32, H, N, On, Stream, V, on  # noqa: E402

U8 = torch.uint8


def embed(at, stream):
    return lambda: flce.embedding_forward(on(at("ids"), N, dtype=I32), on(at("weight"), V, H, dtype=BF16),
                                          ws=on(at("ws"), 256, dtype=U8), stream=stream)


def embed_backward(at, stream):
    return lambda: flce.embedding_backward(on(at("dy"), N, H), on(at("ids"), N, dtype=I32), V, add_to=on(at("add_to"), V, H),
                                           ws=on(at("ws"), 256, dtype=U8), stream=stream)


def orthogonalize(at, stream):
    return lambda: flce.orthogonalize([on(at("x"), H, H), on(at("second"), N, H)], ws=on(at("ws"), 256, dtype=U8),
                                      out=[on(at("out"), H, H, dtype=BF16), on(at("second_out"), N, H, dtype=BF16)],
                                      stream=stream)


def muon_step(at, stream):
    plan = flce.muon_plan([on(at("x"), H, H)], [on(at("x"), H, H)])
    return lambda: flce.muon_step(plan, [on(at("x"), H, H)], grad_scale=on(at("grad_scale"), 1),
                                  ws=on(at("ws"), 256, dtype=U8), stream=stream)


CALLS = {embed: ("ids", "ws"), embed_backward: ("ids", "add_to", "ws"), orthogonalize: ("second", "out", "second_out", "ws"),
         muon_step: ("grad_scale", "ws")}


@pytest.fixture
def current(monkeypatch):
    """GPU 0 is the current device, and the library is out of reach."""
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    for mod in (binding, muon):
        monkeypatch.setattr(mod, "lib", lambda: pytest.fail("not refused"))
        monkeypatch.setattr(mod, "_stream_ptr", lambda *a: None)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))


@pytest.mark.parametrize("call,name", [(c, n) for c, names in CALLS.items() for n in names],
                         ids=lambda v: v if isinstance(v, str) else v.__name__)
def test_a_tensor_of_another_device_is_refused(current, call, name):
    with pytest.raises(ValueError, match="one device"):
        call(lambda which: 1 if which == name else 0, None)()


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_a_device_that_is_not_current_is_refused(current, call):
    with pytest.raises(ValueError, match="current device"):
        call(lambda which: 1, None)()


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_a_stream_of_another_device_is_refused(current, call):
    with pytest.raises(ValueError, match="stream"):
        call(lambda which: 0, Stream(1))()


@pytest.mark.parametrize("call", CALLS, ids=lambda c: c.__name__)
def test_the_current_device_is_taken(current, monkeypatch, call):
    def reached():
        raise KeyError("library")

    for mod in (binding, muon):
        monkeypatch.setattr(mod, "lib", reached)
    with pytest.raises(KeyError):
        call(lambda which: 0, None)()


class Recorded(On):
    """One that keeps the streams its memory is recorded on."""

    def record_stream(self, stream):
        self.__dict__.setdefault("streams", []).append(stream)


def recorded(*shape, dtype=F32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(Recorded)
    t.index = 0
    return t


@pytest.mark.parametrize("stream", [None, Stream(0)], ids=["current", "given"])
def test_a_given_stream_is_recorded_on_what_it_uses(current, monkeypatch, stream):
    """What is freed after a call on another stream than its own must not be reused before its end."""
    class Library:
        def __getattr__(self, name):
            return lambda *a: 0

    for mod in (binding, muon):
        monkeypatch.setattr(mod, "lib", Library)
        monkeypatch.setattr(mod, "_allocating", lambda s: contextlib.nullcontext())
    ids, w, dy, dw, ws, x, y, g, m, p, gs = used = [
        recorded(N, dtype=I32), recorded(V, H), recorded(N, H), recorded(V, H), recorded(256, dtype=U8), recorded(H, H),
        recorded(H, H, dtype=BF16), *(recorded(H, H) for _ in range(3)), recorded(1)]
    new = flce.embedding_forward(ids, w, ws=ws, stream=stream)[0]
    flce.embedding_backward(dy, ids, V, add_to=dw, ws=ws, stream=stream)
    flce.orthogonalize([x], out=[y], ws=ws, stream=stream)
    flce.muon_step(flce.muon_plan([p], [m]), [g], grad_scale=gs, ws=ws, stream=stream)
    for t in used:
        assert bool(getattr(t, "streams", None)) == (stream is not None)
        assert all(s is stream for s in getattr(t, "streams", []))
    assert not hasattr(new, "streams")  # (allocated on it)


def test_gradients_of_another_device_are_refused(current):
    plan = flce.muon_plan([on(0, H, H)], [on(0, H, H)])
    with pytest.raises(ValueError, match="plan's device"):
        flce.muon_step(plan, [on(1, H, H)])
    with pytest.raises(ValueError, match="one device"):
        flce.muon_plan([on(0, H, H), on(1, H, H)], [on(0, H, H), on(1, H, H)])
