"""The calls around the head run on the current device alone: tensors or a stream of another
one are refused on the host, before anything is allocated or launched.  Tensors that say they
are on a device stand in for those of a second GPU; no call gets as far as their memory."""
import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding, optim  # noqa: E402

H, V, N = 64, 100, 8
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


class On(torch.Tensor):
    """A CPU tensor that says it is on GPU `index`."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.index)

    def get_device(self):
        return self.index


def on(index, *shape, dtype=F32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.index = index
    return t


class Stream:
    cuda_stream = 0

    def __init__(self, index):
        self.device = torch.device("cuda", index)


def norm_forward(at, stream):
    return lambda: flce.layernorm_forward(on(at("x"), N, H), on(at("weight"), H), on(at("bias"), H), stream=stream)


def norm_backward(at, stream):
    return lambda: flce.layernorm_backward(on(at("dy"), N, H), on(at("x"), N, H), on(at("weight"), H),
                                           on(at("mean"), N), on(at("rstd"), N), ws=on(at("ws"), 64, dtype=torch.uint8),
                                           stream=stream)


def logprobs(at, stream):
    return lambda: flce.logprobs_forward(on(at("x"), N, H, dtype=BF16), on(at("w"), V, H, dtype=BF16),
                                         on(at("tokens"), N, dtype=I32), ws=on(at("ws"), 64, dtype=torch.uint8),
                                         stream=stream)


def logprobs_backward(at, stream):
    return lambda: flce.logprobs_backward(on(at("x"), N, H, dtype=BF16), on(at("w"), V, H, dtype=BF16),
                                          on(at("tokens"), N, dtype=I32), *(on(at(name), N) for name in
                                                                             ("lse", "entropy", "gl", "ge")),
                                          ws=on(at("ws"), 64, dtype=torch.uint8), stream=stream)


def adamw(at, stream):
    plan = flce.adamw_plan(*([on(at("x"), H)] for _ in range(3)))
    return lambda: flce.adamw_step(plan, [on(at("x"), H)], step=1, grad_scale=on(at("grad_scale"), 1), stream=stream)


CALLS = {norm_forward: ("weight", "bias"), norm_backward: ("dy", "weight", "mean", "rstd", "ws"),
         logprobs: ("w", "tokens", "ws"), logprobs_backward: ("w", "tokens", "lse", "entropy", "gl", "ge", "ws"),
         adamw: ("grad_scale",)}


@pytest.fixture
def current(monkeypatch):
    """GPU 0 is the current device, and the library is out of reach."""
    monkeypatch.setattr(binding, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(binding, "lib", lambda: pytest.fail("not refused"))
    monkeypatch.setattr(optim, "lib", lambda: pytest.fail("not refused"))
    for mod in (binding, optim):
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
    """The same stand-ins get as far as the library where the devices agree."""
    def reached():
        raise KeyError("library")

    for mod in (binding, optim):
        monkeypatch.setattr(mod, "lib", reached)
    binding.token_logprobs_workspace_bytes.cache_clear()
    with pytest.raises(KeyError):
        call(lambda which: 0, None)()
