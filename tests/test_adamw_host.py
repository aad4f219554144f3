"""The AdamW calls' own work on the host, on CPU tensors and with a stand-in for the library's
step (which writes nothing): what they tell autograd, what they hand to the step, and on what
they refuse to run.  With a GPU, the same through the step itself."""
import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import optim  # noqa: E402


class Steps:
    """Stands in for the library: keeps what each step was given."""

    def __init__(self):
        self.rows = []

    def flce_adamw_step(self, table, count, options, grad_scale, stream):
        self.rows.append([{name: getattr(table[i], name) for name, _ in table[i]._fields_} for i in range(count)])
        return 0


@pytest.fixture
def steps(monkeypatch):
    s = Steps()
    monkeypatch.setattr(optim, "lib", lambda: s)
    monkeypatch.setattr(optim, "_check", lambda *a, **k: None)  # (CPU tensors)
    monkeypatch.setattr(optim, "_check_device", lambda *a: None)
    monkeypatch.setattr(optim, "_stream_ptr", lambda *a: None)
    return s


def params(device="cpu"):
    return [torch.nn.Parameter(torch.linspace(-1, 1, n, device=device)) for n in (6, 5)]


def graphs_refuse(ps):
    """A step moves a weight that a graph has saved: its backward pass must not use the new one."""
    opt = flce.AdamW(ps, lr=0.1)
    losses = [(p * p).sum() for p in ps]
    ps[0].grad = torch.ones_like(ps[0])
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        losses[0].backward()
    losses[1].backward()  # no gradient: left alone
    assert torch.equal(ps[1].grad, 2 * ps[1].detach())


def test_graphs_of_old_weights_refuse_their_backward_pass(steps):
    graphs_refuse(params())


@pytest.mark.gpu
def test_graphs_of_old_weights_refuse_their_backward_pass_on_gpu():
    graphs_refuse(params("cuda"))


def test_master_weights_count_as_written(steps):
    w = torch.zeros(8, dtype=torch.bfloat16)
    master = torch.zeros(8, requires_grad=True)
    loss = (master * master).sum()
    plan = flce.adamw_plan([w], [torch.zeros(8)], [torch.zeros(8)], masters=[master])
    flce.adamw_step(plan, [torch.ones(8)], step=1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_a_schedule_of_lr_and_weight_decay_is_followed(steps):
    ps = params()
    opt = flce.AdamW([{"params": ps[:1]}, {"params": ps[1:], "weight_decay": 0.5}], lr=0.1, weight_decay=0.25)
    for p in ps:
        p.grad = torch.ones_like(p)
    opt.step()
    opt.groups[0]["lr"], opt.groups[1]["weight_decay"] = 0.5, 0.125
    opt.step()
    got = [[(r["lr"], r["weight_decay"]) for r in rows] for rows in steps.rows]
    tenth = float(torch.tensor(0.1))
    assert got == [[(tenth, 0.25), (tenth, 0.5)], [(0.5, 0.25), (tenth, 0.125)]]
    opt.plan.set_weight_decay(0.0)
    flce.adamw_step(opt.plan, [p.grad for p in ps], step=3)
    assert [r["weight_decay"] for r in steps.rows[-1]] == [0.0, 0.0]
    for set_one in (opt.plan.set_lr, opt.plan.set_weight_decay):
        with pytest.raises(ValueError):
            set_one([0.1])


@pytest.mark.gpu
def test_weight_decay_changed_between_steps():
    """Zero gradients from zero moments: only the decay moves a weight, by 1 - lr wd."""
    p = torch.nn.Parameter(torch.full((300,), 2.0, device="cuda"))
    opt = flce.AdamW([p], lr=0.5, weight_decay=0.5)
    p.grad = torch.zeros_like(p)
    opt.step()
    opt.groups[0]["weight_decay"] = 0.25
    opt.step()
    assert torch.equal(p.detach(), torch.full_like(p, 2.0 * 0.75 * 0.875))  # exact in fp32


class Recorded(torch.Tensor):
    """A CPU tensor that says it is on a GPU and keeps the streams its memory is recorded on."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = True

    def record_stream(self, stream):
        self.__dict__.setdefault("streams", []).append(stream)


class Stream:
    cuda_stream = 7


def test_a_foreign_stream_is_recorded_on_what_it_uses(steps):
    """Every step: the gradients and grad_scale; once: what the plan holds, and a parameter's
    new storage."""
    def make(n):
        return torch.zeros(n).as_subclass(Recorded)

    held = [make(6) for _ in range(4)]
    plan = flce.adamw_plan(held[:1], held[1:2], held[2:3], masters=held[3:])
    s = Stream()
    for k in range(2):
        grad, scale = make(6), make(1)
        flce.adamw_step(plan, [grad], step=k + 1, grad_scale=scale, stream=s)
        assert [t.streams for t in (grad, scale, *held)] == [[s]] * 6
    moved = make(6)
    plan.set_param(0, moved)
    flce.adamw_step(plan, [None], step=3, stream=s)
    assert moved.streams == [s]
    grad = make(6)
    flce.adamw_step(plan, [grad], step=4)  # the current stream
    assert not hasattr(grad, "streams")


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_freed_right_after_a_step_on_another_stream(bits):
    """The step waits on its stream while the caller frees the gradients and writes to memory
    of the same size: the weights are those of a step that was waited for."""
    n = 1 << 20
    g = torch.Generator().manual_seed(0)
    start, grad = torch.randn(n, generator=g).cuda(), torch.randn(n, generator=g).cuda()
    ends = []
    for early in (False, True):
        p = torch.nn.Parameter(start.clone())
        opt = flce.AdamW([p], lr=0.1, state_bits=bits)
        p.grad = grad.clone()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if early:
            with torch.cuda.stream(s):
                torch.cuda._sleep(20_000_000)  # about 10 ms
        opt.step(stream=s)
        if not early:
            s.synchronize()
        opt.zero_grad()
        for _ in range(4):
            torch.full((n,), 1e6, device="cuda")
        torch.cuda.synchronize()
        ends.append(p.detach().clone())
    assert torch.equal(*ends)


@pytest.mark.gpu
@pytest.mark.parametrize("foreign", [False, True])
def test_gradients_of_other_layouts_are_taken(foreign):
    """A transposed and an expanded gradient step as their contiguous copies do."""
    g = torch.Generator().manual_seed(0)
    start, grad = torch.randn(40, 24, generator=g).cuda(), torch.randn(24, 40, generator=g).cuda().t()
    row = torch.randn(24, generator=g).cuda().expand(40, 24)
    ends = []
    for copy in (True, False):
        ps = [torch.nn.Parameter(start.clone()) for _ in range(3)]
        opt = flce.AdamW(ps, lr=0.1)
        s = torch.cuda.Stream() if foreign else None
        for k, p in enumerate(ps[:2]):
            p.grad = (grad, row)[k].contiguous() if copy else (grad, row)[k]
            assert p.grad.is_contiguous() is copy
        if foreign:
            s.wait_stream(torch.cuda.current_stream())
        opt.step(stream=s)
        torch.cuda.synchronize()
        ends.append([p.detach().clone() for p in ps])
    for a, b in zip(*ends):
        assert torch.equal(a, b)
    assert torch.equal(ends[1][2], start)  # without a gradient
