"""AdamW: the kernels against the formulas in 64 bits, at sizes, types, alignments and
values where they can go wrong, and the calls they refuse.

Tolerances (u = 2^-24).  m and v are sums of two rounded products: 4 u of the sum of
their magnitudes.  The update m / (sqrt(v) c + eps) adds the errors of a root, a
product, a sum and a quotient, some of them by hardware approximations good to 2^-22:
32 u of itself, besides m's and half of v's own; p adds 3 u |p|; bf16 half an ulp
(2^-8).  An e4m3 value is off by half a step when rounded to nearest, by less than one
step when dithered; a step is 2^(e - 3) at exponent e, at least 2^-9.
"""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding  # noqa: E402

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
HYPER = dict(lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)


def rounding_bytes(count, step):
    """The byte that dithers each element's second moment in this step."""
    i = np.arange(count, dtype=np.uint64)
    mask, k = np.uint64(0xFFFFFFFF), np.uint64(0x9E3779B1)
    h = ((i >> np.uint64(2)) * k + np.uint64(step * 0xA511E9B3 & 0xFFFFFFFF)) & mask
    h = ((h ^ (h >> np.uint64(16))) * k) & mask
    h = ((h ^ (h >> np.uint64(13))) * k) & mask
    h ^= h >> np.uint64(16)
    return ((h >> (np.uint64(8) * (i & np.uint64(3)))) & np.uint64(0xFF)).astype(np.float64)


def step64(p, g, m, v, step, gs=1.0, lr=3e-3, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1):
    """The formulas, in 64 bits; returns the new values and the tolerances of fp32 ones."""
    b1, b2 = betas
    p, g, m0, v0 = (np.asarray(t, np.float64) for t in (p, g, m, v))
    g = g * gs
    m = b1 * m0 + (1 - b1) * g
    v = b2 * v0 + (1 - b2) * g * g
    em = 4 * U * (np.abs(b1 * m0) + np.abs((1 - b1) * g)) + 1e-45
    ev = 5 * U * v + 1e-44
    c1, c2 = 1 - b1 ** step, 1 - b2 ** step
    den = np.sqrt(v / c2) + eps
    upd = lr / c1 * m / den
    q = p * (1 - lr * weight_decay) - upd
    e_upd = lr / c1 * em / den + np.abs(upd) * (32 * U + np.where(v > 1e-37, 0.5 * ev / np.maximum(v, 1e-300), 1.0))
    return dict(p=q, m=m, v=v, em=em, ev=ev, ep=e_upd + 3 * U * (np.abs(p) + np.abs(q)))


def e4m3_step(q):
    return np.maximum(2.0 ** -9, 2.0 ** (np.floor(np.log2(np.maximum(np.abs(q), 2.0 ** -9))) - 3))


def blocks(x, fill=0.0):
    n = len(x)
    pad = np.full(-n % 256, fill)
    return np.concatenate([x, pad]).reshape(-1, 256)


class Tensors:
    """One parameter with everything its step needs, on the GPU, optionally one element
    past a vector boundary."""

    def __init__(self, count, dtype=BF16, gdtype=BF16, master=True, bits=32, seed=0, shift=0):
        g = torch.Generator().manual_seed(seed)
        self.count, self.bits, self.shift = count, bits, shift
        w = 0.02 * torch.randn(count, generator=g)
        self.master = self.place(w) if master and dtype == BF16 else None
        self.param = self.place(w.to(dtype))
        self.grad = self.place((1e-3 * torch.randn(count, generator=g) * torch.rand(count, generator=g)).to(gdtype))
        m = 3e-4 * torch.randn(count, generator=g)
        r = 1e-3 * torch.rand(count, generator=g) + 1e-6
        self.m_scale = self.v_scale = None
        if bits == 32:
            self.m, self.v = self.place(m), self.place(r.square())
        else:
            self.m, self.m_scale = self.encode(m)
            self.v, self.v_scale = self.encode(r)

    def place(self, t):
        t = t.cuda()
        return torch.cat([t.new_zeros(self.shift), t])[self.shift:] if self.shift else t

    def encode(self, t):
        b = torch.nn.functional.pad(t, (0, -t.numel() % 256)).view(-1, 256)
        s = b.abs().amax(1) / 448
        q = (b / s.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)[:t.numel()]
        return self.place(q.view(torch.uint8)).view(torch.float8_e4m3fn), s.cuda()

    def moments(self):
        """m and v (not its root) in 64 bits."""
        if self.bits == 32:
            return self.m.double().cpu().numpy(), self.v.double().cpu().numpy()
        out = []
        for q, s in ((self.m, self.m_scale), (self.v, self.v_scale)):
            out.append((blocks(q.cpu().float().double().numpy()) * s.double().cpu().numpy()[:, None])
                       .reshape(-1)[:self.count])
        return out[0], out[1] ** 2

    def start(self):
        w = self.master if self.master is not None else self.param
        return w.double().cpu().numpy(), self.grad.double().cpu().numpy(), *self.moments()


def plan_of(ts, **over):
    scales = None if ts[0].bits == 32 else ([t.m_scale for t in ts], [t.v_scale for t in ts])
    return flce.adamw_plan([t.param for t in ts], [t.m for t in ts], [t.v for t in ts],
                           masters=[t.master for t in ts], scales=scales, **{**HYPER, **over})


def within(got, want, tol, name):
    got = got.double().cpu().numpy() if torch.is_tensor(got) else got
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), f"{name}: {bad.sum()} of {bad.size} outside, worst {np.nanmax(np.abs(got - want)):.3e}"


def check(t, before, step, gs=1.0, **over):
    ref = step64(*before, step, gs, **{**HYPER, **over})
    if t.master is not None:
        within(t.master, ref["p"], ref["ep"], "master")
        assert torch.equal(t.param, t.master.to(t.param.dtype))
    else:
        half = np.abs(ref["p"]) * 2.0 ** -8 if t.param.dtype == BF16 else 0.0
        within(t.param, ref["p"], ref["ep"] * (1 + 2.0 ** -8) + half, "param")
    if t.bits == 32:
        within(t.m, ref["m"], ref["em"], "m")
        within(t.v, ref["v"], ref["ev"], "v")
        return
    r = np.sqrt(ref["v"])
    rnd = rounding_bytes(t.count, step)
    for name, x, q, s in (("m", ref["m"], t.m, t.m_scale), ("r", r, t.v, t.v_scale)):
        top = np.abs(blocks(x)).max(1)
        # the largest magnitude is one of fp32 values that are each a few u off
        within(s, top / 448, 12 * U * top / 448 + 1e-44, name + " scale")
        scale = np.repeat(s.double().cpu().numpy(), 256)[:t.count]
        exact = x / np.where(scale > 0, scale, 1.0)
        code = q.cpu().view(torch.uint8).numpy()
        value = q.cpu().float().double().numpy()
        step8 = e4m3_step(exact)
        if name == "m":
            within(value, exact, 0.5 * step8 * (1 + 1e-4) + 1e-4 * np.abs(exact), "m")
            continue
        assert (value[exact > 0] > 0).all()
        within(value, exact, np.maximum(step8 * (1 + 1e-4), np.where(exact < 2.0 ** -9, 2.0 ** -9, 0)), "r")
        # where the fraction of a step is not within rounding of the threshold, the value is known
        low = np.floor(np.clip(exact, 0, 448) / step8) * step8
        frac = (np.clip(exact, 0, 448) - low) / step8
        # (a value at a grid point may lie a rounding below it, where byte 0 takes it down)
        clear = (np.abs(frac + rnd / 256 - 1) > 1e-3) & (frac > 1e-3)
        want = np.maximum(low + step8 * (frac + rnd / 256 >= 1), np.where(exact > 0, 2.0 ** -9, 0))
        assert clear.mean() > 0.98 or t.count < 500
        np.testing.assert_array_equal(value[clear], want[clear])
        assert (code < 0x7F).all()


SIZES = [1, 7, 8, 255, 256, 257, 4095, 4096, 4097, 5003, 300001]
KINDS = [(BF16, BF16, True), (BF16, F32, True), (BF16, BF16, False), (F32, F32, False), (F32, BF16, False)]


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,gdtype,master", KINDS)
@pytest.mark.parametrize("shift", [0, 1])
def test_one_step_of_every_size(bits, dtype, gdtype, master, shift):
    """All sizes in one call; with shift, every tensor starts one element past a vector
    boundary."""
    ts = [Tensors(n, dtype, gdtype, master, bits, seed=n, shift=shift) for n in SIZES]
    before = [t.start() for t in ts]
    gs = torch.tensor([0.5], device="cuda")
    flce.adamw_step(plan_of(ts), [t.grad for t in ts], step=7, grad_scale=gs)
    for t, b in zip(ts, before):
        check(t, b, 7, gs=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    """950 tensors of many sizes and types, some without a gradient, a few empty."""
    rng = np.random.default_rng(5)
    ts = [Tensors(0 if i % 97 == 5 else int(rng.integers(1, 3000)), *KINDS[i % len(KINDS)], bits, seed=i)
          for i in range(950)]
    before = [t.start() for t in ts]
    grads = [None if i % 50 == 3 else t.grad for i, t in enumerate(ts)]
    held = [t.param.clone() for t in ts]
    flce.adamw_step(plan_of(ts), grads, step=1)
    for i, (t, b) in enumerate(zip(ts, before)):
        if grads[i] is None:
            assert torch.equal(t.param, held[i])
        elif t.count:
            check(t, b, 1)


@pytest.mark.gpu
def test_per_tensor_rates_and_other_hyperparameters():
    ts = [Tensors(5000, F32, F32, seed=i) for i in range(3)]
    before = [t.start() for t in ts]
    lrs, wds = [1e-2, 0.0, 1e-4], [0.0, 0.5, 0.01]
    over = dict(betas=(0.0, 0.999), eps=1e-3)
    flce.adamw_step(plan_of(ts, lr=lrs, weight_decay=wds, **over), [t.grad for t in ts], step=123456)
    for t, b, lr, wd in zip(ts, before, lrs, wds):
        check(t, b, 123456, lr=lr, weight_decay=wd, **over)


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_zero_gradients_from_zero_state(bits):
    """v = 0 and m = 0: the update is 0 / eps, the parameter only decays."""
    t = Tensors(1000, F32, F32, bits=bits)
    for x in (t.grad, t.m.view(torch.uint8) if bits == 8 else t.m, t.v.view(torch.uint8) if bits == 8 else t.v):
        x.zero_()
    want = t.param.double() * (1 - HYPER["lr"] * HYPER["weight_decay"])
    flce.adamw_step(plan_of([t]), [t.grad], step=1)
    within(t.param, want.cpu().numpy(), 2 * U * want.abs().cpu().numpy(), "param")
    assert not t.m.float().any() and not t.v.float().any()
    if bits == 8:
        assert not t.m_scale.any() and not t.v_scale.any()


@pytest.mark.gpu
def test_non_finite_gradients_stay_in_their_block():
    t = Tensors(256 * 6, F32, F32, bits=8, seed=2)
    t.grad[300], t.grad[256 * 4] = float("nan"), float("inf")
    before = t.start()
    flce.adamw_step(plan_of([t]), [t.grad], step=5)
    bad = torch.tensor([0, 1, 0, 0, 1, 0], dtype=torch.bool)
    assert torch.equal(torch.isnan(t.m_scale).cpu(), bad) and torch.equal(torch.isnan(t.v_scale).cpu(), bad)
    clean = Tensors(256 * 6, F32, F32, bits=8, seed=2)
    clean.grad[300] = clean.grad[256 * 4] = 0
    flce.adamw_step(plan_of([clean]), [clean.grad], step=5)
    keep = (~bad).repeat_interleave(256).cuda()
    assert torch.equal(t.param[keep], clean.param[keep])
    assert torch.equal(t.v.view(torch.uint8)[keep], clean.v.view(torch.uint8)[keep])
    assert torch.isnan(t.param[300]) and before is not None


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [1e-30, 1e15])
def test_8bit_moments_of_extreme_gradients(scale):
    """Gradients whose squares leave fp32's range on either side: v flushes to zero or
    becomes infinite, and nothing else in the call is touched."""
    a, b = Tensors(512, F32, F32, bits=8, seed=1), Tensors(512, F32, F32, bits=8, seed=3)
    a.grad.mul_(scale)
    before = b.start()
    flce.adamw_step(plan_of([a, b]), [a.grad, b.grad], step=2)
    check(b, before, 2)
    assert not torch.isnan(a.param).any() or scale > 1


@pytest.mark.gpu
def test_8bit_second_moment_keeps_moving():
    """With rounding to nearest, r could not follow a change below half an 8-bit step (3-6%);
    dithered, its mean does.  g^2 grows by 1.5 in every element: v must reach it."""
    n = 256 * 64
    t = Tensors(n, F32, F32, bits=8, seed=4)
    g = torch.Generator().manual_seed(1)
    size = (1e-3 * (0.2 + torch.rand(n, generator=g))).cuda()
    q, s = t.encode(size.cpu())
    t.v.view(torch.uint8).copy_(q.view(torch.uint8))
    t.v_scale.copy_(s)
    t.grad.copy_(size * math.sqrt(1.5))
    plan = plan_of([t])
    for k in range(300):
        flce.adamw_step(plan, [t.grad], step=k + 1)
    v = t.moments()[1]
    ratio = v / (size.double().cpu().numpy() ** 2)
    # a stationary EMA with steps of 6-12% of r: the mean over elements is exact to a few percent
    assert abs(ratio.mean() / 1.5 - 1) < 0.05, ratio.mean()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last block of a tensor of more than 2^31 elements."""
    n = (1 << 31) + 300
    param = torch.zeros(n, dtype=BF16, device="cuda")
    grad = torch.zeros(n, dtype=BF16, device="cuda")
    m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ms, vs = (torch.zeros((n + 255) // 256, device="cuda") for _ in range(2))
    tail = Tensors(300, BF16, BF16, master=False, bits=8, seed=6)
    param[-300:], grad[-300:] = tail.param, tail.grad
    m.view(torch.uint8)[-300:], v.view(torch.uint8)[-300:] = tail.m.view(torch.uint8), tail.v.view(torch.uint8)
    ms[-2:], vs[-2:] = tail.m_scale, tail.v_scale
    before = tail.start()
    plan = flce.adamw_plan([param], [m], [v], scales=([ms], [vs]), **HYPER)
    flce.adamw_step(plan, [grad], step=9)
    ref = step64(*before, 9, **HYPER)
    within(param[-300:], ref["p"], ref["ep"] + np.abs(ref["p"]) * 2.0 ** -8, "param")
    top = np.abs(blocks(ref["m"])).max(1)
    within(ms[-2:], top / 448, 12 * U * top / 448, "scale")
    assert not param[:-300].any() and not ms[:-2].any()


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_on_another_stream_and_twice_the_same(bits):
    outs = []
    for stream in (None, torch.cuda.Stream()):
        ts = [Tensors(n, BF16, BF16, True, bits, seed=n) for n in (100, 70000)]
        torch.cuda.synchronize()
        plan = plan_of(ts)
        for k in range(3):
            flce.adamw_step(plan, [t.grad for t in ts], step=k + 1, stream=stream)
        torch.cuda.synchronize()
        outs.append([x.view(torch.uint8).clone() for t in ts for x in (t.param, t.master, t.m, t.v)])
    for a, b in zip(*outs):
        assert torch.equal(a, b)


@pytest.mark.gpu
def test_optimizer_follows_the_formulas():
    """Twelve steps of the optimizer object with two groups against 64 bits."""
    g = torch.Generator().manual_seed(0)
    ps = [torch.nn.Parameter((0.1 * torch.randn(s, generator=g)).cuda()) for s in ((40, 33), (17,), (5, 5))]
    opt = flce.AdamW([{"params": ps[:2]}, {"params": ps[2:], "weight_decay": 0.0, "lr": 1e-2}], lr=1e-3,
                     betas=(0.9, 0.99), weight_decay=0.2)
    ref = [(p.detach().double().cpu().numpy(), 0 * p.detach().double().cpu().numpy(), 0.0) for p in ps]
    for k in range(12):
        for p in ps:
            p.grad = torch.randn(p.shape, generator=g).cuda()
        opt.step()
        for i, p in enumerate(ps):
            w, m, v = ref[i]
            r = step64(w, p.grad.cpu().numpy(), m, v, k + 1, lr=1e-2 if i == 2 else 1e-3, betas=(0.9, 0.99),
                       weight_decay=0.0 if i == 2 else 0.2)
            ref[i] = (r["p"], r["m"], r["v"])
            # errors of twelve steps add up
            within(p.detach(), r["p"], 12 * r["ep"] + 1e-9, "param")
    opt.zero_grad()
    assert all(p.grad is None for p in ps)
    held = [p.detach().clone() for p in ps]
    opt.step()  # no gradients: nothing moves
    assert all(torch.equal(a, b.detach()) for a, b in zip(held, ps))


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [32, 8])
def test_optimizer_state_round_trip(bits):
    def make():
        g = torch.Generator().manual_seed(3)
        return [torch.nn.Parameter((0.1 * torch.randn(n, generator=g)).to(BF16).cuda()) for n in (1000, 77)]

    def run(ps, opt, steps, seed):
        g = torch.Generator().manual_seed(seed)
        for _ in range(steps):
            for p in ps:
                p.grad = (1e-2 * torch.randn(p.shape, generator=g)).to(BF16).cuda()
            opt.step()

    a = make()
    oa = flce.AdamW(a, lr=1e-2, state_bits=bits)
    run(a, oa, 4, 1)
    b = make()
    ob = flce.AdamW(b, lr=1e-2, state_bits=bits)
    ob.load_state_dict(oa.state_dict())
    for p, q in zip(b, a):
        p.data = q.detach().clone()  # new storage: the optimizer follows it
    run(a, oa, 3, 2)
    run(b, ob, 3, 2)
    for p, q in zip(a, b):
        assert torch.equal(p.detach(), q.detach())
    with pytest.raises(ValueError):
        flce.AdamW(b, state_bits=40 - bits).load_state_dict(oa.state_dict())


@pytest.mark.gpu
def test_python_refusals():
    t = Tensors(64)
    e = Tensors(64, bits=8)
    plan = plan_of([t])
    for bad in (lambda: flce.adamw_step(plan, [t.grad.half()], step=1), lambda: plan_of([t, e]),
                lambda: flce.adamw_plan([t.param], [t.m.half()], [t.v]),
                lambda: flce.adamw_plan([t.param.half()], [t.m], [t.v]),
                lambda: flce.adamw_plan([t.param], [t.m], [t.v], masters=[t.param])):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: flce.adamw_step(plan, [], step=1), lambda: flce.adamw_step(plan, [t.grad[:63]], step=1),
                lambda: flce.adamw_step(plan, [t.grad.cpu()], step=1),
                lambda: flce.adamw_step(plan, [t.grad], step=1, grad_scale=torch.ones(2, device="cuda")),
                lambda: flce.adamw_plan([t.param], [t.m[:3]], [t.v]), lambda: flce.adamw_plan([t.param], [], [t.v]),
                lambda: flce.adamw_plan([e.param], [e.m], [e.v], scales=([e.m_scale[:0]], [e.v_scale])),
                lambda: flce.adamw_plan([t.param], [t.m], [t.v], lr=[1.0, 2.0]),
                lambda: flce.AdamW([t.param], state_bits=16), lambda: flce.AdamW([t.param, t.param])):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(betas=(1.0, 0.9)), dict(betas=(0.9, -0.1)), dict(eps=-1.0)):
        with pytest.raises(flce.FlceError) as err:
            flce.adamw_step(plan_of([t], **kw), [t.grad], step=1)
        assert err.value.code == 1
    with pytest.raises(flce.FlceError):
        flce.adamw_step(plan, [t.grad], step=0)


def test_host_refusals():
    L, T, O = flce.lib(), binding.AdamwTensor, binding.AdamwOptions
    z = 0x1000
    opt = O(0.9, 0.95, 1e-8, 1, 32)

    def call(t, o=opt, count=1, gs=None):
        return L.flce_adamw_step(ctypes.byref(t) if t is not None else None, count,
                                 ctypes.byref(o) if o is not None else None, gs, None)

    def tensor(**kw):
        base = dict(param=z, grad=z, master=None, exp_avg=z, exp_avg_sq=z, exp_avg_scale=z, exp_avg_sq_scale=z,
                    count=10, lr=1e-3, weight_decay=0.0, param_dtype=0, grad_dtype=0)
        return T(**{**base, **kw})

    assert call(None) == 1 and call(tensor(), None) == 1 and call(tensor(), count=-1) == 1
    assert call(None, count=0) == 0 and call(tensor(count=0, param=None)) == 0
    for kw in (dict(count=-1), dict(param=None), dict(grad=None), dict(exp_avg=None), dict(exp_avg_sq=None),
               dict(param_dtype=2), dict(grad_dtype=-1)):
        assert call(tensor(**kw)) == 1, kw
    for kw in (dict(param=z + 1), dict(grad=z + 1), dict(master=z + 2), dict(exp_avg=z + 2), dict(exp_avg_sq=z + 1),
               dict(param=z + 2, param_dtype=1)):
        assert call(tensor(**kw)) == 3, kw
    eight = O(0.9, 0.95, 1e-8, 1, 8)
    assert call(tensor(exp_avg_scale=None), eight) == 1 and call(tensor(exp_avg_sq_scale=z + 2), eight) == 3
    assert call(tensor(count=1 << 50)) == 2 and call(tensor(), gs=z + 2) == 3
    for o in (O(1.0, 0.9, 0, 1, 32), O(0.9, float("nan"), 0, 1, 32), O(0.9, 0.9, -1, 1, 32), O(0.9, 0.9, 0, 0, 32),
              O(0.9, 0.9, 0, 1, 16)):
        assert call(tensor(), o) == 1


def test_rounding_bytes_are_uniform_and_change_with_the_step():
    a, b = rounding_bytes(1 << 20, 11), rounding_bytes(1 << 20, 12)
    for x in (a, b):
        counts = np.bincount(x.astype(int), minlength=256)
        # chi-square with 255 degrees of freedom: mean 255, deviation 22.6; 8 deviations
        assert ((counts - 4096.0) ** 2 / 4096).sum() < 255 + 8 * 22.6
        for lag in (1, 2, 3, 4, 5, 8, 256, 4096):
            c = np.corrcoef(x[:-lag], x[lag:])[0, 1]
            assert abs(c) < 8 / 1024, (lag, c)
    assert abs(np.corrcoef(a, b)[0, 1]) < 8 / 1024


def test_reference_step_against_a_derivation():
    """step64 with beta1 = beta2 = 0, no decay: the update is lr g / (|g| + eps)."""
    g = np.array([1e-3, -2.0, 0.5])
    r = step64(np.ones(3), g, np.ones(3), np.ones(3), 4, lr=0.1, betas=(0.0, 0.0), eps=1e-8, weight_decay=0.0)
    np.testing.assert_allclose(r["p"], 1 - 0.1 * np.sign(g), rtol=1e-5)
