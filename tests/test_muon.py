"""Newton-Schulz products and the Muon step, against the definition in 64 bits and against the
products' documented roundings done in 64 bits, and the calls they refuse.

Tolerances (u = 2^-24; a rounding is off by half a step: fp16 2^-11, bf16 2^-8, relative).
`rounded` follows the documented arithmetic: operands in fp16 (pairs of it where the header says
so), everything else exact.
  Up to 128 rows or columns every operand carries 22 bits, and what is left are fp32 sums of 3 c / 16
products of 16 terms each, off by 2^-23 of the running sum each time (in either direction: their
root, for c = 1000 14 of them), so that X X^T's eigenvalues move by 14 2^-23 2 / sqrt(r) of the
strongest one, up to an 8th of all in the cases here: 5e-8 for r = 64.  The product of the steps
falls from 486 to 1 while an eigenvalue grows from 0 to about 1 / 486^2, by 486^2 / 2 of itself for
a whole one: 6e-3 of the weakest directions, and 4e-3 of the result's norm at most, the header's
promise.  Without strong directions eigenvalues are as large as their errors' scale, 1 / r: a
hundredth of that.  Element by element five times as much or more: 2^-6 and 2^-9 of the result's
root mean square, besides the result's own rounding.
  After a single step above that size the kernels differ from `rounded` by what fp32 sums and single
other neighbours of fp16 make: less than 2^-11 of the result's root mean square.
  Above 128 rows and after several steps no emulation follows the kernel's roundings: an
off-diagonal element of X X^T is about K^(-1/2) of the terms it sums, so the sum's error of u of
those is K^(1/2) 2^-13 of an fp16 step: one rounding in 2^13 / K^(1/2) goes to the other neighbour
(of 129^2 elements, 20), the next iterates then differ by about a step of fp16 somewhere in every
row, and from there on the two sides' roundings are unrelated.  There the definition itself is what
is compared with: the header's promise of 4e-3 of the result's norm, and element by element, the
noise being a sum of many independent roundings of at most 1.6e-3 root mean square, twice that in
rows of twice the usual size: 2^-6 of the result's root mean square, five of these deviations or
ten (of the 2.3e6 elements of the largest case, 5.7e-7 of a normal distribution or one or two lie
past five, 1e-16 past eight).  Where all singular values are equal all roundings
agree, at most half a step of X, A and P each, times 1.6^k: 3 2^-11 (1.6^5 - 1) / 0.6 = 2.4e-2."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding, muon  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
USUAL = (3.4445, -4.7750, 2.0315)


def triples(coefficients, steps):
    return [coefficients] * steps if isinstance(coefficients[0], float) else coefficients


def exact(u, steps=5, coefficients=USUAL, eps=1e-7):
    """The definition: u [..., R, C] in 64 bits."""
    x = u.double()
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    for a, b, c in triples(coefficients, steps):
        if x.shape[-2] <= x.shape[-1]:
            g = x @ x.mT
            x = a * x + (b * g + c * (g @ g)) @ x
        else:
            g = x.mT @ x
            x = a * x + x @ (b * g + c * (g @ g))
    return x


def rounded(u, steps=5, coefficients=USUAL, eps=1e-7):
    """The same with the operands' roundings."""
    wide = u.shape[-2] <= u.shape[-1]
    x = u.double() if wide else u.double().mT
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + eps)
    r = x.shape[-2]

    def pair(t, scale, low):
        hi = (t * scale).half().double() / scale
        return hi, ((t - hi) * scale).half().double() / scale if low else torch.zeros_like(hi)

    most, top = 0.0, 1.0 + 1 / 256
    for a, b, c in triples(coefficients, steps):  # the scale of P
        s = torch.linspace(0, top, 4097, dtype=torch.float64)
        p = (a + b * s ** 2 + c * s ** 4).abs()
        most, top = max(most, p.max().item()), (p * s).max().item() * (1 + 1 / 256)
    ps = 2.0 ** math.floor(math.log2(60000 / most))
    one = torch.eye(r, dtype=torch.float64, device=u.device)
    x = pair(x, 2.0 ** 14, True)
    for k, (a, b, c) in enumerate(triples(coefficients, steps)):
        g = x[0] @ x[0].mT
        if c:  # the square completed; what rounding the diagonal left is known
            g = g + b / (2 * c) * one
            left = torch.diagonal(g - pair(g, 2.0 ** 13, False)[0], dim1=-2, dim2=-1)
            g = pair(g, 2.0 ** 13, False)[0]
            more = left * (2 * torch.diagonal(g, dim1=-2, dim2=-1) + left)
            p = c * (g @ g) + (a - b * b / (4 * c)) * one + c * torch.diag_embed(more)
        else:
            p = a * one + b * g
        y = pair(p, ps, False)[0] @ x[0] + (a * x[1] if k < 3 else 0)
        x = pair(y, 2.0 ** 14, k + 1 < 3 and k + 1 < steps)
    y = x[0] + x[1]
    return y if wide else y.mT


def matrix(shape, kind="noise", seed=0):
    g = torch.Generator().manual_seed(seed)
    m = torch.randn(shape, generator=g)
    if kind == "strong":  # eight strong directions over noise
        *lead, r, c = shape
        m = torch.randn(*lead, r, 8, generator=g) @ torch.randn(*lead, 8, c, generator=g) + 0.05 * m
    if kind == "same":
        m = torch.eye(shape[-2], shape[-1]).expand(shape)
    return m.contiguous()


def shifted(t, by):
    flat = torch.cat([t.new_zeros(by), t.reshape(-1)])
    return flat[by:].view(t.shape)


def within(got, want, tol, name):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, worst " \
                          f"{((got.double() - want).abs() / tol).max().item():.3g} of it"


def rms(x):
    return x.square().mean((-1, -2), keepdim=True).sqrt()


def model(x, promise=4e-3, strong=False, steps=5, **kw):
    """What the elements are compared with, and by how much they may be off besides the result's rounding."""
    near = exact(x, steps=steps, **kw)
    if min(x.shape[-2:]) <= 128:
        return near, rms(near) * 2.0 ** (-6 if strong else -9)
    if steps == 1:
        near = rounded(x, steps=steps, **kw)
        return near, rms(near) * 2.0 ** -11
    return near, rms(near) * 2.0 ** -6 + near.abs() * (promise if promise > 4e-3 else 0)


def check(x, got, promise=4e-3, strong=False, **kw):
    true = exact(x, **kw)
    near, noise = model(x, promise, strong, **kw)
    within(got, near, near.abs() * 2.0 ** -8 + noise, "elements")
    off = (got.double() - true).square().sum((-1, -2)).sqrt() / true.square().sum((-1, -2)).sqrt()
    assert (off <= promise + 2.0 ** -9).all(), off


# ----------------------------------------------------------------------------- refusals (CPU)


def options(momentum=0.0, nesterov=False, steps=5, coefficients=USUAL, eps=1e-7):
    return muon._options(momentum, nesterov, steps, coefficients, eps)


def ortho(row=(0x1000, 0x2000, 8, 8, 0), o=None, ws=0x100000, nbytes=0, count=1):
    table = (binding.Matrix * 1)(row)
    return flce.lib().flce_orthogonalize(table, count, ctypes.byref(o or options()), ws, nbytes, None)


def test_library_refuses():
    assert ortho() == 4  # (all is well but the workspace's size)
    assert ortho(ws=None) == 1 and ortho(ws=0x100010) == 3 and ortho(count=-1) == 1
    for row, code in (((None, 0x2000, 8, 8, 0), 1), ((0x1000, None, 8, 8, 0), 1), ((0x1001, 0x2000, 8, 8, 0), 3),
                      ((0x1002, 0x2000, 8, 8, 1), 3), ((0x1000, 0x2001, 8, 8, 0), 3), ((0x1000, 0x2000, -1, 8, 0), 1),
                      ((0x1000, 0x2000, 8, 8, 2), 1), ((0x1000, 0x2000, 65537, 65537, 0), 2),
                      ((0x1000, 0x2000, 8, (1 << 24) + 1, 0), 2)):
        assert ortho(row) == code, row
    for over in (dict(eps=0.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(coefficients=(4.5, -4.775, 2.03)),
                 dict(coefficients=(float("nan"), 0.0, 0.0)), dict(coefficients=(1.5, -0.5, 0.05)), dict(coefficients=(1e5, 0.0, 0.0), steps=1),
                 dict(momentum=1.0), dict(momentum=-0.1)):
        assert ortho(o=options(**over)) == 1, over
    o = options()
    for name, value in (("steps", 0), ("steps", 17), ("nesterov", 2), ("coefficients", None)):
        o = options()
        setattr(o, name, value)
        assert ortho(o=o) == 1, name
    for over in (dict(coefficients=(1.875, -1.25, 0.375)), dict(coefficients=(1.5, -0.5, 0.0), steps=12)):
        assert ortho(o=options(**over)) == 4, over
    L = flce.lib()

    def step(ws=0x100000, gs=None, **over):
        row = dict(param=0x1000, grad=0x2000, master=None, momentum=0x3000, rows=8, cols=8, lr=0.1, weight_decay=0.0,
                   scale=1.0, param_dtype=0, grad_dtype=0)
        table = (binding.MuonTensor * 1)(tuple({**row, **over}.values()))
        return L.flce_muon_step(table, 1, ctypes.byref(options(0.9)), gs, ws, 0, None)
    assert step() == 4 and step(gs=0x1002) == 3 and step(ws=None) == 1
    for over in (dict(param=None), dict(grad=None), dict(momentum=None), dict(lr=float("nan")),
                 dict(weight_decay=float("inf")), dict(scale=float("nan")), dict(param_dtype=3), dict(grad_dtype=-1)):
        assert step(**over) == 1, over
    for over in (dict(param=0x1001), dict(grad=0x2002, grad_dtype=1), dict(momentum=0x3002), dict(master=0x4002)):
        assert step(**over) == 3, over


def workspace(*shapes):
    table = (binding.Matrix * max(len(shapes), 1))(*((1, 1, r, c, 0) for r, c in shapes))
    return flce.lib().flce_orthogonalize_workspace_bytes(table, len(shapes))


def test_workspace_size_rules():
    assert workspace() == 256 and workspace((0, 5), (5, 0)) == 256
    assert workspace((-1, 5)) == 0 and workspace((70000, 70000)) == 0
    n = 2048
    assert 10 * n * n <= workspace((n, n)) <= 10 * n * n + 65536
    assert workspace((504, 904)) == workspace((904, 504))
    # rounds of at most 256 matrices, 12 shapes and 4 GiB: more of them need no more room
    assert workspace(*[(200, 200)] * 256) == workspace(*[(200, 200)] * 600)
    assert workspace(*[(4096, 4096)] * 40) <= 4 << 30
    assert workspace(*((200 + i, 300) for i in range(12))) >= workspace(*((200 + i, 300) for i in range(11)))


def test_workspace_of_long_thin_matrices():
    """Their parts of X X^T count towards a round's size."""
    assert workspace(*[(1, 1 << 22)] * 300) <= (4 << 30) + (1 << 20)
    assert workspace((2, 1 << 24)) >= 8 * 2 * (1 << 24) + 64 * 65536


def test_eps_that_fp32_squares_pass_by_is_refused():
    assert ortho(o=options(eps=9e-16)) == 1 and ortho(o=options(eps=1.1e-15)) == 4


@pytest.mark.gpu
@pytest.mark.parametrize("size", [1e-21, 1e-24, 1e-38])
def test_elements_whose_squares_are_lost(size):
    """Each X is u / eps or nearly so.  fp16 ends at 2^-24 / 2^14 = 2^-38: half of that an element."""
    x = torch.randn(100, 200, device="cuda") * size
    for y in (x, x.repeat(2, 1)):
        got = flce.orthogonalize(y, steps=1, eps=1e-15).double()
        near = exact(y.cpu(), steps=1, eps=1e-15).to(got)
        assert (got - near).norm() <= 2.0 ** -6 * near.norm() + 3.4445 * 2.0 ** -39 * x.numel() ** 0.5 * 2


def test_python_refuses_on_cpu():
    for x in (torch.zeros(4, 4), [torch.zeros(4, 4)], torch.zeros(4)):
        with pytest.raises(ValueError):
            flce.orthogonalize(x)
    assert flce.orthogonalize([]) == []
    with pytest.raises(ValueError, match="steps"):
        muon._options(0.0, False, 17, USUAL, 1e-7)
    with pytest.raises(ValueError, match="coefficients"):
        muon._options(0.0, False, 2, [USUAL], 1e-7)
    with pytest.raises(ValueError, match="adjust"):
        muon.shape_factor(3, 4, "none")
    with pytest.raises(ValueError):
        flce.Muon([torch.zeros(4, 4)])
    assert muon.shape_factor(8, 2, "original") == 2 and muon.shape_factor(2, 8, "original") == 1
    assert muon.shape_factor(4, 16, "match_rms_adamw") == 0.8


def test_longer_sums_than_the_accumulator_holds_are_refused():
    for rows, cols, code in ((129, (1 << 20) + 1, 2), ((1 << 20) + 1, 129, 2), (129, 1 << 20, 4), (128, 1 << 24, 4),
                             (1 << 24, 128, 4), ((1 << 24) + 1, 128, 2)):
        assert ortho((0x1000, 0x2000, rows, cols, 0)) == code, (rows, cols)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(2100, 1 << 20), (128, 1 << 24), (1 << 24, 128)])
def test_offsets_beyond_32_bits(rows, cols):
    """A matrix beside itself n times: its singular vectors, n times over, so X's blocks / sqrt(n)."""
    r, n = min(rows, cols), max(rows, cols) // 4096
    x = torch.randn(r, 4096, device="cuda").bfloat16()
    near = exact(x) / n ** 0.5
    big = x.repeat(1, n) if rows < cols else x.t().contiguous().repeat(n, 1)
    got = flce.orthogonalize(big, out=big)
    blocks = [got[:, k:k + 4096] if rows < cols else got[k:k + 4096].t() for k in (0, 4096, n // 2 * 4096, 4096 * (n - 1))]
    for b in blocks:
        assert torch.equal(b, blocks[0])
        assert (b.double() - near).norm() <= 2.0 ** -6 * near.norm()


class Device(torch.Tensor):
    """A CPU tensor that says it is on a GPU."""
    __torch_function__ = torch._C._disabled_torch_function_impl
    is_cuda = True


def test_memory_that_is_written_twice_is_refused():
    a, b, c = (torch.zeros(4, 6).as_subclass(Device) for _ in range(3))
    for lists in (([a, a], [b, c]), ([a, c], [b, b]), ([a], [a]), ([a], [b], [a]), ([a], [b], [b])):
        with pytest.raises(ValueError, match="same memory"):
            flce.muon_plan(*lists)
    flce.muon_plan([a], [b], [c])
    empty = [torch.zeros(0, 6).as_subclass(Device) for _ in range(4)]
    flce.muon_plan(empty[:2], empty[2:])
    y = torch.zeros(4, 6, dtype=BF16).as_subclass(Device)
    with pytest.raises(ValueError, match="same memory"):
        flce.orthogonalize([a, b], out=[y, y])


def test_a_group_of_other_options_is_refused():
    for group in ({"params": [], "momentum": 0.9}, {"lr": 0.1}):
        with pytest.raises(ValueError, match="group"):
            flce.Muon([group])


def test_sizes_of_many_sets_of_gradients_are_not_kept():
    plan = flce.muon_plan(*([torch.zeros(2, 3).as_subclass(Device) for _ in range(8)] for _ in range(2)))
    want = {}
    for k in range(1, 256):
        live = [bool(k >> i & 1) for i in range(8)]
        want[k] = plan.workspace_bytes(live)
        assert len(plan._bytes) <= 64
    assert want[1] == plan.workspace_bytes([True] + 7 * [False]) and want[255] == plan.workspace_bytes()


# ----------------------------------------------------------------------------- orthogonalize


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["noise", "strong", "same"])
@pytest.mark.parametrize("shape", [(8, 8), (1, 1), (1, 7), (7, 1), (64, 1000), (128, 128), (130, 100), (129, 129),
                                   (256, 512), (300, 777), (777, 300), (2, 513, 640), (3, 257, 130), (1024, 1024),
                                   (16, 4096), (9000, 65), (5, 100, 72), (128, 2000),
                                   (1100, 2056)])
def test_orthogonalize(shape, kind):
    for dtype, by in ((BF16, 0), (F32, 1)):
        x = shifted((1e-3 * matrix(shape, kind)).to(dtype).cuda(), by)
        got = flce.orthogonalize(x, check=True)
        assert got.shape == x.shape and got.dtype == BF16
        check(x, got, 2.4e-2 if kind == "same" else 4e-3, kind == "strong")


@pytest.mark.gpu
@pytest.mark.parametrize("steps,coefficients", [(1, USUAL), (2, USUAL), (3, USUAL), (4, USUAL), (12, (1.5, -0.5, 0.0)),
                                                (1, (1.5, -0.5, 0.0)), (1, (3.9, -8.0, 4.5)),
                                                (8, (1.875, -1.25, 0.375)),
                                                (3, [(3.9, -8.0, 4.5), (3.0, -4.0, 1.9), (1.875, -1.25, 0.375)])])
@pytest.mark.parametrize("shape", [(100, 60), (200, 300)])
def test_other_polynomials(shape, steps, coefficients):
    x = matrix(shape).cuda()
    check(x, flce.orthogonalize(x, steps=steps, coefficients=coefficients, check=True), steps=steps,
          coefficients=coefficients)


@pytest.mark.gpu
def test_eps_counts_where_the_norm_is_small():
    x = 1e-9 * matrix((150, 200)).cuda()
    for eps in (1e-7, 1e-12):
        check(x, flce.orthogonalize(x, eps=eps), eps=eps)


@pytest.mark.gpu
def test_lists_of_many_shapes_and_rounds():
    """More shapes and more matrices than one round of launches takes, empty ones among them."""
    shapes = [(130 + 8 * i, 200 + 7 * i) for i in range(14)] + [(40, 24), (24, 40)] * 130 + [(0, 5), (5, 0), (1, 1)]
    xs = [matrix(s, seed=i).to(BF16 if i % 2 else F32).cuda() for i, s in enumerate(shapes)]
    got = flce.orthogonalize(xs, check=True)
    assert [tuple(t.shape) for t in got] == shapes
    for x, y in zip(xs, got):
        if x.numel():
            assert torch.equal(y, flce.orthogonalize(x))
    for i in (0, 13, 14, 15, 273, 276):
        check(xs[i], got[i])


@pytest.mark.gpu
def test_zeros_and_non_finite_matrices():
    x = matrix((6, 140, 150)).cuda()
    clean = flce.orthogonalize(x)
    x[1] = 0
    x[2, 3, 4] = float("nan")
    x[3, 5, 6] = float("inf")
    x[4] *= 1e25  # squares past fp32's range
    got = flce.orthogonalize(x, check=True)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[5], clean[5])
    assert not got[1].any()
    assert torch.isnan(got[2:5]).all()


@pytest.mark.gpu
def test_in_place_same_bits_and_nothing_past_the_workspace():
    x = matrix((2, 300, 260)).to(BF16).cuda()
    want = flce.orthogonalize(x)
    table = (binding.Matrix * 2)((1, 1, 300, 260, 0), (1, 1, 300, 260, 0))
    size = flce.lib().flce_orthogonalize_workspace_bytes(table, 2)
    for fill in (0, 255):
        ws = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
        assert torch.equal(flce.orthogonalize(x, ws=ws[:size]), want)
        assert (ws[size:] == fill).all()
    y = x.clone()
    assert flce.orthogonalize(y, out=y) is y and torch.equal(y, want)
    assert flce.orthogonalize(torch.zeros(0, 4, 4, device="cuda")).shape == (0, 4, 4)


# ----------------------------------------------------------------------------- the step


def build(shapes, dtype, gdtype, master, by=0):
    g = torch.Generator().manual_seed(1)
    ps = [shifted((0.02 * torch.randn(s, generator=g)).to(dtype).cuda(), by) for s in shapes]
    ms = [shifted(1e-3 * matrix(s, seed=i).cuda(), by) for i, s in enumerate(shapes)]
    gs = [shifted((1e-3 * matrix(s, seed=99 + i)).to(gdtype).cuda(), by) for i, s in enumerate(shapes)]
    masters = [p.float() + 1e-6 for p in ps] if master else None
    return ps, ms, gs, masters


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,gdtype,master", [(BF16, BF16, False), (BF16, F32, True), (F32, BF16, False),
                                                 (F32, F32, False)])
@pytest.mark.parametrize("nesterov,by", [(True, 0), (False, 1)])
def test_step(dtype, gdtype, master, nesterov, by):
    shapes = [(200, 136), (136, 200), (300, 300), (16, 40), (7, 5), (300, 300), (1, 9)]
    ps, ms, gs, masters = build(shapes, dtype, gdtype, master, by)
    lr, wd, mu, scale = [0.02 + 0.01 * i for i in range(7)], 0.3, 0.9, torch.full((1,), 0.7, device="cuda")
    plan = flce.muon_plan(ps, ms, masters, lr=lr, weight_decay=wd, momentum=mu, nesterov=nesterov)
    gs[3] = None
    old = [(p.clone(), m.clone(), None if not master else w.clone())
           for p, m, w in zip(ps, ms, masters or [None] * 7)]
    flce.muon_step(plan, gs, grad_scale=scale, check=True)
    for i, s in enumerate(shapes):
        p0, m0, w0 = old[i]
        if gs[i] is None:
            assert torch.equal(ps[i], p0) and torch.equal(ms[i], m0)
            continue
        g = gs[i].double() * scale.double()
        m = mu * m0.double() + (1 - mu) * g
        within(ms[i], m, 4 * U * (m0.double().abs() + g.abs()), f"momentum {i}")
        x, noise = model(mu * m + (1 - mu) * g if nesterov else m)
        rate = lr[i] * math.sqrt(max(1.0, s[0] / s[1]))
        w = (p0 if w0 is None else w0).double()
        want = w * (1 - lr[i] * wd) - rate * x
        tol = rate * (noise + x.abs() * 4 * U) + 4 * U * (w.abs() + want.abs())
        if master:
            within(masters[i], want, tol, f"master {i}")
            assert torch.equal(ps[i], masters[i].to(dtype))
        else:
            within(ps[i], want, tol + want.abs() * torch.finfo(dtype).eps / 2, f"param {i}")


@pytest.mark.gpu
def test_steps_of_the_optimizer():
    """The optimizer object against the plan and step calls; groups, schedules, state."""
    shapes = [(160, 144), (48, 40)]
    ps, _, _, _ = build(shapes, BF16, BF16, False)
    a = [torch.nn.Parameter(p.clone()) for p in ps]
    opt = flce.Muon([{"params": a[:1], "lr": 0.1}, {"params": a[1:], "weight_decay": 0.2}], lr=0.05, adjust="match_rms_adamw")
    opt.step()  # no gradient: nothing
    assert torch.equal(a[0], ps[0])
    masters, momenta = [p.float() for p in ps], [torch.zeros(s, device="cuda") for s in shapes]
    plan = flce.muon_plan(ps, momenta, masters, lr=[0.1, 0.05], weight_decay=[0.0, 0.2], adjust="match_rms_adamw")
    for k in range(3):
        gs = [matrix(s, seed=k).to(BF16).cuda() for s in shapes]
        for p, g in zip(a, gs):
            p.grad = g.t().contiguous().t()  # another layout: copied
        if k == 2:
            opt.groups[0]["lr"] = 0.01
            plan.set_lr([0.01, 0.05])
            b = [torch.nn.Parameter(p.detach().clone()) for p in a]
            other = flce.Muon([{"params": b[:1], "lr": 0.01}, {"params": b[1:], "weight_decay": 0.2}], lr=0.05,
                              adjust="match_rms_adamw")
            other.load_state_dict(opt.state_dict())
            for p, g in zip(b, gs):
                p.grad = g
            other.step()
        opt.step()
        flce.muon_step(plan, gs)
        assert all(torch.equal(p, q) for p, q in zip(a, ps))
        assert all(torch.equal(p, q) for p, q in zip(opt.state["master"], masters))
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(ValueError):
        flce.Muon([a[0], a[0]])
    with pytest.raises(ValueError):
        flce.Muon([torch.nn.Parameter(torch.zeros(3, 4, 5, device="cuda"))])


@pytest.mark.gpu
def test_graphs_of_old_weights_refuse_their_backward_pass():
    ps = [torch.nn.Parameter(matrix((20, 30)).cuda()) for _ in range(2)]
    opt = flce.Muon(ps)
    losses = [(p * p).sum() for p in ps]
    ps[0].grad = torch.ones_like(ps[0])
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        losses[0].backward()
    losses[1].backward()


@pytest.mark.gpu
def test_graph_replays_and_streams():
    shapes = [(200, 136), (136, 200), (64, 64)]
    ps, ms, gs, _ = build(shapes, F32, F32, False)
    qs, ns = [p.clone() for p in ps], [m.clone() for m in ms]
    plan, other = flce.muon_plan(ps, ms), flce.muon_plan(qs, ns)
    ws = torch.empty(plan.workspace_bytes(), dtype=torch.uint8, device="cuda")
    flce.muon_step(plan, gs, ws=ws)
    flce.muon_step(other, gs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        flce.muon_step(plan, gs, ws=ws)
    side = torch.cuda.Stream()
    for k in range(2):
        for g in gs:
            g.mul_(-0.5).add_(1e-4)
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        flce.muon_step(other, gs, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(ps + ms, qs + ns))


@pytest.mark.gpu
def test_python_refuses():
    p, m = torch.zeros(4, 6, device="cuda"), torch.zeros(4, 6, device="cuda")
    plan = flce.muon_plan([p], [m])
    for args in (([p.t()], [m]), ([p], [m[:2]]), ([p], [m.double()]), ([p], []), ([p.half()], [m])):
        with pytest.raises((ValueError, TypeError)):
            flce.muon_plan(*args)
    for g in (torch.zeros(6, 4, device="cuda"), torch.zeros(4, 6), torch.zeros(4, 6, device="cuda").half(),
              torch.zeros(6, 4, device="cuda").t()):
        with pytest.raises((ValueError, TypeError)):
            flce.muon_step(plan, [g])
    with pytest.raises(ValueError):
        flce.muon_step(plan, [])
    with pytest.raises(flce.FlceError):
        flce.muon_step(plan, [m], ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        flce.orthogonalize(p, out=torch.zeros(4, 6, device="cuda"))
    with pytest.raises(ValueError):
        flce.orthogonalize(p.t())
    with pytest.raises(flce.FlceError):
        flce.orthogonalize(p, coefficients=(5.0, 0.0, 0.0))
