"""Embedding rows and their gradient by sorted tokens, against the definition in 64 bits, and the
calls they refuse.

Tolerances (u = 2^-24; e = half a step of the output's type, relative).  A scaled row: one fp32
product, one rounding.  A row of the gradient that sums c terms in fp32, in whatever parts: c u of
the sum of their magnitudes, then a product or a multiply-add and one rounding."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def within(got, want, tol, name):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} of {bad.numel()} outside, at {bad.nonzero()[0].tolist()}"


def shifted(t, by):
    """t's values at an address `by` elements past an allocation's start."""
    flat = torch.cat([t.new_zeros(by), t.reshape(-1)])
    return flat[by:].view(t.shape)


def tokens(n, v, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    if kind == "one":  # every token the same id
        return torch.full((n,), v // 2, dtype=torch.int32)
    if kind == "zipf":
        p = 1.0 / (torch.arange(v, dtype=torch.float64) + 1.0)
        return torch.multinomial(p, n, replacement=True, generator=g).to(torch.int32)
    if kind == "ends":
        return torch.where(torch.rand(n, generator=g) < 0.5, 0, v - 1).to(torch.int32)
    return torch.randint(0, v, (n,), generator=g).to(torch.int32)


def gradient64(dy, ids, v, scale, pad=None):
    """The gradient, the magnitudes that enter each of its sums, and how many."""
    keep = (ids >= 0) & (ids < v) & (ids != (-1 if pad is None else pad))
    at, d = ids[keep].long(), dy[keep].double()
    zero = torch.zeros(v, dy.shape[1], dtype=torch.float64, device=dy.device)
    total = zero.index_add(0, at, d) * scale
    size = zero.index_add(0, at, d.abs()) * abs(scale)
    count = torch.bincount(at, minlength=v).double()[:, None]
    return total, size, count


# ----------------------------------------------------------------------------- refusals (CPU)


def _call(name, q, a=0x1000, b=0x2000, c=0x3000, ws=0x100000, nbytes=1 << 30, add=0):
    L = flce.lib()
    q = ctypes.byref(q) if q is not None else None
    if name == "forward":
        return L.flce_embedding_forward(q, a, b, c, ws, nbytes, None)
    return L.flce_embedding_backward(q, a, b, c, add, ws, nbytes, None)


@pytest.mark.parametrize("name", ["forward", "backward"])
def test_library_refuses(name):
    E = binding.Embedding
    ok = dict(n=10, h=8, v=100, scale=1.0, padding_idx=-1, w_dtype=0, y_dtype=0)
    assert _call(name, None) == 1
    for over in (dict(n=-1), dict(h=0), dict(v=0), dict(scale=float("nan")), dict(scale=float("inf")),
                 dict(padding_idx=-2), dict(padding_idx=100), dict(w_dtype=2), dict(y_dtype=-1)):
        assert _call(name, E(**{**ok, **over})) == 1, over
    for over in (dict(n=(1 << 30) + 1), dict(v=(1 << 20) + 1), dict(h=(1 << 20) + 1)):
        assert _call(name, E(**{**ok, **over})) == 2, over
    for which in "abc":
        assert _call(name, E(**ok), **{which: None}) == 1
        assert _call(name, E(**ok), **{which: 0x1001}) == 3
    assert _call(name, E(**ok), ws=None) == 1 and _call(name, E(**ok), ws=0x100010) == 3
    assert _call(name, E(**ok), nbytes=128) == 4
    if name == "forward":
        assert _call(name, E(**{**ok, "y_dtype": 1})) == 1  # y has W's type
    else:
        assert _call(name, E(**ok), add=2) == 1
        assert _call(name, E(**ok), nbytes=flce.embedding_workspace_bytes(10, 8, 100) - 1) == 4


def test_workspace_size_rules():
    ws = flce.embedding_workspace_bytes
    assert ws(-1, 8, 8) == ws(1, 0, 8) == ws(1, 8, 0) == 0
    assert ws(32, 4096, 100) < ws(33, 4096, 100)  # up to 32 tokens need no parts
    n, h, v = 131072, 4096, 131072
    for n, tile in ((n, 64), (16384, 32)):
        least = 4 * (v + 4 * n) + 2 * (n // tile) * 4 * h
        assert least <= ws(n, h, v) <= least + 700000


def test_python_refuses_on_cpu():
    ids, w = torch.zeros(4, dtype=torch.int32), torch.zeros(10, 8)
    with pytest.raises(ValueError):
        flce.embedding_forward(ids, w)
    with pytest.raises(TypeError):
        flce.embedding_forward(ids.long(), w)
    with pytest.raises(ValueError, match="padding_idx"):
        flce.embedding(ids, w, padding_idx=10)
    with pytest.raises(ValueError):
        flce.embedding_backward(torch.zeros(4, 8), ids, 10)


def test_ids_that_are_no_integers_are_refused():
    """(Converted, 1.9 would be row 1, and an unsigned 2^32 + 1 too.)"""
    for dtype in (F32, BF16, torch.bool, torch.uint64):
        with pytest.raises(TypeError, match="integers"):
            flce.embedding(torch.zeros(4).to(dtype), torch.zeros(10, 8))


def test_a_padding_id_from_the_end_is_refused():
    class Device(torch.Tensor):
        __torch_function__ = torch._C._disabled_torch_function_impl
        is_cuda = True

    ids, dy = torch.zeros(4, dtype=torch.int32).as_subclass(Device), torch.zeros(4, 8).as_subclass(Device)
    with pytest.raises(ValueError, match="padding_idx"):
        flce.embedding_backward(dy, ids, 10, padding_idx=-1)


# ----------------------------------------------------------------------------- forward


SIZES = [(1, 1, 1), (4, 4096, 1000), (3, 7, 5), (1000, 40, 300), (257, 1031, 129), (5000, 96, 50), (20, 2, 3)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,h,v", SIZES)
@pytest.mark.parametrize("by", [0, 1])
def test_forward(n, h, v, dtype, by):
    g = torch.Generator().manual_seed(n + h)
    w = shifted(torch.randn(v, h, generator=g).to(dtype).cuda(), by)
    ids = tokens(n, v, "uniform").cuda()
    for scale in (1.0, -3.7):
        y, ws = flce.embedding_forward(ids, w, scale=scale, check=True)
        want = w.double()[ids.long()] * float(torch.tensor(scale, dtype=F32))
        within(y, want, want.abs() * (half_step(dtype) * 1.001 + U), "y")
        if scale == 1.0:
            assert torch.equal(y, w[ids.long()])


@pytest.mark.gpu
def test_forward_of_nothing_and_of_ids_outside():
    w = torch.randn(10, 16, device="cuda")
    y, ws = flce.embedding_forward(torch.zeros(0, dtype=torch.int32, device="cuda"), w, check=True)
    assert y.shape == (0, 16)
    for bad in (10, -1, 2 ** 31 - 1, -2 ** 31):
        ids = torch.tensor([3, bad, 4], dtype=torch.int32, device="cuda")
        y, ws = flce.embedding_forward(ids, w)
        assert flce.read_device_status(ws) == 5
        assert torch.equal(y[::2], w[[3, 4]])
    y, ws = flce.embedding_forward(ids[:1], w, ws=ws)
    assert flce.read_device_status(ws) == 0  # each call starts a clear word


@pytest.mark.gpu
@pytest.mark.parametrize("n", [16383, 16384, 16385, 40000])
def test_forward_finds_an_id_outside_wherever_it_stands(n):
    w = torch.randn(50, 8, device="cuda")
    ids = torch.randint(0, 50, (n,), device="cuda", dtype=torch.int32)
    ws = torch.full((256,), 255, dtype=torch.uint8, device="cuda")
    y, _ = flce.embedding_forward(ids, w, ws=ws, check=True)
    assert torch.equal(y, w[ids.long()])
    for at in {0, min(16383, n - 1), min(16384, n - 1), n // 2, n - 1}:
        bad = ids.clone()
        bad[at] = 50
        ws.fill_(255)
        y, _ = flce.embedding_forward(bad, w, ws=ws)
        assert flce.read_device_status(ws) == 5
        want = w[ids.long()]
        want[at] = 0
        assert torch.equal(y, want)


@pytest.mark.gpu
def test_forward_of_offsets_beyond_32_bits():
    v, h = 70000, 40000  # 2.8e9 elements
    w = torch.empty(v, h, dtype=BF16, device="cuda")
    w[-1] = torch.arange(h, device="cuda") % 250
    w[1] = -(torch.arange(h, device="cuda") % 250)
    ids = torch.tensor([v - 1, 1, v - 1], dtype=torch.int32, device="cuda")
    y, _ = flce.embedding_forward(ids, w, check=True)
    assert torch.equal(y, w[ids.long()])


# ----------------------------------------------------------------------------- gradient


def check_gradient(n, h, v, kind, dtype, wtype, pad=None, scale=0.37, by=0, old=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    dy = shifted(torch.randn(n, h, generator=g).to(dtype).cuda(), by)
    ids = tokens(n, v, kind, seed).cuda()
    add_to = None if old is None else shifted(old, by)
    before = None if old is None else add_to.double().clone()
    dw, ws = flce.embedding_backward(dy, ids, v, scale=scale, padding_idx=pad, add_to=add_to, dtype=wtype, check=True)
    total, size, count = gradient64(dy, ids, v, float(torch.tensor(scale, dtype=F32)), pad)
    want = total if old is None else total + before
    within(dw, want, size * U * (count + 4) + want.abs() * (half_step(wtype) * 1.001 + U), "dweight")
    return dw


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,wtype", [(BF16, BF16), (F32, F32), (BF16, F32), (F32, BF16)])
@pytest.mark.parametrize("n,h,v,kind", [
    (1, 1, 1, "one"), (5, 8, 3, "uniform"), (32, 24, 4, "one"), (33, 24, 4, "one"), (64, 1031, 9, "one"),
    (65, 5, 2, "ends"), (1000, 40, 300, "zipf"), (2000, 264, 7, "zipf"), (5003, 129, 5000, "zipf"),
    (100, 16, 40000, "uniform"), (31, 2050, 31, "uniform"), (9000, 9, 700, "ends")])
def test_gradient(n, h, v, kind, dtype, wtype):
    check_gradient(n, h, v, kind, dtype, wtype)
    check_gradient(n, h, v, kind, dtype, wtype, by=1, seed=1)
    check_gradient(n, h, v, kind, dtype, wtype, pad=v // 2, seed=2)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n,h,v,kind", [(1, 8, 5, "one"), (700, 72, 3000, "zipf"), (3000, 61, 20, "zipf"),
                                        (4097, 16, 2, "ends")])
@pytest.mark.parametrize("by", [0, 1])
def test_gradient_added(n, h, v, kind, dtype, by):
    """Rows of the vocabulary without a token keep their bits, NaNs included."""
    old = torch.randn(v, h, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    ids = tokens(n, v, kind).cuda()
    check_gradient(n, h, v, kind, dtype, dtype, by=by, old=old)
    old[:] = float("nan")
    dy = torch.ones(n, h, dtype=dtype, device="cuda")
    kept = shifted(old, by)
    kept[ids.long()] = 0
    dw, _ = flce.embedding_backward(dy, ids, v, add_to=kept, check=True)
    assert dw.data_ptr() == kept.data_ptr()
    count = torch.bincount(ids.long(), minlength=v)
    assert torch.isnan(dw[count == 0]).all() and not torch.isnan(dw[count > 0]).any()


@pytest.mark.gpu
@pytest.mark.parametrize("n,v", [(200000, 3), (131072, 131072), (70001, 151936)])
def test_gradient_of_many_tokens(n, v):
    check_gradient(n, 8, v, "zipf", BF16, F32, seed=5)
    check_gradient(n, 3, v, "one", F32, F32, seed=5)


@pytest.mark.gpu
def test_gradient_of_large_vocabularies():
    check_gradient(3000, 8, 400000, "uniform", BF16, BF16)
    check_gradient(70000, 8, 1 << 20, "uniform", BF16, BF16)


@pytest.mark.gpu
def test_gradient_of_nothing():
    dy = torch.zeros(0, 8, device="cuda")
    ids = torch.zeros(0, dtype=torch.int32, device="cuda")
    dw, _ = flce.embedding_backward(dy, ids, 5, check=True)
    assert dw.shape == (5, 8) and not dw.any()
    old = torch.full((5, 8), 2.0, device="cuda")
    flce.embedding_backward(dy, ids, 5, add_to=old, check=True)
    assert (old == 2).all()
    # every token padding
    ids = torch.full((100,), 3, dtype=torch.int32, device="cuda")
    dw, _ = flce.embedding_backward(torch.full((100, 8), float("nan"), device="cuda"), ids, 5, padding_idx=3, check=True)
    assert not dw.any()


@pytest.mark.gpu
def test_gradient_skips_ids_outside_and_says_so():
    ids = torch.tensor([3, -1, 4, 10, 2 ** 31 - 1, -2 ** 31, 3], dtype=torch.int32, device="cuda")
    dy = torch.randn(7, 16, device="cuda")
    dw, ws = flce.embedding_backward(dy, ids, 10)
    assert flce.read_device_status(ws) == 5
    assert torch.equal(dw[3], dy[0] + dy[6]) and torch.equal(dw[4], dy[2])
    assert not dw[[0, 1, 2, 5, 6, 7, 8, 9]].any()
    flce.embedding_backward(dy[:1], ids[:1], 10, ws=ws)
    assert flce.read_device_status(ws) == 0


@pytest.mark.gpu
def test_non_finite_rows_stay_in_their_own():
    n, h, v = 4000, 24, 50
    ids = tokens(n, v, "zipf").cuda()
    dy = torch.randn(n, h, device="cuda")
    clean, _ = flce.embedding_backward(dy, ids, v)
    for value in (float("nan"), float("inf")):
        hurt = dy.clone()
        hurt[17, 5] = value
        dw, _ = flce.embedding_backward(hurt, ids, v)
        same = torch.ones(v, h, dtype=torch.bool, device="cuda")
        same[ids[17].long(), 5] = False
        assert torch.equal(dw[same], clean[same]) and not torch.isfinite(dw[~same]).any()


@pytest.mark.gpu
def test_same_bits_whatever_the_workspace_holds():
    n, h, v = 20000, 136, 1000
    ids, dy = tokens(n, v, "zipf").cuda(), torch.randn(n, h, device="cuda")
    size = flce.embedding_workspace_bytes(n, h, v)
    got = []
    for fill in (0, 255, 0x7f):
        ws = torch.full((size + 512,), fill, dtype=torch.uint8, device="cuda")
        dw, _ = flce.embedding_backward(dy, ids, v, ws=ws[:size], check=True)
        assert (ws[size:] == fill).all()
        got.append(dw)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ----------------------------------------------------------------------------- as a user has them


@pytest.mark.gpu
def test_autograd():
    """The gradient that autograd gets, against the formula's and against differences."""
    w = torch.randn(30, 12, device="cuda", requires_grad=True)
    ids = torch.randint(0, 30, (3, 7), device="cuda")
    c = torch.randn(3, 7, 12, device="cuda")
    y = flce.embedding(ids, w, scale=1.5, padding_idx=4)
    assert y.shape == (3, 7, 12)
    (y * c).sum().backward()
    total, size, count = gradient64(c.view(21, 12), ids.view(-1).int(), 30, 1.5, pad=4)
    within(w.grad, total, size * U * (count + 4), "gradient")
    d = torch.randn_like(w)
    d[4] = 0
    f = [(flce.embedding(ids, w.detach() + s * d, scale=1.5).double() * c).sum() for s in (0.25, -0.25)]
    # linear in w: differences are exact but for the roundings of w + s d and of the products
    assert abs((f[0] - f[1]) / 0.5 - (total * d).sum()) <= 8 * U * ((w.detach().abs() + d.abs()) * size).sum()
    # an upstream gradient that is one number spread out
    w.grad = None
    flce.embedding(ids, w).sum().backward()
    assert torch.equal(w.grad.sum(1), 12.0 * torch.bincount(ids.view(-1), minlength=30))


@pytest.mark.gpu
def test_completes_the_gradient_of_a_tied_head():
    """One matrix embeds and projects: the head's dW, then the embedding's part added in place,
    against both products in 64 bits from the same bf16 values.  bf16 holds dW twice and G once."""
    n, h, v = 300, 64, 500
    w = (0.1 * torch.randn(v, h, device="cuda")).to(BF16)
    ids, labels = tokens(n, v, "zipf").cuda(), tokens(n, v, "uniform", 1).cuda()
    x, _ = flce.embedding_forward(ids, w, scale=8.0)
    _, _, dx, dw, _ = flce.fwd_bwd(x, w, labels)
    head = dw.clone()
    flce.embedding_backward(dx, ids, v, scale=8.0, add_to=dw, check=True)
    total, size, count = gradient64(dx, ids, v, 8.0)
    want = head.double() + total
    within(dw, want, size * U * (count + 4) + want.abs() * (half_step(BF16) * 1.001 + U), "dW")
    w64 = w.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy((w64[ids.long()] * 8.0) @ w64.t(), labels.long())
    loss.backward()
    assert (dw.double() - w64.grad).norm() <= 4 * 2.0 ** -8 * w64.grad.norm()


@pytest.mark.gpu
def test_graph_replays_and_streams():
    n, h, v = 500, 40, 90
    w = torch.randn(v, h, device="cuda").to(BF16)
    ids, dy = tokens(n, v, "zipf").cuda(), torch.randn(n, h, device="cuda").to(BF16)
    ws = torch.empty(flce.embedding_workspace_bytes(n, h, v), dtype=torch.uint8, device="cuda")
    flce.embedding_forward(ids, w, ws=ws)
    flce.embedding_backward(dy, ids, v, ws=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = flce.embedding_forward(ids, w, scale=2.0, ws=ws)
        dw, _ = flce.embedding_backward(dy, ids, v, scale=2.0, ws=ws)
    for seed in (7, 8):
        ids.copy_(tokens(n, v, "zipf", seed))
        graph.replay()
        assert torch.equal(y, flce.embedding_forward(ids, w, scale=2.0)[0])
        assert torch.equal(dw, flce.embedding_backward(dy, ids, v, scale=2.0)[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y2, _ = flce.embedding_forward(ids, w, scale=2.0, stream=side)
    dw2, _ = flce.embedding_backward(dy, ids, v, scale=2.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, y2) and torch.equal(dw, dw2)


@pytest.mark.gpu
def test_python_refuses():
    w = torch.zeros(10, 8, device="cuda")
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    dy = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError):
        flce.embedding_forward(ids, w.t())
    with pytest.raises(ValueError):
        flce.embedding_forward(ids[::2], w)
    with pytest.raises(TypeError):
        flce.embedding_forward(ids, w.half())
    with pytest.raises(ValueError):
        flce.embedding_forward(ids.cpu(), w)
    with pytest.raises(ValueError):
        flce.embedding_backward(dy[:3], ids, 10)
    with pytest.raises(ValueError):
        flce.embedding_backward(dy, ids, 10, add_to=w[:9])
    with pytest.raises(TypeError):
        flce.embedding_backward(dy, ids, 10, add_to=w, dtype=BF16)
    with pytest.raises(flce.FlceError):
        flce.embedding_backward(dy, ids, 10, padding_idx=10)
    with pytest.raises(flce.FlceError):
        flce.embedding_backward(dy, ids, 10, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
