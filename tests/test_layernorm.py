"""Layer norm: the kernels against the formula in 64 bits, at the sizes, types,
alignments and values where they can go wrong, and the calls they refuse.

Tolerances (u = 2^-24, the unit roundoff of fp32).  A sum of m terms in fp32 is off
by at most m u times the sum of their magnitudes; the kernels sum a row or a column
in partial sums no longer than ``chain`` additions, so

  mean:  chain u mean|x|                     (plus one rounding)
  rstd:  relative 0.5 (the variance's relative error) <= 2 (chain + 4) u, once the
         mean's own error e adds e^2 to the variance
  y:     |weight| rstd (the mean's error + 2 u |x - mean|) + relative errors, then half
         an ulp of the output type (2^-8 relative in bf16, whose significand has 8 bits)
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding  # noqa: E402

U = 2.0 ** -24
CHAIN = 300  # additions on the longest path of a sum over a row of at most 65536 elements: h / 256 and the tree


def reference(x, weight, bias, eps, dy=None):
    """64-bit forward, or with dy backward: the formulas themselves."""
    x, w = x.double(), weight.double()
    mean = x.mean(1, keepdim=True)
    rstd = ((x - mean).square().mean(1, keepdim=True) + eps) ** -0.5
    xhat = (x - mean) * rstd
    if dy is None:
        y = xhat * w + (0 if bias is None else bias.double())
        return y, mean[:, 0], rstd[:, 0]
    dy = dy.double()
    u = dy * w
    dx = rstd * (u - u.mean(1, keepdim=True) - xhat * (u * xhat).mean(1, keepdim=True))
    return dx, (dy * xhat).sum(0), dy.sum(0)


def half_ulp(ref, dtype):
    return ref.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else U) + 1e-38


def make(n, h, dtype, wdtype, seed=0, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, generator=g) * (0.5 + torch.rand(n, 1, generator=g)) + offset
    w = 1 + 0.3 * torch.randn(h, generator=g)
    b = 0.2 * torch.randn(h, generator=g)
    dy = torch.randn(n, h, generator=g)
    return [t.to(d) for t, d in ((x, dtype), (w, wdtype), (b, wdtype), (dy, dtype))]


def assert_within(got, want, tol, name):
    got, want = got.double().cpu(), want.double().cpu()
    bad = (got - want).abs() > tol.double().cpu()
    assert not bad.any(), f"{name}: {int(bad.sum())} outside, worst {(got - want).abs().max():.3e}"


def check_forward(x, w, b, eps, got):
    y, mean, rstd = got
    ry, rmean, rrstd = reference(x, w, b, eps)
    xd = x.double()
    mean_err = (CHAIN + 2) * U * xd.abs().mean(1) + U * rmean.abs()
    assert_within(mean, rmean, mean_err, "mean")
    # variance about a mean that is e off: + e^2; its own sum's relative error (CHAIN + 4) u
    rel = (CHAIN + 6) * U + mean_err.square() * rrstd.square()
    assert_within(rstd, rrstd, rrstd * rel, "rstd")
    wd = w.double().abs()
    dev = (xd - rmean[:, None]).abs()
    tol = wd * rrstd[:, None] * (mean_err[:, None] + dev * (rel[:, None] + 4 * U)) + 2 * U * ry.abs()
    if b is not None:
        tol = tol + 2 * U * (wd * rrstd[:, None] * dev + b.double().abs())
    assert_within(y, ry, tol + half_ulp(ry, x.dtype), "y")


def check_backward(x, w, dy, mean, rstd, got):
    """Against the formula with the same mean and rstd (they are inputs of the call)."""
    dx, dweight, dbias = got
    xd, wd, d = x.double(), w.double(), dy.double()
    rs = rstd.double()[:, None]
    xhat = (xd - mean.double()[:, None]) * rs
    u = d * wd
    m1, m2 = u.mean(1, keepdim=True), (u * xhat).mean(1, keepdim=True)
    ref = rs * (u - m1 - xhat * m2)
    e1 = (CHAIN + 3) * U * u.abs().mean(1, keepdim=True)
    e2 = (CHAIN + 6) * U * (u * xhat).abs().mean(1, keepdim=True)
    xerr = 3 * U * xhat.abs() + U * (xd.abs() + mean.double().abs()[:, None]) * rs
    tol = rs * (e1 + e2 * xhat.abs() + xerr * m2.abs() + 6 * U * (u.abs() + m1.abs() + (xhat * m2).abs()))
    assert_within(dx, ref, tol + half_ulp(ref, x.dtype), "dx")
    n = x.shape[0]
    col = (min(n, 600 + n // 100) + 4) * U  # rows in one chain, the chains' joining
    rw, rb = (d * xhat).sum(0), d.sum(0)
    assert_within(dweight, rw, col * (d * xhat).abs().sum(0) + (d.abs() * xerr).sum(0) + half_ulp(rw, w.dtype) + 1e-38,
                  "dweight")
    if dbias is not None:
        assert_within(dbias, rb, col * d.abs().sum(0) + half_ulp(rb, w.dtype) + 1e-38, "dbias")


TYPES = [(torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float32, torch.float32),
         (torch.float32, torch.bfloat16)]
SIZES = [(1, 1), (1, 8), (3, 7), (2, 16), (5, 1000), (257, 2048), (33, 4096), (64, 8192), (17, 16392), (9, 20001),
         (300, 1031), (2, 65536), (4099, 24), (1000, 520), (777, 1544), (2500, 4096),
         (7000, 1), (5000, 33), (3000, 250), (2000, 999), (1500, 2049), (900, 4100), (700, 4089), (400, 8185), (300, 16377)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", SIZES)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_forward_and_backward(n, h, dtype, wdtype):
    x, w, b, dy = make(n, h, dtype, wdtype, seed=n + h)
    gx, gw, gb, gdy = (t.cuda() for t in (x, w, b, dy))
    y, mean, rstd = flce.layernorm_forward(gx, gw, gb, eps=1e-5)
    check_forward(gx, gw, gb, 1e-5, (y, mean, rstd))
    dx, dweight, dbias, ws = flce.layernorm_backward(gdy, gx, gw, mean, rstd)
    check_backward(gx, gw, gdy, mean, rstd, (dx, dweight, dbias))
    again = flce.layernorm_backward(gdy, gx, gw, mean, rstd, ws=ws)[:3]
    for a, c in zip((dx, dweight, dbias), again):
        assert torch.equal(a, c)  # fixed order of every sum


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_bias(dtype):
    x, w, _, dy = (t.cuda() for t in make(37, 264, dtype, torch.float32))
    got = flce.layernorm_forward(x, w)
    check_forward(x, w, None, 1e-5, got)
    dx, dweight, dbias, _ = flce.layernorm_backward(dy, x, w, got[1], got[2], bias=False)
    assert dbias is None
    check_backward(x, w, dy, got[1], got[2], (dx, dweight, None))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("h,pitch,at", [(512, 4096, 0), (512, 1027, 3), (505, 1024, 1), (4096, 4104, 8), (64, 65, 1)])
def test_rows_of_a_larger_tensor(dtype, h, pitch, at):
    """Row pitches and offsets that leave rows unaligned for vector loads."""
    n = 21
    _, w, b, dy = (t.cuda() for t in make(n, h, dtype, torch.float32, seed=pitch))
    big = torch.randn(n, pitch, generator=torch.Generator().manual_seed(at)).to(dtype).cuda()
    x = big[:, at:at + h]
    got = flce.layernorm_forward(x, w, b)
    check_forward(x, w, b, 1e-5, got)
    dx, dweight, dbias, _ = flce.layernorm_backward(dy, x, w, got[1], got[2])
    check_backward(x, w, dy, got[1], got[2], (dx, dweight, dbias))


# many rows whose length no 16-byte access divides, at every width of the kernels that take them
PHASES = [(13000, 250), (8000, 501), (6500, 761), (8193, 137), (8200, 999), (8201, 1501), (9000, 2041), (1600, 2060),
          (1600, 3001), (1100, 4003), (1027, 5001), (500, 7001)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h", PHASES)
@pytest.mark.parametrize("dtype,wdtype", TYPES)
def test_rows_at_every_phase(n, h, dtype, wdtype):
    test_forward_and_backward(n, h, dtype, wdtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_a_larger_tensor_at_every_phase(dtype):
    """A pitch that leaves x's rows at the phases of contiguous ones."""
    n, h, pitch, at = 2100, 2051, 2067, 8
    _, w, b, dy = (t.cuda() for t in make(n, h, dtype, torch.float32, seed=pitch))
    big = torch.randn(n, pitch, generator=torch.Generator().manual_seed(at)).to(dtype).cuda()
    x = big[:, at:at + h]
    got = flce.layernorm_forward(x, w, b)
    check_forward(x, w, b, 1e-5, got)
    dx, dweight, dbias, _ = flce.layernorm_backward(dy, x, w, got[1], got[2])
    check_backward(x, w, dy, got[1], got[2], (dx, dweight, dbias))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,h", [(2100, 2051), (9000, 509)])
def test_non_finite_rows_do_not_reach_their_neighbours(dtype, n, h):
    """An access at a row's start may hold the end of the row before."""
    x, w, b, dy = (t.cuda() for t in make(n, h, dtype, torch.float32))
    clean = flce.layernorm_forward(x, w, b)
    clean_dx = flce.layernorm_backward(dy, x, w, clean[1], clean[2])[0]
    bad = torch.arange(3, n, 17, device="cuda")
    x2, dy2 = x.clone(), dy.clone()
    x2[bad], dy2[bad] = float("nan"), float("inf")
    got = flce.layernorm_forward(x2, w, b)
    dx = flce.layernorm_backward(dy2, x2, w, clean[1], clean[2])[0]
    keep = torch.ones(n, dtype=torch.bool, device="cuda")
    keep[bad] = False
    for a, c in zip(got, clean):
        assert torch.equal(a[keep], c[keep])
    assert torch.equal(dx[keep], clean_dx[keep])


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["weight", "dy"])
def test_unaligned_vectors(which):
    """weight, bias and dy that start between vector boundaries."""
    n, h = 19, 1024
    x, w, b, dy = (t.cuda() for t in make(n, h, torch.bfloat16, torch.bfloat16))
    if which == "weight":
        w, b = (torch.cat([t[:1], t])[1:] for t in (w, b))
        assert w.data_ptr() % 16 == 2
    else:
        dy = torch.cat([dy.flatten()[:1], dy.flatten()])[1:].view(n, h)
    got = flce.layernorm_forward(x, w, b)
    check_forward(x, w, b, 1e-5, got)
    dx, dweight, dbias, _ = flce.layernorm_backward(dy, x, w, got[1], got[2])
    check_backward(x, w, dy, got[1], got[2], (dx, dweight, dbias))


@pytest.mark.gpu
@pytest.mark.parametrize("h", [7, 512, 4096, 16400])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_constant_rows_and_large_offsets(h, dtype):
    """Variance zero leaves rstd = 1 / sqrt(eps) and y = bias; an offset 100 times the
    spread is taken out before the squares are summed."""
    x, w, b, _ = make(8, h, dtype, torch.float32, seed=3)
    x[0] = 0
    x[1] = 2.0
    x[2:5] = (x[2:5].float() + 100).to(dtype)
    x, w, b = x.cuda(), w.cuda(), b.cuda()
    y, mean, rstd = flce.layernorm_forward(x, w, b, eps=1e-6)
    check_forward(x, w, b, 1e-6, (y, mean, rstd))
    assert float(rstd[0]) == pytest.approx(1e3, rel=1e-6)
    assert torch.equal(y[0], b.to(dtype))


@pytest.mark.gpu
@pytest.mark.parametrize("h", [33, 1024, 20000])
def test_non_finite_rows_stay_by_themselves(h):
    x, w, b, dy = (t.cuda() for t in make(9, h, torch.bfloat16, torch.float32))
    clean = flce.layernorm_forward(x, w, b)
    x2 = x.clone()
    x2[2, h // 2], x2[5, 0], x2[7, h - 1] = float("inf"), float("nan"), float("-inf")
    y, mean, rstd = flce.layernorm_forward(x2, w, b)
    rest = [0, 1, 3, 4, 6, 8]
    for r in (2, 5, 7):
        assert torch.isnan(y[r]).all()
    for a, c in zip((y, mean, rstd), clean):
        assert torch.equal(a[rest], c[rest])
    dx, _, _, _ = flce.layernorm_backward(dy, x2, w, mean, rstd)
    dx0, _, _, _ = flce.layernorm_backward(dy, x, w, clean[1], clean[2])
    assert torch.equal(dx[rest], dx0[rest]) and not torch.isfinite(dx[[2, 5, 7]].float()).any()


@pytest.mark.gpu
def test_empty_batch():
    w = torch.ones(64, device="cuda")
    x = torch.empty(0, 64, device="cuda")
    y, mean, rstd = flce.layernorm_forward(x, w, w)
    assert y.shape == (0, 64) and mean.numel() == rstd.numel() == 0
    dx, dweight, dbias, _ = flce.layernorm_backward(x, x, w, mean, rstd)
    assert dx.shape == (0, 64) and not dweight.any() and not dbias.any()


@pytest.mark.gpu
def test_offsets_past_32_bits():
    """The last rows of an x of more than 2^31 elements."""
    h, n = 8192, (1 << 18) + 40
    x = torch.empty(n, h, dtype=torch.bfloat16, device="cuda")
    tail, w, b, _ = (t.cuda() for t in make(16, h, torch.bfloat16, torch.float32))
    x[:-16] = 1.0
    x[-16:] = tail
    y, mean, rstd = flce.layernorm_forward(x, w, b)
    check_forward(tail, w, b, 1e-5, (y[-16:], mean[-16:], rstd[-16:]))
    assert torch.equal(y[0], b.to(torch.bfloat16))
    dx, dweight, dbias, _ = flce.layernorm_backward(x, x, w, mean, rstd)  # dy = x
    check_backward(tail, w, tail, mean[-16:], rstd[-16:], (dx[-16:], *reference_dw(tail, mean[-16:], rstd[-16:], w)))
    # constant rows have xhat = 0: only the tail reaches dweight; dbias counts the ones
    rw = (tail.double() * (tail.double() - mean[-16:].double()[:, None]) * rstd[-16:].double()[:, None]).sum(0)
    assert_within(dweight, rw, rw.abs() * 1e-5 + 1e-4, "dweight")
    rb = tail.double().sum(0) + (n - 16)
    assert_within(dbias, rb, rb.abs() * (600 + n // 100) * U, "dbias")


def reference_dw(tail, mean, rstd, w):
    """Column sums of the tail itself, so that check_backward's comparison of them is an identity."""
    d = tail.double()
    xhat = (d - mean.double()[:, None]) * rstd.double()[:, None]
    return (d * xhat).sum(0).to(w.dtype), d.sum(0).to(w.dtype)


@pytest.mark.gpu
def test_on_another_stream():
    x, w, b, dy = (t.cuda() for t in make(2000, 2048, torch.bfloat16, torch.float32))
    want = flce.layernorm_forward(x, w, b)
    want_b = flce.layernorm_backward(dy, x, w, want[1], want[2])[:3]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = flce.layernorm_forward(x, w, b, stream=s)
    got_b = flce.layernorm_backward(dy, x, w, got[1], got[2], stream=s)[:3]
    torch.cuda.current_stream().wait_stream(s)
    for a, c in zip(got + got_b, want + want_b):
        assert torch.equal(a, c)


@pytest.mark.gpu
def test_autograd_against_differences():
    """The wrapper's gradients of sum(c y) against central differences of the 64-bit
    forward, along random directions: the differences' own error is O(step^2)."""
    x, w, b, c = (t.cuda() for t in make(6, 96, torch.float32, torch.float32, seed=8))
    shaped = [t.clone().requires_grad_() for t in (x.view(2, 3, 96), w, b)]
    (flce.layer_norm(*shaped, eps=1e-5) * c.view(2, 3, 96)).sum().backward()

    def value(xv, wv, bv):
        return float((reference(xv, wv, bv, 1e-5)[0] * c.double()).sum())

    g = torch.Generator().manual_seed(1)
    base = [t.double() for t in (x, w, b)]
    for k in range(3):
        for _ in range(4):
            d = torch.randn(base[k].shape, generator=g, dtype=torch.float64).cuda()
            lo, hi = list(base), list(base)
            lo[k], hi[k] = base[k] - 1e-4 * d, base[k] + 1e-4 * d
            slope = (value(*hi) - value(*lo)) / 2e-4
            got = float((shaped[k].grad.reshape(base[k].shape).double() * d).sum())
            assert got == pytest.approx(slope, rel=1e-4, abs=1e-3)


@pytest.mark.gpu
def test_python_refusals_on_gpu():
    x, w, b, dy = (t.cuda() for t in make(4, 64, torch.bfloat16, torch.float32))
    for bad in (lambda: flce.layernorm_forward(x.half(), w), lambda: flce.layernorm_forward(x, w.double())):
        with pytest.raises(TypeError):
            bad()
    y, mean, rstd = flce.layernorm_forward(x, w, b)
    for bad in (lambda: flce.layernorm_forward(x, w[:63]), lambda: flce.layernorm_forward(x[None], w),
                lambda: flce.layernorm_forward(x.t(), w[:4]), lambda: flce.layernorm_forward(x, w, b.bfloat16()),
                lambda: flce.layernorm_forward(x[:1].expand(4, 64), w), lambda: flce.layernorm_forward(x, w.cpu()),
                lambda: flce.layernorm_backward(dy.float(), x, w, mean, rstd),
                lambda: flce.layernorm_backward(dy[:3], x, w, mean, rstd),
                lambda: flce.layernorm_backward(dy, x, w, mean[:3], rstd),
                lambda: flce.layernorm_backward(dy, x, w, mean, rstd.double())):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(flce.FlceError) as e:
        flce.layernorm_backward(dy, x, w, mean, rstd, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.code == 4


def test_host_refusals():
    """Bad arguments come back as errors before any GPU call."""
    L, Q = flce.lib(), binding.Norm
    z = 0x1000

    def fwd(q, x=z, w=z, b=z, y=z, mean=z, rstd=z):
        return L.flce_layernorm_forward(ctypes.byref(q), x, w, b, y, mean, rstd, None)

    def bwd(q, dy=z, x=z, w=z, mean=z, rstd=z, dx=z, dw=z, db=z, ws=0x100000, nbytes=1 << 30):
        return L.flce_layernorm_backward(ctypes.byref(q), dy, x, w, mean, rstd, dx, dw, db, ws, nbytes, None)

    ok = Q(4, 64, 64, 1e-5, 0, 1)
    assert L.flce_layernorm_forward(None, z, z, z, z, z, z, None) == 1
    for q in (Q(-1, 64, 64, 1e-5, 0, 1), Q(4, 0, 64, 1e-5, 0, 1), Q(4, 64, 63, 1e-5, 0, 1), Q(4, 64, 64, -1.0, 0, 1),
              Q(4, 64, 64, float("nan"), 0, 1), Q(4, 64, 64, 1e-5, 2, 1), Q(4, 64, 64, 1e-5, 0, -1)):
        assert fwd(q) == 1 and bwd(q) == 1
        assert L.flce_layernorm_workspace_bytes(ctypes.byref(q)) == 0
    for q in (Q(4, (1 << 20) + 1, 1 << 21, 1e-5, 0, 1), Q(1 << 33, 64, 1024, 1e-5, 0, 1)):
        assert fwd(q) == 2 and bwd(q) == 2
    for name in ("x", "w", "y", "mean", "rstd"):
        assert fwd(ok, **{name: None}) == 1
        assert fwd(ok, **{name: z + 1}) == 3
    assert fwd(ok, b=z + 2) == 3
    for name in ("dy", "x", "w", "mean", "rstd", "dx", "dw", "ws"):
        assert bwd(ok, **{name: None}) == 1
        assert bwd(ok, **{name: z + 1}) == 3
    assert bwd(ok, nbytes=16) == 4
    assert fwd(Q(0, 64, 64, 1e-5, 0, 1), x=None, y=None, mean=None, rstd=None) == 0  # nothing to do
    assert fwd(Q(0, 64, 64, 1e-5, 0, 1), w=None) == 1
    n = flce.layernorm_workspace_bytes
    assert n(131072, 4096) % 256 == 0 and n(131072, 4096) < 1 << 25 and n(1, 1) >= 256


def test_reference_backward_against_differences():
    """The 64-bit backward used above against central differences of the 64-bit forward."""
    x, w, b, c = (t.double() for t in make(3, 17, torch.float32, torch.float32, seed=5))
    dx, dw, db = reference(x, w, b, 1e-3, dy=c)
    rng = np.random.default_rng(0)
    for grad, k in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        for _ in range(5):
            d = torch.from_numpy(rng.standard_normal(tuple(args[k].shape)))
            hi, lo = list(args), list(args)
            hi[k], lo[k] = args[k] + 1e-5 * d, args[k] - 1e-5 * d
            slope = ((reference(*hi, 1e-3)[0] - reference(*lo, 1e-3)[0]) * c).sum() / 2e-5
            assert float((grad * d).sum()) == pytest.approx(float(slope), rel=1e-6, abs=1e-7)
