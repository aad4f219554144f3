"""Token log probabilities, entropies and top alternatives: the kernels against the
definition in 64 bits, at the sizes and values where they can go wrong, and the calls
they refuse.

Most inputs lie on 8-bit grids (x in steps of 2^-5, w in a power-of-two step), so that
every logit is an fp32 number whatever the order of its sum: then the alternatives have
one right answer (the lowest id first among equal logits), and the tolerances are those
of the softmax alone (u = 2^-24).  A row's sum of exponentials runs over at most
``chain`` = V / 128 + 100 additions in a thread and then the joining of partial sums; an
exponential is good to 2^-21 and to |t - m| u, t - m its distance from the maximum in
log2 units.  So
  lse:      (chain + 16) u + 6 u |lse|
  logprob:  the same with |z - lse| in the last term, and 2 u max|z|: one rounding of a
            scaled logit and of the maximum it is taken against
  entropy:  (chain + 16) u (1 + mean|t - m|) + 8 u (entropy + mean|t - m|)
G, the gradient's [N, V] factor, is held in bf16 (2^-8 relative): dX and dW are within
2^-8 of the products of magnitudes, and half an ulp of their own.
"""
import ctypes
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from helpers import LSE_ATOL  # noqa: E402
from lm_head_cross_gb300 import binding  # noqa: E402

U = 2.0 ** -24
BF16 = torch.bfloat16


def grid_inputs(n, h, v, seed=0, ties=True):
    g = torch.Generator().manual_seed(seed)
    step = 2.0 ** -(5 + math.ceil(math.log2(h) / 2))
    kw = torch.randn(v, h, generator=g).mul_(60).round_().clamp_(-127, 127)
    if ties and v > 3:  # equal rows: equal logits, near each other and far apart
        kw[v - 1], kw[v // 2] = kw[0], kw[1]
        kw[2] = kw[1]
    tok = torch.randint(0, v, (n,), generator=g)
    lean = torch.rand(n, 1, generator=g) * (max(math.log(v) - 1, 0) / (h * 60 * step))
    x = torch.randn(n, h, generator=g) + lean * kw[tok] / 60
    x = (x * 32).round_().clamp_(-127, 127) / 32
    return x.to(BF16).cuda(), (kw * step).to(BF16).cuda(), tok.to(torch.int32).cuda()


def reference(x, w, tok, k, temperature, ignore_index=-100):
    """The definition in 64 bits, on the GPU in row blocks."""
    out = {"logprob": [], "entropy": [], "lse": [], "ids": [], "top": [], "dist": [], "zmax": []}
    wd = w.double()
    for lo in range(0, x.shape[0], 512):
        raw = x[lo:lo + 512].double() @ wd.t()
        z = raw / temperature
        lse = torch.logsumexp(z, 1)
        lp = z - lse[:, None]
        p = lp.exp()
        out["lse"].append(lse)
        out["entropy"].append(-(p * lp).sum(1))
        out["dist"].append((p * (z.amax(1, keepdim=True) - z)).sum(1) / math.log(2))
        out["zmax"].append(z.abs().amax(1))
        if tok is not None:
            t = tok[lo:lo + 512].long()
            ok = t != ignore_index
            got = lp.gather(1, torch.where(ok, t, 0)[:, None])[:, 0]
            out["logprob"].append(torch.where(ok, got, 0.0))
        if k:
            top = raw.sort(dim=1, descending=True, stable=True)  # stable: the lowest id first
            out["ids"].append(top.indices[:, :k])
            out["top"].append(lp.gather(1, top.indices[:, :k]))
    return {key: torch.cat(v) if v else None for key, v in out.items()}


def within(got, want, tol, name):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), f"{name}: {int(bad.sum())} outside, worst {(got.double() - want).abs().max():.3e}"


def check(r, x, w, tok, k, temperature, ignore_index=-100):
    ref = reference(x, w, tok, min(k, w.shape[0]), temperature, ignore_index)
    base = (w.shape[0] / 128 + 116) * U
    within(r.lse, ref["lse"], base + 6 * U * ref["lse"].abs(), "lse")
    within(r.entropy, ref["entropy"], base * (1 + ref["dist"]) + 8 * U * (ref["entropy"] + ref["dist"]), "entropy")
    lp_tol = lambda z, m: base + 6 * U * z.abs() + 4 * U * m  # noqa: E731
    if tok is None:
        assert r.logprob is None
    else:
        within(r.logprob, ref["logprob"], lp_tol(ref["logprob"], ref["zmax"]), "logprob")
        assert (r.logprob[tok == ignore_index] == 0).all()
    if k == 0:
        assert r.top_ids is None and r.top_logprobs is None
        return
    have = min(k, w.shape[0])
    assert torch.equal(r.top_ids[:, :have].long(), ref["ids"])
    within(r.top_logprobs[:, :have], ref["top"], lp_tol(ref["top"], ref["zmax"][:, None]), "top_logprobs")
    if have < k:
        assert (r.top_ids[:, have:] == -1).all() and (r.top_logprobs[:, have:] == -math.inf).all()


CASES = [
    # n, h, v, k, temperature
    (1, 8, 1, 1, 1.0), (1, 8, 2, 16, 1.0), (3, 72, 5, 8, 0.5), (1, 64, 17, 16, 2.0), (2, 128, 100, 0, 1.0),
    (1, 2048, 4099, 5, 1.0), (1, 4096, 32000, 16, 0.7), (7, 200, 1000, 3, 1.0), (15, 1544, 2050, 16, 1.3),
    (16, 64, 131072, 8, 1.0), (17, 512, 3001, 1, 1.0), (32, 2048, 777, 2, 0.7), (33, 136, 20000, 16, 1.0),
    (64, 1024, 8191, 8, 1.0), (65, 72, 300, 4, 1.0), (100, 4096, 5003, 0, 1.3), (127, 8, 256, 16, 1.0),
    (128, 512, 257, 5, 1.0), (129, 512, 4097, 16, 0.7), (200, 256, 40009, 7, 1.0), (256, 128, 1024, 16, 1.0),
    (257, 512, 4099, 16, 2.0), (513, 128, 777, 0, 1.0), (777, 264, 40009, 16, 1.3), (1000, 64, 2050, 1, 1.0),
    (2600, 72, 5001, 16, 1.0), (3000, 2048, 1023, 0, 0.7),
    (300, 2056, 5003, 16, 1.0), (700, 1032, 9001, 8, 1.3), (135, 4096, 3001, 3, 1.0),
    (20, 72, 50001, 0, 1.0), (40, 72, 50001, 16, 1.0), (20, 4104, 39001, 16, 0.7), (60, 4096, 39001, 0, 1.0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,v,k,temperature", CASES)
def test_forward(n, h, v, k, temperature):
    x, w, tok = grid_inputs(n, h, v, seed=n + v)
    tok[::5] = -100
    r, ws = flce.logprobs_forward(x, w, tok, top=k, temperature=temperature, check=True)
    check(r, x, w, tok, k, temperature)
    again, _ = flce.logprobs_forward(x, w, tok, top=k, temperature=temperature, ws=ws)
    for a, b in zip(r, again):
        assert a is None or torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 40, 300])
def test_without_tokens_and_with_an_ignore_index_in_the_vocabulary(n):
    x, w, tok = grid_inputs(n, 256, 3000, seed=n)
    r, _ = flce.logprobs_forward(x, w, top=4, check=True)
    check(r, x, w, None, 4, 1.0)
    tok[: max(1, n // 3)] = 7
    r, _ = flce.logprobs_forward(x, w, tok, ignore_index=7, check=True)
    check(r, x, w, tok, 0, 1.0, ignore_index=7)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [2, 60, 400])
def test_edge_tokens_and_all_ignored(n):
    v = 5000
    x, w, tok = grid_inputs(n, 128, v, seed=3)
    tok[0], tok[1] = 0, v - 1
    r, _ = flce.logprobs_forward(x, w, tok, check=True)
    check(r, x, w, tok, 0, 1.0)
    tok[:] = -100
    r, _ = flce.logprobs_forward(x, w, tok, top=2, check=True)
    assert not r.logprob.any()
    check(r, x, w, tok, 2, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 20, 300])
def test_every_logit_equal(n):
    """Equal weights: entropy ln V, alternatives 0 .. k - 1."""
    v, k = 3333, 16
    x, w, tok = grid_inputs(n, 64, v, ties=False)
    w[:] = w[0]
    r, _ = flce.logprobs_forward(x, w, tok, top=k, check=True)
    assert torch.equal(r.top_ids, torch.arange(k, device="cuda", dtype=torch.int32).expand(n, k))
    within(r.entropy, torch.full((n,), math.log(v), device="cuda", dtype=torch.float64), (v / 128 + 116) * U, "entropy")
    within(r.logprob, torch.full((n,), -math.log(v), device="cuda", dtype=torch.float64),
           (v / 128 + 116 + 100) * U, "logprob")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 50, 300])
@pytest.mark.parametrize("temperature", [0.01, 100.0])
def test_peaked_and_flat(n, temperature):
    """A low temperature leaves one token with nearly all of the mass: log probabilities of
    -100s and an entropy near 0; a high one an entropy near ln V."""
    x, w, tok = grid_inputs(n, 512, 4000, seed=9)
    r, _ = flce.logprobs_forward(x, w, tok, top=3, temperature=temperature, check=True)
    check(r, x, w, tok, 3, temperature)
    assert (r.entropy >= -1e-6).all()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 60, 300])
def test_certain_tokens_stay_on_their_side_of_zero(n):
    """One logit far above all others, at scales whose product with log2 e rounds: log
    probability at most 0, entropy at least 0, both within rounding of it."""
    v = 700
    x = torch.linspace(1, 9, n, device="cuda")[:, None].expand(n, 64).to(BF16).contiguous()
    w = torch.zeros(v, 64, dtype=BF16, device="cuda")
    w[123] = 0.77
    r, _ = flce.logprobs_forward(x, w, torch.full((n,), 123, dtype=torch.int32, device="cuda"), top=2, check=True)
    assert (r.logprob <= 0).all() and (r.top_logprobs <= 0).all() and (r.entropy >= 0).all()
    check(r, x, w, torch.full((n,), 123, dtype=torch.int32, device="cuda"), 2, 1.0)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 90, 500])
def test_inputs_off_the_grid(n):
    """Ordinary bf16 values: the logits' own fp32 sums are within the library's promise."""
    g = torch.Generator().manual_seed(n)
    x, w = torch.randn(n, 1032, generator=g).to(BF16).cuda(), (0.05 * torch.randn(5003, 1032, generator=g)).to(BF16).cuda()
    tok = torch.randint(0, 5003, (n,), generator=g).to(torch.int32).cuda()
    r, _ = flce.logprobs_forward(x, w, tok, top=5, check=True)
    ref = reference(x, w, tok, 5, 1.0)
    for a, b in ((r.lse, ref["lse"]), (r.logprob, ref["logprob"]), (r.entropy, ref["entropy"]),
                 (r.top_logprobs, ref["top"])):
        within(a, b, LSE_ATOL, "off the grid")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [4, 70, 300])
def test_non_finite_rows_stay_by_themselves(n):
    x, w, tok = grid_inputs(n, 128, 2000, seed=1)
    clean, _ = flce.logprobs_forward(x, w, tok, top=3)
    x[n // 2, 5] = float("nan")
    r, _ = flce.logprobs_forward(x, w, tok, top=3, check=True)
    keep = torch.arange(n, device="cuda") != n // 2
    for a, b in zip(r, clean):
        assert torch.equal(a[keep], b[keep])
    for a in (r.lse, r.entropy, r.logprob):
        assert torch.isnan(a[n // 2])


@pytest.mark.gpu
@pytest.mark.parametrize("n", [3, 128, 260])
def test_an_infinite_weight_bans_its_token(n):
    """A logit of minus infinity has probability 0 and no share in the entropy."""
    x, w, tok = grid_inputs(n, 64, 1000, seed=2, ties=False)
    x[:, 0] = 1.0
    w2 = w.clone()
    w2[11, 0] = w2[999, 0] = -float("inf")
    tok[:] = 5
    r, _ = flce.logprobs_forward(x, w2, tok, top=4, check=True)
    keep = [j for j in range(1000) if j not in (11, 999)]
    ref = reference(x, w[keep], tok, 4, 1.0)
    base = (1000 / 128 + 116) * U
    within(r.lse, ref["lse"], base + 6 * U * ref["lse"].abs(), "lse")
    within(r.entropy, ref["entropy"], base * (1 + ref["dist"]) + 8 * U * (ref["entropy"] + ref["dist"]), "entropy")
    ids = torch.tensor(keep, device="cuda")[ref["ids"]]
    assert torch.equal(r.top_ids.long(), ids)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 8, 40, 100, 260])
@pytest.mark.parametrize("v,banned", [(3000, 700), (90000, 40000)])
def test_whole_ranges_of_banned_tokens(n, v, banned):
    """Blocks of logits that are all minus infinity, first or last in a range: they add nothing."""
    x, w, tok = grid_inputs(n, 64, v, seed=3, ties=False)
    x[:, 0] = 1.0
    w2 = w.clone()
    w2[:banned, 0] = w2[v - 300:, 0] = -float("inf")
    tok[:] = banned + 5
    r, _ = flce.logprobs_forward(x, w2, tok, top=4, check=True)
    ref = reference(x, w[banned:v - 300], tok - banned, 4, 1.0)
    base = (v / 128 + 116) * U
    within(r.lse, ref["lse"], base + 6 * U * ref["lse"].abs(), "lse")
    within(r.entropy, ref["entropy"], base * (1 + ref["dist"]) + 8 * U * (ref["entropy"] + ref["dist"]), "entropy")
    assert torch.equal(r.top_ids.long(), ref["ids"] + banned)


@pytest.mark.gpu
@pytest.mark.parametrize("n", [4, 100, 600])
@pytest.mark.parametrize("bad", [3000, -1, -101, 2 ** 31 - 1])
def test_tokens_out_of_range_are_reported(n, bad):
    x, w, tok = grid_inputs(n, 64, 3000)
    tok[n - 2] = bad
    _, ws = flce.logprobs_forward(x, w, tok, top=1)
    assert flce.read_device_status(ws) == 5
    r, _ = flce.logprobs_forward(x, w, tok.clamp(0, 2999), ws=ws, check=True)  # the next call is clean
    check(r, x, w, tok.clamp(0, 2999), 0, 1.0)
    _, _, wsb = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, torch.ones_like(r.lse))
    assert flce.read_device_status(wsb) == 5


@pytest.mark.gpu
def test_empty_batch():
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.zeros(100, 64, dtype=BF16, device="cuda")
    tok = torch.empty(0, dtype=torch.int32, device="cuda")
    r, _ = flce.logprobs_forward(x, w, tok, top=3)
    assert r.logprob.shape == r.lse.shape == (0,) and r.top_ids.shape == (0, 3)
    dX, dW, _ = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, r.lse, r.lse)
    assert dX.shape == (0, 64) and not dW.any()


@pytest.mark.gpu
@pytest.mark.parametrize("n", [16, 600])
def test_on_another_stream(n):
    x, w, tok = grid_inputs(n, 512, 9000)
    want, _ = flce.logprobs_forward(x, w, tok, top=5)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got, _ = flce.logprobs_forward(x, w, tok, top=5, stream=s)
    torch.cuda.current_stream().wait_stream(s)
    for a, b in zip(got, want):
        assert torch.equal(a, b)


# ----------------------------------------------------------------------------- gradients


def gradients64(x, w, tok, gl, ge, temperature, ignore_index=-100):
    """The formula: dz, and the products with magnitudes that bound bf16's share."""
    xd, wd = x.double(), w.double()
    z = xd @ wd.t() / temperature
    lp = torch.log_softmax(z, 1)
    p = lp.exp()
    ent = -(p * lp).sum(1, keepdim=True)
    dz = torch.zeros_like(z)
    if gl is not None:
        ok = tok != ignore_index
        g = torch.where(ok, gl.double(), 0.0)[:, None]
        dz = dz - g * p
        dz.scatter_add_(1, torch.where(ok, tok.long(), 0)[:, None], g)
    if ge is not None:
        dz = dz - ge.double()[:, None] * p * (lp + ent)
    dz = dz / temperature
    return dz @ wd, dz.t() @ xd, dz.abs() @ wd.abs(), dz.abs().t() @ xd.abs()


GRADS = [(1, 8, 3, 1.0), (5, 64, 100, 0.5), (256, 128, 1024, 1.0), (300, 264, 1000, 1.0), (70, 512, 9000, 1.3),
         (1000, 72, 8200, 0.7), (129, 1544, 2050, 1.0)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,v,temperature", GRADS)
@pytest.mark.parametrize("which", ["logprob", "entropy", "both"])
def test_gradients(n, h, v, temperature, which):
    x, w, tok = grid_inputs(n, h, v, seed=n)
    tok[1::4] = -100
    g = torch.Generator().manual_seed(7)
    gl = torch.randn(n, generator=g).cuda() if which != "entropy" else None
    ge = torch.randn(n, generator=g).cuda() if which != "logprob" else None
    r, _ = flce.logprobs_forward(x, w, tok, temperature=temperature)
    dX, dW, ws = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, gl, ge, temperature=temperature, check=True)
    rX, rW, mX, mW = gradients64(x, w, tok, gl, ge, temperature)
    # p (a + b log2 p) sums terms that may cancel: dz's own fp32 error is small against its
    # magnitudes' row maximum; 1e-5 of the largest product bounds it
    for got, ref, mag, name in ((dX, rX, mX, "dX"), (dW, rW, mW, "dW")):
        within(got, ref, 2.0 ** -8 * (mag * (1 + 2.0 ** -8) + ref.abs()) + 1e-5 * mag.max() + 1e-30, name)
        assert (got.double() - ref).norm() <= 2.0 ** -8 * math.sqrt(2) * ref.norm() + 1e-20, name
    if which == "logprob":
        assert not dX[1::4].any()  # masked rows


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,v", [(8000, 72, 20000), (1000, 64, 70000), (20, 1032, 60000), (17000, 8, 9000)])
def test_gradients_over_several_chunks_and_parts(n, h, v):
    """Vocabularies of several chunks (the last a narrow one), with dX in parts and without."""
    x, w, tok = grid_inputs(n, h, v, seed=n)
    g = torch.Generator().manual_seed(3)
    gl, ge = (torch.randn(n, generator=g).cuda() / n for _ in range(2))
    r, _ = flce.logprobs_forward(x, w, tok)
    dX, dW, ws = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, gl, ge, check=True)
    rX, rW, mX, mW = gradients64(x, w, tok, gl, ge, 1.0)
    for got, ref, mag, name in ((dX, rX, mX, "dX"), (dW, rW, mW, "dW")):
        within(got, ref, 2.0 ** -8 * (mag * (1 + 2.0 ** -8) + ref.abs()) + 1e-5 * mag.max() + 1e-30, name)
        assert (got.double() - ref).norm() <= 2.0 ** -8 * math.sqrt(2) * ref.norm() + 1e-20, name
    again = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, gl, ge, ws=ws)
    assert torch.equal(dX, again[0]) and torch.equal(dW, again[1])  # parts join in a fixed order


@pytest.mark.gpu
def test_gradients_agree_with_the_cross_entropy():
    """-logprob summed is the cross-entropy: its gradients come from the same products."""
    x, w, tok = grid_inputs(500, 256, 5000, seed=1)
    tok[::7] = -100
    _, _, dX, dW, _ = flce.fwd_bwd(x, w, tok, reduction="sum")
    r, _ = flce.logprobs_forward(x, w, tok)
    pX, pW, _ = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, torch.full((500,), -1.0, device="cuda"))
    for a, b in ((pX, dX), (pW, dW)):
        assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()


@pytest.mark.gpu
def test_autograd_against_differences():
    """token_logprobs with a shift: gradients of sum(c logprob) + sum(d entropy) against
    central differences of the 64-bit value along random directions.  bf16 gradients are
    good to 2^-8 in norm, and an inner product with a random direction inherits that."""
    B, S, h, v = 2, 9, 64, 300
    x, w, tok = grid_inputs(B * S, h, v, seed=4)
    xs = x.view(B, S, h).clone().requires_grad_()
    ws_ = w.clone().requires_grad_()
    tokens = tok.view(B, S).long()
    g = torch.Generator().manual_seed(2)
    c, d = (torch.randn(B, S, generator=g).cuda() for _ in range(2))
    r = flce.token_logprobs(xs, ws_, tokens, top=2, temperature=0.8, shift=1)
    assert r.logprob.shape == (B, S) and r.top_ids.shape == (B, S, 2) and (r.logprob[:, -1] == 0).all()
    assert not r.lse.requires_grad and not r.top_logprobs.requires_grad
    ((c * r.logprob).sum() + (d * r.entropy).sum()).backward()

    def value(xv, wv):
        lp = torch.log_softmax(xv @ wv.t() / 0.8, -1)
        picked = lp[:, :-1].gather(2, tokens[:, 1:, None])[..., 0]
        return float((c[:, :-1] * picked).sum() - (d * (lp.exp() * lp).sum(-1)).sum())

    base = [x.view(B, S, h).double(), w.double()]
    for k, grad in ((0, xs.grad), (1, ws_.grad)):
        for _ in range(3):
            e = torch.randn(base[k].shape, generator=g, dtype=torch.float64).cuda()
            hi, lo = list(base), list(base)
            hi[k], lo[k] = base[k] + 1e-5 * e, base[k] - 1e-5 * e
            slope = (value(*hi) - value(*lo)) / 2e-5
            assert abs(float((grad.double() * e).sum()) - slope) <= 2.0 ** -6 * float(grad.double().norm() * 4)
    only = flce.token_logprobs(xs, ws_, tokens)
    only.entropy.sum().backward()  # one output's gradient alone
    assert torch.isfinite(xs.grad.float()).all()


@pytest.mark.gpu
def test_python_refusals():
    x, w, tok = grid_inputs(8, 64, 100)
    for bad in (lambda: flce.logprobs_forward(x.float(), w), lambda: flce.logprobs_forward(x, w, tok.long())):
        with pytest.raises(TypeError):
            bad()
    r, _ = flce.logprobs_forward(x, w, tok)
    for bad in (lambda: flce.logprobs_forward(x[0], w), lambda: flce.logprobs_forward(x, w[:, :56]),
                lambda: flce.logprobs_forward(x[:, :32], w[:, :32]), lambda: flce.logprobs_forward(x, w, tok[:7]),
                lambda: flce.logprobs_forward(x, w, tok, shift=1, seq_len=3),
                lambda: flce.logprobs_backward(x, w, None, r.lse, r.entropy, r.lse),
                lambda: flce.logprobs_backward(x, w, tok, r.lse, None, None, r.lse),
                lambda: flce.logprobs_backward(x, w, tok, r.lse[:3], r.entropy, r.lse),
                lambda: flce.token_logprobs(x, w, tok, shift=1)):
        with pytest.raises(ValueError):
            bad()
    for kw in (dict(top=17), dict(top=-1), dict(temperature=0.0), dict(temperature=float("nan")),
               dict(temperature=-1.0), dict(ws=torch.empty(256, dtype=torch.uint8, device="cuda"))):
        with pytest.raises(flce.FlceError):
            flce.logprobs_forward(x, w, tok, **kw)


def test_host_refusals():
    L, P = flce.lib(), binding.Problem
    z, ok = 0x1000, P(8, 64, 100, -100, 2)

    def fwd(p=ok, k=2, t=1.0, X=z, W=z, tok=z, lp=z, ent=z, lse=z, ids=z, tlp=z, ws=0x100000, nbytes=1 << 30):
        return L.flce_token_logprobs(ctypes.byref(p) if p else None, k, t, X, W, tok, lp, ent, lse, ids, tlp, ws,
                                     nbytes, None)

    def bwd(p=ok, t=1.0, X=z, W=z, tok=z, lse=z, ent=z, gl=z, ge=z, dX=z, dW=z, ws=0x100000, nbytes=1 << 40):
        return L.flce_token_logprobs_backward(ctypes.byref(p) if p else None, t, X, W, tok, lse, ent, gl, ge, dX, dW,
                                              ws, nbytes, None)

    assert fwd(p=None) == 1 and bwd(p=None) == 1
    for kw in (dict(k=-1), dict(k=17), dict(t=0.0), dict(t=float("inf")), dict(t=float("nan")), dict(X=None),
               dict(W=None), dict(lse=None), dict(ws=None), dict(ids=None), dict(tlp=None), dict(tok=None)):
        assert fwd(**kw) == 1, kw
    for kw in (dict(X=z + 8), dict(W=z + 8), dict(tok=z + 2), dict(lp=z + 2), dict(ent=z + 1), dict(lse=z + 2),
               dict(ids=z + 2), dict(tlp=z + 2), dict(ws=0x100010)):
        assert fwd(**kw) == 3, kw
    assert fwd(p=P(8, 12, 100, -100, 2)) == 2 and fwd(nbytes=256) == 4
    for kw in (dict(t=-1.0), dict(X=None), dict(W=None), dict(lse=None), dict(dX=None), dict(dW=None), dict(tok=None),
               dict(ent=None), dict(ws=None)):
        assert bwd(**kw) == 1, kw
    for kw in (dict(X=z + 8), dict(dX=z + 8), dict(gl=z + 2), dict(ge=z + 2), dict(ws=0x100010)):
        assert bwd(**kw) == 3, kw
    assert bwd(nbytes=256) == 4
    size = flce.token_logprobs_workspace_bytes
    assert size(8192, 2048, 32000) == size(8192, 64, 131072) < 4 << 20  # independent of H and V
    assert size(64, 2048, 32000, 16) > size(64, 2048, 32000, 0) > 0
    assert size(8, 64, 100, 17) == size(8, 12, 100) == size(-1, 64, 100) == 0


def test_reference_gradient_against_differences():
    """The 64-bit gradient used above against central differences of the 64-bit value."""
    g = torch.Generator().manual_seed(0)
    x, w = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((4, 6), (11, 6)))
    tok = torch.tensor([0, 10, -100, 3])
    gl, ge = torch.randn(4, generator=g).double(), torch.randn(4, generator=g).double()
    rX, rW, _, _ = gradients64(x, w, tok, gl, ge, 0.9)

    def value(x, w):
        lp = torch.log_softmax(x @ w.t() / 0.9, 1)
        ok = tok != -100
        return float((gl * ok * lp.gather(1, torch.where(ok, tok, 0)[:, None])[:, 0]).sum()
                     - (ge * (lp.exp() * lp).sum(1)).sum())

    for grad, k in ((rX, 0), (rW, 1)):
        for _ in range(6):
            d = torch.from_numpy(np.random.default_rng(k).standard_normal(tuple((x, w)[k].shape)))
            hi, lo = [x, w], [x, w]
            hi[k], lo[k] = hi[k] + 1e-6 * d, lo[k] - 1e-6 * d
            assert float((grad * d).sum()) == pytest.approx((value(*hi) - value(*lo)) / 2e-6, rel=1e-6, abs=1e-8)
