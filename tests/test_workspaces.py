"""Workspaces hold no promise about what they hold: every call gives the same bits from one of
zeros and from one of NaN bytes, and writes nothing past the size that it asked for."""
import random

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300.binding import logprobs_backward_workspace_bytes  # noqa: E402
from test_layernorm import make  # noqa: E402
from test_logprobs import grid_inputs  # noqa: E402

pytestmark = pytest.mark.gpu

GUARD = 1 << 16


def bits(t):
    return None if t is None else t.contiguous().view(torch.uint8)


def same_from_any_workspace(nbytes, call):
    """call(ws) -> tensors, from zeros and from NaN bytes, with guard bytes behind both."""
    outs = []
    for fill in (0x00, 0xFF):
        held = torch.full((nbytes + GUARD,), fill, dtype=torch.uint8, device="cuda")
        outs.append([bits(t) for t in call(held[:nbytes])])
        assert (held[nbytes:] == fill).all(), "written past the workspace"
    for a, b in zip(*outs):
        assert (a is None and b is None) or torch.equal(a, b)


def log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def head_shape(rng, most):
    h, v = 8 * log_int(rng, 1, 256), log_int(rng, 1, 150000)
    return max(1, min(log_int(rng, 1, 6000), most // (h * v))), h, v


@pytest.mark.parametrize("seed", range(40))
def test_token_logprobs(seed):
    rng = random.Random(seed)
    n, h, v = head_shape(rng, 10 ** 12)
    k = rng.choice([0, 1, 5, 16])
    x, w, tok = grid_inputs(n, h, v, seed=seed)
    tok[::7] = -100
    call = lambda ws: flce.logprobs_forward(x, w, tok, top=k, temperature=0.9, ws=ws, check=True)[0]  # noqa: E731
    same_from_any_workspace(flce.token_logprobs_workspace_bytes(n, h, v, k), call)


@pytest.mark.parametrize("seed", range(40))
def test_token_logprobs_backward(seed):
    rng = random.Random(1000 + seed)
    n, h, v = head_shape(rng, 3 * 10 ** 11)
    if seed < 12:  # dX in parts over several chunks
        n, h, v = rng.randint(1, 1100), 8 * rng.randint(1, 32), rng.randint(131073, 300000)
    x, w, tok = grid_inputs(n, h, v, seed=seed)
    tok[::7] = -100
    r, _ = flce.logprobs_forward(x, w, tok)
    gl, ge = torch.rand(n, device="cuda"), torch.rand(n, device="cuda")
    same_from_any_workspace(logprobs_backward_workspace_bytes(n, h, v), lambda ws: flce.logprobs_backward(
        x, w, tok, r.lse, r.entropy, gl, ge, ws=ws, check=True)[:2])


@pytest.mark.parametrize("seed", range(40))
def test_layernorm_backward(seed):
    rng = random.Random(2000 + seed)
    h = log_int(rng, 1, 40000)
    n = max(1, min(log_int(rng, 1, 40000), (1 << 25) // h))
    x, w, b, dy = (t.cuda() for t in make(n, h, rng.choice([torch.bfloat16, torch.float32]),
                                          rng.choice([torch.bfloat16, torch.float32]), seed=seed))
    _, mean, rstd = flce.layernorm_forward(x, w, b)
    same_from_any_workspace(flce.layernorm_workspace_bytes(n, h),
                            lambda ws: flce.layernorm_backward(dy, x, w, mean, rstd, ws=ws)[:3])


@pytest.mark.parametrize("seed", range(16))
@pytest.mark.parametrize("rowchunk", [False, True])
def test_cross_entropy(seed, rowchunk):
    rng = random.Random(3000 + seed)
    n, h, v = head_shape(rng, 10 ** 11)
    if rowchunk and n * v > 1 << 29:
        n = max(1, (1 << 29) // v)
    x, w, tok = grid_inputs(n, h, v, seed=seed)
    tok[::7] = -100
    size = (flce.workspace_bytes_rowchunk if rowchunk else flce.workspace_bytes)(n, h, v)
    same_from_any_workspace(size, lambda ws: flce.fwd_bwd(x, w, tok, ws=ws, check=True, rowchunk=rowchunk)[:4])
