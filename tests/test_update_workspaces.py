"""The embedding's gradient and Muon's calls from workspaces of any content, at drawn sizes: the same
bits, nothing written past the size; and the debug build's index checks through both."""
import ctypes
import os
import random
import subprocess
import sys

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300 import binding  # noqa: E402
from test_embedding import tokens  # noqa: E402
from test_muon import matrix  # noqa: E402
from test_workspaces import log_int, same_from_any_workspace  # noqa: E402

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("seed", range(40))
def test_embedding_backward(seed):
    rng = random.Random(seed)
    n, v = log_int(rng, 1, 200000), log_int(rng, 1, 300000)
    h = max(1, min(log_int(rng, 1, 3000), (1 << 27) // max(n, v)))
    kind, dtype, wtype = rng.choice(["zipf", "uniform", "one", "ends"]), rng.choice([BF16, F32]), rng.choice([BF16, F32])
    ids = tokens(n, v, kind, seed).cuda()
    dy = torch.randn(n, h, device="cuda").to(dtype)
    old = torch.randn(v, h, device="cuda").to(wtype)
    pad = rng.choice([None, v // 2])
    size = flce.embedding_workspace_bytes(n, h, v)
    same_from_any_workspace(size, lambda ws: [flce.embedding_backward(dy, ids, v, padding_idx=pad, dtype=wtype, ws=ws,
                                                                      check=True)[0]])
    same_from_any_workspace(size, lambda ws: [flce.embedding_backward(dy, ids, v, padding_idx=pad, add_to=old.clone(),
                                                                      ws=ws, check=True)[0]])


@pytest.mark.parametrize("seed", range(40))
def test_orthogonalize(seed):
    rng = random.Random(seed)
    shapes = []
    for _ in range(rng.randint(1, 5)):
        r = log_int(rng, 1, 1500)
        shapes += [(r, log_int(rng, 1, 3000))] * rng.randint(1, 3)
    xs = [matrix(s, seed=i).to(rng.choice([BF16, F32])).cuda() for i, s in enumerate(shapes)]
    table = (binding.Matrix * len(xs))(*((1, 1, *s, 0) for s in shapes))
    size = flce.lib().flce_orthogonalize_workspace_bytes(table, len(xs))
    steps = rng.randint(1, 6)
    same_from_any_workspace(size, lambda ws: flce.orthogonalize(xs, steps=steps, ws=ws, check=True))


@pytest.mark.parametrize("seed", range(10))
def test_muon_step(seed):
    rng = random.Random(seed)
    shapes = [(log_int(rng, 1, 700), log_int(rng, 1, 700)) for _ in range(rng.randint(1, 8))]
    dtype = rng.choice([BF16, F32])
    gs = [matrix(s, seed=i).to(rng.choice([BF16, F32])).cuda() for i, s in enumerate(shapes)]

    def call(ws):
        ps, ms = [matrix(s).to(dtype).cuda() for s in shapes], [matrix(s).cuda() for s in shapes]
        flce.muon_step(flce.muon_plan(ps, ms, nesterov=seed % 2 == 0), gs, ws=ws, check=True)
        return ps + ms
    plan = flce.muon_plan([matrix(s).to(dtype).cuda() for s in shapes], [matrix(s).cuda() for s in shapes])
    same_from_any_workspace(plan.workspace_bytes(), call)


def test_too_small_a_workspace_is_refused():
    x = torch.randn(300, 200, device="cuda")
    table = (binding.Matrix * 1)((1, 1, 300, 200, 1))
    size = flce.lib().flce_orthogonalize_workspace_bytes(table, 1)
    with pytest.raises(flce.FlceError, match="workspace"):
        flce.orthogonalize(x, ws=torch.empty(size - 1, dtype=torch.uint8, device="cuda"))
    assert ctypes.sizeof(binding.Matrix) == 40


def test_debug_build_runs_clean():
    here = os.path.dirname(os.path.abspath(__file__))
    lib = os.path.join(os.path.dirname(flce.lib_path()), "libflce_debug.so")
    assert os.path.exists(lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", os.path.join(here, "test_embedding.py"),
                        os.path.join(here, "test_muon.py"), "-k", "gradient or forward or orthogonalize or step or rounds"],
                       env=dict(os.environ, FLCE_LIB=lib), capture_output=True, text=True, timeout=600,
                       cwd=os.path.dirname(here))
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-2000:])
