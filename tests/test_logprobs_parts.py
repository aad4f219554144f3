"""The gradients of token log probabilities where dX is summed in parts over several
chunks of the vocabulary, on workspaces that hold NaN bytes before the call: a part that
no chunk stored shows at once.  And the plan of chunks and parts itself, on the host."""
import os
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from lm_head_cross_gb300.binding import logprobs_backward_workspace_bytes  # noqa: E402
from test_logprobs import gradients64, grid_inputs, within  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# last chunks that, cut anew into as many parts, would fill more than the first chunk does
# (50 and 51, 30 and 31, 147 and 152, 37 and 38), fewer, and none at all
SHAPES = [(40, 768, 250002), (700, 128, 128256), (1161, 112, 94416), (728, 160, 105002), (200, 64, 140800),
          (980, 64, 70784), (256, 256, 256000), (1000, 64, 70000), (300, 264, 1000), (100, 512, 60000)]


@pytest.mark.gpu
@pytest.mark.parametrize("n,h,v", SHAPES)
def test_no_part_is_read_that_was_not_stored(n, h, v):
    """Tolerances as in test_logprobs: dz is held in bf16, 2^-8 of the products of
    magnitudes, and half an ulp of the result."""
    x, w, tok = grid_inputs(n, h, v, seed=n + h)
    g = torch.Generator().manual_seed(5)
    gl, ge = (torch.randn(n, generator=g).cuda() / n for _ in range(2))
    r, _ = flce.logprobs_forward(x, w, tok)
    ws = torch.full((logprobs_backward_workspace_bytes(n, h, v),), 0xFF, dtype=torch.uint8, device="cuda")
    dX, dW, _ = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, gl, ge, ws=ws, check=True)
    rX, rW, mX, mW = gradients64(x, w, tok, gl, ge, 1.0)
    for got, ref, mag, name in ((dX, rX, mX, "dX"), (dW, rW, mW, "dW")):
        within(got, ref, 2.0 ** -8 * (mag * (1 + 2.0 ** -8) + ref.abs()) + 1e-5 * mag.max() + 1e-30, name)
        assert (got.double() - ref).norm() <= 2.0 ** -8 * 2 ** 0.5 * ref.norm() + 1e-20, name
    again = flce.logprobs_backward(x, w, tok, r.lse, r.entropy, gl, ge, ws=ws, check=True)
    assert torch.equal(dX, again[0]) and torch.equal(dW, again[1])


PLAN_CHECK = r"""
#include <cstdio>
#include "flce_internal.h"
using namespace flce;
int main() {
  long long cases = 0, in_parts = 0;
  for (int h = 8; h <= 8192; h += h < 64 ? 8 : h < 1024 ? 104 : 1032)
    for (int j = 0; j < 40; ++j) {
      const int v = j == 0 ? 250002 : j == 1 ? 128256 : j == 2 ? 1 : 300 + 7691 * j + 37 * h % 300;
      for (int n = 1; n <= 8192; ++n, ++cases) {
        const ScorePlan p = score_plan(n, h, v);
        const int first = v < p.chunk ? v : p.chunk;
        in_parts += p.parts > 1;
        bool ok = p.splits(first) == p.parts && p.part_k % kBK == 0 && 4ll * n * h * (p.parts - 1) < 1ll << 26;
        for (long long c0 = 0; c0 < v; c0 += p.chunk) {
          const int cw = static_cast<int>(v - c0 < p.chunk ? v - c0 : p.chunk);
          const int s = p.splits(cw);  // each of the chunk's parts is stored, and holds at least one id
          ok = ok && s >= 1 && s <= p.parts && static_cast<long long>(s - 1) * p.part_k < cw;
        }
        if (!ok) return printf("n %d h %d v %d: chunk %d parts %d part_k %d\n", n, h, v, p.chunk, p.parts, p.part_k), 1;
      }
    }
  printf("ok %lld %lld\n", cases, in_parts);
}
"""


def test_no_chunk_fills_more_parts_than_the_first(tmp_path):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "plan.cpp", tmp_path / "plan"
    src.write_text(PLAN_CHECK)
    cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    r = subprocess.run([cxx, "-std=c++17", "-O2", "-I", os.path.join(ROOT, "lm_head_cross_gb300", "csrc"),
                        "-I", os.path.join(ROOT, "include"), "-I", os.path.join(cuda, "include"), str(src), "-o",
                        str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stdout
    word, cases, in_parts = r.stdout.split()
    assert word == "ok" and int(cases) > 1_000_000 and int(in_parts) > 100_000
