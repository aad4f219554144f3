"""The debug build (FLCE_DEBUG_CHECKS) through the token log probabilities: few and many
rows, every alternative count, forward and backward; no index check fires and the results
are those of the release build's tests.  In a child process, which loads that library."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

import lm_head_cross_gb300 as flce  # noqa: E402


def test_debug_build_runs_clean_on_token_logprobs():
    here = os.path.dirname(os.path.abspath(__file__))
    lib = os.path.join(os.path.dirname(flce.lib_path()), "libflce_debug.so")
    assert os.path.exists(lib)
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-m", "gpu", os.path.join(here, "test_logprobs.py"),
                        "-k", "test_forward or test_gradients or out_of_range"],
                       env=dict(os.environ, FLCE_LIB=lib), capture_output=True, text=True, timeout=600,
                       cwd=os.path.dirname(here))
    assert r.returncode == 0, (r.stdout[-3000:], r.stderr[-2000:])
