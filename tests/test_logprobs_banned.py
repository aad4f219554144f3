"""The alternatives of rows with fewer logits above minus infinity than are asked for: the
banned ids follow, lowest first, as equal logits do everywhere; -1 stands only past the
vocabulary's end.  And of rows with NaN logits, whose ids stay ids of the vocabulary."""
import math

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402
from test_logprobs import U, grid_inputs, within  # noqa: E402

pytestmark = pytest.mark.gpu

# a few rows, up to 128, and more: with the alternatives' wide and narrow epilogues (H = 64, 1544)
ROWS = [(1, 64), (8, 64), (9, 64), (40, 512), (100, 64), (260, 64), (300, 1544)]


def banned_inputs(n, h, v, live):
    x, w, _ = grid_inputs(n, h, v, seed=n + v, ties=False)
    x[:, 0] = 1.0
    ban = torch.ones(v, dtype=torch.bool, device="cuda")
    ban[live] = False
    w[ban, 0] = -math.inf
    return x, w


@pytest.mark.parametrize("n,h", ROWS)
@pytest.mark.parametrize("v,live", [(3000, [0, 2, 5, 2999]), (40009, [39000, 1, 20000]), (70001, []), (5, [1, 3]),
                                    (1000, [3, 4, 5, 6, 7, 8, 9, 10, 11, 12, 13, 14, 15, 999])])
def test_banned_ids_follow_in_order(n, h, v, live):
    x, w = banned_inputs(n, h, v, live)
    k = 16 if v > 5 else 8
    r, _ = flce.logprobs_forward(x, w, top=k, check=True)
    raw = x.double() @ w.double().t()
    order = raw.sort(dim=1, descending=True, stable=True).indices[:, :k]  # stable: the lowest id first
    have = min(k, v)
    assert torch.equal(r.top_ids[:, :have].long(), order)
    assert (r.top_ids[:, have:] == -1).all() and (r.top_logprobs[:, have:] == -math.inf).all()
    if not live:
        assert torch.isnan(r.top_logprobs).all()  # minus infinity less minus infinity
        return
    lp = (raw - torch.logsumexp(raw, 1, keepdim=True)).gather(1, order)
    tol = (v / 128 + 116) * U + 6 * U * lp[:, :len(live)].abs() + 4 * U * raw[:, live].abs().amax(1, keepdim=True)
    within(r.top_logprobs[:, :len(live)], lp[:, :len(live)], tol, "live")
    assert (r.top_logprobs[:, len(live):have] == -math.inf).all()


@pytest.mark.parametrize("n,h", ROWS)
def test_alternatives_of_a_nan_row_stay_in_the_vocabulary(n, h):
    x, w, tok = grid_inputs(n, h, 3000, seed=n)
    x[n // 2, 5] = float("nan")
    r, _ = flce.logprobs_forward(x, w, tok, top=9, check=True)
    ids = r.top_ids[n // 2].long()
    assert ((ids >= 0) & (ids < 3000)).all() and ids.unique().numel() == 9
    assert torch.isnan(r.top_logprobs[n // 2]).all()
