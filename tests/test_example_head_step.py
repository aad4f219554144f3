"""The example that trains and serves a model's end: norm, token log probabilities,
optimizer, and decoding with alternatives, together."""
import importlib.util
import math
import os

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("head_step", os.path.join(ROOT, "examples", "head_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [8, 32])
def test_trains_and_generates(bits):
    ex = _example()
    vocab = 512
    batch, follow = ex.synthetic_batch(vocab, 32, 128)
    model = ex.Bigram(vocab, 128)
    history = ex.train(model, batch, 80, state_bits=bits)
    assert abs(history[0] - math.log(vocab)) < 0.5  # near uniform at the start
    # 90% of the tokens follow their predecessor's successor, the rest is uniform: on new data the
    # best is about -0.9 ln 0.9 - 0.1 ln(0.1 / V) = 0.95 nats, on the one batch it trains on less
    assert history[-1] < 1.6 and all(math.isfinite(h) for h in history)
    tokens, logprobs = ex.generate(model, batch[:, 0], 24)
    chain = torch.cat([batch[:, :1], tokens], 1)
    right = (follow[chain[:, :-1]] == chain[:, 1:]).float().mean().item()
    assert right > 0.8 and (logprobs <= 0).all()


@pytest.mark.gpu
def test_one_step_against_plain_torch():
    """The gradients of one training step against the same step in 32-bit torch from the
    same bf16 weights.  bf16 holds the hidden states, dz, dX and dW (2^-8 relative each):
    4 of them in a chain give 2^-6 in norm."""
    ex = _example()
    batch, _ = ex.synthetic_batch(300, 4, 33)
    model = ex.Bigram(300, 64)
    flce = ex.flce
    r = flce.token_logprobs(model.hidden(batch), model.head, batch, shift=1)
    (-r.logprob.sum() + 0.1 * r.entropy.sum()).backward()
    emb, w, b, head = (t.detach().float().requires_grad_() for t in
                       (model.embed, model.norm_weight, model.norm_bias, model.head))
    y = torch.nn.functional.layer_norm(emb[batch], (64,), w, b)
    lp = torch.log_softmax(y @ head.t(), -1)
    picked = lp[:, :-1].gather(2, batch[:, 1:, None]).sum()
    (-picked - 0.1 * (lp.exp() * lp).sum()).backward()
    for mine, ref in zip((model.embed, model.norm_weight, model.norm_bias, model.head), (emb, w, b, head)):
        err = (mine.grad.float() - ref.grad).norm() / ref.grad.norm()
        assert err < 2.0 ** -6, err
