"""A training step of a small model through the library's calls together: a matrix that embeds and
projects, a hidden layer between, the loss with its gradient, the embedding's part added to the
head's, AdamW on the shared matrix and the norm, Muon on the hidden matrices; against the same step
in 64 bits from the same starting values."""
import math

import pytest

torch = pytest.importorskip("torch")

import lm_head_cross_gb300 as flce  # noqa: E402

BF16 = torch.bfloat16


def newton_schulz(u):
    x = u / (u.square().sum().sqrt() + 1e-7)
    tall = x.shape[0] > x.shape[1]
    x = x.t() if tall else x
    for _ in range(5):
        g = x @ x.t()
        x = 3.4445 * x + (-4.7750 * g + 2.0315 * g @ g) @ x
    return x.t() if tall else x


def model(vocab, hidden, inner, device="cuda"):
    g = torch.Generator().manual_seed(0)
    make = lambda *s, by=1.0: (by * torch.randn(*s, generator=g)).to(device)  # noqa: E731
    return {"tied": make(vocab, hidden, by=0.05).to(BF16), "up": make(inner, hidden, by=hidden ** -0.5).to(BF16),
            "down": make(hidden, inner, by=inner ** -0.5).to(BF16), "norm": torch.ones(hidden, device=device)}


@pytest.mark.gpu
@pytest.mark.parametrize("vocab,hidden,inner,batch,length", [(500, 64, 200, 4, 33), (1000, 256, 130, 2, 128)])
def test_step_of_a_tied_model(vocab, hidden, inner, batch, length):
    """bf16 holds the activations (five of them in a chain), the logits' gradient and both products:
    2^-8 each, 2^-5 of a gradient's norm.  AdamW's first step moves every weight by lr whatever its
    gradient's size, and Muon's by an orthogonal matrix's elements, so there the sign and the
    direction count: the share of AdamW's elements whose sign a 2^-5 error can turn, and half of
    Muon's step (the gradient's weak directions, which that error outweighs, count as
    much as strong ones)."""
    p = model(vocab, hidden, inner)
    scale = math.sqrt(hidden)
    tokens = torch.randint(0, vocab, (batch, length), generator=torch.Generator().manual_seed(1)).cuda()
    ids = tokens.view(-1).to(torch.int32)
    start = {k: v.clone() for k, v in p.items()}

    # the library's step
    up, down, norm = (p[k].clone().requires_grad_() for k in ("up", "down", "norm"))
    x0, _ = flce.embedding_forward(ids, p["tied"], scale=scale, check=True)
    x0.requires_grad_()
    y = flce.layer_norm(x0 + torch.relu(x0 @ up.t()) @ down.t(), norm)
    y2 = y.detach()
    loss, _, dy, dtied, ws = flce.fwd_bwd(y2, p["tied"], ids, shift=1, seq_len=length, check=True)
    y.backward(dy)
    flce.embedding_backward(x0.grad, ids, vocab, scale=scale, add_to=dtied, check=True)
    got = {"tied": dtied, "up": up.grad, "down": down.grad, "norm": norm.grad}
    tied = torch.nn.Parameter(p["tied"].clone())
    tied.grad = dtied
    for q in (up, down, norm):
        q.requires_grad_(False)
    norm_p = torch.nn.Parameter(norm.clone())
    norm_p.grad = got["norm"]
    adam = flce.AdamW([tied, norm_p], lr=1e-3, weight_decay=0.0)
    hidden_p = [torch.nn.Parameter(up.clone()), torch.nn.Parameter(down.clone())]
    for q, k in zip(hidden_p, ("up", "down")):
        q.grad = got[k]
    muon = flce.Muon(hidden_p, lr=0.02, momentum=0.95)
    adam.step()
    muon.step()

    # the same in 64 bits
    w = {k: v.double().requires_grad_() for k, v in start.items()}
    x = scale * w["tied"][tokens.view(-1)]
    z = torch.nn.functional.layer_norm(x + torch.relu(x @ w["up"].t()) @ w["down"].t(), (hidden,), w["norm"])
    logits = (z @ w["tied"].t()).view(batch, length, vocab)
    want = torch.nn.functional.cross_entropy(logits[:, :-1].reshape(-1, vocab), tokens[:, 1:].reshape(-1))
    want.backward()
    assert abs(loss.item() - want.item()) <= 2.0 ** -6 * want.item()
    for k, g in got.items():
        ref = w[k].grad
        assert (g.double() - ref).norm() <= 2.0 ** -5 * ref.norm(), k
    moved = tied.detach().double() - start["tied"].double()
    ref = -1e-3 * w["tied"].grad.sign()
    # (bf16 weights: the master weights moved by lr, their rounding by that or by a step of bf16)
    master = adam.state["master"][0].double() - start["tied"].double()
    clear = w["tied"].grad.abs() > 2.0 ** -4 * w["tied"].grad.abs().mean()
    assert (master[clear] - ref[clear]).abs().max() <= 1e-3 * 2.5 and ((master - ref)[clear].abs() > 1e-4).double().mean() < 0.05
    assert moved.abs().max() <= 1e-3 + 2.0 ** -8 * start["tied"].double().abs().max()
    for i, k in enumerate(("up", "down")):
        r, c = start[k].shape
        u = w[k].grad * (1 - 0.95) * 1.95  # momentum from zero, Nesterov
        step = 0.02 * math.sqrt(max(1.0, r / c)) * newton_schulz(u)
        off = muon.state["master"][i].double() - (start[k].double() - step)
        own = 0.02 * math.sqrt(max(1.0, r / c)) * newton_schulz(got[k].double() * (1 - 0.95) * 1.95)
        exact_of_own = muon.state["master"][i].double() - (start[k].double() - own)
        assert exact_of_own.norm() <= 4e-3 * own.norm() and off.norm() <= 2.0 ** -1 * step.norm(), k
    assert torch.equal(hidden_p[0], muon.state["master"][0].to(BF16))
