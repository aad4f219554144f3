#!/usr/bin/env python3
"""The end of a language model, trained and served through the library.

A small bigram model (an embedding in place of a transformer's trunk) runs the calls that
surround the LM head as a program would use them together:

  training   layer_norm -> token_logprobs (log probabilities and entropies of the next
             tokens) -> backward through both -> AdamW over every parameter, moments in 8
             bits, gradients clipped by their global norm through grad_scale;
  serving    layernorm_forward -> logprobs_forward for single tokens with the top
             alternatives, sampling the next token from them.

    python examples/head_step.py [--steps 60] [--hidden 256] [--vocab 1024] [--state-bits 8]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import lm_head_cross_gb300 as flce  # noqa: E402


class Bigram:
    """Embedding, final norm, head; bf16 weights, fp32 norm parameters."""

    def __init__(self, vocab, hidden, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def param(t, dtype):
            return t.to(device=device, dtype=dtype).requires_grad_()

        self.embed = param(torch.randn(vocab, hidden, generator=g), torch.bfloat16)
        self.norm_weight = param(torch.ones(hidden), torch.float32)
        self.norm_bias = param(torch.zeros(hidden), torch.float32)
        self.head = param(0.02 * torch.randn(vocab, hidden, generator=g), torch.bfloat16)

    def groups(self):
        """AdamW's parameter groups: no weight decay on the norm."""
        return [{"params": [self.embed, self.head]},
                {"params": [self.norm_weight, self.norm_bias], "weight_decay": 0.0}]

    def hidden(self, tokens):
        return flce.layer_norm(self.embed[tokens], self.norm_weight, self.norm_bias)


def train(model, batch, steps, lr=2e-2, entropy_bonus=1e-3, clip=1.0, state_bits=8):
    """Maximises the batch's log likelihood with a small entropy bonus; position t of each
    sequence is scored against the token at t + 1.  Returns each step's mean negative log
    likelihood (read back once, at the end)."""
    opt = flce.AdamW(model.groups(), lr=lr, betas=(0.9, 0.95), weight_decay=0.01, state_bits=state_bits)
    history = []
    scored = batch.shape[0] * (batch.shape[1] - 1)
    for _ in range(steps):
        r = flce.token_logprobs(model.hidden(batch), model.head, batch, shift=1)
        nll = -r.logprob.sum() / scored
        (nll - entropy_bonus * r.entropy.mean()).backward()
        norm = torch.stack([p.grad.float().norm() for p in opt.params]).norm()
        opt.step(grad_scale=(clip / norm).clamp(max=1.0).reshape(1))
        opt.zero_grad()
        history.append(nll.detach())
    return torch.stack(history).tolist()


@torch.no_grad()
def generate(model, prompt, length, top=8, temperature=0.8, seed=0):
    """Samples `length` tokens for each sequence from its top alternatives.  Returns the tokens
    [B, length] and their log probabilities under the full distribution."""
    g = torch.Generator(device=prompt.device).manual_seed(seed)
    token, tokens, logprobs, ws = prompt, [], [], None
    for _ in range(length):
        y, _, _ = flce.layernorm_forward(model.embed[token], model.norm_weight, model.norm_bias)
        r, ws = flce.logprobs_forward(y, model.head, top=top, temperature=temperature, ws=ws)
        pick = torch.multinomial(r.top_logprobs.exp(), 1, generator=g)
        token = r.top_ids.gather(1, pick)[:, 0].long()
        tokens.append(token)
        logprobs.append(r.top_logprobs.gather(1, pick)[:, 0])
    return torch.stack(tokens, 1), torch.stack(logprobs, 1)


def synthetic_batch(vocab, batch, length, device="cuda", seed=1):
    """Sequences that mostly follow one successor for each token."""
    g = torch.Generator().manual_seed(seed)
    follow = torch.randperm(vocab, generator=g)
    out = torch.randint(0, vocab, (batch, 1), generator=g)
    for _ in range(length - 1):
        stray = torch.randint(0, vocab, (batch, 1), generator=g)
        keep = torch.rand(batch, 1, generator=g) < 0.9
        out = torch.cat([out, torch.where(keep, follow[out[:, -1:]], stray)], 1)
    return out.to(device), follow.to(device)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--hidden", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=1024)
    ap.add_argument("--batch", type=int, default=32)
    ap.add_argument("--length", type=int, default=128)
    ap.add_argument("--state-bits", type=int, choices=(8, 32), default=8)
    a = ap.parse_args()
    batch, follow = synthetic_batch(a.vocab, a.batch, a.length)
    model = Bigram(a.vocab, a.hidden)
    history = train(model, batch, a.steps, state_bits=a.state_bits)
    for step in sorted({0, a.steps // 4, a.steps // 2, a.steps - 1}):
        print(f"step {step:4d}  negative log likelihood {history[step]:.4f}")
    tokens, logprobs = generate(model, batch[:4, 0], 16)
    chain = torch.cat([batch[:4, :1], tokens], 1)
    right = (follow[chain[:, :-1]] == chain[:, 1:]).float().mean().item()
    print(f"generated {tokens.shape[1]} tokens for {tokens.shape[0]} sequences: {100 * right:.0f}% follow the data's "
          f"successor, mean log probability {logprobs.mean().item():.3f}")


if __name__ == "__main__":
    main()
