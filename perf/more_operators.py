"""The cases on which the operators at a training step's two ends are measured.

Two operators, each with what trains it or what it trains, next to the LM head, its
gradient and AdamW:

  embedding     rows of a vocabulary matrix, scaled; and the matrix's gradient, summed token
                by token, as a new tensor or added to the gradient that the head, which may
                share the matrix, has already left there;
  Muon          the update of a model's other matrices: momentum, orthogonalised by
                Newton-Schulz products; alone (``orthogonalize``) and as an optimizer step.

``run`` computes a case in plain 32-bit torch operations where ``own`` is false and
through this library's entry points where it is true.  ``exact`` gives the definition
in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2, "fp32": 4}

#: Newton-Schulz: X <- a X + (b X X^T + c (X X^T)^2) X
STEPS, COEFFICIENTS, EPS = 5, (3.4445, -4.7750, 2.0315), 1e-7


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding step of four sequences: launch latency, nothing else
        dict(name="emb_fwd_decode", op="emb_fwd", n=4, h=4096, v=128256, dtype="bf16"),
        # the rows of a 128K-token batch over the largest vocabulary
        dict(name="emb_fwd_128k", op="emb_fwd", n=131072, h=4096, v=131072, dtype="bf16"),
        # an ordinary training step with an embedding of its own: a whole new gradient
        dict(name="emb_bwd_8k", op="emb_bwd", n=8192, h=2048, v=32000, dtype="bf16", pad=0.0, add=False),
        # 32-bit training of padded batches, a width and a vocabulary that nothing divides
        dict(name="emb_bwd_odd_fp32", op="emb_bwd", n=5003, h=1031, v=40009, dtype="fp32", pad=0.3, add=False),
        # the largest workload with tied matrices: added to the head's gradient
        dict(name="emb_tied_128k", op="emb_bwd", n=131072, h=4096, v=131072, dtype="bf16", pad=0.0, add=True),
        # one small matrix: launch latency
        dict(name="ortho_128", op="ortho", count=1, rows=128, cols=128, dtype="bf16"),
        # a few wide matrices that no tile divides, in 32 bits
        dict(name="ortho_odd", op="ortho", count=3, rows=777, cols=1544, dtype="fp32"),
        # one large square matrix
        dict(name="ortho_4096", op="ortho", count=1, rows=4096, cols=4096, dtype="bf16"),
        # every matrix of a small model's 16 layers (112 of them, five shapes), one optimizer step
        dict(name="muon_model", op="muon", layers=16, h=512, gdtype="bf16", nesterov=True),
        # four layers of a model of ordinary width, gradients in 32 bits
        dict(name="muon_2k", op="muon", layers=4, h=2048, gdtype="fp32", nesterov=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["emb_fwd", "emb_bwd", "emb_bwd", "ortho", "ortho", "muon"])
    if op in ("emb_fwd", "emb_bwd"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        h = _log_int(rng, 8, 4096)
        if rng.random() < 0.6:
            h = (h + 7) // 8 * 8
        v = _log_int(rng, 100, 131072)
        n = _log_int(rng, 1, min(131072, 131072 * 4096 // h) // (2 if dtype == "fp32" else 1))
        if op == "emb_fwd":
            return dict(op=op, n=n, h=h, v=v, dtype=dtype)
        if dtype == "fp32" and v * h > 131072 * 2048:
            v = 131072 * 2048 // h
        return dict(op=op, n=n, h=h, v=v, dtype=dtype, pad=rng.choice([0.0, 0.0, 0.3]), add=rng.random() < 0.5)
    if op == "ortho":
        rows, cols = _log_int(rng, 2, 4096), _log_int(rng, 2, 4096)
        most = 2.5e12 / _products(rows, cols)
        count = _log_int(rng, 1, max(1, min(32, int(most))))
        return dict(op=op, count=count, rows=rows, cols=cols, dtype=rng.choice(["bf16", "fp32"]))
    h = _log_int(rng, 24, 2048)
    return dict(op=op, layers=rng.randint(1, 4 if h > 1024 else 8), h=h, gdtype=rng.choice(["bf16", "fp32"]),
                nesterov=rng.random() < 0.7)


def _products(rows, cols):
    """Operations of one matrix: X X^T and its square are symmetric, half of each is enough."""
    r, c = min(rows, cols), max(rows, cols)
    return STEPS * (r * (r + 1) * c + r * (r + 1) * r + 2 * r * r * c)


def _layer_shapes(h):
    """A decoder layer's matrices: queries, keys, values, output; the gated feed-forward's three."""
    f = 2 * h + h // 3
    return [(h, h), (h // 4 + 1, h), (h // 4 + 1, h), (h, h), (f, h), (f, h), (h, f)]


#: every matrix starts at a multiple of this many elements of a flat buffer, as buckets lay them out
ALIGN = 256


def _layout(case):
    at, spans = 0, []
    for shape in _layer_shapes(case["h"]) * case["layers"]:
        spans.append((at, shape))
        at += (math.prod(shape) + ALIGN - 1) // ALIGN * ALIGN
    return at, spans


def _token_weights(v):
    """Frequencies of a vocabulary's tokens, most frequent first."""
    return 1.0 / (np.arange(v, dtype=np.float64) + 2.7) ** 1.07


def _distinct(case):
    """Rows of the vocabulary that n tokens are expected to touch."""
    p = _token_weights(case["v"])
    return float(np.sum(-np.expm1(case["n"] * (1 - case.get("pad", 0.0)) * np.log1p(-p / p.sum()))))


def work(case):
    op = case["op"]
    if op in ("emb_fwd", "emb_bwd"):
        n, h, v, s = case["n"], case["h"], case["v"], SIZE[case["dtype"]]
        if op == "emb_fwd":
            return {"bytes": int((_distinct(case) + n) * h * s) + 4 * n, "flops": n * h}
        rows = n * (1 - case["pad"])
        written = 2 * _distinct(case) if case["add"] else v
        return {"bytes": int((rows + written) * h * s) + 4 * n, "flops": int(rows * h)}
    if op == "ortho":
        count = case["count"] * case["rows"] * case["cols"]
        return {"bytes": count * (SIZE[case["dtype"]] + 2), "flops": case["count"] * _products(case["rows"], case["cols"])}
    shapes = _layer_shapes(case["h"]) * case["layers"]
    count = sum(math.prod(x) for x in shapes)  # gradient in, momentum in and out, weights in and out
    return {"bytes": count * (SIZE[case["gdtype"]] + 8 + 4), "flops": sum(_products(*x) for x in shapes) + 10 * count}


# ----------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _tokens(case, g):
    """Token ids by frequency, the frequent ones anywhere in the vocabulary; the end of a padded
    batch's share of them is one id."""
    n, v = case["n"], case["v"]
    cdf = torch.from_numpy(np.cumsum(_token_weights(v))).to(DEV)
    rank = torch.searchsorted(cdf, torch.rand(n, device=DEV, generator=g, dtype=torch.float64) * cdf[-1])
    ids = torch.randperm(v, device=DEV, generator=g)[rank.clamp_max_(v - 1)]
    if case.get("pad"):
        ids[torch.rand(n, device=DEV, generator=g) < case["pad"]] = v // 2
    return ids.to(torch.int32)


def _matrices(shape, g):
    """Momenta or gradients [..., R, C]: a few strong directions of decreasing size over noise
    whose size differs by row and column, as the gradients of trained layers have."""
    *lead, r, c = shape
    k = min(16, r, c)
    noise = torch.randn(*lead, r, c, device=DEV, generator=g)
    noise *= 0.5 + torch.rand(*lead, r, 1, device=DEV, generator=g)
    noise *= 0.5 + torch.rand(*lead, 1, c, device=DEV, generator=g)
    left = torch.randn(*lead, r, k, device=DEV, generator=g) / (1.0 + torch.arange(k, device=DEV))
    return (noise + left @ torch.randn(*lead, k, c, device=DEV, generator=g)) * 1e-4


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("emb_fwd", "emb_bwd"):
        n, h, v, dt = case["n"], case["h"], case["v"], DTYPES[case["dtype"]]
        s["ids"], s["scale"] = _tokens(case, g), math.sqrt(h)
        if op == "emb_fwd":
            s["weight"] = torch.empty(v, h, device=DEV).normal_(0, 0.02, generator=g).to(dt)
            return s
        s["dy"] = torch.empty(n, h, device=DEV).normal_(0, 1e-3, generator=g).to(dt)
        s["pad"] = v // 2 if case["pad"] else None
        if case["add"]:
            s["dw"] = torch.empty(v, h, device=DEV).normal_(0, 1e-2, generator=g).to(dt)
        return s
    if op == "ortho":
        s["x"] = _matrices((case["count"], case["rows"], case["cols"]), g).to(DTYPES[case["dtype"]])
        return s
    total, spans = _layout(case)
    s["param"] = torch.zeros(total, device=DEV, dtype=torch.bfloat16)
    s["momentum"] = torch.zeros(total, device=DEV)
    s["grad"] = torch.zeros(total, device=DEV, dtype=DTYPES[case["gdtype"]])
    for at, (r, c) in spans:
        cut = slice(at, at + r * c)
        s["param"][cut] = torch.empty(r * c, device=DEV).normal_(0, 0.02, generator=g).to(torch.bfloat16)
        s["momentum"][cut] = _matrices((r, c), g).view(-1)
        s["grad"][cut] = 2 * (s["momentum"][cut] + _matrices((r, c), g).view(-1)).to(s["grad"].dtype)
    s["grad_scale"] = torch.full((1,), 0.5, device=DEV)
    s["lr"], s["weight_decay"], s["mu"] = 0.02, 0.1, 0.95
    return s


# ----------------------------------------------------------------------------- the library's calls


def _views(s, name):
    return [s[name][at:at + r * c].view(r, c) for at, (r, c) in _layout(s["case"])[1]]


def _run_own(s):
    import lm_head_cross_gb300 as flce

    case, op = s["case"], s["case"]["op"]
    if op == "emb_fwd":
        return flce.embedding_forward(s["ids"], s["weight"], scale=s["scale"])[0]
    if op == "emb_bwd":
        return flce.embedding_backward(s["dy"], s["ids"], case["v"], scale=s["scale"], padding_idx=s["pad"],
                                       add_to=s.get("dw"))[0]
    if op == "ortho":
        return flce.orthogonalize(s["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
    if "plan" not in s:  # the handle that a training program makes once for its matrices
        s["plan"] = flce.muon_plan(_views(s, "param"), _views(s, "momentum"), lr=s["lr"],
                                   weight_decay=s["weight_decay"], momentum=s["mu"], nesterov=case["nesterov"],
                                   steps=STEPS, coefficients=COEFFICIENTS, eps=EPS)
        s["grads"] = _views(s, "grad")
    flce.muon_step(s["plan"], s["grads"], grad_scale=s["grad_scale"])
    return {"param": s["param"], "momentum": s["momentum"]}


# ----------------------------------------------------------------------------- plain forms


def _newton_schulz(x):
    """x [..., R, C] in 32 bits, on the side of the smaller products."""
    flip = x.shape[-2] > x.shape[-1]
    if flip:
        x = x.transpose(-1, -2)
    x = x / (x.square().sum((-1, -2), keepdim=True).sqrt() + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        gram = x @ x.transpose(-1, -2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(-1, -2) if flip else x


def _by_shape(case):
    """{shape: where its matrices start in the flat buffers}."""
    found = {}
    for at, shape in _layout(case)[1]:
        found.setdefault(shape, []).append(at)
    return found


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "emb_fwd":
        return (s["weight"][s["ids"].long()].float() * s["scale"]).to(s["weight"].dtype)
    if op == "emb_bwd":
        ids, dy = s["ids"].long(), s["dy"].float()
        if s["pad"] is not None:
            dy = torch.where((ids == s["pad"])[:, None], 0.0, dy)
        total = torch.zeros(case["v"], case["h"], device=DEV).index_add_(0, ids, dy).mul_(s["scale"])
        if not case["add"]:
            return total.to(s["dy"].dtype)
        s["dw"].copy_(total.add_(s["dw"]))
        return s["dw"]
    if op == "ortho":
        return _newton_schulz(s["x"].float()).to(torch.bfloat16)
    mu = s["mu"]
    g = s["grad"].float() * s["grad_scale"]
    s["momentum"].mul_(mu).add_(g, alpha=1 - mu)
    u = s["momentum"] * mu + g * (1 - mu) if case["nesterov"] else s["momentum"]
    for (r, c), starts in _by_shape(case).items():
        at = torch.tensor(starts, device=DEV)[:, None] + torch.arange(r * c, device=DEV)
        step = _newton_schulz(u[at].view(-1, r, c)).reshape(-1, r * c)
        rate = s["lr"] * math.sqrt(max(1.0, r / c))
        s["param"][at] = (s["param"][at].float() * (1 - s["lr"] * s["weight_decay"]) - rate * step).to(torch.bfloat16)
    return {"param": s["param"], "momentum": s["momentum"]}


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- definitions in 64 bits


def _exact_polynomial(m):
    """One matrix in 64 bits: its singular values' odd polynomial, applied as products on the right
    for tall and on the left for wide ones."""
    x = m.double()
    x = x / (torch.linalg.vector_norm(x) + EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        if x.shape[0] <= x.shape[1]:
            q = torch.einsum("ik,jk->ij", x, x)
            x = a * x + torch.addmm(b * q, q, q, alpha=c) @ x
        else:
            q = torch.einsum("ki,kj->ij", x, x)
            x = a * x + x @ torch.addmm(b * q, q, q, alpha=c)
    return x


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "emb_fwd":
        return torch.index_select(s["weight"], 0, s["ids"]).double().mul_(s["scale"])
    if op == "emb_bwd":
        # tokens in sorted order, each token's rows added up in turn
        ids, order = torch.sort(s["ids"].long(), stable=True)
        keep = torch.ones_like(ids, dtype=torch.bool) if s["pad"] is None else ids != s["pad"]
        ids, order = ids[keep], order[keep]
        out = torch.zeros(case["v"], case["h"], dtype=torch.float64, device=DEV)
        rows = 1 << 15
        for lo in range(0, ids.numel(), rows):
            out.index_put_((ids[lo:lo + rows],), s["dy"][order[lo:lo + rows]].double(), accumulate=True)
        out *= s["scale"]
        return out + s["dw"].double() if case["add"] else out
    if op == "ortho":
        return torch.stack([_exact_polynomial(m) for m in s["x"]])
    param, momentum = s["param"].double(), s["momentum"].double()
    g = s["grad"].double() * s["grad_scale"].double()
    momentum += (1 - s["mu"]) * (g - momentum)
    u = momentum + (1 - s["mu"]) * (g - momentum) if case["nesterov"] else momentum
    for at, (r, c) in _layout(case)[1]:
        cut = slice(at, at + r * c)
        step = _exact_polynomial(u[cut].view(r, c)).view(-1)
        param[cut] -= s["lr"] * (s["weight_decay"] * param[cut] + max(1.0, r / c) ** 0.5 * step)
    return {"param": param, "momentum": momentum}
