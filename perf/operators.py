"""The cases on which the operators around the LM head are measured.

Three operators that a program calls next to the fused linear cross-entropy:

  layer norm        the final norm that makes the head's input, forward and backward
                    with the reduction of the weight's and bias's gradients;
  token logprobs    log probabilities of given tokens under softmax(x W^T / T), with
                    the distribution's entropy and its top alternatives, from single
                    tokens to whole batches, and the gradients of both;
  AdamW             one step over many tensors, with moments in 32 or in 8 bits.

``run`` computes a case in plain 32-bit torch operations where ``own`` is false and
through this library's entry points where it is true.  ``exact`` gives the definition
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ----------------------------------------------------------------------------- cases


def listed():
    return [
        # one decoding step of four sequences: launch latency, nothing else
        dict(name="ln_fwd_decode", op="ln_fwd", n=4, h=4096, dtype="bf16", wdtype="bf16"),
        # the final norm of a 128K-token batch, the head's largest workload
        dict(name="ln_fwd_128k", op="ln_fwd", n=131072, h=4096, dtype="bf16", wdtype="bf16"),
        # the backward pass of the final norm in an ordinary training step
        dict(name="ln_bwd_8k", op="ln_bwd", n=8192, h=2048, dtype="bf16", wdtype="fp32"),
        # 32-bit activations and a width that no vector load divides
        dict(name="ln_bwd_odd_fp32", op="ln_bwd", n=5003, h=1031, dtype="fp32", wdtype="fp32"),
        # one token of one sequence: the head's weights are read once, that is all
        dict(name="lp_decode_1", op="lp", n=1, h=2048, v=32000, top=5, temperature=1.0, tokens=True),
        # a serving batch that reports the sampled token and eight alternatives
        dict(name="lp_serve_64", op="lp", n=64, h=4096, v=128256, top=8, temperature=0.7, tokens=True),
        # scoring a ragged batch over a vocabulary that no tile divides, with the most alternatives
        dict(name="lp_score_ragged", op="lp", n=777, h=1544, v=40009, top=16, temperature=1.3, tokens=True),
        # scoring 8K prompt tokens: likelihoods and entropies alone
        dict(name="lp_score_8k", op="lp", n=8192, h=2048, v=32000, top=0, temperature=1.0, tokens=True),
        # a small policy step: log probabilities and entropies, forward and backward
        dict(name="lp_step_256", op="lp_step", n=256, h=128, v=1024, temperature=1.0, ignore=0.1),
        # an ordinary policy step with masked (prompt) tokens and an entropy bonus
        dict(name="lp_step_4k", op="lp_step", n=4096, h=4096, v=32000, temperature=1.0, ignore=0.25),
        # every parameter of a small model: 149 tensors of very different sizes, moments in 32 bits
        dict(name="adamw_model", op="adamw", layers=16, h=512, v=32000, dtype="bf16", gdtype="bf16", master=True,
             bits=32),
        # the head of the 128K vocabulary with the final norm, moments in 8 bits
        dict(name="adamw_head_8bit", op="adamw", layers=0, h=4096, v=128256, dtype="bf16", gdtype="bf16", master=True,
             bits=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "lp", "lp_step", "adamw"])
    if op in ("ln_fwd", "ln_bwd"):
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        h = _log_int(rng, 8, 8192)
        if rng.random() < 0.6:
            h = (h + 7) // 8 * 8
        most = 131072 * 4096 // (2 if dtype == "fp32" or op == "ln_bwd" else 1)
        n = _log_int(rng, 1, min(131072, most // h))
        return dict(op=op, n=n, h=h, dtype=dtype, wdtype=rng.choice(["bf16", "fp32"]))
    if op in ("lp", "lp_step"):
        most = 8192 * 2048 * 32000 if op == "lp" else 4096 * 4096 * 32000
        h = 8 * _log_int(rng, 8, 512)
        v = _log_int(rng, 100, 131072)
        n = _log_int(rng, 1, max(1, min(8192, most // (h * v), 8192 * 64000 // v)))
        t = rng.choice([1.0, 1.0, 0.7, 1.3])
        if op == "lp_step":
            return dict(op=op, n=n, h=h, v=v, temperature=t, ignore=rng.choice([0.0, 0.1, 0.5]))
        return dict(op=op, n=n, h=h, v=v, top=rng.randint(0, 16), temperature=t, tokens=rng.random() < 0.8)
    dtype = rng.choice(["bf16", "fp32"])
    h = _log_int(rng, 64, 2048) if rng.random() < 0.3 else 8 * _log_int(rng, 8, 256)
    return dict(op=op, layers=rng.randint(0, 8), h=h, v=_log_int(rng, 100, 65536), dtype=dtype,
                gdtype=rng.choice([dtype, "fp32"]), master=dtype == "bf16" and rng.random() < 0.7,
                bits=rng.choice([8, 32]))


def _adamw_shapes(case):
    """A decoder's parameters: per layer two norms, the four attention matrices and the
    gated feed-forward's three; then the final norm's weight and bias and the head."""
    h, f = case["h"], 2 * case["h"] + case["h"] // 3
    layer = [(h,), (h, h), (h // 4 + 1, h), (h // 4 + 1, h), (h, h), (h,), (f, h), (f, h), (h, f)]
    return layer * case["layers"] + [(h,), (h,), (case["v"], h)] + [(7,), (1,)] * (case["layers"] > 0)


#: every tensor starts at a multiple of this many elements of a flat buffer, as buckets lay them out
ALIGN = 256


def _adamw_layout(case):
    at, spans = 0, []
    for shape in _adamw_shapes(case):
        count = math.prod(shape)
        spans.append((at, count, shape))
        at += (count + ALIGN - 1) // ALIGN * ALIGN
    return at, spans


def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp32": 4}
    if op in ("ln_fwd", "ln_bwd"):
        n, h, s, ws = case["n"], case["h"], size[case["dtype"]], size[case["wdtype"]]
        if op == "ln_fwd":  # x, weight, bias in; y, mean, rstd out
            return {"bytes": 2 * n * h * s + 2 * h * ws + 8 * n, "flops": 8 * n * h}
        return {"bytes": 3 * n * h * s + 3 * h * ws + 8 * n, "flops": 16 * n * h}
    if op == "lp":
        n, h, v = case["n"], case["h"], case["v"]
        return {"bytes": 2 * (n + v) * h + 4 * n * (3 + bool(case["tokens"])) + 8 * n * case["top"],
                "flops": 2 * n * h * v + 6 * n * v}
    if op == "lp_step":  # the logits, dX and dW: three products
        n, h, v = case["n"], case["h"], case["v"]
        return {"bytes": 4 * (n + v) * h + 24 * n, "flops": 6 * n * h * v + 12 * n * v}
    count = sum(c for _, c, _ in _adamw_layout(case)[1])
    s = size[case["gdtype"]] + size[case["dtype"]] * (1 if case["master"] else 2) + (8 if case["master"] else 0)
    s += 16 if case["bits"] == 32 else 4 + 16 / 256
    return {"bytes": s * count, "flops": 16 * count}


# ----------------------------------------------------------------------------- inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _head_inputs(case, g):
    """Hidden states and head weights on 8-bit grids, as an 8-bit-quantised checkpoint
    holds them in bf16: x in steps of 2^-5, w in a power-of-two step that keeps the logits'
    spread near that of a trained head.  Every logit is then a 32-bit number without
    rounding, whatever the order of its sum, so that the alternatives' ids have one right
    answer (equal logits occur: the lowest id goes first).  Each row leans towards its
    token by a random amount, from not at all to better than even odds."""
    n, h, v = case["n"], case["h"], case["v"]
    step = 2.0 ** -(5 + math.ceil(math.log2(h) / 2))
    kw = torch.empty(v, h, device=DEV, dtype=torch.float32).normal_(0, 60, generator=g).round_().clamp_(-127, 127)
    tok = torch.randint(0, v, (n,), device=DEV, generator=g)
    lean = torch.rand(n, 1, device=DEV, generator=g) * ((math.log(v) - 1) / (h * 60 * step))
    x = torch.randn(n, h, device=DEV, generator=g) + lean * kw[tok] / 60
    x = (x * 32).round_().clamp_(-127, 127) / 32
    return x.to(torch.bfloat16), (kw * step).to(torch.bfloat16), tok.to(torch.int32)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": case}
    if op in ("ln_fwd", "ln_bwd"):
        n, h, dt, wdt = case["n"], case["h"], DTYPES[case["dtype"]], DTYPES[case["wdtype"]]
        # residual-stream statistics: a spread that differs by row, an offset, a few large columns
        col = 1 + 6 * (torch.rand(h, device=DEV, generator=g) < 0.01).float()
        x = torch.randn(n, h, device=DEV, generator=g) * (0.5 + torch.rand(n, 1, device=DEV, generator=g)) * col + 0.2
        s["x"] = x.to(dt)
        s["weight"] = (1 + 0.2 * torch.randn(h, device=DEV, generator=g)).to(wdt)
        s["bias"] = (0.1 * torch.randn(h, device=DEV, generator=g)).to(wdt)
        s["eps"] = 1e-5
        if op == "ln_bwd":
            s["dy"] = (1e-3 * torch.randn(n, h, device=DEV, generator=g)).to(dt)
            xf = s["x"].float()
            s["mean"] = xf.mean(1)
            s["rstd"] = torch.rsqrt(xf.var(1, unbiased=False) + s["eps"])
        return s
    if op in ("lp", "lp_step"):
        s["x"], s["w"], tok = _head_inputs(case, g)
        if op == "lp":
            s["tokens"] = tok if case["tokens"] else None
        else:
            n = case["n"]
            skip = torch.rand(n, device=DEV, generator=g) < case["ignore"]
            s["tokens"] = torch.where(skip, torch.full_like(tok, -100), tok)
            # a policy step's upstream gradients: -advantage / n on the log probabilities, a
            # small bonus on the entropies, none where the token is masked
            s["g_logprob"] = torch.randn(n, device=DEV, generator=g) / n
            s["g_entropy"] = torch.where(skip, 0.0, -0.01 / n)
        return s
    total, spans = _adamw_layout(case)
    dt, gdt = DTYPES[case["dtype"]], DTYPES[case["gdtype"]]
    gap = torch.ones(total, dtype=torch.bool, device=DEV)
    for at, count, _ in spans:
        gap[at:at + count] = False
    master = torch.empty(total, device=DEV).normal_(0, 0.02, generator=g).masked_fill_(gap, 0)
    s["param"] = master.to(dt)
    s["master"] = master if case["master"] else None
    grad = torch.empty(total, device=DEV).normal_(0, 1e-3, generator=g)
    grad.mul_(torch.rand(total, device=DEV, generator=g).pow_(2)).masked_fill_(gap, 0)
    s["grad"] = grad.to(gdt)
    m = torch.empty(total, device=DEV).normal_(0, 3e-4, generator=g).masked_fill_(gap, 0)
    r = torch.empty(total, device=DEV).uniform_(1e-5, 1e-3, generator=g).masked_fill_(gap, 0)
    if case["bits"] == 32:
        s["exp_avg"], s["exp_avg_sq"] = m, r.square_()
    else:  # e4m3 values with one scale for 256 elements; the second moment as its root
        for name, t in (("exp_avg", m), ("exp_avg_sq", r)):
            scale = t.view(-1, 256).abs().amax(1) / 448
            s[name] = (t.view(-1, 256) / scale.clamp_min(1e-30)[:, None]).to(torch.float8_e4m3fn).view(-1)
            s[name + "_scale"] = scale
    s["grad_scale"] = torch.full((1,), 0.5, device=DEV)
    s["lr"], s["betas"], s["eps"], s["weight_decay"], s["step"] = 3e-4, (0.9, 0.95), 1e-8, 0.1, 1000
    return s


# ----------------------------------------------------------------------------- the library's calls


def _views(s, name, per=1):
    t = s[name]
    if t is None:
        return None
    if per > 1:
        return [t[at // per:(at + count + per - 1) // per] for at, count, _ in _adamw_layout(s["case"])[1]]
    return [t[at:at + count].view(shape) for at, count, shape in _adamw_layout(s["case"])[1]]


def _run_own(s):
    import lm_head_cross_gb300 as flce

    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        y, mean, rstd = flce.layernorm_forward(s["x"], s["weight"], s["bias"], eps=s["eps"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dx, dweight, dbias, _ = flce.layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op in ("lp", "lp_step"):
        r, ws = flce.logprobs_forward(s["x"], s["w"], s["tokens"], top=case.get("top", 0),
                                      temperature=case["temperature"])
        if op == "lp":
            return {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse, "top_ids": r.top_ids,
                    "top_logprobs": r.top_logprobs}
        dx, dw, _ = flce.logprobs_backward(s["x"], s["w"], s["tokens"], r.lse, r.entropy, s["g_logprob"],
                                           s["g_entropy"], temperature=case["temperature"])
        return {"logprob": r.logprob, "entropy": r.entropy, "dx": dx, "dw": dw}
    if "plan" not in s:  # the handle that a training program makes once for its tensors
        bits = case["bits"]
        s["plan"] = flce.adamw_plan(
            _views(s, "param"), _views(s, "exp_avg"), _views(s, "exp_avg_sq"), masters=_views(s, "master"),
            scales=None if bits == 32 else (_views(s, "exp_avg_scale", 256), _views(s, "exp_avg_sq_scale", 256)),
            lr=s["lr"], betas=s["betas"], eps=s["eps"], weight_decay=s["weight_decay"])
        s["grads"] = _views(s, "grad")
    s["step"] += 1
    flce.adamw_step(s["plan"], s["grads"], step=s["step"], grad_scale=s["grad_scale"])
    return _adamw_out(s)


def _adamw_out(s):
    names = ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")
    return {k: s[k] for k in names if s.get(k) is not None}


# ----------------------------------------------------------------------------- plain forms


def _top_alternatives(z, k):
    """Ids of each row's k largest values, the lowest id first among equals: the order of
    (value, -id) as one 64-bit key."""
    bits = (z + 0.0).view(torch.int32).to(torch.int64)
    bits = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF)
    key = bits * (1 << 32) + ((1 << 32) - 1 - torch.arange(z.shape[1], device=z.device))
    return torch.topk(key, k, dim=1).indices


def _softmax_stats(z):
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    lse = m + torch.log(total)
    entropy = torch.log(total) - (e * (z - m)).sum(1, keepdim=True) / total
    return lse, entropy


def _plain_adamw_8bit_encode(s, m, r, step):
    """Moments as e4m3 with one scale for 256 elements.  The first moment is rounded to
    nearest; the root of the second by a hash of (step, element), up with a probability
    equal to the fraction passed, so that its running mean keeps moving by less than one
    8-bit step; it never becomes zero unless it is."""
    mb, rb = m.view(-1, 256), r.view(-1, 256)
    for name, t in (("exp_avg", mb), ("exp_avg_sq", rb)):
        top = t.abs().amax(1)
        s[name + "_scale"].copy_(top * (1.0 / 448.0))
        inv = torch.where(top > 0, 448.0 / top, torch.zeros_like(top))
        q = (t * inv[:, None]).clamp_(-448.0, 448.0).view(-1)
        if name == "exp_avg":
            s[name].copy_(q.to(torch.float8_e4m3fn))
            continue
        # elements count from their own tensor's start
        h = _element_index(s) >> 2
        mask, k = 0xFFFFFFFF, 0x9E3779B1
        h = (h * k + (step * 0xA511E9B3 & mask)) & mask
        h = ((h ^ (h >> 16)) * k) & mask
        h = ((h ^ (h >> 13)) * k) & mask
        h = h ^ (h >> 16)
        rnd = ((h >> (8 * (_element_index(s) & 3))) & 0xFF) << 12
        low = q < 2.0 ** -6  # below the normal numbers the steps are equal: shifted up by 2^-6 they are those above it
        bits = torch.where(low, q + 2.0 ** -6, q).view(torch.int32).to(torch.int64)
        code = ((bits + rnd) >> 20) - (120 << 3) - torch.where(low, 8, 0)
        code = torch.where(q > 0, code.clamp_min(1), code)
        s[name].copy_(code.to(torch.uint8).view(torch.float8_e4m3fn))


def _element_index(s):
    """Each element's place in its own tensor (the flat buffer's gaps count on)."""
    if "index" not in s:
        total, spans = _adamw_layout(s["case"])
        starts = torch.tensor([at for at, _, _ in spans], device=DEV)
        at = torch.arange(total, device=DEV)
        s["index"] = at - starts[torch.searchsorted(starts, at, right=True) - 1]
    return s["index"]


def _run_plain_adamw(s):
    case = s["case"]
    b1, b2 = s["betas"]
    s["step"] += 1
    bc1, bc2 = 1 - b1 ** s["step"], 1 - b2 ** s["step"]
    g = s["grad"].float() * s["grad_scale"]
    if case["bits"] == 32:
        m, v = s["exp_avg"], s["exp_avg_sq"]
    else:
        m = (s["exp_avg"].float().view(-1, 256) * s["exp_avg_scale"][:, None]).view(-1)
        v = (s["exp_avg_sq"].float().view(-1, 256) * s["exp_avg_sq_scale"][:, None]).square_().view(-1)
    m = m * b1 + g * (1 - b1)
    v = v * b2 + g * g * (1 - b2)
    r = torch.sqrt(v)
    p = s["master"] if s["master"] is not None else s["param"].float()
    p = p * (1 - s["lr"] * s["weight_decay"]) - (s["lr"] / bc1) * m / (r * (1 / math.sqrt(bc2)) + s["eps"])
    if s["master"] is not None:
        s["master"].copy_(p)
    s["param"].copy_(p)
    if case["bits"] == 32:
        s["exp_avg"].copy_(m)
        s["exp_avg_sq"].copy_(v)
    else:
        _plain_adamw_8bit_encode(s, m, r, s["step"])
    return _adamw_out(s)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "ln_fwd":
        x = s["x"].float()
        mean = x.mean(1)
        c = x - mean[:, None]
        rstd = 1 / torch.sqrt((c * c).mean(1) + s["eps"])
        y = c * rstd[:, None] * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}
    if op == "ln_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        gw = dy * s["weight"].float()
        dx = rstd * (gw - gw.mean(1, keepdim=True) - xhat * (gw * xhat).mean(1, keepdim=True))
        wdt = s["weight"].dtype
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(wdt), "dbias": dy.sum(0).to(wdt)}
    if op == "adamw":
        return _run_plain_adamw(s)
    x, w, it = s["x"].float(), s["w"].float(), 1.0 / case["temperature"]
    raw = x @ w.t()
    z = raw * it
    lse, entropy = _softmax_stats(z)
    out = {"logprob": None, "entropy": entropy[:, 0]}
    if s["tokens"] is not None:
        tok = s["tokens"].long()
        given = tok != -100
        out["logprob"] = torch.where(given, z.gather(1, tok.clamp_min(0)[:, None])[:, 0] - lse[:, 0], 0.0)
    if op == "lp":
        out["lse"] = lse[:, 0]
        out["top_ids"] = out["top_logprobs"] = None
        if case["top"]:
            k = min(case["top"], z.shape[1])
            ids = _top_alternatives(raw, k)
            out["top_ids"], out["top_logprobs"] = ids.to(torch.int32), z.gather(1, ids) - lse
        return out
    # d logprob / dz_j = [j = token] - p_j;  d entropy / dz_j = -p_j (log p_j + entropy)
    lp = z - lse
    gl = torch.where(given, s["g_logprob"], 0.0)[:, None]
    ge = s["g_entropy"][:, None]
    dz = torch.exp(lp) * (-gl - ge * (lp + entropy))
    dz.scatter_add_(1, tok.clamp_min(0)[:, None], gl)
    dz = dz * it
    out["dx"], out["dw"] = (dz @ w).to(torch.bfloat16), (dz.t() @ x).to(torch.bfloat16)
    return out


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ----------------------------------------------------------------------------- definitions in 64 bits


def _exact_norm(s, op):
    """Row by row blocks: the centred, scaled row and, backward, the Jacobian's product."""
    x, w, b = s["x"], s["weight"].double(), s["bias"].double()
    h = x.shape[1]
    ys, means, rstds, dxs = [], [], [], []
    dweight, dbias = torch.zeros_like(w), torch.zeros_like(w)
    for lo in range(0, x.shape[0], 16384):
        a = x[lo:lo + 16384].double()
        if op == "ln_fwd":
            mu = a.sum(1, keepdim=True) / h
            inv = ((a - mu).pow(2).sum(1, keepdim=True) / h + s["eps"]).pow(-0.5)
            ys.append((a - mu) * inv * w + b)
            means.append(mu[:, 0])
            rstds.append(inv[:, 0])
            continue
        inv = s["rstd"][lo:lo + 16384].double()[:, None]
        n = (a - s["mean"][lo:lo + 16384].double()[:, None]) * inv
        d = s["dy"][lo:lo + 16384].double()
        dweight += torch.einsum("ij,ij->j", d, n)
        dbias += d.sum(0)
        u = d * w
        dxs.append(inv * (u - (u.sum(1, keepdim=True) + n * (u * n).sum(1, keepdim=True)) / h))
    if op == "ln_fwd":
        return {"y": torch.cat(ys), "mean": torch.cat(means), "rstd": torch.cat(rstds)}
    return {"dx": torch.cat(dxs), "dweight": dweight, "dbias": dbias}


def _exact_head(s, case):
    x, w = s["x"].double(), s["w"].double()
    n, t = x.shape[0], case["temperature"]
    rows = max(1, (1 << 27) // w.shape[0])
    got = {"logprob": [], "entropy": [], "lse": [], "top": []}
    step = case["op"] == "lp_step"
    dx, dw = [], torch.zeros_like(w) if step else None
    for lo in range(0, n, rows):
        z = (x[lo:lo + rows] @ w.t()) / t
        lse = torch.logsumexp(z, dim=1)
        logp = z - lse[:, None]
        p = logp.exp()
        entropy = -(p * logp).sum(1)
        got["entropy"].append(entropy)
        got["lse"].append(lse)
        if not step and case["top"]:
            got["top"].append(logp.sort(dim=1, descending=True).values[:, :case["top"]])
        if s["tokens"] is None:
            continue
        tok = s["tokens"][lo:lo + rows].long()
        at = torch.nonzero(tok >= 0)[:, 0]
        lpt = torch.zeros(tok.shape[0], dtype=torch.float64, device=x.device)
        lpt[at] = logp[at, tok[at]]
        got["logprob"].append(lpt)
        if step:
            gl = torch.zeros_like(lpt)
            gl[at] = s["g_logprob"][lo:lo + rows].double()[at]
            ge = s["g_entropy"][lo:lo + rows].double()
            dz = -p * gl[:, None] - ge[:, None] * p * (logp + entropy[:, None])
            dz[at, tok[at]] += gl[at]
            dx.append(dz @ w / t)
            dw += dz.t() @ x[lo:lo + rows] / t
    cat = lambda v: torch.cat(v) if v else None  # noqa: E731
    if step:
        return {"logprob": cat(got["logprob"]), "entropy": cat(got["entropy"]), "dx": cat(dx), "dw": dw}
    return {"logprob": cat(got["logprob"]), "entropy": cat(got["entropy"]), "lse": cat(got["lse"]), "top_ids": None,
            "top_logprobs": cat(got["top"])}


def _exact_adamw(s, case):
    """Decoupled weight decay and bias-corrected moments.  The 8-bit moments themselves are
    a rounding to a grid and have no value here; their scales have."""
    b1, b2 = s["betas"]
    t = s["step"] + 1
    eight = case["bits"] == 8
    out = {k: [] for k in ("param", "master", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale")}
    total, block = s["grad"].numel(), 1 << 26
    for lo in range(0, total, block):
        cut = slice(lo, min(total, lo + block))
        cell = slice(lo // 256, (min(total, lo + block)) // 256)
        g = s["grad"][cut].double() * s["grad_scale"].double()
        m, v = s["exp_avg"][cut].double(), s["exp_avg_sq"][cut].double()
        if eight:
            m = m * s["exp_avg_scale"][cell].double().repeat_interleave(256)
            v = (v * s["exp_avg_sq_scale"][cell].double().repeat_interleave(256)) ** 2
        m = m + (1 - b1) * (g - m)
        v = v + (1 - b2) * (g * g - v)
        p = (s["master"] if s["master"] is not None else s["param"])[cut].double()
        p = p - s["lr"] * (s["weight_decay"] * p + (m / (1 - b1 ** t)) / ((v / (1 - b2 ** t)).sqrt() + s["eps"]))
        out["param"].append(p)
        if s["master"] is not None:
            out["master"].append(p)
        if eight:
            out["exp_avg_scale"].append(m.abs().view(-1, 256).max(1).values / 448)
            out["exp_avg_sq_scale"].append(v.sqrt().view(-1, 256).max(1).values / 448)
        else:
            out["exp_avg"].append(m)
            out["exp_avg_sq"].append(v)
    return {k: torch.cat(v) if v else None for k, v in out.items()}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] in ("ln_fwd", "ln_bwd"):
        return _exact_norm(s, case["op"])
    if case["op"] == "adamw":
        return _exact_adamw(s, case)
    return _exact_head(s, case)
