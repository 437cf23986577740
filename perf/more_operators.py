"""Timed cases of the operators at the two ends of a training step's matrices: the loss that starts
the backward pass, and the direction that the optimizer's projected step takes.

  xent_fwd, xent_bwd   softmax cross entropy of hidden states against a large vocabulary, straight
                       from the output head's weights: loss and log-sum-exp of every token, and the
                       gradients of the hidden states and of the weights, in pieces of the
                       vocabulary, so that no matrix of all logits exists
  ortho                momentum of weight gradients and its orthogonalised direction by
                       Newton-Schulz products, for several matrices of one shape at once

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own``
true it calls the package's entry points. ``exact`` evaluates the definitions in 64 bits."""
import math

import torch

own = False

DEV = "cuda"
COEFFICIENTS = (3.4445, -4.7750, 2.0315)   # of X <- aX + b(XX')X + c(XX')^2 X
STEPS = 5
BETA = 0.95
NO_TARGET = -100


def listed():
    return [
        # one token scored against a vocabulary of 32768: the weights are read once, pure bandwidth
        {"name": "xent-fwd-1x2048x32768", "op": "xent_fwd", "tokens": 1, "d": 2048, "vocab": 32768,
         "masked": 0.0},
        # a prompt of odd length scored, hidden size that is no multiple of 64, odd vocabulary
        {"name": "xent-fwd-777x1000x50021", "op": "xent_fwd", "tokens": 777, "d": 1000,
         "vocab": 50021, "masked": 0.0},
        # the training micro-batch: two sequences of 4096 tokens, hidden size 2048
        {"name": "xent-fwd-8192x2048x131072", "op": "xent_fwd", "tokens": 8192, "d": 2048,
         "vocab": 131072, "masked": 0.02},
        # few tokens trained: the backward pass at its most bandwidth-bound
        {"name": "xent-bwd-64x2048x32768", "op": "xent_bwd", "tokens": 64, "d": 2048,
         "vocab": 32768, "masked": 0.0, "lse": False},
        # a ragged batch whose prompts carry no loss, with a penalty on the log-sum-exp
        {"name": "xent-bwd-1003x1000x50021", "op": "xent_bwd", "tokens": 1003, "d": 1000,
         "vocab": 50021, "masked": 0.5, "lse": True},
        # one sequence of 4096 tokens, a middle-sized vocabulary
        {"name": "xent-bwd-4096x2048x65536", "op": "xent_bwd", "tokens": 4096, "d": 2048,
         "vocab": 65536, "masked": 0.02, "lse": True},
        # the training micro-batch backward
        {"name": "xent-bwd-8192x2048x131072", "op": "xent_bwd", "tokens": 8192, "d": 2048,
         "vocab": 131072, "masked": 0.02, "lse": False},
        # one small projection: launches count
        {"name": "ortho-1x128x512", "op": "ortho", "count": 1, "rows": 128, "cols": 512,
         "momentum": True},
        # odd, tall matrices, plain gradients without momentum
        {"name": "ortho-3x1000x333", "op": "ortho", "count": 3, "rows": 1000, "cols": 333,
         "momentum": False},
        # a layer's down projection by itself
        {"name": "ortho-1x2048x6144", "op": "ortho", "count": 1, "rows": 2048, "cols": 6144,
         "momentum": True},
        # the attention output projections of all 28 layers
        {"name": "ortho-28x2048x2048", "op": "ortho", "count": 28, "rows": 2048, "cols": 2048,
         "momentum": True},
        # the gate_up projections of four layers: tall
        {"name": "ortho-4x12288x2048", "op": "ortho", "count": 4, "rows": 12288, "cols": 2048,
         "momentum": True},
    ]


def _log_int(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), max(lo, hi))


def draw(rng):
    op = rng.choice(["xent_fwd", "xent_bwd", "ortho"])
    if op == "ortho":
        rows, cols = _log_int(rng, 16, 12288), _log_int(rng, 16, 12288)
        if rng.random() < 0.5:
            rows, cols = max(16, rows // 64 * 64), max(16, cols // 64 * 64)
        short, long = min(rows, cols), max(rows, cols)
        short = min(short, 4096)
        rows, cols = (short, long) if rows <= cols else (long, short)
        most = 2.4e11 // (short * short * (long + short))    # about 28 matrices of 2048 x 2048
        return {"op": op, "count": _log_int(rng, 1, int(min(28, max(1, most)))), "rows": rows,
                "cols": cols, "momentum": rng.random() < 0.75}
    tokens, d = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096)
    if rng.random() < 0.75:
        d = max(64, d // 64 * 64)
    vocab = min(_log_int(rng, 500, 131072), 2 ** 41 // (tokens * d))
    c = {"op": op, "tokens": tokens, "d": d, "vocab": vocab,
         "masked": rng.choice([0.0, 0.02, 0.5])}
    if op == "xent_bwd":
        c["lse"] = rng.random() < 0.5
    return c


def work(c):
    if c["op"] == "ortho":
        n = c["count"] * c["rows"] * c["cols"]
        short, long = min(c["rows"], c["cols"]), max(c["rows"], c["cols"])
        # XX' and its square are symmetric: half of their products; their product with X whole
        step = short * short * long + short ** 3 + 2 * short * short * long
        return {"bytes": n * (4 + 2) + (8 * n if c["momentum"] else 0),
                "flops": c["count"] * STEPS * step}
    t, d, v = c["tokens"], c["d"], c["vocab"]
    if c["op"] == "xent_fwd":
        return {"bytes": 2 * (t + v) * d + 16 * t, "flops": 2 * t * d * v}
    # the logits are not kept: they are multiplied out again, then both gradients
    return {"bytes": 4 * (t + v) * d + (20 if c["lse"] else 16) * t, "flops": 6 * t * d * v}


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _hidden(c, g):
    """Hidden states that know their target to different degrees (its logit is raised by 0 to 16),
    head weights of standard deviation 0.02, targets, and which tokens have none."""
    t, d, v = c["tokens"], c["d"], c["vocab"]
    w = (0.02 * torch.randn((v, d), generator=g, device=DEV)).bfloat16()
    targets = torch.randint(0, v, (t,), generator=g, device=DEV)
    lift = 16 * torch.rand((t, 1), generator=g, device=DEV) / (d * 4e-4)
    h = (torch.randn((t, d), generator=g, device=DEV) + lift * w[targets].float()).bfloat16()
    if c["masked"]:
        targets[torch.rand(t, generator=g, device=DEV) < c["masked"]] = NO_TARGET
    return h, w, targets


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "ortho":
        n, rows, cols = c["count"], c["rows"], c["cols"]
        rank = max(1, min(rows, cols) // 8)

        def gradient():
            # what a weight gradient looks like: a few strong directions over a floor of noise
            left = torch.randn((n, rows, rank), generator=g, device=DEV)
            right = torch.randn((n, rank, cols), generator=g, device=DEV)
            fall = torch.arange(1, rank + 1, device=DEV, dtype=torch.float32) ** -0.5
            return 1e-4 * (torch.bmm(left * fall, right)
                           + 0.5 * torch.randn((n, rows, cols), generator=g, device=DEV))

        s["g"] = gradient()
        if c["momentum"]:
            s["m"] = 0.3 * gradient() + 0.2 * s["g"]
            s["m_out"] = torch.empty_like(s["m"])
        return s
    s["h"], s["w"], s["targets"] = _hidden(c, g)
    if c["op"] == "xent_bwd":
        t = c["tokens"]
        lse = _lse(s["h"], s["w"])
        s["lse"] = torch.where(s["targets"] >= 0, lse, torch.zeros_like(lse))
        # the mean over the tokens that have a target, weighted per token
        s["dloss"] = (0.5 + torch.rand(t, generator=g, device=DEV)) / t
        s["dlse"] = 2e-4 * s["lse"] / t if c["lse"] else None
    return s


def _lse(h, w):
    return torch.cat([torch.logsumexp(h[i:i + 1024].float() @ w.float().t(), 1)
                      for i in range(0, len(h), 1024)])


# ------------------------------------------------------------------ plain forms
def _plain_xent_fwd(h, w, targets):
    has = targets >= 0
    logits = h.float() @ w.float().t()
    top = logits.max(1).values
    lse = top + (logits - top[:, None]).exp().sum(1).log()
    at = logits.gather(1, targets.clamp_min(0)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return torch.where(has, lse - at, zero), torch.where(has, lse, zero)


def _plain_xent_bwd(h, w, targets, lse, dloss, dlse):
    has = targets >= 0
    hf, wf = h.float(), w.float()
    p = ((hf @ wf.t()) - lse[:, None]).exp_()
    p *= (dloss if dlse is None else dloss + dlse)[:, None]
    rows = torch.arange(len(h), device=h.device)
    at = targets.clamp_min(0)
    p[rows, at] -= dloss
    p = torch.where(has[:, None], p, torch.zeros_like(p))
    return (p @ wf).bfloat16(), (p.t() @ hf).bfloat16()


def _plain_ortho(g, m):
    a, b, c = COEFFICIENTS
    x = g
    if m is not None:
        m = BETA * m + (1 - BETA) * g
        x = BETA * m + (1 - BETA) * g
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    norm = x.double().square().sum((1, 2), keepdim=True).sqrt().float()
    x = x / norm
    for _ in range(STEPS):
        gram = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * gram + c * torch.bmm(gram, gram), x)
    if tall:
        x = x.transpose(1, 2).contiguous()
    return x.bfloat16(), m


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from blockwise_fp8_gemm_x128_amd import binding as puro
        if op == "xent_fwd":
            return list(puro.puro_linear_xent_fwd(s["h"], s["w"], s["targets"]))
        if op == "xent_bwd":
            return list(puro.puro_linear_xent_bwd(s["h"], s["w"], s["targets"], s["lse"],
                                                  s["dloss"], s["dlse"]))
        u = torch.empty_like(s["g"], dtype=torch.bfloat16)
        if "m" not in s:
            puro.puro_newton_schulz(s["g"].unbind(0), us=u.unbind(0))
            return [u]
        puro.puro_newton_schulz(s["g"].unbind(0), s["m"].unbind(0), us=u.unbind(0),
                                ms_out=s["m_out"].unbind(0), beta=BETA)
        return [u, s["m_out"]]
    if op == "xent_fwd":
        return list(_plain_xent_fwd(s["h"], s["w"], s["targets"]))
    if op == "xent_bwd":
        return list(_plain_xent_bwd(s["h"], s["w"], s["targets"], s["lse"], s["dloss"], s["dlse"]))
    u, m = _plain_ortho(s["g"], s.get("m"))
    return [u] if m is None else [u, m]


# ------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The definitions in 64 bits, a block of tokens (a matrix) at a time."""
    s = prepare(case, seed)
    if case["op"] == "ortho":
        return _exact_ortho(s)
    h, w, targets = s["h"].double(), s["w"].double(), s["targets"]
    blocks = range(0, len(h), 512)
    if case["op"] == "xent_fwd":
        loss = torch.zeros(len(h), dtype=torch.float64, device=DEV)
        lse = torch.zeros_like(loss)
        for i in blocks:
            l = torch.matmul(h[i:i + 512], w.t())
            for_all = torch.logsumexp(l, 1)
            y = targets[i:i + 512]
            own_logit = (h[i:i + 512] * w[y.clamp(min=0)]).sum(1)
            lse[i:i + 512] = for_all * (y >= 0)
            loss[i:i + 512] = (for_all - own_logit) * (y >= 0)
        return [loss, lse]
    dloss = s["dloss"].double()
    every = dloss + (s["dlse"].double() if s["dlse"] is not None else 0)
    dh, dw = torch.zeros_like(h), torch.zeros_like(w)
    for i in blocks:
        part, y = slice(i, i + 512), targets[i:i + 512]
        keep = (y >= 0).double()[:, None]
        soft = torch.exp(torch.matmul(h[part], w.t()) - s["lse"][part].double()[:, None])
        soft = soft * every[part][:, None] * keep
        hot = dloss[part][:, None] * keep
        at = y.clamp(min=0)
        dh[part] = torch.matmul(soft, w) - hot * w[at]
        dw += torch.matmul(soft.t(), h[part])
        dw.index_add_(0, at, -hot * h[part])
    return [dh, dw]


def _exact_ortho(s):
    a, b, c = COEFFICIENTS
    us, ms = [], []
    for i in range(s["case"]["count"]):
        v = s["g"][i].double()
        if "m" in s:
            ms.append(BETA * s["m"][i].double() + (1 - BETA) * v)
            v = BETA * ms[-1] + (1 - BETA) * v
        x = v / torch.linalg.matrix_norm(v)
        for _ in range(STEPS):
            if x.shape[0] > x.shape[1]:     # the polynomial from the right: the same matrix
                k = torch.matmul(x.t(), x)
                x = torch.matmul(x, a * torch.eye(len(k), dtype=k.dtype, device=DEV)
                                 + torch.matmul(k, b * torch.eye(len(k), dtype=k.dtype, device=DEV)
                                                + c * k))
            else:
                k = torch.matmul(x, x.t())
                kx = torch.matmul(k, x)
                x = a * x + b * kx + c * torch.matmul(k, kx)
        us.append(x)
    return [torch.stack(us)] + ([torch.stack(ms)] if ms else [])
