"""Timed cases of the operators that stand between the blockwise-FP8 GEMMs of a training step.

  norm_fwd, norm_bwd    the norm after a block, its gate and residual scale, and the norm before
                        the next block, in one pass; forward with the next GEMM's FP8 operand and
                        the 8-bit checkpoints, backward from checkpoints or from bf16
  swiglu_fwd, swiglu_bwd, swiglu_bwd_fp8
                        the gated activation of the MLP; forward with the down projection's FP8
                        operand and the 8-bit checkpoint, backward to a bf16 gradient, or straight
                        to the FP8 operands of the data- and weight-gradient GEMMs
  pack, unpack, transpose
                        8-bit activation checkpoints (E4M3, one scale per 128 columns): written,
                        read back, and requantised along the rows for the weight gradient

With ``own`` false ``run`` computes them in elementary torch operations in 32 bits; with ``own``
true it calls the package's entry points. ``exact`` evaluates the definitions in 64 bits (codes as
the unrounded scaled values)."""
import math

import torch

own = False

DEV = "cuda"
G = 128           # columns (or rows) per scale
EPS = 1e-6
ALPHA, BETA = 0.75, 0.9375
FP8 = torch.float8_e4m3fn


def listed():
    return [
        # one token through the block boundary: pure latency
        {"name": "norm-fwd-1x2048", "op": "norm_fwd", "rows": 1, "cols": 2048, "res": "bf16",
         "gate": "channel", "n": "fp8", "ckpt": True, "pow2": False},
        # a micro-batch of two 4096-token sequences, hidden size 2048, as the training step runs it
        {"name": "norm-fwd-8192x2048", "op": "norm_fwd", "rows": 8192, "cols": 2048, "res": "bf16",
         "gate": "channel", "n": "fp8", "ckpt": True, "pow2": False},
        # ragged batch, hidden size that ends inside a group, fp32 residual stream, gate per token
        {"name": "norm-fwd-1021x1000", "op": "norm_fwd", "rows": 1021, "cols": 1000, "res": "fp32",
         "gate": "token", "n": "bf16", "ckpt": False, "pow2": False},
        # the same micro-batch backward, from the 8-bit checkpoints
        {"name": "norm-bwd-8192x2048", "op": "norm_bwd", "rows": 8192, "cols": 2048, "res": "bf16",
         "gate": "channel", "saved": "fp8"},
        # odd hidden size, wide rows, fp32 stream, a gate of its own for every element, from bf16
        {"name": "norm-bwd-333x5121", "op": "norm_bwd", "rows": 333, "cols": 5121, "res": "fp32",
         "gate": "full", "saved": "bf16"},
        # the MLP activation of the micro-batch (width 6144)
        {"name": "swiglu-fwd-8192x6144", "op": "swiglu_fwd", "rows": 8192, "f": 6144,
         "pow2": False},
        # ragged batch and width, no checkpoint: backward from the bf16 projections
        {"name": "swiglu-bwd-1003x1537", "op": "swiglu_bwd", "rows": 1003, "f": 1537,
         "saved": "bf16"},
        # one 128-token tile: the smallest batch the weight-gradient GEMM takes
        {"name": "swiglu-bwd-fp8-128x6144", "op": "swiglu_bwd_fp8", "rows": 128, "f": 6144,
         "pow2": False},
        # four sequences of 4096 tokens: the largest batch of the single-layer configurations
        {"name": "swiglu-bwd-fp8-16384x6144", "op": "swiglu_bwd_fp8", "rows": 16384, "f": 6144,
         "pow2": False},
        # an fp32 stream checkpointed for four sequences
        {"name": "pack-16384x2048-fp32", "op": "pack", "rows": 16384, "cols": 2048,
         "dtype": "fp32", "pad": 0, "pow2": False},
        # a checkpoint of odd sizes read back as bf16
        {"name": "unpack-2047x4111", "op": "unpack", "rows": 2047, "cols": 4111, "dtype": "bf16"},
        # the forward operand of the down projection turned into the weight gradient's
        {"name": "transpose-8192x6144", "op": "transpose", "rows": 8192, "cols": 6144,
         "pow2": False},
    ]


MOST_ELEMENTS = 64 * 1024 * 1024      # 10 to 14 bytes an element: below the largest listed case


def _log_int(rng, lo, hi):
    while True:
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        if v not in (1536, 3072):
            return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "swiglu_fwd", "swiglu_bwd", "swiglu_bwd_fp8", "pack",
                     "unpack", "transpose"])
    rows = _log_int(rng, 1, 16384)
    c = {"op": op, "rows": rows}
    if op in ("norm_fwd", "norm_bwd"):
        c["cols"] = min(_log_int(rng, 64, 8192), MOST_ELEMENTS // rows)
        if rng.random() < 0.5:
            c["cols"] = max(64, c["cols"] // 64 * 64)
        c["res"] = rng.choice(["bf16", "fp32"])
        c["gate"] = rng.choice(["none", "channel", "token", "full"])
        if op == "norm_fwd":
            c["n"] = rng.choice(["fp8", "bf16"])
            c["ckpt"] = rng.random() < 0.5
            c["pow2"] = rng.random() < 0.25
        else:
            c["saved"] = rng.choice(["fp8", "bf16"])
    elif op == "swiglu_bwd_fp8":
        c["rows"] = G * _log_int(rng, 1, 128)
        c["f"] = G * min(_log_int(rng, 1, 96), MOST_ELEMENTS // c["rows"] // G)
        c["pow2"] = rng.random() < 0.25
    elif op in ("swiglu_fwd", "swiglu_bwd"):
        c["f"] = min(_log_int(rng, 64, 12288), MOST_ELEMENTS // rows)
        if op == "swiglu_fwd":
            c["pow2"] = rng.random() < 0.25
        else:
            c["saved"] = rng.choice(["fp8", "bf16"])
    else:
        c["cols"] = min(_log_int(rng, 64, 12288), MOST_ELEMENTS // rows)
        if op == "pack":
            c["pad"] = rng.choice([0, 0, 8, 13])
        if op in ("pack", "transpose"):
            c["pow2"] = rng.random() < 0.25
        if op in ("pack", "unpack"):
            c["dtype"] = rng.choice(["bf16", "fp32"])
    for k in ("rows", "cols", "f"):
        if c.get(k) in (1536, 3072):
            c[k] += G
    return c


def _chunks(n):
    return (n + G - 1) // G


def work(c):
    op, rows = c["op"], c["rows"]
    if op in ("norm_fwd", "norm_bwd"):
        cols = c["cols"]
        n, rb = rows * cols, 2 if c["res"] == "bf16" else 4
        scale = 4 * rows * _chunks(cols)
        gate = {"none": 0, "channel": 4 * cols, "token": 4 * rows, "full": 2 * n}[c["gate"]]
        if op == "norm_fwd":
            b = n * (2 + rb + rb) + 8 * cols + gate + 8 * rows
            b += n + scale if c["n"] == "fp8" else 2 * n
            b += 2 * (n + scale) if c["ckpt"] else 0
            return {"bytes": b, "flops": 12 * n}
        saved = 2 * (n + scale) if c["saved"] == "fp8" else n * (2 + rb)
        return {"bytes": saved + n * (rb + 2) + n * (rb + 2) + 16 * cols + 2 * gate + 8 * rows,
                "flops": 30 * n}
    if op.startswith("swiglu"):
        f = c["f"]
        n, scale = rows * f, 4 * rows * _chunks(f)
        if op == "swiglu_fwd":
            return {"bytes": 4 * n + 3 * (n + scale), "flops": 8 * n}
        if op == "swiglu_bwd":
            return {"bytes": 2 * n + (2 * (n + scale) if c["saved"] == "fp8" else 4 * n) + 4 * n,
                    "flops": 14 * n}
        return {"bytes": 2 * n + 2 * (n + scale) + 5 * n + 4 * (5 * n // G), "flops": 20 * n}
    cols = c["cols"]
    n, scale = rows * cols, 4 * rows * _chunks(cols)
    if op == "transpose":
        return {"bytes": 2 * n + scale + 4 * cols * _chunks(rows), "flops": 4 * n}
    return {"bytes": n + scale + n * (2 if c["dtype"] == "bf16" else 4), "flops": 2 * n}


# ------------------------------------------------------------------ plain forms
def _grouped(x):
    """[rows, cols] -> [rows, chunks, G], zeros after the last column."""
    rows, cols = x.shape
    pad = _chunks(cols) * G - cols
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.reshape(rows, -1, G)


def _power(e):
    """2^e as fp32, -127 < e < 128, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _encode(x, pow2):
    """fp32 [rows, cols] -> E4M3 codes (as float8) [rows, cols], scales [chunks, rows]."""
    rows, cols = x.shape
    v = _grouped(x)
    amax = v.abs().amax(2, keepdim=True)
    a = torch.clamp(amax, min=2.0 ** -119)
    if pow2:
        m, e = torch.frexp(a)                       # a = m 2^e, 1/2 <= m < 1; 448 = (7/8) 2^9
        e = torch.clamp(e - 9 + (m > 0.875).to(e.dtype), min=-127)
        s = torch.where(e > -127, _power(e), torch.full_like(a, 2.0 ** -127))
        r = _power(-e)
    else:
        s, r = a / 448.0, torch.full_like(a, 448.0) / a     # each one rounding
    one = torch.ones_like(a)
    s, r = torch.where(amax == 0, one, s), torch.where(amax == 0, one, r)
    q = torch.clamp(v * r, -448.0, 448.0).to(FP8)
    return q.reshape(rows, -1)[:, :cols].contiguous(), s[:, :, 0].t().contiguous()


def _decode(q, s):
    """uint8 codes [rows, cols], scales [chunks, rows] -> fp32."""
    cols = q.shape[1]
    return q.view(FP8).float() * s.t().repeat_interleave(G, 1)[:, :cols]


def _decode_halves(q, s):
    f, k = q.shape[1] // 2, s.shape[0] // 2
    return _decode(q[:, :f].contiguous(), s[:k]), _decode(q[:, f:].contiguous(), s[k:])


def _gate(st):
    g = st["gate"]
    if g is None:
        return 1.0
    return g.float()


def _plain_norm_fwd(st):
    c = st["case"]
    y, r = st["y"].float(), st["r"].float()
    rstd_y = torch.rsqrt((y * y).mean(1) + EPS)
    p = y * rstd_y[:, None] * st["w_post"]
    t = BETA * r + ALPHA * _gate(st) * p
    rstd_r = torch.rsqrt((t * t).mean(1) + EPS)
    n = t * rstd_r[:, None] * st["w_pre"]
    o = {"r_out": t.to(st["r"].dtype), "rstd_y": rstd_y, "rstd_r": rstd_r}
    if c["n"] == "fp8":
        o["nq"], o["ns"] = _encode(n, c["pow2"])
    else:
        o["n"] = n.to(torch.bfloat16)
    if c["ckpt"]:
        o["yq"], o["ys"] = _encode(y, c["pow2"])
        o["rq"], o["rs"] = _encode(t, c["pow2"])
    return o


def _plain_norm_bwd(st):
    c = st["case"]
    if c["saved"] == "fp8":
        y, t = _decode(*st["y_saved"]), _decode(*st["r_saved"])
    else:
        y, t = st["y_saved"].float(), st["r_saved"].float()
    g = _gate(st)
    dn, dro = st["dn"].float(), st["dr_out"].float()
    yh, th = y * st["rstd_y"][:, None], t * st["rstd_r"][:, None]
    a = st["w_pre"] * dn
    grad = dro + st["rstd_r"][:, None] * (a - th * (th * a).mean(1, keepdim=True))
    dp = ALPHA * g * grad
    b = st["w_post"] * dp
    dy = st["rstd_y"][:, None] * (b - yh * (yh * b).mean(1, keepdim=True))
    o = {"dr": (BETA * grad).to(st["dr_out"].dtype), "dy": dy.to(torch.bfloat16),
         "dw_post": (dp * yh).sum(0), "dw_pre": (dn * th).sum(0)}
    if c["gate"] != "none":
        dg = ALPHA * yh * st["w_post"] * grad
        o["dgate"] = {"channel": lambda: dg.sum(0), "token": lambda: dg.sum(1, keepdim=True),
                      "full": lambda: dg.to(torch.bfloat16)}[c["gate"]]()
    return o


def _plain_swiglu_fwd(st):
    f = st["case"]["f"]
    g, u = st["gu"][:, :f].float(), st["gu"][:, f:].float()
    h = g * torch.sigmoid(g) * u
    o = {}
    o["hq"], o["hs"] = _encode(h, st["case"]["pow2"])
    gq, gs = _encode(g, st["case"]["pow2"])
    uq, us = _encode(u, st["case"]["pow2"])
    o["guq"] = torch.cat([gq.view(torch.uint8), uq.view(torch.uint8)], 1).view(FP8)
    o["gus"] = torch.cat([gs, us], 0)
    return o


def _plain_swiglu_grads(st):
    f = st["case"]["f"]
    if st["case"].get("saved", "fp8") == "fp8":
        g, u = _decode_halves(*st["gu_saved"])
    else:
        g, u = st["gu_saved"][:, :f].float(), st["gu_saved"][:, f:].float()
    dh = st["dh"].float()
    sig = torch.sigmoid(g)
    return dh * u * sig * (1 + g * (1 - sig)), dh * g * sig, g * sig * u


def _plain(st):
    op = st["case"]["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(st)
    if op == "norm_bwd":
        return _plain_norm_bwd(st)
    if op == "swiglu_fwd":
        return _plain_swiglu_fwd(st)
    if op == "swiglu_bwd":
        dg, du, _ = _plain_swiglu_grads(st)
        return {"dgu": torch.cat([dg, du], 1).to(torch.bfloat16)}
    if op == "swiglu_bwd_fp8":
        dg, du, h = _plain_swiglu_grads(st)
        dgu, p = torch.cat([dg, du], 1), st["case"]["pow2"]
        o = {}
        o["dguq"], o["dgus"] = _encode(dgu, p)
        o["dgutq"], o["dguts"] = _encode(dgu.t().contiguous(), p)
        o["htq"], o["hts"] = _encode(h.t().contiguous(), p)
        return o
    if op == "pack":
        q, s = _encode(st["x"].float(), st["case"]["pow2"])
        return {"q": q, "s": s}
    if op == "unpack":
        x = _decode(*st["saved"])
        return {"x": x.to(torch.bfloat16) if st["case"]["dtype"] == "bf16" else x}
    q, s = _encode(_decode(*st["saved"]).t().contiguous(), st["case"]["pow2"])
    return {"qt": q, "st": s}


# ------------------------------------------------------------------ the package's entry points
def _own(st):
    from blockwise_fp8_gemm_x128_amd import binding as puro
    c = st["case"]
    op, out = c["op"], st["out"]
    if op == "norm_fwd":
        o = puro.puro_block_norm_fwd(st["y"], st["r"], st["w_post"], st["w_pre"], st["gate"],
                                     alpha=ALPHA, beta=BETA, eps=EPS, pow2=c["pow2"], out=out)
        r_out, n, nq, ns, rstd_y, rstd_r, yq, ys, rq, rs = o
        d = {"r_out": r_out, "rstd_y": rstd_y, "rstd_r": rstd_r}
        if c["n"] == "fp8":
            d["nq"], d["ns"] = nq.view(FP8), ns
        else:
            d["n"] = n
        if c["ckpt"]:
            d["yq"], d["ys"], d["rq"], d["rs"] = yq.view(FP8), ys, rq.view(FP8), rs
        return d
    if op == "norm_bwd":
        o = puro.puro_block_norm_bwd(st["dr_out"], st["dn"], st["y_saved"], st["r_saved"],
                                     st["rstd_y"], st["rstd_r"], st["w_post"], st["w_pre"],
                                     st["gate"], alpha=ALPHA, beta=BETA, out=out)
        d = {"dr": o[0], "dy": o[1], "dw_post": o[2], "dw_pre": o[3]}
        if c["gate"] != "none":
            d["dgate"] = o[4]
        return d
    if op == "swiglu_fwd":
        _, hq, hs, guq, gus = puro.puro_swiglu_fwd(st["gu"], pow2=c["pow2"], out=out)
        return {"hq": hq.view(FP8), "hs": hs, "guq": guq.view(FP8), "gus": gus}
    if op == "swiglu_bwd":
        return {"dgu": puro.puro_swiglu_bwd(st["dh"], st["gu_saved"], dgu=out)}
    if op == "swiglu_bwd_fp8":
        o = puro.puro_swiglu_bwd_fp8(st["dh"], st["gu_saved"], pow2=c["pow2"], out=out)
        return {"dguq": o[0].view(FP8), "dgus": o[1], "dgutq": o[2].view(FP8), "dguts": o[3],
                "htq": o[4].view(FP8), "hts": o[5]}
    if op == "pack":
        q, s = puro.puro_ckpt_pack(st["x"], *out, pow2=c["pow2"])
        return {"q": q.view(FP8), "s": s}
    if op == "unpack":
        return {"x": puro.puro_ckpt_unpack(*st["saved"], x=out)}
    qt, s = puro.puro_ckpt_transpose(*st["saved"], *out, pow2=c["pow2"])
    return {"qt": qt.view(FP8), "st": s}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ inputs
def _acts(gen, rows, cols, std=1.0):
    """Activations: Gaussian, one channel in a hundred 20 times larger, one row in 64 (padding)
    zero."""
    x = torch.randn((rows, cols), generator=gen, device=DEV) * std
    big = torch.rand((cols,), generator=gen, device=DEV) < 0.01
    x = torch.where(big, 20.0 * x, x)
    if rows > 1:
        x[torch.rand((rows,), generator=gen, device=DEV) < 1 / 64] = 0.0
    return x


def _empty(shape, dtype):
    return torch.empty(shape, dtype=dtype, device=DEV)


def _codes(rows, cols):
    return _empty((rows, cols), torch.uint8), _empty((_chunks(cols), rows), torch.float32)


def _saved(x):
    q, s = _encode(x, False)
    return q.view(torch.uint8), s


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    op, rows, st = c["op"], c["rows"], {"case": c}
    bf16 = torch.bfloat16
    if op in ("norm_fwd", "norm_bwd"):
        cols = c["cols"]
        res = bf16 if c["res"] == "bf16" else torch.float32
        y, r = _acts(gen, rows, cols), _acts(gen, rows, cols, 4.0)
        st["w_post"] = 1 + 0.1 * torch.randn((cols,), generator=gen, device=DEV)
        st["w_pre"] = 1 + 0.1 * torch.randn((cols,), generator=gen, device=DEV)
        st["gate"] = {
            "none": lambda: None,
            "channel": lambda: 0.5 + 0.1 * torch.randn((cols,), generator=gen, device=DEV),
            "token": lambda: torch.sigmoid(torch.randn((rows, 1), generator=gen, device=DEV)),
            "full": lambda: torch.sigmoid(torch.randn((rows, cols), generator=gen,
                                                      device=DEV)).to(bf16)}[c["gate"]]()
        if op == "norm_fwd":
            st["y"], st["r"] = y.to(bf16), r.to(res)
            none2 = (None, None)
            st["out"] = (_empty((rows, cols), res),
                         _empty((rows, cols), bf16) if c["n"] == "bf16" else None,
                         *(_codes(rows, cols) if c["n"] == "fp8" else none2),
                         _empty((rows,), torch.float32), _empty((rows,), torch.float32),
                         *(_codes(rows, cols) if c["ckpt"] else none2),
                         *(_codes(rows, cols) if c["ckpt"] else none2))
            return st
        st["rstd_y"] = torch.rsqrt((y * y).mean(1) + EPS)
        st["rstd_r"] = torch.rsqrt((r * r).mean(1) + EPS)
        if c["saved"] == "fp8":
            st["y_saved"], st["r_saved"] = _saved(y), _saved(r)
        else:
            st["y_saved"], st["r_saved"] = y.to(bf16), r.to(res)
        st["dn"] = _acts(gen, rows, cols, 1e-3).to(bf16)
        st["dr_out"] = _acts(gen, rows, cols, 1e-3).to(res)
        dgate = {"none": lambda: None, "channel": lambda: _empty((cols,), torch.float32),
                 "token": lambda: _empty((rows, 1), torch.float32),
                 "full": lambda: _empty((rows, cols), bf16)}[c["gate"]]()
        st["out"] = (_empty((rows, cols), res), _empty((rows, cols), bf16),
                     _empty((cols,), torch.float32), _empty((cols,), torch.float32), dgate)
        return st
    if op.startswith("swiglu"):
        f = c["f"]
        gu = _acts(gen, rows, 2 * f)
        if op == "swiglu_fwd":
            st["gu"] = gu.to(bf16)
            guq, gus = _empty((rows, 2 * f), torch.uint8), _empty((2 * _chunks(f), rows),
                                                                   torch.float32)
            st["out"] = (None, *_codes(rows, f), guq, gus)
            return st
        if c.get("saved", "fp8") == "fp8":
            gq, gs = _saved(gu[:, :f].to(bf16).float())
            uq, us = _saved(gu[:, f:].to(bf16).float())
            st["gu_saved"] = (torch.cat([gq, uq], 1), torch.cat([gs, us], 0))
        else:
            st["gu_saved"] = gu.to(bf16)
        st["dh"] = _acts(gen, rows, f, 1e-3).to(bf16)
        if op == "swiglu_bwd":
            st["out"] = _empty((rows, 2 * f), bf16)
        else:
            st["out"] = (*_codes(rows, 2 * f), *_codes(2 * f, rows), *_codes(f, rows))
        return st
    cols = c["cols"]
    x = _acts(gen, rows, cols)
    if op == "pack":
        dt = bf16 if c["dtype"] == "bf16" else torch.float32
        wide = torch.zeros((rows, cols + c["pad"]), dtype=dt, device=DEV)
        wide[:, :cols] = x.to(dt)
        st["x"], st["out"] = wide[:, :cols], _codes(rows, cols)
        return st
    st["saved"] = _saved(x.to(bf16).float())
    if op == "unpack":
        st["out"] = _empty((rows, cols), bf16 if c["dtype"] == "bf16" else torch.float32)
    else:
        st["out"] = _codes(cols, rows)
    return st


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_codes(x, pow2):
    """Unrounded scaled values (what a code stands for before its rounding) and scales of float64
    [rows, cols], group by group along the columns."""
    rows, cols = x.shape
    k = -(-cols // G)
    scales = torch.empty((k, rows), dtype=torch.float64, device=x.device)
    vals = torch.empty_like(x)
    for j in range(k):
        part = x[:, j * G:(j + 1) * G]
        top = part.abs().max(1).values
        a = torch.where(top < 2.0 ** -119, torch.full_like(top, 2.0 ** -119), top)
        s = a / 448
        if pow2:
            m, e = torch.frexp(s)               # the power of two at or above s
            s = torch.where(m == 0.5, s, s / m)
        s = torch.where(top == 0, torch.ones_like(s), s)
        vals[:, j * G:(j + 1) * G] = part / s[:, None]
        scales[j] = s
    return vals, scales


def _exact_value(q, s):
    x = q.view(FP8).to(torch.float64)
    for j in range(s.shape[0]):
        x[:, j * G:(j + 1) * G] *= s[j].double()[:, None]
    return x


def _exact_pair(saved, f):
    if isinstance(saved, tuple):
        k = saved[1].shape[0] // 2
        return (_exact_value(saved[0][:, :f].contiguous(), saved[1][:k]),
                _exact_value(saved[0][:, f:].contiguous(), saved[1][k:]))
    return saved[:, :f].double(), saved[:, f:].double()


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    op, rows = c["op"], c["rows"]
    o = {}
    if op in ("norm_fwd", "norm_bwd"):
        wp, wn = st["w_post"].double(), st["w_pre"].double()
        gate = torch.ones((1, 1), dtype=torch.float64, device=DEV)
        if st["gate"] is not None:
            gate = st["gate"].double()
    if op == "norm_fwd":
        y, r = st["y"].double(), st["r"].double()
        iy = (y.square().sum(1) / c["cols"] + EPS) ** -0.5
        t = r * BETA + (gate * ALPHA) * (y * iy[:, None] * wp)
        it = (t.square().sum(1) / c["cols"] + EPS) ** -0.5
        n = t * it[:, None] * wn
        o = {"r_out": t, "rstd_y": iy, "rstd_r": it}
        if c["n"] == "fp8":
            o["nq"], o["ns"] = _exact_codes(n, c["pow2"])
        else:
            o["n"] = n
        if c["ckpt"]:
            o["yq"], o["ys"] = _exact_codes(y, c["pow2"])
            o["rq"], o["rs"] = _exact_codes(t, c["pow2"])
    elif op == "norm_bwd":
        if c["saved"] == "fp8":
            y, t = _exact_value(*st["y_saved"]), _exact_value(*st["r_saved"])
        else:
            y, t = st["y_saved"].double(), st["r_saved"].double()
        iy, it = st["rstd_y"].double()[:, None], st["rstd_r"].double()[:, None]
        dn, d = st["dn"].double(), c["cols"]
        # the gradient of t * it with it depending on t, then back through the gate to y
        total = st["dr_out"].double() + it * wn * dn - it ** 3 * t * (t * wn * dn).sum(
            1, keepdim=True) / d
        dp = total * gate * ALPHA
        dy = iy * wp * dp - iy ** 3 * y * (y * wp * dp).sum(1, keepdim=True) / d
        o = {"dr": BETA * total, "dy": dy, "dw_post": (dp * y * iy).sum(0),
             "dw_pre": (dn * t * it).sum(0)}
        if c["gate"] != "none":
            dg = ALPHA * total * y * iy * wp
            o["dgate"] = (dg if c["gate"] == "full" else
                          dg.sum(0) if c["gate"] == "channel" else
                          dg.sum(1, keepdim=True))
    elif op == "swiglu_fwd":
        f = c["f"]
        g, u = st["gu"][:, :f].double(), st["gu"][:, f:].double()
        o["hq"], o["hs"] = _exact_codes(u * g / (1 + torch.exp(-g)), c["pow2"])
        a, b = _exact_codes(g, c["pow2"]), _exact_codes(u, c["pow2"])
        o["guq"], o["gus"] = torch.cat([a[0], b[0]], 1), torch.cat([a[1], b[1]], 0)
    elif op.startswith("swiglu"):
        g, u = _exact_pair(st["gu_saved"], c["f"])
        dh = st["dh"].double()
        e = torch.exp(-g)
        dg, du = dh * u * (1 + e + g * e) / (1 + e) ** 2, dh * g / (1 + e)
        dgu = torch.cat([dg, du], 1)
        if op == "swiglu_bwd":
            return {"dgu": dgu}
        o["dguq"], o["dgus"] = _exact_codes(dgu, c["pow2"])
        o["dgutq"], o["dguts"] = _exact_codes(dgu.t().contiguous(), c["pow2"])
        o["htq"], o["hts"] = _exact_codes((u * g / (1 + e)).t().contiguous(), c["pow2"])
    elif op == "pack":
        o["q"], o["s"] = _exact_codes(st["x"].double(), c["pow2"])
    elif op == "unpack":
        o["x"] = _exact_value(*st["saved"])
    else:
        o["qt"], o["st"] = _exact_codes(_exact_value(*st["saved"]).t().contiguous(), c["pow2"])
    return o
