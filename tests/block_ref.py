"""Plain 64-bit forms (numpy) of the operators between the GEMMs, with a bound on the fp32
kernels' error beside each result.

The bounds follow from the operations: u = 2^-24 is one fp32 rounding; a sum of D products over a
team runs through at most 16 terms in a lane, 6 lane steps and 16 waves, so with its products and
the reciprocal square root it is off by less than 64 u = 2^-18 of the sum of magnitudes (K below).
bf16 results carry 2^-8 of themselves on top (half a step of 2^-7, 8 significant bits, with the
values below 2^-126 rounded in steps of 2^-133), E4M3 codes 2^-4 of themselves or half the subnormal
step, 2^-10, times their scale."""
from __future__ import annotations

import numpy as np
import torch

K = 2.0 ** -18
BF16 = 2.0 ** -8
G = 128


def f64(t) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def bf16_err(x) -> np.ndarray:
    return BF16 * np.abs(x) + 2.0 ** -134


def out_err(x, dtype):
    return bf16_err(x) if dtype == torch.bfloat16 else 2.0 ** -24 * np.abs(x) + 2.0 ** -150


# ------------------------------------------------------------------ 8-bit groups, bit for bit
def groups(n):
    return -(-n // G)


def encode(x: torch.Tensor, pow2=False):
    """fp32 [rows, cols] (any values) -> (codes uint8, scales fp32 [groups, rows]) by the rule in
    fp32, each step one rounding; E4M3 rounding by torch's cast."""
    x = x.detach().cpu().float()
    rows, cols = x.shape
    q = torch.empty((rows, cols), dtype=torch.uint8)
    s = torch.empty((groups(cols), rows), dtype=torch.float32)
    for j in range(groups(cols)):
        part = x[:, j * G:(j + 1) * G]
        fin = torch.isfinite(part)
        amax = torch.where(fin, part.abs(), torch.zeros(())).amax(1)
        a = torch.clamp(amax, min=2.0 ** -119)
        if pow2:
            e = np.ceil(np.log2(a.double().numpy() / 448.0) - 1e-12)
            e = np.where(448.0 * 2.0 ** e < a.double().numpy(), e + 1, e)
            e = np.where(448.0 * 2.0 ** (e - 1) >= a.double().numpy(), e - 1, e)
            e = np.maximum(e, -127)
            sc = torch.from_numpy((2.0 ** e).astype(np.float32))
            r = torch.from_numpy((2.0 ** -e).astype(np.float32))
        else:
            sc, r = a / 448.0, torch.full_like(a, 448.0) / a  # (a scalar over a tensor rounds twice)
        one = torch.ones(())
        sc, r = torch.where(amax == 0, one, sc), torch.where(amax == 0, one, r)
        v = torch.clamp(torch.where(fin, part, torch.zeros(())) * r[:, None], -448.0, 448.0)
        c = v.to(torch.float8_e4m3fn).view(torch.uint8)
        sign = torch.signbit(part).to(torch.uint8) * 0x80
        # torch's cast drops no sign of zero, but the zero put in for a non-finite element has none
        c = torch.where(fin, torch.where(part == 0, sign, c), sign | 0x7F)
        q[:, j * G:(j + 1) * G] = c
        s[j] = sc
    return q, s


def decode32(q, s) -> torch.Tensor:
    """value(q) * s in fp32 (one rounding)."""
    q, s = q.detach().cpu(), s.detach().cpu()
    v = q.contiguous().view(torch.float8_e4m3fn).float()
    return v * s.t().repeat_interleave(G, 1)[:, :q.shape[1]]


def check_codes(q, s, ref, err, pow2, what):
    """Codes and scales of computed values against their 64-bit reference with error bound err:
    the scale follows the group's largest magnitude, and every decoded value is within half an
    E4M3 step."""
    q, s = q.cpu(), s.cpu().double().numpy()
    rows, cols = ref.shape
    val = q.contiguous().view(torch.float8_e4m3fn).double().numpy()
    assert s.shape == (groups(cols), rows), what
    for j in range(groups(cols)):
        sl = slice(j * G, (j + 1) * G)
        amax, slack = np.abs(ref[:, sl]).max(1), err[:, sl].max(1)
        sj = s[j]
        zero = (amax <= slack) & (sj == 1.0)
        if pow2:
            m, _ = np.frexp(sj)
            ok = (m == 0.5) & ((448 * sj * (1 + 2.0 ** -22) + slack >= amax)) & (
                (224 * sj * (1 - 2.0 ** -22) - slack < amax) | (sj <= 2.0 ** -126))
        else:
            ok = np.abs(448 * sj - amax) <= slack + 2.0 ** -22 * amax + 2.0 ** -119
        assert np.all(ok | zero), (what, "scale", j, sj[~(ok | zero)][:4], amax[~(ok | zero)][:4])
        d = np.abs(val[:, sl] * sj[:, None] - ref[:, sl])
        lim = (2.0 ** -4 * np.abs(ref[:, sl]) + 2.0 ** -10 * sj[:, None]) * (1 + 2.0 ** -18) \
            + 1.0625 * err[:, sl]
        assert np.all(d <= lim), (what, "codes", j, float((d - lim).max()))


def close(got, ref, err, what):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    d = np.abs(got - ref)
    assert np.all(d <= err), (what, float(np.nanmax(d / np.maximum(err, 1e-300))),
                              int((~(d <= err)).sum()))


# ------------------------------------------------------------------ block norm
def gate64(gate):
    return np.ones((1, 1)) if gate is None else f64(gate)


def norm_fwd(y, r, w_post, w_pre, gate, alpha, beta, eps):
    """All arguments float64 arrays (y/w_post or w_pre None). Returns ({name: value}, {name: error
    bound}) without the output roundings."""
    v, e = {}, {}
    t, et = beta * r, 2.0 ** -24 * np.abs(beta * r)
    if y is not None:
        v["rstd_y"] = 1.0 / np.sqrt((y * y).mean(1) + eps)
        e["rstd_y"] = K * v["rstd_y"]
        p = alpha * gate * y * v["rstd_y"][:, None] * w_post
        t = t + p
        et = K * (np.abs(beta * r) + np.abs(p)) * 1.25
    v["r_out"], e["r_out"] = t, et
    if w_pre is not None:
        rr = 1.0 / np.sqrt((t * t).mean(1) + eps)
        err_rr = rr * (rr * rr * (np.abs(t) * et).mean(1) + K)
        v["rstd_r"], e["rstd_r"] = rr, err_rr
        v["n"] = t * rr[:, None] * w_pre
        e["n"] = np.abs(w_pre) * (rr[:, None] * et + np.abs(t) * err_rr[:, None]) * 1.01 \
            + 2.0 ** -22 * np.abs(v["n"])
    return v, e


def norm_bwd(dr_out, dn, y, t, ry, rr, w_post, w_pre, gate, alpha, beta, axes):
    """Gradients, float64, from the stored activations; `axes`: the axes dgate is summed over
    (None: no gate). Returns (values, bounds)."""
    v, e = {}, {}
    shape = (dr_out if dr_out is not None else dn).shape
    D = shape[1]
    d = np.zeros(shape) if dr_out is None else dr_out
    G_, eG = d, np.zeros(shape)
    rh, m1 = np.zeros(shape), np.zeros((shape[0], 1))
    magA = np.abs(d)
    if dn is not None:
        rh = t * rr[:, None]
        x = w_pre * dn
        k1 = rr[:, None] * (rh * x).sum(1, keepdims=True) / D
        m1 = rr[:, None] * np.abs(rh * x).sum(1, keepdims=True) / D
        magA = magA + np.abs(rr[:, None] * x)
        G_ = d + rr[:, None] * x - rh * k1
        eG = K * (magA + np.abs(rh) * m1)
        v["dw_pre"] = (dn * rh).sum(0)
        e["dw_pre"] = K * np.abs(dn * rh).sum(0) + 2.0 ** -120
    v["dr"] = beta * G_
    e["dr"] = abs(beta) * eG + 2.0 ** -24 * np.abs(v["dr"])
    if y is not None:
        yh = y * ry[:, None]
        q = yh * w_post * gate
        dp = alpha * gate * G_
        qG = (q * G_).sum(1, keepdims=True)
        eQ = K * (np.abs(q) * magA).sum(1, keepdims=True) + 2 * K * m1 * np.abs(q * rh).sum(
            1, keepdims=True)
        v["dy"] = ry[:, None] * (w_post * dp - yh * alpha * qG / D)
        e["dy"] = np.abs(ry[:, None]) * (np.abs(w_post * alpha * gate) * eG
                                         + np.abs(yh * alpha) * eQ / D
                                         + K * (np.abs(w_post * dp) + np.abs(yh * alpha * qG) / D))
        v["dw_post"] = (dp * yh).sum(0)
        e["dw_post"] = (np.abs(alpha * gate * yh) * eG + 2 * K * np.abs(dp * yh)).sum(0) \
            + 2.0 ** -120
        if axes is not None:
            dg = alpha * w_post * yh * G_
            edg = np.abs(alpha * w_post * yh) * eG + 2 * K * np.abs(dg)
            if axes == 1:  # over columns: through the same three sums as dy
                p = alpha * yh * w_post
                edg = K * np.abs(p) * magA + 2 * K * m1 * np.abs(p * rh) + 2 * K * np.abs(dg)
            v["dgate"] = dg if axes == () else dg.sum(axes, keepdims=axes == 1)
            e["dgate"] = (edg if axes == () else edg.sum(axes, keepdims=axes == 1)) + 2.0 ** -120
    return v, e


# ------------------------------------------------------------------ gated activation
def swiglu(g, u):
    """h, float64, and its bound: the exponent's argument is off by |g| 2^-23, the exponential,
    the sum and the reciprocal by an ulp each."""
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-g))
    rel = (np.abs(g) + 4) * 2.0 ** -22
    h = g * sig * u
    return h, np.abs(h) * (rel + 2.0 ** -22) + np.abs(g * u) * 2.0 ** -120


def swiglu_bwd(dh, g, u):
    with np.errstate(over="ignore"):
        sig = 1.0 / (1.0 + np.exp(-g))
    rel = (np.abs(g) + 4) * 2.0 ** -22
    dg = dh * u * sig * (1 + g * (1 - sig))
    du = dh * g * sig
    tiny = 2.0 ** -120
    eg = np.abs(dh * u) * sig * ((1 + np.abs(g) * (1 - sig)) * (rel + 2.0 ** -21)
                                 + np.abs(g) * (sig * rel + 2.0 ** -23)) \
        + np.abs(dh * u) * (1 + np.abs(g)) * tiny
    eu = np.abs(du) * (rel + 2.0 ** -22) + np.abs(dh * g) * tiny
    return dg, du, eg, eu
