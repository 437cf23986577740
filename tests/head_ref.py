"""The output head's cross entropy and the orthogonalised direction in 64 bits, with the bounds that
the kernels' roundings allow, written from the definitions.

Cross entropy. Products of two bf16 values are exact in fp32, so a logit's error is that of a sum of
d terms: at most d steps of 2^-23 (a step per addition, whichever way the adder rounds) of the sum of
magnitudes, e_l. lse inherits the largest e_l of its row, a relative error of the sum of exponentials
(at most 2^9 additions and roundings of 2^-24 on any path through tile, join and logarithm: 2^-15),
and three roundings of values of the size of lse or the logits. Backward, P has the relative error of
its exponential (e_l, and roundings of its argument and factors) and half a step of bf16, 2^-8; the
gradients take those through their sums, add their own summation, and half a step of bf16 if
rounded.

Orthogonalisation. The bound is not elementary: `ortho_rounded` runs the steps with every operand
rounded to fp16 where the kernels round it (sums exact), and the kernels have to lie within twice that
run's distance from the exact steps (their sums round too, far below fp16), plus u's rounding: the
larger distance of its two orders of the steps. (Short sides are held to the same, though their
operands are two halves wide.)"""
import numpy as np
import torch

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def xent_fwd(h, w, targets):
    """(loss, lse, bound of loss, bound of lse), float64."""
    h, w = h.double(), w.double()
    v = w.shape[0]
    has = (targets >= 0) & (targets < v)
    l = h @ w.t()
    e = h.shape[1] * 2.0 ** -23 * (h.abs() @ w.abs().t())
    top = l.max(1, keepdim=True).values
    lse = (top + (l - top).exp().sum(1, keepdim=True).log())[:, 0]
    at = l.gather(1, targets.clamp(0, v - 1)[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    size = lse.abs() + l.abs().max(1).values + 1
    b = e.max(1).values + 2.0 ** -15 + 2.0 ** -21 * size
    return (torch.where(has, lse - at, zero), torch.where(has, lse, zero),
            torch.where(has, 2 * b, zero), torch.where(has, b, zero))


def xent_bwd(h, w, targets, lse, dloss, dlse, dw_before=None):
    """(dh, dw, bound of dh in bf16, bound of dw in fp32), float64; bf16's rounding of dw is not in
    its bound. Rows of h without a target do not enter."""
    v = w.shape[0]
    has = (targets >= 0) & (targets < v)
    h = torch.where(has[:, None], h.double(), torch.zeros((), dtype=torch.float64, device=h.device))
    w = w.double()
    l = h @ w.t()
    e = (h.shape[1] * 2.0 ** -23 * (h.abs() @ w.abs().t())
         + 2.0 ** -21 * (l.abs() + lse.double().abs()[:, None] + 1))
    lse = torch.where(has, lse.double(), torch.zeros_like(lse, dtype=torch.float64))
    hot = torch.where(has, dloss.double(), torch.zeros_like(lse))
    every = hot if dlse is None else hot + torch.where(has, dlse.double(), torch.zeros_like(lse))
    soft = (l - lse[:, None]).exp() * every[:, None]
    soft = torch.where(has[:, None], soft, torch.zeros_like(soft))
    p = soft.clone()
    rows = torch.arange(len(h), device=h.device)
    p[rows, targets.clamp(0, v - 1)] -= hot
    dp = soft.abs() * torch.expm1(e) + 2.0 ** -8 * p.abs()
    dp[rows, targets.clamp(0, v - 1)] += 2.0 ** -8 * (soft * torch.expm1(e)).abs()[
        rows, targets.clamp(0, v - 1)] + 2.0 ** -23 * hot.abs()
    dh, dw = p @ w, p.t() @ h
    bh = dp @ w.abs() + v * 2.0 ** -23 * (p.abs() @ w.abs())
    bw = dp.t() @ h.abs() + (len(h) + 1) * 2.0 ** -23 * (p.abs().t() @ h.abs())
    if dw_before is not None:
        dw = dw + dw_before.double()
        bw = bw + 2.0 ** -23 * dw.abs()
    return dh, dw, bh + 2.0 ** -8 * (dh.abs() + bh), bw


def momentum(g, m, beta, nesterov):
    """(new momentum or None, v) in float64 of the fp32 beta and 1 - beta."""
    g = g.double()
    if m is None:
        return None, g
    b = float(np.float32(beta))
    rest = float(np.float32(1.0) - np.float32(beta))
    m = b * m.double() + rest * g
    return m, (b * m + rest * g if nesterov else m)


def ortho(v, steps=5, coefficients=COEFFICIENTS):
    """The steps on one float64 matrix."""
    a, b, c = (float(np.float32(k)) for k in coefficients)
    tall = v.shape[0] > v.shape[1]
    x = v.t() if tall else v
    norm = torch.linalg.matrix_norm(x)
    x = x / norm if norm > 0 else x
    for _ in range(steps):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.t() if tall else x


def ortho_rounded(v, steps=5, coefficients=COEFFICIENTS, grouped=False):
    """The same with every operand in fp16 where the kernels hold it so (sums exact): step by step with
    X in two halves until the last two steps, or by matrices of three steps (X in two halves), then two."""
    a, b, c = (float(np.float32(k)) for k in coefficients)
    tall = v.shape[0] > v.shape[1]
    x = v.t() if tall else v
    norm = torch.linalg.matrix_norm(x)
    x = x / norm if norm > 0 else x

    def half(t, scale):
        return (t * scale).half().double() / scale

    eye = torch.eye(x.shape[0], dtype=x.dtype, device=x.device)
    done = 0
    while done < steps:
        g = 1 if not grouped else 3 if done == 0 else min(2, steps - done)
        both = done == 0 if grouped else steps - done > 2
        hi = half(x, 4096.0)
        lo = half(x - hi, 4096.0 * 2048.0)
        gram = half(hi @ hi.t(), 16384.0)
        poly = b * gram + c * (gram @ gram)
        q, rest = poly, a
        for k in range(1, g):
            poly = half(poly, 2048.0)
            if k > 1:
                q, rest = a * q + rest * poly + poly @ q, rest * a
            q = half(q, 2048.0 if k == 1 else 512.0)
            t = half(a * gram + poly @ gram, 16384.0)
            gram = half(a * t + t @ poly, 16384.0)
            poly = b * gram + c * (gram @ gram)
        if g > 1:
            poly = half(poly, 2048.0)
            q, rest = a * q + rest * poly + poly @ q, rest * a
        scale = 2048.0 if g == 1 else 512.0 if both else 1024.0
        x = rest * (hi + lo) + half(q, scale) @ hi if both else half(rest * eye + q, scale) @ hi
        done += g
    return x.t() if tall else x
