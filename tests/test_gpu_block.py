"""GPU tests of the operators between the GEMMs against their plain 64-bit forms (block_ref.py,
where the tolerances are derived): the block norm forward and backward, the gated activation, and
8-bit checkpoints, whose bytes are checked exactly wherever their input is exact."""
import sys

import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
EPS = 1e-6


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def rnd(shape, seed, std=1.0, dtype=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


def acts(rows, cols, seed, dtype=BF16, std=1.0):
    """Activations with a zero row, a zero group and a large channel where there is room."""
    x = rnd((rows, cols), seed, std).cpu()
    if cols > 3:
        x[:, cols // 3] *= 30.0
    if rows > 2:
        x[rows // 2] = 0.0
        x[0, :128] = 0.0
    return x.to(dtype).to(DEV)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8).cpu(), b.contiguous().view(torch.uint8).cpu())


def gate_of(kind, rows, cols, seed):
    return {"none": lambda: None, "channel": lambda: rnd((cols,), seed, 0.5),
            "token": lambda: rnd((rows, 1), seed, 0.5),
            "full": lambda: rnd((rows, cols), seed, 0.5, BF16)}[kind]()


AXES = {"none": None, "channel": 0, "token": 1, "full": ()}
SIZES = [(1, 1), (1, 2048), (3, 7), (37, 100), (5, 128), (130, 129), (33, 256), (9, 500),
         (17, 1000), (70, 2051), (261, 2048), (6, 5120), (4, 8191), (3, 8200), (2, 16384)]
# rows of three to fourteen groups of columns and of many waves, several to a block, and blocks of
# unequal length
GROUPED = [(5, 300), (9001, 384), (2500, 600), (3777, 768), (1700, 896), (2311, 1152), (1, 1200),
           (1303, 1280), (1111, 1600), (1040, 1792), (600, 7100)]


# ------------------------------------------------------------------ 8-bit checkpoints
@pytest.mark.parametrize("rows,cols", SIZES + [(1, 12288), (300, 384)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pow2", [False, True])
def test_pack_unpack_transpose(puro, rows, cols, dtype, pow2):
    say("ckpt", rows, cols, dtype, pow2)
    x = acts(rows, cols, rows + cols, dtype)
    q, s = puro.puro_ckpt_pack(x, pow2=pow2)
    rq, rs = ref.encode(x, pow2)
    assert same(q, rq) and same(s, rs)
    val = ref.decode32(rq, rs)
    assert same(puro.puro_ckpt_unpack(q, s, dtype=F32), val)
    assert same(puro.puro_ckpt_unpack(q, s), val.to(BF16))
    qt, st = puro.puro_ckpt_transpose(q, s, pow2=pow2)
    tq, ts = ref.encode(val.t().contiguous(), pow2)
    assert same(qt, tq) and same(st, ts)


@pytest.mark.parametrize("pow2", [False, True])
def test_pack_is_the_quantiser_on_whole_groups(puro, pow2):
    x = acts(256, 384, 5)
    sfx = "_pow2" if pow2 else ""
    q, s = getattr(puro, "puro_quant_act_1x128" + sfx)(x)
    cq, cs = puro.puro_ckpt_pack(x, pow2=pow2)
    assert same(q, cq) and same(s, cs)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pow2", [False, True])
def test_special_values(puro, dtype, pow2):
    """Infinities and NaN of either sign, zero groups, groups below the least scale, -0."""
    x = rnd((40, 300), 11).cpu()
    x[0, 3], x[0, 4], x[1, 200], x[2, 290] = float("inf"), -float("inf"), float("nan"), -0.0
    x[3] = float("nan")
    x[4] = 0.0
    x[5] = 2.0 ** -125
    x[6, :] = -0.0
    x[7, 256:] = -float("inf")
    x = x.to(dtype).to(DEV)
    q, s = puro.puro_ckpt_pack(x, pow2=pow2)
    rq, rs = ref.encode(x, pow2)
    nan = torch.isnan(x).cpu()
    assert same(s, rs)
    assert torch.equal(q.cpu()[~nan], rq[~nan])
    assert torch.equal(q.cpu()[nan] & 0x7F, rq[nan] & 0x7F)    # a NaN's sign has no meaning
    qt, st = puro.puro_ckpt_transpose(q, s, pow2=pow2)
    tq, ts = ref.encode(ref.decode32(q, s).t().contiguous(), pow2)
    assert same(st, ts)
    m = (tq & 0x7F) == 0x7F
    assert torch.equal(qt.cpu()[~m], tq[~m]) and torch.equal(qt.cpu()[m] & 0x7F, tq[m] & 0x7F)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pow2", [False, True])
def test_both_ends_of_the_range(puro, dtype, pow2):
    """Groups up to the largest finite values and down to subnormal ones, alone and mixed."""
    x = rnd((130, 260), 12).cpu()
    x[0] *= 2.0 ** 125
    x[1] = torch.finfo(dtype).max
    x[2, ::2], x[2, 1::2] = torch.finfo(dtype).max, 2.0 ** -130
    x[3] *= 2.0 ** -127
    x[4] = 2.0 ** -133
    x[5] *= 2.0 ** -119
    x[6, 7] = -torch.finfo(dtype).max
    x = x.to(dtype).to(DEV)
    q, s = puro.puro_ckpt_pack(x, pow2=pow2)
    rq, rs = ref.encode(x, pow2)
    assert same(s, rs) and same(q, rq)
    qt, st = puro.puro_ckpt_transpose(q, s, pow2=pow2)
    tq, ts = ref.encode(ref.decode32(q, s).t().contiguous(), pow2)
    assert same(st, ts)
    m = (tq & 0x7F) == 0x7F
    assert torch.equal(qt.cpu()[~m], tq[~m]) and torch.equal(qt.cpu()[m] & 0x7F, tq[m] & 0x7F)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("off", [0, 1, 3, 8])
def test_strided_rows(puro, dtype, off):
    """Rows inside a wider matrix at any element offset; what lies around them stays."""
    rows, cols = 70, 203
    wide = rnd((rows, 300), 21, dtype=dtype)
    x = wide[:, off:off + cols]
    q, s = puro.puro_ckpt_pack(x)
    rq, rs = ref.encode(x.contiguous())
    assert same(q, rq) and same(s, rs)
    before = wide.clone()
    puro.puro_ckpt_unpack(q, s, x=x)
    before[:, off:off + cols] = ref.decode32(rq, rs).to(dtype).to(DEV)
    assert same(wide, before)


def test_offsets_past_32_bits(puro):
    """2.2e9 elements: the last rows of pack, unpack and transpose as of a small matrix."""
    rows, cols = (1 << 20) + 5, 2100
    x = torch.empty((rows, cols), dtype=BF16, device=DEV)
    x.fill_(0.5)
    x[-300:] = acts(300, cols, 31)
    q, s = puro.puro_ckpt_pack(x)
    rq, rs = ref.encode(x[-300:])
    assert same(q[-300:], rq) and same(s[:, -300:], rs)
    assert torch.all(q[:-300] == 0x7E).item() and torch.all(s[:, :-300] == s[0, 0]).item()
    y = puro.puro_ckpt_unpack(q, s)
    assert same(y[-300:], ref.decode32(rq, rs).to(BF16))
    del x, y
    qt, st = puro.puro_ckpt_transpose(q, s)
    tail = rows % 128 + 128
    tq, ts = ref.encode(ref.decode32(q[-tail:], s[:, -tail:]).t().contiguous())
    assert same(qt[:, -tail:], tq) and same(st[-2:], ts)


# ------------------------------------------------------------------ block norm
def check_fwd(puro, rows, cols, res, kind, n, ckpt, pow2, half="both", inplace=False):
    say("norm fwd", rows, cols, res, kind, n, ckpt, pow2, half)
    y, r = acts(rows, cols, 1), acts(rows, cols, 2, res, 4.0)
    wo, wp = rnd((cols,), 3), rnd((cols,), 4)
    post, pre = half != "pre", half != "post"
    gate = gate_of(kind, rows, cols, 5) if post else None
    alpha, beta = 0.75, 0.9375
    r0 = r.clone()
    kw = dict(alpha=alpha, beta=beta, eps=EPS, n=n, ckpt=ckpt, pow2=pow2)
    args = (y if post else None, r, wo if post else None, wp if pre else None, gate)
    o = puro.puro_block_norm_fwd(*args, **kw)
    if inplace:
        o2 = puro.puro_block_norm_fwd(*args, **kw, out=o._replace(r_out=r))
        assert o2.r_out is r
        o = o2
    else:
        assert same(r, r0)
    v, e = ref.norm_fwd(ref.f64(y) if post else None, ref.f64(r0), ref.f64(wo),
                        ref.f64(wp) if pre else None, ref.gate64(gate), alpha, beta, EPS)
    ref.close(o.r_out, v["r_out"], e["r_out"] + ref.out_err(v["r_out"], res) * 1.01, "r_out")
    if post:
        ref.close(o.rstd_y, v["rstd_y"], e["rstd_y"], "rstd_y")
        if ckpt:
            yq, ys = ref.encode(y, pow2)
            assert same(o.yq, yq) and same(o.ys, ys)
    if pre:
        ref.close(o.rstd_r, v["rstd_r"], e["rstd_r"], "rstd_r")
        if n != "fp8":
            ref.close(o.n, v["n"], e["n"] + ref.bf16_err(v["n"]) * 1.01, "n")
        if n != "bf16":
            ref.check_codes(o.nq, o.ns, v["n"], e["n"], pow2, "n")
    if ckpt:
        ref.check_codes(o.rq, o.rs, v["r_out"], e["r_out"], pow2, "r")
    return o


@pytest.mark.parametrize("rows,cols", SIZES + GROUPED)
@pytest.mark.parametrize("res", [BF16, F32])
def test_norm_fwd_sizes(puro, rows, cols, res):
    check_fwd(puro, rows, cols, res, "channel", "both", True, False)


@pytest.mark.parametrize("kind", ["none", "token", "full"])
@pytest.mark.parametrize("rows,cols,res", [(19, 200, F32), (130, 2048, BF16), (7, 8195, BF16)])
def test_norm_fwd_gates(puro, kind, rows, cols, res):
    check_fwd(puro, rows, cols, res, kind, "fp8", False, True)


@pytest.mark.parametrize("half", ["post", "pre"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (50, 520), (1100, 2048), (6, 9000)])
def test_norm_fwd_halves(puro, half, rows, cols):
    check_fwd(puro, rows, cols, BF16, "channel", "both", True, False, half)


@pytest.mark.parametrize("rows,cols,res", [(21, 96, F32), (300, 2048, BF16), (5, 10000, F32)])
def test_norm_fwd_in_place(puro, rows, cols, res):
    check_fwd(puro, rows, cols, res, "full", "bf16", True, False, inplace=True)


def bwd_inputs(puro, rows, cols, res, kind, saved, half="both", seed=7):
    y, t = acts(rows, cols, seed), acts(rows, cols, seed + 1, res, 4.0)
    d = {"wo": rnd((cols,), seed + 2), "wp": rnd((cols,), seed + 3),
         "dn": acts(rows, cols, seed + 4, BF16, 1e-3), "dro": acts(rows, cols, seed + 5, res, 1e-3),
         "gate": gate_of(kind, rows, cols, seed + 6)}
    d["ry"] = torch.rsqrt(y.float().square().mean(1) + EPS)
    d["rr"] = torch.rsqrt(t.float().square().mean(1) + EPS)
    if saved == "fp8":
        d["y"], d["t"] = puro.puro_ckpt_pack(y), puro.puro_ckpt_pack(t)
        d["y64"], d["t64"] = (ref.f64(ref.decode32(*d[k])) for k in ("y", "t"))
    else:
        d["y"], d["t"] = y, t
        d["y64"], d["t64"] = ref.f64(y), ref.f64(t)
    if half == "pre":
        d["y"] = d["ry"] = d["wo"] = d["gate"] = d["y64"] = None
    if half == "post":
        d["t"] = d["rr"] = d["wp"] = d["dn"] = d["t64"] = None
    return d


def bwd_ref(d, kind, alpha, beta):
    n = lambda k: None if d[k] is None else ref.f64(d[k])  # noqa: E731
    return ref.norm_bwd(n("dro"), n("dn"), d["y64"], d["t64"], n("ry"), n("rr"), n("wo"), n("wp"),
                        ref.gate64(d["gate"]), alpha, beta,
                        AXES[kind] if d["gate"] is not None else None)


def bwd_call(puro, d, alpha, beta, **kw):
    return puro.puro_block_norm_bwd(d["dro"], d["dn"], d["y"], d["t"], d["ry"], d["rr"], d["wo"],
                                    d["wp"], d["gate"], alpha=alpha, beta=beta, **kw)


def check_bwd(o, v, e, res, kind):
    ref.close(o.dr, v["dr"], e["dr"] + ref.out_err(v["dr"], res) * 1.01, "dr")
    if "dy" in v:
        ref.close(o.dy, v["dy"], e["dy"] + ref.bf16_err(v["dy"]) * 1.01, "dy")
        ref.close(o.dw_post, v["dw_post"], e["dw_post"], "dw_post")
    if "dw_pre" in v:
        ref.close(o.dw_pre, v["dw_pre"], e["dw_pre"], "dw_pre")
    if "dgate" in v:
        extra = ref.bf16_err(v["dgate"]) * 1.01 if kind == "full" else 0.0
        ref.close(o.dgate, v["dgate"], e["dgate"] + extra, "dgate")


@pytest.mark.parametrize("rows,cols", SIZES + GROUPED + [(3000, 64), (2100, 2048)])
@pytest.mark.parametrize("res,saved", [(BF16, "fp8"), (F32, "asis")])
def test_norm_bwd_sizes(puro, rows, cols, res, saved):
    say("norm bwd", rows, cols, res, saved)
    d = bwd_inputs(puro, rows, cols, res, "channel", saved)
    v, e = bwd_ref(d, "channel", 0.75, 0.9375)
    check_bwd(bwd_call(puro, d, 0.75, 0.9375), v, e, res, "channel")


@pytest.mark.parametrize("kind", ["none", "token", "full"])
@pytest.mark.parametrize("rows,cols,res,saved", [(19, 200, F32, "fp8"), (700, 2048, BF16, "asis"),
                                                 (7, 8195, BF16, "fp8")])
def test_norm_bwd_gates(puro, kind, rows, cols, res, saved):
    say("norm bwd", rows, cols, res, saved, kind)
    d = bwd_inputs(puro, rows, cols, res, kind, saved)
    v, e = bwd_ref(d, kind, 0.75, 0.9375)
    check_bwd(bwd_call(puro, d, 0.75, 0.9375), v, e, res, kind)


@pytest.mark.parametrize("half", ["post", "pre"])
@pytest.mark.parametrize("rows,cols", [(1, 64), (50, 520), (1100, 2048), (300, 9000)])
def test_norm_bwd_halves(puro, half, rows, cols):
    d = bwd_inputs(puro, rows, cols, BF16, "channel", "fp8", half)
    v, e = bwd_ref(d, "channel", 1.5, 1.0)
    check_bwd(bwd_call(puro, d, 1.5, 1.0), v, e, BF16, "channel")


def test_norm_bwd_without_the_streams_gradient(puro):
    """dr_out absent counts as zero."""
    d = bwd_inputs(puro, 33, 640, F32, "channel", "asis")
    d["dro"] = None
    v, e = bwd_ref(d, "channel", 0.75, 0.9375)
    check_bwd(bwd_call(puro, d, 0.75, 0.9375), v, e, F32, "channel")


@pytest.mark.parametrize("rows,cols,res", [(21, 96, F32), (300, 2048, BF16), (5, 10000, F32)])
def test_norm_bwd_in_place_and_accumulate(puro, rows, cols, res):
    d = bwd_inputs(puro, rows, cols, res, "channel", "fp8")
    a = bwd_call(puro, d, 0.75, 0.9375)
    out = tuple(t.clone() for t in a)
    stream = d["dro"].clone()
    d["dro"] = stream
    b = bwd_call(puro, d, 0.75, 0.9375, accumulate=True, out=(stream, *out[1:]))
    assert same(b.dr, a.dr) and same(b.dy, a.dy)
    for x, y in ((b.dw_post, a.dw_post), (b.dw_pre, a.dw_pre), (b.dgate, a.dgate)):
        assert torch.equal(x, y + y)


def test_norm_empty(puro):
    """No rows: nothing to write, and gradients of zero rows are zero (or what was there)."""
    z = torch.empty((0, 256), dtype=BF16, device=DEV)
    w = torch.ones(256, device=DEV)
    none = torch.empty(0, device=DEV)
    o = puro.puro_block_norm_fwd(z, z, w, w, w)
    assert o.r_out.shape == (0, 256)
    g = puro.puro_block_norm_bwd(z, z, z, z, none, none, w, w, w)
    assert torch.all(g.dw_post == 0) and torch.all(g.dw_pre == 0) and torch.all(g.dgate == 0)
    g.dw_pre.fill_(3.0)
    g = puro.puro_block_norm_bwd(z, z, z, z, none, none, w, w, w, accumulate=True, out=g)
    assert torch.all(g.dw_pre == 3.0) and torch.all(g.dw_post == 0)
    e = torch.empty((5, 0), dtype=BF16, device=DEV)
    q, s = puro.puro_ckpt_pack(e)
    assert q.shape == (5, 0) and s.shape == (0, 5)
    assert puro.puro_swiglu_bwd(e, torch.empty((5, 0), dtype=BF16, device=DEV)).shape == (5, 0)


@pytest.mark.parametrize("kind", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("res,saved", [(BF16, "fp8"), (F32, "asis")])
def test_norm_bwd_wide_rows(puro, kind, res, saved):
    """More than 8192 columns, and several rows to a block."""
    rows, cols = 520, 8328
    say("norm bwd wide", kind, res, saved)
    d = bwd_inputs(puro, rows, cols, res, kind, saved)
    v, e = bwd_ref(d, kind, 0.75, 0.9375)
    check_bwd(bwd_call(puro, d, 0.75, 0.9375), v, e, res, kind)


@pytest.mark.parametrize("rows,cols", [(3, 256), (1, 100), (5, 5), (3, 600)])
def test_norm_bwd_infinite_gradient_in_the_last_row(puro, rows, cols):
    """An infinite element of dn in the last row makes its column of dw_pre infinite, with the sign
    of its normalised activation, not NaN, and no other column: lanes without a row of their own,
    which there are at these sizes, add nothing."""
    d = bwd_inputs(puro, rows, cols, F32, "none", "asis", half="pre")
    d["t"][-1] = rnd((cols,), 3).abs() + 0.5
    d["dn"][-1, 1] = float("inf")
    o = bwd_call(puro, d, 1.0, 1.0)
    assert o.dw_pre[1].item() == float("inf")
    assert torch.isfinite(o.dw_pre[torch.arange(cols, device=DEV) != 1]).all()


@pytest.mark.parametrize("value", [float("inf"), -float("inf")])
def test_norm_infinite_residual_stays_in_its_row(puro, value):
    """An infinity in the residual stream: its row's statistics fail, no other row changes, and the
    checkpoints keep their finite elements."""
    rows, cols = 9, 1000
    y, r = acts(rows, cols, 1), acts(rows, cols, 2, F32)
    w = rnd((cols,), 3)
    a = puro.puro_block_norm_fwd(y, r, w, w)
    r2 = r.clone()
    r2[3, 500] = value
    b = puro.puro_block_norm_fwd(y, r2, w, w)
    keep = [i for i in range(rows) if i != 3]
    for k in ("r_out", "nq", "yq", "rq", "rstd_y", "rstd_r"):
        assert same(getattr(a, k)[keep], getattr(b, k)[keep]), k
    assert same(a.yq, b.yq) and same(a.ys, b.ys)
    other = [i for i in range(cols) if i // 128 != 500 // 128]
    assert same(a.rq[3, other], b.rq[3, other]) and torch.isfinite(b.rs).all()
    assert (b.rq[3, 500].item() & 0x7F) == 0x7F


def test_norm_nonfinite_row_stays_in_its_row(puro):
    """A NaN in one row of y makes that row's outputs NaN and changes no other row."""
    rows, cols = 40, 2048
    y, r = acts(rows, cols, 1), acts(rows, cols, 2)
    w = rnd((cols,), 3)
    a = puro.puro_block_norm_fwd(y, r, w, w, n="both")
    y2 = y.clone()
    y2[7, 100] = float("nan")
    b = puro.puro_block_norm_fwd(y2, r, w, w, n="both")
    keep = [i for i in range(rows) if i != 7]
    for k in ("r_out", "n", "nq", "yq", "rq", "rstd_y", "rstd_r"):
        assert same(getattr(a, k)[keep], getattr(b, k)[keep]), k
    assert torch.isnan(b.n[7].float()).all() and torch.isnan(b.r_out[7].float()).all()
    assert torch.all((b.nq[7] & 0x7F) == 0x7F) and torch.all(b.ns[:, 7] == 1.0)
    assert torch.equal(b.yq[7, 101:], a.yq[7, 101:])     # y's checkpoint loses one element only


# ------------------------------------------------------------------ gated activation
SW_SIZES = [(1, 1), (1, 6144), (3, 100), (64, 128), (65, 129), (129, 1537), (200, 640)]


def gu_of(rows, f, seed=41):
    x = acts(rows, 2 * f, seed, F32, 2.0)
    x[rows - 1, 0] = 120.0
    x[0, f - 1] = -120.0
    return x.to(BF16)


@pytest.mark.parametrize("rows,f", SW_SIZES)
@pytest.mark.parametrize("pow2", [False, True])
def test_swiglu_fwd(puro, rows, f, pow2):
    say("swiglu fwd", rows, f, pow2)
    gu = gu_of(rows, f)
    o = puro.puro_swiglu_fwd(gu, h=True, pow2=pow2)
    h, e = ref.swiglu(ref.f64(gu[:, :f]), ref.f64(gu[:, f:]))
    ref.close(o.h, h, e + ref.bf16_err(h) * 1.01, "h")
    ref.check_codes(o.hq, o.hs, h, e, pow2, "h")
    gq, gs = ref.encode(gu[:, :f], pow2)
    uq, us = ref.encode(gu[:, f:], pow2)
    assert same(o.guq, torch.cat([gq, uq], 1)) and same(o.gus, torch.cat([gs, us], 0))
    only = puro.puro_swiglu_fwd(gu, h=True, fp8=False, ckpt=False)
    assert only.hq is None and only.guq is None and same(only.h, o.h)


def saved_gu(puro, gu, f, saved, pow2=False):
    if saved == "asis":
        return gu, ref.f64(gu[:, :f]), ref.f64(gu[:, f:])
    o = puro.puro_swiglu_fwd(gu, fp8=False, pow2=pow2)
    k = o.gus.shape[0] // 2
    return ((o.guq, o.gus), ref.f64(ref.decode32(o.guq[:, :f], o.gus[:k])),
            ref.f64(ref.decode32(o.guq[:, f:], o.gus[k:])))


@pytest.mark.parametrize("rows,f", SW_SIZES)
@pytest.mark.parametrize("saved", ["fp8", "asis"])
def test_swiglu_bwd(puro, rows, f, saved):
    say("swiglu bwd", rows, f, saved)
    gu, dh = gu_of(rows, f), acts(rows, f, 43, BF16, 1e-3)
    src, g, u = saved_gu(puro, gu, f, saved)
    dg, du, eg, eu = ref.swiglu_bwd(ref.f64(dh), g, u)
    want, err = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    ref.close(puro.puro_swiglu_bwd(dh, src), want, err + ref.bf16_err(want) * 1.01, "dgu")


@pytest.mark.parametrize("rows,f", [(128, 128), (256, 384), (128, 6144), (640, 256)])
@pytest.mark.parametrize("saved", ["fp8", "asis"])
@pytest.mark.parametrize("pow2", [False, True])
def test_swiglu_bwd_fp8(puro, rows, f, saved, pow2):
    say("swiglu bwd fp8", rows, f, saved, pow2)
    gu, dh = gu_of(rows, f), acts(rows, f, 43, BF16, 1e-3)
    src, g, u = saved_gu(puro, gu, f, saved, pow2)
    dg, du, eg, eu = ref.swiglu_bwd(ref.f64(dh), g, u)
    want, err = np.concatenate([dg, du], 1), np.concatenate([eg, eu], 1)
    o = puro.puro_swiglu_bwd_fp8(dh, src, pow2=pow2)
    ref.check_codes(o.dguq, o.dgus, want, err, pow2, "dgu")
    ref.check_codes(o.dgutq, o.dguts, want.T, err.T, pow2, "dgu transposed")
    h, e = ref.swiglu(g, u)
    ref.check_codes(o.htq, o.hts, h.T, e.T, pow2, "h transposed")


@pytest.mark.parametrize("rows,f", [(256, 256), (1664, 1024)])    # split by tensor, and whole
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_swiglu_bwd_fp8_nonfinite(puro, rows, f, value):
    """A NaN or infinite gradient element: NaN codes at its own places only, in both orientations,
    and scales that leave it out."""
    gu, dh = gu_of(rows, f), acts(rows, f, 43, BF16, 1e-3)
    gu[130, 9], gu[130, f + 9] = 0.75, -1.5      # du = dh silu(g) and dg = dh u silu'(g) both not 0
    a = puro.puro_swiglu_bwd_fp8(dh, gu)
    dh2 = dh.clone()
    dh2[130, 9] = value
    b = puro.puro_swiglu_bwd_fp8(dh2, gu)
    bad = torch.zeros((rows, 2 * f), dtype=torch.bool, device=DEV)
    bad[130, 9] = bad[130, f + 9] = True
    for x, m in ((b.dguq, bad), (b.dgutq, bad.t())):
        assert torch.all((x[m] & 0x7F) == 0x7F) and torch.all((x[~m] & 0x7F) != 0x7F)
    assert same(a.htq, b.htq) and same(a.hts, b.hts)
    keep = torch.ones(rows, dtype=torch.bool, device=DEV)
    keep[130] = False
    assert same(a.dguq[keep], b.dguq[keep])
    zero = dh.clone()           # the scales are those without the element
    zero[130, 9] = 0.0
    z = puro.puro_swiglu_bwd_fp8(zero, gu)
    assert same(b.dgus, z.dgus) and same(b.dguts, z.dguts)


# ------------------------------------------------------------------ large offsets
def test_rows_past_32_bits(puro):
    """2.2e9 elements a tensor: the last rows come out as those of a small matrix."""
    rows, cols, n = (1 << 20) + 5, 2100, 300

    def big(small):
        x = torch.empty((rows, cols), dtype=small.dtype, device=DEV)
        x.fill_(0.5)
        x[-n:] = small
        return x

    y, r, dn = acts(n, cols, 1), acts(n, cols, 2), acts(n, cols, 3, BF16, 1e-3)
    wo, wp = rnd((cols,), 4), rnd((cols,), 5)
    a = puro.puro_block_norm_fwd(y, r, wo, wp)
    b = puro.puro_block_norm_fwd(big(y), big(r), wo, wp)
    for k in ("r_out", "nq", "rstd_y", "rstd_r", "yq", "rq"):
        assert same(getattr(a, k), getattr(b, k)[-n:]), k
    for k in ("ns", "ys", "rs"):
        assert same(getattr(a, k), getattr(b, k)[:, -n:]), k
    ga = puro.puro_block_norm_bwd(r, dn, (a.yq, a.ys), (a.rq, a.rs), a.rstd_y, a.rstd_r, wo, wp)
    gb = puro.puro_block_norm_bwd(big(r), big(dn), (b.yq, b.ys), (b.rq, b.rs), b.rstd_y, b.rstd_r,
                                  wo, wp)
    assert same(ga.dr, gb.dr[-n:]) and same(ga.dy, gb.dy[-n:])
    del b, gb
    torch.cuda.empty_cache()
    gu, dh = y, dn[:, :cols // 2].contiguous()
    wide = torch.empty((rows, cols // 2), dtype=BF16, device=DEV)
    wide.fill_(0.5)
    wide[-n:] = dh
    ha, hb = puro.puro_swiglu_fwd(gu), puro.puro_swiglu_fwd(big(gu))
    assert same(ha.hq, hb.hq[-n:]) and same(ha.guq, hb.guq[-n:]) and same(ha.gus, hb.gus[:, -n:])
    assert same(puro.puro_swiglu_bwd(dh, (ha.guq, ha.gus)),
                puro.puro_swiglu_bwd(wide, (hb.guq, hb.gus))[-n:])


# ------------------------------------------------------------------ how they are called
def test_results_repeat(puro):
    d = bwd_inputs(puro, 1500, 2048, BF16, "channel", "fp8")
    a, b = bwd_call(puro, d, 1.0, 1.0), bwd_call(puro, d, 1.0, 1.0)
    for x, y in zip(a, b):
        assert same(x, y)


def test_native_calls_and_checked_calls_agree(puro, monkeypatch):
    """The binding's one-step native call and its way around it, argument by argument, make the same
    call: also taken for what the native one leaves alone (a list for a pair, 1 for True)."""
    rows, f, cols = 256, 384, 1024
    y, r, w = acts(rows, cols, 1), acts(rows, cols, 2, F32), rnd((cols,), 3)
    gu, dh = gu_of(rows, f), acts(rows, f, 43, BF16, 1e-3)
    d = bwd_inputs(puro, rows, cols, BF16, "token", "fp8")

    def calls(as_pair, flag):
        a = puro.puro_block_norm_fwd(y, r, w, w, rnd((rows, 1), 4), 0.5, 0.25, 1e-5, n="both",
                                     pow2=flag)
        h = puro.puro_swiglu_fwd(gu, h=True, pow2=flag)
        pair = as_pair((h.guq, h.gus))
        e = dict(d, y=as_pair(d["y"]), t=as_pair(d["t"]))
        g = bwd_call(puro, e, 0.75, 0.9375)
        g2 = bwd_call(puro, dict(e, dro=None), 0.75, 0.9375, accumulate=flag, out=g._replace(
            **{k: getattr(g, k).clone() for k in g._fields}))
        q, s = puro.puro_ckpt_pack(r[:, 5:900], pow2=flag)
        return (*a, *h, *g, *g2, puro.puro_swiglu_bwd(dh, pair),
                *puro.puro_swiglu_bwd_fp8(dh, pair, pow2=flag), q, s,
                puro.puro_ckpt_unpack(q, s, dtype=F32), *puro.puro_ckpt_transpose(q, s, pow2=flag))

    native = calls(tuple, True)
    made = []
    real = puro._call
    monkeypatch.setattr(puro, "_call", lambda name, *a: (made.append(name), real(name, *a))[1])
    assert len(native) == len(calls(tuple, True)) and not made
    checked = calls(list, 1)
    assert len(made) >= 8
    for a, b in zip(native, checked):
        assert same(a, b)


def test_other_stream_and_graph(puro):
    """The calls run on torch's current stream and can be captured; replays, with eager work
    between them, give the eager bytes."""
    rows, f, cols = 256, 512, 1024
    y, r = acts(rows, cols, 1), acts(rows, cols, 2)
    w = rnd((cols,), 3)
    gu, dh = gu_of(rows, f), acts(rows, f, 43, BF16, 1e-3)
    d = bwd_inputs(puro, rows, cols, BF16, "channel", "fp8")
    ws = puro.block_norm_workspace(rows, cols, DEV)

    def once(o=(None,) * 4):
        return (puro.puro_block_norm_fwd(y, r, w, w, w, out=o[0]),
                puro.puro_swiglu_fwd(gu, out=o[1]),
                puro.puro_swiglu_bwd_fp8(dh, gu, out=o[2]),
                bwd_call(puro, d, 1.0, 1.0, workspace=ws, out=o[3]))

    want = once()
    flat = lambda o: [t for part in o for t in part if t is not None]  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        got = once()
    torch.cuda.synchronize()
    assert all(same(a, b) for a, b in zip(flat(want), flat(got)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        once(got)
    for _ in range(3):
        for t in flat(got):
            t.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(flat(want), flat(got)))
        once()


def test_binding_refusals(puro):
    from blockwise_fp8_gemm_x128_amd import PuroError
    x, w = acts(8, 256, 1), rnd((256,), 2)
    rstd = torch.ones(8, device=DEV)
    q, s = puro.puro_ckpt_pack(x)
    bad = [
        lambda: puro.puro_ckpt_pack(x.half()),
        lambda: puro.puro_ckpt_pack(x.t()),
        lambda: puro.puro_ckpt_pack(x, q[:4]),
        lambda: puro.puro_ckpt_unpack(q, s[:1]),
        lambda: puro.puro_ckpt_unpack(q, s, dtype=torch.float16),
        lambda: puro.puro_ckpt_transpose(q, s, qt=q),
        lambda: puro.puro_block_norm_fwd(x.float(), x, w, w),
        lambda: puro.puro_block_norm_fwd(x, x, w[:128], w),
        lambda: puro.puro_block_norm_fwd(x, x, w, w.to(BF16)),
        lambda: puro.puro_block_norm_fwd(x, x, w, w, gate=w[:8]),
        lambda: puro.puro_block_norm_fwd(x, x, w, w, gate=x.float()),
        lambda: puro.puro_block_norm_fwd(x, x, w, w, eps=0.0),
        lambda: puro.puro_block_norm_fwd(x, x, w, w, n="fp4"),
        lambda: puro.puro_block_norm_fwd(x, x, None, None),
        lambda: puro.puro_block_norm_bwd(x, x, None, x, rstd, rstd, w, w),
        lambda: puro.puro_block_norm_bwd(x, x.float(), x, x, rstd, rstd, w, w),
        lambda: puro.puro_block_norm_bwd(x, x, (q, s[:1]), x, rstd, rstd, w, w),
        lambda: puro.puro_block_norm_bwd(x, x, x, x, rstd[:4], rstd, w, w),
        lambda: puro.puro_block_norm_bwd(x, x, x, x, rstd, rstd, w, w, accumulate=True),
        lambda: puro.puro_block_norm_bwd(x, x, x, x, rstd, rstd, w, w,
                                         workspace=torch.empty(8, dtype=torch.uint8, device=DEV)),
        lambda: puro.puro_swiglu_fwd(x[:, :255]),
        lambda: puro.puro_swiglu_fwd(x, fp8=False, ckpt=False),
        lambda: puro.puro_swiglu_bwd(x, x),
        lambda: puro.puro_swiglu_bwd_fp8(x[:, :128].contiguous(), x),   # 8 rows
    ]
    for i, call in enumerate(bad):
        with pytest.raises(PuroError):
            call()
            say("not refused:", i)
