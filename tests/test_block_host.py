"""Host-side checks of the operators between the GEMMs (no GPU): their 64-bit reference forms
against differences and hand values, and the refusals of the C entry points. No call here reaches
a kernel launch."""
import ctypes
import os

import numpy as np
import pytest
import torch

import block_ref as ref

NULL, SHAPE, ALIGN, ARG = 1, 2, 3, 5
P, MIS = 0x10000, 0x10001  # never dereferenced: every call below fails validation first


@pytest.fixture(scope="module")
def L():
    from blockwise_fp8_gemm_x128_amd import _lib
    from blockwise_fp8_gemm_x128_amd.build import LIB_PATH, build
    if not os.path.exists(LIB_PATH):
        build(verbose=False)
    return _lib.lib()


# ------------------------------------------------------------------ the reference forms
def _directional(f, x, g, seed, h=1e-5):
    """(f(x + h v) - f(x - h v)) / 2h against <g, v> for a random direction v."""
    v = np.random.default_rng(seed).standard_normal(x.shape)
    num = (f(x + h * v) - f(x - h * v)) / (2 * h)
    return num, float((g * v).sum())


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 5), (7, 129)])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("half", ["both", "post", "pre"])
def test_norm_gradients_match_differences(rows, cols, gate, half):
    """Central differences of the 64-bit forward form. Step 1e-5 on values of order 1: a
    truncation error of order h^2 = 1e-10 and a rounding error of order 1e-16/1e-5 times the sum's
    terms, so 1e-6 of the gradient's scale is far above both."""
    rng = np.random.default_rng(rows * 1000 + cols)
    draw = lambda *s: rng.standard_normal(s)  # noqa: E731
    y, r, wo, wp = draw(rows, cols), draw(rows, cols), draw(cols), draw(cols)
    g = {"none": np.ones((1, 1)), "channel": draw(1, cols), "token": draw(rows, 1),
         "full": draw(rows, cols)}[gate]
    axes = {"none": None, "channel": 0, "token": 1, "full": ()}[gate]
    alpha, beta, eps = 0.7, 1.3, 1e-3
    a, b = draw(rows, cols), draw(rows, cols)  # the gradients of r_out and n
    post, pre = half != "pre", half != "post"
    if not post:
        y, g, axes = None, np.ones((1, 1)), None

    def loss(y=y, r=r, wo=wo, wp=wp, g=g):
        v, _ = ref.norm_fwd(y, r, wo, wp if pre else None, g, alpha, beta, eps)
        return (a * v["r_out"]).sum() + ((b * v["n"]).sum() if pre else 0.0)

    v, _ = ref.norm_fwd(y, r, wo, wp if pre else None, g, alpha, beta, eps)
    grads, _ = ref.norm_bwd(a, b if pre else None, y, v["r_out"], v.get("rstd_y"),
                            v.get("rstd_r"), wo, wp, g, alpha, beta, axes)
    args = [("dr", "r", r)]
    if post:
        args += [("dy", "y", y), ("dw_post", "wo", wo)]
        if axes is not None:
            args.append(("dgate", "g", g))
    if pre:
        args.append(("dw_pre", "wp", wp))
    for name, arg, x in args:
        grad = np.reshape(grads[name], x.shape)
        num, want = _directional(lambda t: loss(**{arg: t}), x, grad, 5)
        scale = np.abs(grad).sum() + 1.0
        assert abs(num - want) <= 1e-6 * scale, (name, num, want)


def test_swiglu_gradients_match_differences():
    rng = np.random.default_rng(3)
    g, u, dh = (rng.standard_normal((5, 40)) * 3 for _ in range(3))
    dg, du, _, _ = ref.swiglu_bwd(dh, g, u)
    for x, grad, f in ((g, dg, lambda t: (dh * ref.swiglu(t, u)[0]).sum()),
                       (u, du, lambda t: (dh * ref.swiglu(g, t)[0]).sum())):
        num, want = _directional(f, x, grad, 9)
        assert abs(num - want) <= 1e-6 * np.abs(grad).sum()


def test_norm_forward_hand_values():
    # y = (3, 4): mean square 25/2; with eps = 0 its norm is y sqrt(2)/5
    y, r = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    v, _ = ref.norm_fwd(y, r, np.array([1.0, 2.0]), np.array([1.0, 1.0]), np.array([[0.5]]), 2.0,
                        3.0, 0.0)
    s = np.sqrt(2.0) / 5
    t = np.array([[3 + 3 * s, -3 + 8 * s]])
    assert np.allclose(v["r_out"], t, rtol=1e-14)
    assert np.allclose(v["n"], t / np.sqrt((t * t).mean()), rtol=1e-14)


def test_encode_rule_hand_values():
    x = torch.zeros((2, 130))
    x[0, 0], x[0, 1], x[0, 2] = 448.0, -1.0, float("nan")
    x[0, 3], x[0, 128] = float("-inf"), -896.0
    q, s = ref.encode(x)
    assert s.tolist() == [[1.0, 1.0], [2.0, 1.0]]
    assert q[0, :4].tolist() == [0x7E, 0xB8, 0x7F, 0xFF] and q[0, 128].item() == 0xFE
    assert q[1].sum().item() == 0
    # below the least amax: s = 2^-119/448, and 2^-130 * 448 * 2^119 = 1.75 * 2^-3 = code 0x26
    q, s = ref.encode(torch.full((1, 1), 2.0 ** -130))
    assert s.item() == float(np.float32(2.0 ** -119) / np.float32(448)) and q.item() == 0x26
    _, s = ref.encode(torch.tensor([[449.0]]), pow2=True)
    assert s.item() == 2.0
    _, s = ref.encode(torch.tensor([[448.0]]), pow2=True)
    assert s.item() == 1.0


# ------------------------------------------------------------------ refusals
def test_ckpt_refusals(L):
    pack, unpack, tr = L.puro_ckpt_pack, L.puro_ckpt_unpack, L.puro_ckpt_transpose
    assert pack(P, 0, -1, 8, 8, 0, P, P, None) == SHAPE
    assert pack(P, 0, 8, (1 << 24) + 1, 1 << 25, 0, P, P, None) == SHAPE
    assert pack(P, 0, 1 << 24, 1 << 24, 1 << 24, 0, P, P, None) == SHAPE    # too many blocks
    assert pack(P, 2, 8, 8, 8, 0, P, P, None) == ARG                        # unknown type
    assert pack(P, 0, 8, 8, 7, 0, P, P, None) == ARG                        # rows overlap
    assert pack(P, 0, 8, 8, 8, 2, P, P, None) == ARG                        # pow2 not 0/1
    assert pack(None, 0, 8, 8, 8, 0, P, P, None) == NULL
    assert pack(P, 0, 8, 8, 8, 0, None, P, None) == NULL
    assert pack(P, 0, 8, 8, 8, 0, P, None, None) == NULL
    assert pack(MIS, 0, 8, 8, 8, 0, P, P, None) == ALIGN                    # odd bf16 address
    assert pack(P + 2, 1, 8, 8, 8, 0, P, P, None) == ALIGN                  # fp32 off by 2
    assert pack(P, 0, 8, 8, 8, 0, P + 8, P, None) == ALIGN
    assert pack(None, 0, 0, 8, 8, 0, None, None, None) == 0
    assert pack(None, 1, 8, 0, 0, 0, None, None, None) == 0
    assert unpack(P, P, 8, 8, P, 3, 8, None) == ARG
    assert unpack(P, P, 8, 8, P, 0, 4, None) == ARG
    assert unpack(P, P, 8, 8, None, 0, 8, None) == NULL
    assert unpack(None, P, 8, 8, P, 0, 8, None) == NULL
    assert unpack(P, MIS, 8, 8, P, 0, 8, None) == ALIGN
    assert unpack(None, None, 8, 0, None, 0, 0, None) == 0
    assert tr(P, P, 8, -8, 0, P, P, None) == SHAPE
    assert tr(P, P, 8, 8, -1, P, P, None) == ARG
    assert tr(P, P, 8, 8, 0, None, P, None) == NULL
    assert tr(P, P, 8, 8, 0, MIS, P, None) == ALIGN
    assert tr(None, None, 0, 8, 0, None, None, None) == 0


def test_swiglu_refusals(L):
    fwd, bwd, fp8 = L.puro_swiglu_fwd, L.puro_swiglu_bwd, L.puro_swiglu_bwd_fp8
    assert fwd(P, -1, 8, P, P, P, P, P, 0, None) == SHAPE
    assert fwd(P, 8, 8, P, P, P, P, P, 7, None) == ARG
    assert fwd(None, 8, 8, P, P, P, P, P, 0, None) == NULL
    assert fwd(P, 8, 8, None, None, None, None, None, 0, None) == NULL      # nothing asked for
    assert fwd(P, 8, 8, None, P, None, None, None, 0, None) == NULL         # codes, no scales
    assert fwd(P, 8, 8, None, None, None, None, P, 0, None) == NULL
    assert fwd(P, 8, 8, MIS, None, None, None, None, 0, None) == ALIGN
    assert fwd(None, 0, 8, None, None, None, None, None, 0, None) == 0
    assert bwd(P, P, P, P, 8, 8, P, None) == ARG                            # both sources
    assert bwd(P, None, P, None, 8, 8, P, None) == NULL
    assert bwd(P, None, None, None, 8, 8, P, None) == NULL
    assert bwd(None, P, None, None, 8, 8, P, None) == NULL
    assert bwd(P, P, None, None, 8, 8, None, None) == NULL
    assert bwd(P, MIS, None, None, 8, 8, P, None) == ALIGN
    assert bwd(P, P, None, None, 1 << 25, 8, P, None) == SHAPE
    assert bwd(None, None, None, None, 8, 0, None, None) == 0
    out = (P,) * 6
    assert fp8(P, P, None, None, 100, 128, 0, *out, None) == SHAPE          # rows not 128 x
    assert fp8(P, P, None, None, 128, 96, 0, *out, None) == SHAPE
    assert fp8(P, P, None, None, 128, 128, 2, *out, None) == ARG
    assert fp8(P, None, P, None, 128, 128, 0, *out, None) == NULL
    for i in range(6):
        o = list(out)
        o[i] = None
        assert fp8(P, P, None, None, 128, 128, 0, *o, None) == NULL
        o[i] = MIS
        assert fp8(P, P, None, None, 128, 128, 0, *o, None) == ALIGN
    assert fp8(None, None, None, None, 0, 128, 0, *((None,) * 6), None) == 0


def _fwd(**kw):
    from blockwise_fp8_gemm_x128_amd._lib import PuroBlockNorm
    d = dict(rows=8, cols=64, residual_type=0, gate_kind=0, pow2=0, alpha=1.0, beta=1.0, eps=1e-6,
             y=P, r=P, w_post=P, w_pre=P, r_out=P, n=P, rstd_y=P, rstd_r=P)
    d.update(kw)
    return ctypes.byref(PuroBlockNorm(**d))


def _bwd(**kw):
    from blockwise_fp8_gemm_x128_amd._lib import PuroBlockNormGrad
    d = dict(rows=8, cols=64, residual_type=0, gate_kind=0, accumulate=0, alpha=1.0, beta=1.0,
             dr_out=P, dn=P, y=P, r=P, rstd_y=P, rstd_r=P, w_post=P, w_pre=P, dr=P, dy=P,
             dw_post=P, dw_pre=P)
    d.update(kw)
    return ctypes.byref(PuroBlockNormGrad(**d))


@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=16385)), (SHAPE, dict(rows=(1 << 24) + 1)),
    (ARG, dict(gate_kind=4)), (ARG, dict(gate_kind=-1)), (ARG, dict(residual_type=2)),
    (ARG, dict(pow2=2)), (ARG, dict(eps=0.0)), (ARG, dict(eps=float("nan"))),
    (ARG, dict(alpha=float("inf"))), (ARG, dict(beta=float("nan"))),
    (NULL, dict(y=None)), (NULL, dict(r=None)), (NULL, dict(r_out=None)),
    (NULL, dict(rstd_y=None)), (NULL, dict(rstd_r=None)), (NULL, dict(n=None)),
    (NULL, dict(gate_kind=1)), (NULL, dict(nq=P)), (NULL, dict(ns=P)), (NULL, dict(ys=P)),
    (NULL, dict(rq=P)), (NULL, dict(w_post=None, y=None, w_pre=None, n=None)),
    (ARG, dict(w_post=None)),                      # y without its norm's weight
    (ARG, dict(w_post=None, y=None, gate_kind=1, gate=P)),
    (ARG, dict(w_pre=None)),                       # n without its norm's weight
    (ALIGN, dict(y=MIS)), (ALIGN, dict(r=MIS)), (ALIGN, dict(r_out=MIS)), (ALIGN, dict(n=MIS)),
    (ALIGN, dict(nq=P, ns=MIS)), (ALIGN, dict(gate_kind=2, gate=MIS)),
    (0, dict(rows=0, y=None, r=None, r_out=None, n=None)), (0, dict(cols=0, w_post=None, y=None)),
])
def test_norm_fwd_refusals(L, status, kw):
    assert L.puro_block_norm_fwd(_fwd(**kw), None) == status


@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(rows=-1)), (SHAPE, dict(cols=16385)), (ARG, dict(gate_kind=9)),
    (ARG, dict(accumulate=2)), (ARG, dict(residual_type=-1)), (ARG, dict(alpha=float("nan"))),
    (ARG, dict(yq=P, ys=P)), (ARG, dict(rq=P, rs=P)),          # both forms of an activation
    (ARG, dict(y=None, yq=P, ys=P)), (ARG, dict(r=None, rq=P, rs=P)),   # one of each form
    (ARG, dict(w_post=None)), (ARG, dict(w_pre=None)),
    (NULL, dict(y=None)), (NULL, dict(y=None, yq=P)), (NULL, dict(y=None, ys=P)),
    (NULL, dict(r=None)), (NULL, dict(r=None, rq=P)), (NULL, dict(dn=None)), (NULL, dict(dy=None)),
    (NULL, dict(rstd_y=None)), (NULL, dict(rstd_r=None)), (NULL, dict(gate_kind=1, gate=P)),
    (NULL, dict(gate_kind=3, dgate=P)),
    (NULL, dict(w_pre=None, dn=None, r=None, dw_pre=None, dr_out=None)),
    (NULL, dict(w_pre=None, dn=None, r=None, dw_pre=None, w_post=None, y=None, dy=None,
                dw_post=None)),
    (ALIGN, dict(dr_out=MIS)), (ALIGN, dict(dr=MIS)), (ALIGN, dict(dy=MIS)),
    (ALIGN, dict(dw_post=MIS)), (ALIGN, dict(dw_pre=MIS)),
    (0, dict(cols=0)),
])
def test_norm_bwd_refusals(L, status, kw):
    assert L.puro_block_norm_bwd(_bwd(**kw), P, None) == status


def test_norm_workspace(L):
    assert L.puro_block_norm_bwd(_bwd(), None, None) == NULL
    assert L.puro_block_norm_bwd(_bwd(), MIS, None) == ALIGN
    assert L.puro_block_norm_fwd(None, None) == NULL
    ws = L.puro_block_norm_workspace
    assert ws(0, 64) == 0 and ws(8, 0) == 0 and ws(8, 16385) == 0
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                             "include", "puro.h")).read()
    assert "#define PURO_NORM_MAX_BLOCKS 512" in text and "#define PURO_NORM_MAX_COLS 16384" in text
    for rows, cols in ((1, 1), (8192, 2048), (1 << 24, 16384)):
        assert 0 < ws(rows, cols) <= 512 * 2 * cols * 4


def test_binding_refuses_host_tensors():
    from blockwise_fp8_gemm_x128_amd import PuroError
    from blockwise_fp8_gemm_x128_amd import binding as puro
    x = torch.zeros((4, 8), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 8), dtype=torch.uint8), torch.ones((1, 4))
    w = torch.ones(8)
    for call in (lambda: puro.puro_ckpt_pack(x), lambda: puro.puro_ckpt_unpack(q, s),
                 lambda: puro.puro_ckpt_transpose(q, s), lambda: puro.puro_swiglu_fwd(x),
                 lambda: puro.puro_swiglu_bwd(x, (q, s)),
                 lambda: puro.puro_block_norm_fwd(x, x, w, w),
                 lambda: puro.puro_block_norm_bwd(x, x, x, x, w, w, w, w),
                 lambda: puro.puro_block_norm_bwd(None, None, x, x, w, w, w, w)):
        with pytest.raises(PuroError):
            call()


def test_binding_refuses_sparse_tensors():
    """A tensor without strides has no answer to "is it contiguous": torch's exception for that must
    not leave the native checks as one of C++."""
    from blockwise_fp8_gemm_x128_amd import PuroError
    from blockwise_fp8_gemm_x128_amd import binding as puro
    dev = torch.device("cuda", 0)
    q = torch.zeros((4, 8), dtype=torch.uint8).to_sparse_csr()
    with pytest.raises(PuroError, match="q: must be contiguous"):
        puro._PACK.pointers(dev, 4, 8, 1, q, None)
    with pytest.raises(PuroError, match="x: expected a bf16 or fp32 matrix"):
        puro._need_rows(torch.zeros((4, 8)).to_sparse_csr(), "x", dev)


def test_native_calls_leave_what_they_do_not_take():
    """Nothing but tensors on the device in their places is taken: the native calls return None,
    without an exception, and the binding's own checks then say what was wrong."""
    from blockwise_fp8_gemm_x128_amd import binding as puro
    nat = puro._load_native()
    x, none = torch.zeros((4, 8), dtype=torch.bfloat16), (None,)
    csr = torch.zeros((4, 8), dtype=torch.uint8).to_sparse_csr()
    for bad in (x, csr, None, 3, "x", (x, x)):
        assert nat.ckpt_pack(bad, x, x, False) is None
        assert nat.ckpt_unpack(bad, x, x) is None
        assert nat.ckpt_transpose(bad, x, x, x, False) is None
        assert nat.norm_fwd(x, bad, x, x, None, 1.0, 1.0, 1e-6, False, none * 10) is None
        assert nat.norm_bwd(bad, x, x, x, x, x, x, x, None, 1.0, 1.0, False, None, none * 5) is None
        assert nat.swiglu_fwd(bad, False, none * 5) is None
        assert nat.swiglu_bwd(bad, (x, x), x) is None
        assert nat.swiglu_bwd_fp8(bad, (x, x), False, none * 6) is None
    assert nat.ckpt_pack(x) is None                      # too few arguments
    assert nat.swiglu_fwd(x, False, none) is None        # too few outputs
    with pytest.raises(TypeError):
        nat.bind(None)
