"""Python binding of libpuro's C ABI: same names, argument marshalling only.

Each function takes torch tensors that live on a HIP device, checks dtype / shape / contiguity
/ device, allocates missing outputs with torch (device memory is PyTorch's job here), and calls
the C entry point with raw device pointers on the current torch stream. Every step of the
computation runs in libpuro's HIP kernels; there is no other code path.
"""
from __future__ import annotations

import ctypes
import struct
from typing import NamedTuple, Optional

import torch

from ._lib import (GATE_CHANNEL, GATE_FULL, GATE_NONE, GATE_TOKEN, NS_GROUP_MAX,
                   OPT_WORKSPACE_BYTES, TYPE_BF16, TYPE_FP32, W_GROUP_MAX, PuroAdamWParams,
                   PuroBlockNorm, PuroBlockNormGrad, PuroError, PuroLinearXent, PuroLinearXentGrad,
                   PuroNewtonSchulzParams, PuroNsItem, PuroWItem, check, lib)

FP8 = torch.uint8  # E4M3 codes travel as raw bytes


# torch's current stream as its raw handle, without the Stream object around it where torch offers
# that (1.8 us less per call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(dev: Optional[torch.device]) -> int:
    """torch's current stream on a tensor's device; None: on the current device."""
    if _raw_stream is not None and dev is not None:
        return _raw_stream(dev.index)
    return torch.cuda.current_stream(dev).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, shape, dev) -> None:
    # the whole check at once first: it is what nearly every call passes, a dozen times a call
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape
            and t.layout is torch.strided and t.is_contiguous() and t.device == dev):
        return
    if not isinstance(t, torch.Tensor):
        raise PuroError(f"{name}: expected a torch.Tensor")
    if t.dtype != dtype:
        raise PuroError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise PuroError(f"{name}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.layout is not torch.strided or not t.is_contiguous():
        raise PuroError(f"{name}: must be contiguous")
    if t.device != dev:
        raise PuroError(f"{name}: on {t.device}, expected {dev}")


def _dev(t: torch.Tensor) -> torch.device:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise PuroError("inputs must be torch tensors on a HIP device")
    return t.device


def _out(t, name, dtype, shape, dev):
    if t is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    _need(t, name, dtype, shape, dev)
    return t


def _need_workspace(t, need: int, dev) -> None:
    """Scratch memory of `need` bytes: of a view, the bytes of its elements are not the bytes behind
    its address (expanded rows share theirs, a stepped view's lie apart)."""
    if not isinstance(t, torch.Tensor):
        raise PuroError("workspace: expected a torch.Tensor")
    if (t.device != dev or t.layout is not torch.strided or not t.is_contiguous()
            or t.numel() * t.element_size() < need):
        raise PuroError(f"workspace: {need} contiguous bytes on {dev} needed")


def puro_quant_act_1x128(x: torch.Tensor, q=None, s=None, _fn="puro_quant_act_1x128"):
    """x bf16 [rows, cols] -> (q uint8 E4M3 [rows, cols], s fp32 [cols/128, rows])."""
    dev = _dev(x)
    rows, cols = x.shape
    _need(x, "x", torch.bfloat16, (rows, cols), dev)
    q = _out(q, "q", FP8, (rows, cols), dev)
    s = _out(s, "s", torch.float32, (cols // 128, rows), dev)
    check(getattr(lib(), _fn)(x.data_ptr(), rows, cols, q.data_ptr(), s.data_ptr(),
                              _stream(dev)))
    return q, s


def puro_quant_w_128x128(w: torch.Tensor, q=None, s=None, _fn="puro_quant_w_128x128"):
    """w bf16 [n, k] -> (q uint8 E4M3 [n, k], s fp32 [n/128, k/128])."""
    dev = _dev(w)
    n, k = w.shape
    _need(w, "w", torch.bfloat16, (n, k), dev)
    q = _out(q, "q", FP8, (n, k), dev)
    s = _out(s, "s", torch.float32, (n // 128, k // 128), dev)
    check(getattr(lib(), _fn)(w.data_ptr(), n, k, q.data_ptr(), s.data_ptr(), _stream(dev)))
    return q, s


def w_group_items(ws, qs, ss):
    """ctypes array of puro_w_item for weights ws [n, k] and outputs qs, ss (checked)."""
    if len(ws) > W_GROUP_MAX:
        raise PuroError(f"at most {W_GROUP_MAX} matrices per grouped call")
    if not (len(ws) == len(qs) == len(ss)):
        raise PuroError("ws, qs and ss must have the same length")
    items = (PuroWItem * max(len(ws), 1))()
    for i, (w, q, s) in enumerate(zip(ws, qs, ss)):
        dev = _dev(w)
        n, k = w.shape
        _need(w, f"w[{i}]", torch.bfloat16, (n, k), dev)
        _need(q, f"q[{i}]", FP8, (n, k), dev)
        _need(s, f"s[{i}]", torch.float32, (n // 128, k // 128), dev)
        items[i] = PuroWItem(w.data_ptr(), n, k, q.data_ptr(), s.data_ptr())
    return items


def puro_quant_w_128x128_group(ws, qs=None, ss=None, _fn="puro_quant_w_128x128_group"):
    """Several bf16 weights [n, k] quantised in one launch -> (list of q, list of s), each as
    from puro_quant_w_128x128."""
    if not ws:
        return [], []
    dev = _dev(ws[0])
    qs = qs or [torch.empty(w.shape, dtype=FP8, device=dev) for w in ws]
    ss = ss or [torch.empty((w.shape[0] // 128, w.shape[1] // 128), dtype=torch.float32,
                            device=dev) for w in ws]
    items = w_group_items(ws, qs, ss)
    check(getattr(lib(), _fn)(items, len(ws), _stream(dev)))
    return qs, ss


def puro_quant_transpose(x: torch.Tensor, qt=None, st=None, _fn="puro_quant_transpose"):
    """x bf16 [rows, cols] -> (qt uint8 E4M3 [cols, rows], st fp32 [rows/128, cols])."""
    dev = _dev(x)
    rows, cols = x.shape
    _need(x, "x", torch.bfloat16, (rows, cols), dev)
    qt = _out(qt, "qt", FP8, (cols, rows), dev)
    st = _out(st, "st", torch.float32, (rows // 128, cols), dev)
    check(getattr(lib(), _fn)(x.data_ptr(), rows, cols, qt.data_ptr(), st.data_ptr(),
                              _stream(dev)))
    return qt, st


def puro_quant_dual_1x128(x: torch.Tensor, q=None, s=None, qt=None, st=None,
                          _fn="puro_quant_dual_1x128"):
    """x bf16 [rows, cols] -> (q [rows, cols], s [cols/128, rows], qt [cols, rows],
    st [rows/128, cols]): the outputs of puro_quant_act_1x128 and puro_quant_transpose from one
    read of x."""
    dev = _dev(x)
    rows, cols = x.shape
    _need(x, "x", torch.bfloat16, (rows, cols), dev)
    q = _out(q, "q", FP8, (rows, cols), dev)
    s = _out(s, "s", torch.float32, (cols // 128, rows), dev)
    qt = _out(qt, "qt", FP8, (cols, rows), dev)
    st = _out(st, "st", torch.float32, (rows // 128, cols), dev)
    check(getattr(lib(), _fn)(x.data_ptr(), rows, cols, q.data_ptr(), s.data_ptr(),
                              qt.data_ptr(), st.data_ptr(), _stream(dev)))
    return q, s, qt, st


def puro_fp8_gemm_fwd(xq, sx, wq, sw, y=None, _fn="puro_fp8_gemm_fwd"):
    """Y bf16 [M, N] from xq [M, K], sx [K/128, M], wq [N, K], sw [N/128, K/128]."""
    dev = _dev(xq)
    M, K = xq.shape
    N = wq.shape[0]
    _need(xq, "xq", FP8, (M, K), dev)
    _need(sx, "sx", torch.float32, (K // 128, M), dev)
    _need(wq, "wq", FP8, (N, K), dev)
    _need(sw, "sw", torch.float32, (N // 128, K // 128), dev)
    y = _out(y, "y", torch.bfloat16, (M, N), dev)
    check(getattr(lib(), _fn)(xq.data_ptr(), sx.data_ptr(), wq.data_ptr(), sw.data_ptr(),
                              y.data_ptr(), M, N, K, _stream(dev)))
    return y


def puro_fp8_gemm_dgrad(dyq, sdy, wq, sw, dx=None, _fn="puro_fp8_gemm_dgrad"):
    """dX bf16 [M, K] from dyq [M, N], sdy [N/128, M], wq [N, K], sw [N/128, K/128]."""
    dev = _dev(dyq)
    M, N = dyq.shape
    K = wq.shape[1]
    _need(dyq, "dyq", FP8, (M, N), dev)
    _need(sdy, "sdy", torch.float32, (N // 128, M), dev)
    _need(wq, "wq", FP8, (N, K), dev)
    _need(sw, "sw", torch.float32, (N // 128, K // 128), dev)
    dx = _out(dx, "dx", torch.bfloat16, (M, K), dev)
    check(getattr(lib(), _fn)(dyq.data_ptr(), sdy.data_ptr(), wq.data_ptr(), sw.data_ptr(),
                              dx.data_ptr(), M, N, K, _stream(dev)))
    return dx


def puro_fp8_gemm_wgrad(dytq, sdyt, xtq, sxt, dw=None, accumulate: bool = False,
                        _fn="puro_fp8_gemm_wgrad"):
    """dW fp32 [N, K] (= or +=) from dytq [N, M], sdyt [M/128, N], xtq [K, M], sxt [M/128, K]."""
    dev = _dev(dytq)
    N, M = dytq.shape
    K = xtq.shape[0]
    _need(dytq, "dytq", FP8, (N, M), dev)
    _need(sdyt, "sdyt", torch.float32, (M // 128, N), dev)
    _need(xtq, "xtq", FP8, (K, M), dev)
    _need(sxt, "sxt", torch.float32, (M // 128, K), dev)
    if accumulate and dw is None:
        raise PuroError("accumulate=True needs an existing dw")
    dw = _out(dw, "dw", torch.float32, (N, K), dev)
    check(getattr(lib(), _fn)(dytq.data_ptr(), sdyt.data_ptr(), xtq.data_ptr(),
                              sxt.data_ptr(), dw.data_ptr(), M, N, K, 1 if accumulate else 0,
                              _stream(dev)))
    return dw


def optim_workspace(dev) -> torch.Tensor:
    """Device workspace for the optimizer-step entry points (PURO_OPT_WORKSPACE_BYTES)."""
    return torch.empty(OPT_WORKSPACE_BYTES, dtype=torch.uint8, device=dev)


def puro_frobenius_norm(w: torch.Tensor, norm=None, workspace=None):
    """||w||_F of an fp32 tensor -> fp32 device tensor of shape (1,)."""
    dev = _dev(w)
    _need(w, "w", torch.float32, tuple(w.shape), dev)
    norm = _out(norm, "norm", torch.float32, (1,), dev)
    if workspace is None:
        workspace = optim_workspace(dev)
    else:
        _need_workspace(workspace, OPT_WORKSPACE_BYTES, dev)
    check(lib().puro_frobenius_norm(w.data_ptr(), w.numel(), norm.data_ptr(), workspace.data_ptr(),
                                    _stream(dev)))
    return norm


def puro_hyperball_step(w: torch.Tensor, u: torch.Tensor, lr: float, radius: torch.Tensor,
                        w_bf16=None, workspace=None):
    """In place: w <- (w - lr*u) * radius / ||w - lr*u||_F; returns the bf16 copy of w."""
    dev = _dev(w)
    n = w.numel()
    _need(w, "w", torch.float32, tuple(w.shape), dev)
    _need(u, "u", torch.float32, tuple(w.shape), dev)
    _need(radius, "radius", torch.float32, (1,), dev)
    w_bf16 = _out(w_bf16, "w_bf16", torch.bfloat16, tuple(w.shape), dev)
    if workspace is None:
        workspace = optim_workspace(dev)
    else:
        _need_workspace(workspace, OPT_WORKSPACE_BYTES, dev)
    check(lib().puro_hyperball_step(w.data_ptr(), u.data_ptr(), n, float(lr), radius.data_ptr(),
                                    w_bf16.data_ptr(), workspace.data_ptr(), _stream(dev)))
    return w_bf16


def puro_hyperball_step_u16(w: torch.Tensor, u: torch.Tensor, lr: float, radius: torch.Tensor,
                            w_bf16=None, workspace=None):
    """puro_hyperball_step with the direction in bf16, as puro_newton_schulz writes it."""
    dev = _dev(w)
    _need(w, "w", torch.float32, tuple(w.shape), dev)
    _need(u, "u", torch.bfloat16, tuple(w.shape), dev)
    _need(radius, "radius", torch.float32, (1,), dev)
    w_bf16 = _out(w_bf16, "w_bf16", torch.bfloat16, tuple(w.shape), dev)
    if workspace is None:
        workspace = optim_workspace(dev)
    else:
        _need_workspace(workspace, OPT_WORKSPACE_BYTES, dev)
    with torch.cuda.device(dev):
        check(lib().puro_hyperball_step_u16(w.data_ptr(), u.data_ptr(), w.numel(), float(lr),
                                            radius.data_ptr(), w_bf16.data_ptr(),
                                            workspace.data_ptr(), _stream(dev)))
    return w_bf16


def puro_hyperball_step_noalloc(w: torch.Tensor, u: torch.Tensor, lr: float,
                                radius: torch.Tensor, w_bf16: torch.Tensor):
    """puro_hyperball_step with the library's own scratch instead of a workspace; the bf16
    output is required (this path allocates nothing)."""
    dev = _dev(w)
    _need(w, "w", torch.float32, tuple(w.shape), dev)
    _need(u, "u", torch.float32, tuple(w.shape), dev)
    _need(radius, "radius", torch.float32, (1,), dev)
    _need(w_bf16, "w_bf16", torch.bfloat16, tuple(w.shape), dev)
    check(lib().puro_hyperball_step_noalloc(w.data_ptr(), u.data_ptr(), w.numel(), float(lr),
                                            radius.data_ptr(), w_bf16.data_ptr(), _stream(dev)))
    return w_bf16


def adamw_params(lr, beta1, beta2, eps, weight_decay, step) -> PuroAdamWParams:
    return PuroAdamWParams(lr, beta1, beta2, eps, weight_decay, int(step))


def puro_adamw_step(p, g, m, v, lr, beta1, beta2, eps, weight_decay, step, p_bf16=None,
                    want_bf16: bool = False):
    """In place AdamW step on fp32 p, m, v with gradient g; returns the bf16 copy of p if
    p_bf16 is given or want_bf16 is set, else None."""
    dev = _dev(p)
    shape = tuple(p.shape)
    for t, name in ((p, "p"), (g, "g"), (m, "m"), (v, "v")):
        _need(t, name, torch.float32, shape, dev)
    if p_bf16 is None and want_bf16:
        p_bf16 = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    if p_bf16 is not None:
        _need(p_bf16, "p_bf16", torch.bfloat16, shape, dev)
    hp = adamw_params(lr, beta1, beta2, eps, weight_decay, step)
    check(lib().puro_adamw_step(p.data_ptr(), g.data_ptr(), m.data_ptr(), v.data_ptr(),
                                p.numel(), ctypes.byref(hp),
                                None if p_bf16 is None else p_bf16.data_ptr(), _stream(dev)))
    return p_bf16


# ---------------------------------------------------------------- between the GEMMs
# 8-bit checkpoints are pairs (codes uint8 [rows, cols], scales fp32 [ceil(cols/128), rows]).
#
# These operators take up to fifteen tensors, and small calls are launch-bound, so their checks and
# addresses come from one native call (csrc/args.cpp) per operator call; where it finds a tensor
# that is not as specified, _need says what is wrong with it.
_TYPES = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_FP32}
_DTYPES = {"b": torch.bfloat16, "f": torch.float32, "q": FP8}
_LETTERS = {torch.bfloat16: "b", torch.float32: "f"}


class _Spec:
    """Expected tensors of a call, "name:tfij" each: t the type (b bf16, f fp32, q codes), f whether
    it is required (!) or may be None (?), i and j which of the call's sizes d0, d1, d2 and 1 (3)
    its sizes are (- for a vector)."""

    def __init__(self, text: str):
        pairs = [item.split(":") for item in text.split()]
        self.names = [n for n, _ in pairs]
        self.code = "".join(c for _, c in pairs).encode()

    def pointers(self, dev, d0, d1, d2, *tensors):
        p = (_native or _load_native()).ptrs(self.code, dev.index, d0, d1, d2, *tensors)
        if type(p) is not int:
            return p
        kind, need, *dims = self.code[4 * p:4 * p + 4].decode()
        name = self.names[p]
        if tensors[p] is None:
            raise PuroError(f"{name}: required")
        shape = tuple((d0, d1, d2, 1)[int(i)] for i in dims if i != "-")
        _need(tensors[p], name, _DTYPES[kind], shape, dev)
        raise PuroError(f"{name}: not as expected")


# The module of native checks and calls. Its calls return the entry point's status, or None for
# arguments that are not as they must be: then the binding's own checks say which.
_native = None


def _load_native():
    global _native
    try:
        from . import _args
    except ImportError as e:
        raise PuroError("the binding's native checks are not built (%s); run `python -m "
                        "blockwise_fp8_gemm_x128_amd.build`" % e) from e
    _args.bind(_raw_stream or (lambda i: torch.cuda.current_stream(i).cuda_stream),
               *(ctypes.cast(getattr(lib(), "puro_" + name), ctypes.c_void_p).value
                 for name in ("ckpt_pack", "ckpt_unpack", "ckpt_transpose", "block_norm_fwd",
                              "block_norm_workspace", "block_norm_bwd", "swiglu_fwd", "swiglu_bwd",
                              "swiglu_bwd_fp8", "linear_xent_fwd_workspace", "linear_xent_fwd",
                              "linear_xent_bwd_workspace", "linear_xent_bwd",
                              "newton_schulz_workspace", "newton_schulz")))
    _native = _args
    return _args


def _done(st) -> bool:
    """Whether a native call was made; raises its error."""
    if st:
        check(st)
    return st is not None


def _call(name, *args) -> None:
    """A C entry point of these operators, its status checked."""
    st = (_entry.get(name) or _load_entry(name))(*args)
    if st:
        check(st)


_entry = {}  # the C entry points by name


def _load_entry(name):
    fn = _entry[name] = getattr(lib(), name)
    return fn


def _groups(n: int) -> int:
    return (n + 127) // 128


def _new_codes(rows, cols, dev):
    return (torch.empty((rows, cols), dtype=FP8, device=dev),
            torch.empty((_groups(cols), rows), dtype=torch.float32, device=dev))


def _matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise PuroError(f"{name}: expected a matrix")
    return t.shape


def _need_rows(x, name, dev):
    """A 2-D bf16 or fp32 matrix with unit column stride; returns (type, row stride)."""
    if (not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in _TYPES
            or x.layout is not torch.strided):
        raise PuroError(f"{name}: expected a bf16 or fp32 matrix")
    if x.device != dev:
        raise PuroError(f"{name}: on {x.device}, expected {dev}")
    rows, cols = x.shape
    ld, unit = x.stride()
    if rows <= 1:
        ld = cols
    if (cols > 1 and unit != 1) or ld < cols:
        raise PuroError(f"{name}: columns must be adjacent and rows must not overlap")
    return _TYPES[x.dtype], ld


_PACK = _Spec("q:q!01 s:f!20")
_TRANSPOSE = _Spec("checkpoint:q!01 scales:f!20 qt:q!10")


def puro_ckpt_pack(x: torch.Tensor, q=None, s=None, pow2: bool = False):
    """8-bit checkpoint of x, bf16 or fp32 [rows, cols] (any sizes, rows may be strided) ->
    (q uint8 E4M3 [rows, cols], s fp32 [ceil(cols/128), rows])."""
    if q is None or s is None:
        new = _new_codes(*_matrix(x, "x"), _dev(x))
        q, s = new[0] if q is None else q, new[1] if s is None else s
    if _done((_native or _load_native()).ckpt_pack(x, q, s, pow2)):
        return q, s
    dev = _dev(x)
    kind, ld = _need_rows(x, "x", dev)
    rows, cols = x.shape
    p = _PACK.pointers(dev, rows, cols, _groups(cols), q, s)
    _call("puro_ckpt_pack", x.data_ptr(), kind, rows, cols, ld, bool(pow2), *p, _stream(dev))
    return q, s


def puro_ckpt_unpack(q, s, x=None, dtype=torch.bfloat16):
    """The values a checkpoint stands for, as `dtype` (bf16 or fp32) or into x (rows may be
    strided)."""
    if x is None:
        x = torch.empty(_matrix(q, "checkpoint"), dtype=dtype, device=_dev(q))
    if _done((_native or _load_native()).ckpt_unpack(q, s, x)):
        return x
    dev = _dev(q)
    rows, cols = _matrix(q, "checkpoint")
    kind, ld = _need_rows(x, "x", dev)
    if x.shape != (rows, cols):
        raise PuroError(f"x: shape {tuple(x.shape)}, expected {(rows, cols)}")
    p = _PACK.pointers(dev, rows, cols, _groups(cols), q, s)
    _call("puro_ckpt_unpack", *p, rows, cols, x.data_ptr(), kind, ld, _stream(dev))
    return x


def puro_ckpt_transpose(q, s, qt=None, st=None, pow2: bool = False):
    """Checkpoint [rows, cols] -> checkpoint of its transpose (qt uint8 [cols, rows], st fp32
    [ceil(rows/128), cols]): a forward GEMM operand becomes the weight gradient's."""
    if qt is None or st is None:
        rows, cols = _matrix(q, "checkpoint")
        new = _new_codes(cols, rows, _dev(q))
        qt, st = new[0] if qt is None else qt, new[1] if st is None else st
    if _done((_native or _load_native()).ckpt_transpose(q, s, qt, st, pow2)):
        return qt, st
    dev = _dev(q)
    rows, cols = _matrix(q, "checkpoint")
    p = _TRANSPOSE.pointers(dev, rows, cols, _groups(cols), q, s, qt)
    _need(st, "st", torch.float32, (_groups(rows), cols), dev)
    _call("puro_ckpt_transpose", p[0], p[1], rows, cols, bool(pow2), p[2], st.data_ptr(),
          _stream(dev))
    return qt, st


class BlockNorm(NamedTuple):
    """Outputs of puro_block_norm_fwd; None where left out."""
    r_out: Optional[torch.Tensor]    # residual type [rows, cols]
    n: Optional[torch.Tensor]        # bf16 [rows, cols]
    nq: Optional[torch.Tensor]       # n as an FP8 operand
    ns: Optional[torch.Tensor]
    rstd_y: Optional[torch.Tensor]   # fp32 [rows]
    rstd_r: Optional[torch.Tensor]
    yq: Optional[torch.Tensor]       # checkpoint of y
    ys: Optional[torch.Tensor]
    rq: Optional[torch.Tensor]       # checkpoint of r_out
    rs: Optional[torch.Tensor]


class BlockNormGrads(NamedTuple):
    """Outputs of puro_block_norm_bwd; None where left out."""
    dr: Optional[torch.Tensor]
    dy: Optional[torch.Tensor]
    dw_post: Optional[torch.Tensor]
    dw_pre: Optional[torch.Tensor]
    dgate: Optional[torch.Tensor]


# puro_block_norm and puro_block_norm_grad packed as bytes, a third of the time of filling a ctypes
# structure field by field.
_NORM = struct.Struct("@qqiiifff15P")
_NORM_GRAD = struct.Struct("@qqiiiff18P")
assert _NORM.size == ctypes.sizeof(PuroBlockNorm)
assert _NORM_GRAD.size == ctypes.sizeof(PuroBlockNormGrad)

# How a gate is specified, by its kind.
_GATES = {GATE_NONE: "f?1-", GATE_CHANNEL: "f!1-", GATE_TOKEN: "f!03", GATE_FULL: "b!01"}
_NORM_FWD = {(dtype, kind): _Spec(
    f"y:b?01 r:{r}!01 w_post:f?1- w_pre:f?1- gate:{g} r_out:{r}?01 n:b?01 nq:q?01 ns:f?20 "
    "rstd_y:f?0- rstd_r:f?0- yq:q?01 ys:f?20 rq:q?01 rs:f?20")
    for dtype, r in _LETTERS.items() for kind, g in _GATES.items()}
_NORM_BWD = {(dtype, kind): _Spec(
    f"dr_out:{r}?01 dn:b?01 y:b?01 y:q?01 y:f?20 r_out:{r}?01 r_out:q?01 r_out:f?20 rstd_y:f?0- "
    f"rstd_r:f?0- w_post:f?1- w_pre:f?1- gate:{g} dr:{r}?01 dy:b?01 dw_post:f?1- dw_pre:f?1- "
    f"dgate:{g}") for dtype, r in _LETTERS.items() for kind, g in _GATES.items()}


def _gate_kind(gate) -> int:
    """fp32 [cols] is a gate per channel, fp32 [rows, 1] one per token, bf16 [rows, cols] one per
    element."""
    if gate is None:
        return GATE_NONE
    if not isinstance(gate, torch.Tensor):
        raise PuroError("gate: expected a torch.Tensor")
    if gate.dim() == 1:
        return GATE_CHANNEL
    return GATE_TOKEN if gate.dtype is torch.float32 else GATE_FULL


def puro_block_norm_fwd(y, r, w_post, w_pre, gate=None, alpha: float = 1.0, beta: float = 1.0,
                        eps: float = 1e-6, n: str = "fp8", ckpt: bool = True,
                        pow2: bool = False, out=None) -> BlockNorm:
    """r_out = beta r + alpha gate * rmsnorm(y) w_post; n = rmsnorm(r_out) w_pre, in one pass.

    y bf16 [rows, cols] (None: only the norm before a block, r_out = beta r), r bf16 or fp32
    [rows, cols], w_post / w_pre fp32 [cols] (w_pre None: only the norm after a block), gate None,
    fp32 [cols], fp32 [rows, 1] or bf16 [rows, cols]. `n`: "fp8" (codes and scales, the next
    GEMM's operand), "bf16" or "both"; `ckpt`: also 8-bit checkpoints of y and r_out. `out`: the
    ten outputs to write (a BlockNorm or a tuple in its order, None to leave one out) instead of
    new ones; out.r_out may be r."""
    if out is None:
        if n not in ("fp8", "bf16", "both"):
            raise PuroError("n: expected 'fp8', 'bf16' or 'both'")
        dev = _dev(r)
        rows, cols = _matrix(r, "r")
        post, pre, none, f32 = y is not None, w_pre is not None, (None, None), torch.float32
        out = BlockNorm(
            torch.empty_like(r) if post or beta != 1.0 else None,
            torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
            if pre and n != "fp8" else None,
            *(_new_codes(rows, cols, dev) if pre and n != "bf16" else none),
            torch.empty((rows,), dtype=f32, device=dev) if post else None,
            torch.empty((rows,), dtype=f32, device=dev) if pre else None,
            *(_new_codes(rows, cols, dev) if post and ckpt else none),
            *(_new_codes(rows, cols, dev) if ckpt else none))
    elif type(out) is not BlockNorm:
        out = BlockNorm(*out)
    if _done((_native or _load_native()).norm_fwd(y, r, w_post, w_pre, gate, alpha, beta, eps,
                                                  pow2, out)):
        return out
    dev = _dev(r)
    rows, cols = _matrix(r, "r")
    dtype = r.dtype
    if dtype not in _TYPES:
        raise PuroError("r: expected bf16 or fp32")
    kind = _gate_kind(gate)
    p = _NORM_FWD[dtype, kind].pointers(dev, rows, cols, (cols + 127) // 128, y, r,
                                        None if y is None else w_post, w_pre, gate, *out)
    _call("puro_block_norm_fwd", _NORM.pack(rows, cols, _TYPES[dtype], kind, bool(pow2), alpha,
                                            beta, eps, *p), _stream(dev))
    return out


def _saved(x, name, wanted):
    """A saved activation, as it was or as its checkpoint (codes, scales): (x, q, s)."""
    if not wanted:
        return None, None, None
    if isinstance(x, (tuple, list)):
        if len(x) != 2:
            raise PuroError(f"{name}: expected a (codes, scales) pair")
        return None, x[0], x[1]
    if x is None:
        raise PuroError(f"{name}: required")
    return x, None, None


def block_norm_workspace(rows: int, cols: int, dev) -> torch.Tensor:
    """Device workspace of puro_block_norm_bwd for these sizes."""
    size = lib().puro_block_norm_workspace(rows, cols)
    return torch.empty(max(size, 16), dtype=torch.uint8, device=dev)


def _residual(dr_out, r_out, given):
    """The residual stream's type in a backward call that makes its own dr: that of the tensors of
    that type, or, where r_out is a checkpoint and dr_out absent, the one given. It is not guessed:
    every earlier boundary takes its type from this dr."""
    known = next((t.dtype for t in (dr_out, r_out) if isinstance(t, torch.Tensor)), given)
    if known is None:
        raise PuroError("residual_dtype: required where r_out is a checkpoint and dr_out None "
                        "(or give out.dr)")
    if given is not None and (given != known or given not in _TYPES):
        raise PuroError(f"residual_dtype: {given}, expected {known} (bf16 or fp32)")
    return known


def puro_block_norm_bwd(dr_out, dn, y, r_out, rstd_y, rstd_r, w_post, w_pre, gate=None,
                        alpha: float = 1.0, beta: float = 1.0, accumulate: bool = False,
                        workspace=None, out=None, residual_dtype=None) -> BlockNormGrads:
    """Gradients of puro_block_norm_fwd from those of r_out (dr_out, None for zero) and n (dn
    bf16, None if w_pre was). y and r_out: the saved tensors, or both as their checkpoints,
    (codes, scales) pairs; rstd_y None: the norm after the block was left out. accumulate adds
    dw_post, dw_pre and a channel gate's gradient to `out`'s. `out`: the five outputs to write
    (None to skip; out.dr may be dr_out). residual_dtype: the residual stream's type, for a new dr
    where neither dr_out nor r_out as it was says it (the last boundary, from checkpoints)."""
    lead = dr_out if dr_out is not None else dn
    if lead is None:
        raise PuroError("dr_out and dn: at least one is required")
    post, pre = rstd_y is not None, dn is not None
    if out is None:
        if accumulate:
            raise PuroError("accumulate=True needs existing gradients in out")
        dev = _dev(lead)
        rows, cols = _matrix(lead, "dr_out")
        vec = lambda: torch.empty((cols,), dtype=torch.float32, device=dev)  # noqa: E731
        out = BlockNormGrads(torch.empty((rows, cols),
                                         dtype=_residual(dr_out, r_out, residual_dtype),
                                         device=dev),
                             torch.empty((rows, cols), dtype=torch.bfloat16, device=dev)
                             if post else None, vec() if post else None, vec() if pre else None,
                             torch.empty_like(gate) if gate is not None else None)
    else:
        if type(out) is not BlockNormGrads:
            out = BlockNormGrads(*out)
        if residual_dtype is not None:
            _residual(out.dr, None, residual_dtype)
    if _done((_native or _load_native()).norm_bwd(dr_out, dn, y, r_out, rstd_y, rstd_r, w_post,
                                                  w_pre, gate, alpha, beta, accumulate, workspace,
                                                  out)):
        return out
    dev = _dev(lead)
    rows, cols = _matrix(lead, "dr_out")
    # (of neither: nothing of the residual type is read or written)
    res = next((t.dtype for t in (dr_out, r_out, out[0]) if isinstance(t, torch.Tensor)),
               torch.bfloat16)
    if res not in _TYPES:
        raise PuroError("dr_out: expected bf16 or fp32")
    kind = _gate_kind(gate)
    saved = *_saved(y, "y", post), *_saved(r_out, "r_out", pre)
    p = _NORM_BWD[res, kind].pointers(
        dev, rows, cols, (cols + 127) // 128, dr_out, dn, *saved, rstd_y, rstd_r if pre else None,
        w_post if post else None, w_pre if pre else None, gate, *out)
    need = lib().puro_block_norm_workspace(rows, cols)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    _call("puro_block_norm_bwd", _NORM_GRAD.pack(rows, cols, _TYPES[res], kind, bool(accumulate),
                                                 alpha, beta, *p), workspace.data_ptr(),
          _stream(dev))
    return out


class SwiGLU(NamedTuple):
    """Outputs of puro_swiglu_fwd; None where left out."""
    h: Optional[torch.Tensor]        # bf16 [rows, f]
    hq: Optional[torch.Tensor]       # h as an FP8 operand
    hs: Optional[torch.Tensor]
    guq: Optional[torch.Tensor]      # checkpoint of gu: codes [rows, 2f]
    gus: Optional[torch.Tensor]      # scales [2 ceil(f/128), rows], g's groups first


class SwiGLUOperands(NamedTuple):
    """Outputs of puro_swiglu_bwd_fp8: the FP8 operands of the GEMMs that follow."""
    dguq: torch.Tensor               # dgu [rows, 2f]: gate_up's data gradient
    dgus: torch.Tensor
    dgutq: torch.Tensor              # dgu transposed [2f, rows]: gate_up's weight gradient
    dguts: torch.Tensor
    htq: torch.Tensor                # h transposed [f, rows]: down's weight gradient
    hts: torch.Tensor


# Sizes d0 rows, d1 f, d2 2f for the tensors; the scales' first sizes are checked apart.
_SWIGLU_FWD = _Spec("gu:b!02 h:b?01 hq:q?01 guq:q?02")
_SWIGLU_BWD = _Spec("dh:b!01 gu:b?02 gu:q?02 dgu:b?02")
_SWIGLU_FP8 = _Spec("dh:b!01 gu:b?02 gu:q?02 dguq:q!02 dgutq:q!20 htq:q!10")
_GU_SCALES = _Spec("hs:f?10 gus:f?20")
_FP8_SCALES = _Spec("gus:f?20 dgus:f!20")
_FP8_T_SCALES = _Spec("dguts:f!01 hts:f!02")


def puro_swiglu_fwd(gu, h: bool = False, fp8: bool = True, ckpt: bool = True, pow2: bool = False,
                    out=None) -> SwiGLU:
    """h = u g sigmoid(g) from gu = [g | u], bf16 [rows, 2f]. `h`: h in bf16; `fp8`: h as the down
    projection's operand; `ckpt`: an 8-bit checkpoint of gu. `out`: the five outputs to write
    (None to leave one out) instead of new ones."""
    if out is None:
        dev = _dev(gu)
        rows, cols = _matrix(gu, "gu")
        f, k, none = cols // 2, (cols // 2 + 127) // 128, (None, None)
        out = SwiGLU(torch.empty((rows, f), dtype=torch.bfloat16, device=dev) if h else None,
                     *(_new_codes(rows, f, dev) if fp8 else none),
                     *((torch.empty((rows, cols), dtype=FP8, device=dev),
                        torch.empty((2 * k, rows), dtype=torch.float32, device=dev))
                       if ckpt else none))
    elif type(out) is not SwiGLU:
        out = SwiGLU(*out)
    if _done((_native or _load_native()).swiglu_fwd(gu, pow2, out)):
        return out
    dev = _dev(gu)
    rows, cols = _matrix(gu, "gu")
    if cols % 2:
        raise PuroError(f"gu: {cols} columns, expected an even number (g and u)")
    f, k = cols // 2, (cols // 2 + 127) // 128
    p, ph, hq, guq = _SWIGLU_FWD.pointers(dev, rows, f, cols, gu, out[0], out[1], out[3])
    hs, gus = _GU_SCALES.pointers(dev, rows, k, 2 * k, out[2], out[4])
    _call("puro_swiglu_fwd", p, rows, f, ph, hq, hs, guq, gus, bool(pow2), _stream(dev))
    return out


def puro_swiglu_bwd(dh, gu, dgu=None):
    """dgu bf16 [rows, 2f] from dh bf16 [rows, f] and gu: bf16 [rows, 2f], or its checkpoint as a
    (codes, scales) pair."""
    if dgu is None:
        rows, f = _matrix(dh, "dh")
        dgu = torch.empty((rows, 2 * f), dtype=torch.bfloat16, device=_dev(dh))
    if _done((_native or _load_native()).swiglu_bwd(dh, gu, dgu)):
        return dgu
    dev = _dev(dh)
    rows, f = _matrix(dh, "dh")
    x, q, s = _saved(gu, "gu", True)
    p = _SWIGLU_BWD.pointers(dev, rows, f, 2 * f, dh, x, q, dgu)
    ps = 0
    if s is not None:
        _need(s, "gu", torch.float32, (2 * ((f + 127) // 128), rows), dev)
        ps = s.data_ptr()
    _call("puro_swiglu_bwd", p[0], p[1], p[2], ps, rows, f, p[3], _stream(dev))
    return dgu


def puro_swiglu_bwd_fp8(dh, gu, pow2: bool = False, out=None) -> SwiGLUOperands:
    """puro_swiglu_bwd straight to the FP8 operands of gate_up's data and weight gradients, and
    h's transposed copy for down's weight gradient. rows and f: multiples of 128. `out`: the six
    outputs to write instead of new ones."""
    if out is None:
        dev = _dev(dh)
        rows, f = _matrix(dh, "dh")
        out = SwiGLUOperands(*_new_codes(rows, 2 * f, dev), *_new_codes(2 * f, rows, dev),
                             *_new_codes(f, rows, dev))
    elif type(out) is not SwiGLUOperands:
        out = SwiGLUOperands(*out)
    if _done((_native or _load_native()).swiglu_bwd_fp8(dh, gu, pow2, out)):
        return out
    dev = _dev(dh)
    rows, f = _matrix(dh, "dh")
    if rows % 128 or f % 128:
        raise PuroError(f"dh: shape {(rows, f)}, expected multiples of 128")
    x, q, s = _saved(gu, "gu", True)
    p = _SWIGLU_FP8.pointers(dev, rows, f, 2 * f, dh, x, q, out[0], out[2], out[4])
    gus, dgus = _FP8_SCALES.pointers(dev, rows, f, f // 64, s, out[1])
    dguts, hts = _FP8_T_SCALES.pointers(dev, rows // 128, 2 * f, f, out[3], out[5])
    _call("puro_swiglu_bwd_fp8", p[0], p[1], p[2], gus, rows, f, bool(pow2), p[3], dgus, p[4],
          dguts, p[5], hts, _stream(dev))
    return out


# ---------------------------------------------------------------- update direction
NS_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def ns_workspace(count: int, rows: int, cols: int, dev) -> torch.Tensor:
    """Device workspace of puro_newton_schulz for `count` matrices [rows, cols]."""
    return torch.empty(lib().puro_newton_schulz_workspace(count, rows, cols), dtype=torch.uint8,
                       device=dev)


def puro_newton_schulz(gs, ms=None, us=None, ms_out=None, beta: float = 0.95,
                       nesterov: bool = True, scale: float = 1.0, steps: int = 5,
                       coefficients=NS_COEFFICIENTS, workspace=None):
    """Directions u (a list of bf16 [rows, cols]) of the gradients gs, fp32 matrices of one shape (a
    list, at most 64): their momentum ms (fp32, updated in place, or into ms_out; None: none),
    orthogonalised by Newton-Schulz products and scaled."""
    gs = list(gs)
    if not gs:
        return []
    if ms is None and ms_out is not None:
        raise PuroError("ms_out needs ms")
    coefficients = tuple(coefficients)
    if len(coefficients) != 3:
        raise PuroError(f"coefficients: {len(coefficients)}, expected 3")
    ms = None if ms is None else list(ms)
    ms_out = ms if ms_out is None else list(ms_out)
    if us is None:
        us = [torch.empty(_matrix(g, "g"), dtype=torch.bfloat16, device=_dev(g)) for g in gs]
    else:
        us = list(us)
    if _done((_native or _load_native()).newton_schulz(
            gs, ms, ms_out, us, beta, nesterov, scale, steps, coefficients, workspace)):
        return us
    if len(gs) > NS_GROUP_MAX:
        raise PuroError(f"at most {NS_GROUP_MAX} matrices per grouped call")
    dev = _dev(gs[0])
    rows, cols = shape = _matrix(gs[0], "g[0]")
    for name, ts in (("ms", ms), ("ms_out", ms_out), ("us", us)):
        if ts is not None and len(ts) != len(gs):
            raise PuroError(f"{name}: {len(ts)} matrices, expected {len(gs)}")
    items = (PuroNsItem * len(gs))()
    for i, (item, g, u) in enumerate(zip(items, gs, us)):
        _need(g, f"g[{i}]", torch.float32, shape, dev)
        _need(u, f"u[{i}]", torch.bfloat16, shape, dev)
        item.g, item.u = g.data_ptr(), u.data_ptr()
        if ms is not None:
            _need(ms[i], f"m[{i}]", torch.float32, shape, dev)
            _need(ms_out[i], f"m_out[{i}]", torch.float32, shape, dev)
            item.m, item.m_out = ms[i].data_ptr(), ms_out[i].data_ptr()
    hp = PuroNewtonSchulzParams(int(steps), int(bool(nesterov)), float(beta), float(scale),
                                (ctypes.c_float * 3)(*coefficients))
    need = lib().puro_newton_schulz_workspace(len(gs), rows, cols)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    with torch.cuda.device(dev):
        check(lib().puro_newton_schulz(items, len(gs), rows, cols, ctypes.byref(hp),
                                       workspace.data_ptr() or None, _stream(dev)))
    return us


# ---------------------------------------------------------------- output head
def _need_bf16_rows(x, name, dev):
    """_need_rows for bf16 alone; returns the row stride."""
    kind, ld = _need_rows(x, name, dev)
    if kind != TYPE_BF16:
        raise PuroError(f"{name}: dtype {x.dtype}, expected {torch.bfloat16}")
    return ld


def _head(h, w, targets):
    """Checks of the head's inputs; returns (device, tokens, d, vocab, ldh, ldw)."""
    dev = _dev(h)
    ldh = _need_bf16_rows(h, "h", dev)
    ldw = _need_bf16_rows(w, "w", dev)
    (tokens, d), vocab = h.shape, w.shape[0]
    if w.shape[1] != d:
        raise PuroError(f"w: shape {tuple(w.shape)}, expected {(vocab, d)}")
    _need(targets, "targets", torch.int64, (tokens,), dev)
    return dev, tokens, d, vocab, ldh, ldw


def _with_workspace(name, desc, workspace, dev) -> None:
    """Calls `name` with its structure and workspace, allocated if there is none."""
    need = getattr(lib(), name + "_workspace")(ctypes.byref(desc))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _need_workspace(workspace, need, dev)
    with torch.cuda.device(dev):
        check(getattr(lib(), name)(ctypes.byref(desc), workspace.data_ptr() or None, _stream(dev)))


def puro_linear_xent_fwd(h, w, targets, loss=None, lse=None, workspace=None):
    """Softmax cross entropy of hidden states h, bf16 [tokens, d], against the output head's weights
    w, bf16 [vocab, d] (rows of both may be strided), without the matrix of all logits -> (loss, lse),
    fp32 [tokens]. targets: int64 [tokens]; a target outside [0, vocab) is none (loss and lse 0)."""
    if loss is None or lse is None:
        tokens = _matrix(h, "h")[0]
        new = [torch.empty((tokens,), dtype=torch.float32, device=_dev(h)) for _ in range(2)]
        loss, lse = new[0] if loss is None else loss, new[1] if lse is None else lse
    if _done((_native or _load_native()).xent_fwd(h, w, targets, loss, lse, workspace)):
        return loss, lse
    dev, tokens, d, vocab, ldh, ldw = _head(h, w, targets)
    _need(loss, "loss", torch.float32, (tokens,), dev)
    _need(lse, "lse", torch.float32, (tokens,), dev)
    desc = PuroLinearXent(tokens, d, vocab, ldh, ldw, h.data_ptr(), w.data_ptr(),
                          targets.data_ptr(), loss.data_ptr(), lse.data_ptr())
    _with_workspace("puro_linear_xent_fwd", desc, workspace, dev)
    return loss, lse


def puro_linear_xent_bwd(h, w, targets, lse, dloss, dlse=None, dh=None, dw=None,
                         dw_dtype=torch.bfloat16, accumulate: bool = False, want_dh: bool = True,
                         want_dw: bool = True, workspace=None):
    """The gradients (dh bf16 [tokens, d], dw bf16 or fp32 [vocab, d]) from those of loss (dloss) and
    lse (dlse, or None), fp32 [tokens]. dw has dw_dtype, or the type of the dw given; accumulate
    adds to an existing fp32 dw. want_dh, want_dw: False leaves that gradient out (None)."""
    if accumulate and dw is None:
        raise PuroError("accumulate=True needs an existing dw")
    if isinstance(dw, torch.Tensor):
        dw_dtype = dw.dtype
    if dw_dtype not in _TYPES:
        raise PuroError(f"dw: dtype {dw_dtype}, expected bf16 or fp32")
    if not want_dh:
        dh = None
    elif dh is None:
        dh = torch.empty(_matrix(h, "h"), dtype=torch.bfloat16, device=_dev(h))
    if not want_dw:
        dw = None
    elif dw is None:
        dw = torch.empty(_matrix(w, "w"), dtype=dw_dtype, device=_dev(w))
    if _done((_native or _load_native()).xent_bwd(h, w, targets, lse, dloss, dlse, dh, dw,
                                                  accumulate, workspace)):
        return dh, dw
    dev, tokens, d, vocab, ldh, ldw = _head(h, w, targets)
    _need(lse, "lse", torch.float32, (tokens,), dev)
    _need(dloss, "dloss", torch.float32, (tokens,), dev)
    if dlse is not None:
        _need(dlse, "dlse", torch.float32, (tokens,), dev)
    if dh is not None:
        _need(dh, "dh", torch.bfloat16, (tokens, d), dev)
    if dw is not None:
        _need(dw, "dw", dw_dtype, (vocab, d), dev)
    desc = PuroLinearXentGrad(tokens, d, vocab, ldh, ldw, _TYPES[dw_dtype], int(bool(accumulate)),
                              h.data_ptr(), w.data_ptr(), targets.data_ptr(), lse.data_ptr(),
                              dloss.data_ptr(), None if dlse is None else dlse.data_ptr(),
                              None if dh is None else dh.data_ptr(),
                              None if dw is None else dw.data_ptr())
    _with_workspace("puro_linear_xent_bwd", desc, workspace, dev)
    return dh, dw


def _pow2_variant(base):
    name = base.__name__ + "_pow2"

    def f(*args, **kwargs):
        return base(*args, _fn=name, **kwargs)

    f.__name__ = name
    f.__doc__ = (base.__doc__ or "") + "\n\n    Power-of-two scales (the library's E8M0 variant)."
    return f


puro_quant_act_1x128_pow2 = _pow2_variant(puro_quant_act_1x128)
puro_quant_w_128x128_pow2 = _pow2_variant(puro_quant_w_128x128)
puro_quant_w_128x128_group_pow2 = _pow2_variant(puro_quant_w_128x128_group)
puro_quant_transpose_pow2 = _pow2_variant(puro_quant_transpose)
puro_quant_dual_1x128_pow2 = _pow2_variant(puro_quant_dual_1x128)
puro_fp8_gemm_fwd_pow2 = _pow2_variant(puro_fp8_gemm_fwd)
puro_fp8_gemm_dgrad_pow2 = _pow2_variant(puro_fp8_gemm_dgrad)
puro_fp8_gemm_wgrad_pow2 = _pow2_variant(puro_fp8_gemm_wgrad)


def puro_set_debug(level: int) -> None:
    """Debug level of the library (0: off; 1 or more: every quantiser and GEMM call checks its
    inputs on the device first and raises PuroError with PURO_ERR_INPUT on data outside the
    contract)."""
    lib().puro_set_debug(int(level))


def puro_debug_level() -> int:
    """Current debug level (initially the PURO_DEBUG environment variable, else 0)."""
    return int(lib().puro_debug_level())


def puro_gemm_kernel_name(op: str, M: int, N: int, K: int, pow2: bool = False) -> str:
    """Name of the kernel function puro_fp8_gemm_<op> (op: 'fwd', 'dgrad' or 'wgrad') launches
    for these sizes on the current device, or '' if it would launch nothing."""
    code = {"fwd": 0, "dgrad": 1, "wgrad": 2}[op]
    res = lib().puro_gemm_kernel_name(code, M, N, K, int(bool(pow2)))
    return res.decode() if res else ""


def prepare(name: str, *args, stream=None):
    """Pre-marshalled call of a C entry point for hot loops: tensors become raw device
    pointers, `stream` (a torch.cuda.Stream; default the current torch stream) is bound, and the
    returned zero-argument callable only crosses into the C ABI (which still validates) and
    checks the status."""
    fn = getattr(lib(), name)
    dev = None
    conv = []
    for a in args:
        if isinstance(a, torch.Tensor):
            dev = dev or a.device
            conv.append(a.data_ptr())
        else:
            conv.append(a)
    conv.append(stream.cuda_stream if stream is not None else _stream(dev))

    keep = tuple(args)  # tensors and ctypes arrays the raw arguments point into

    def call():
        # `keep` holds the tensors: their device memory must outlive every launch of this call
        # (including replays of a captured graph), not just the moment of preparation.
        st = fn(*conv)
        if st != 0:
            check(st)

    call.tensors = keep
    return call
