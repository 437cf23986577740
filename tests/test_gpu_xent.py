"""The output head's cross entropy on the GPU, forward and backward, against the definitions in 64
bits (tests/head_ref.py, which derives the bounds)."""
import pytest
import torch

import head_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# (tokens, d, vocab): a single one of each, sizes that end inside a tile, a chunk or an 8-byte group, and
# each tile shape
SIZES = [(1, 64, 1), (1, 1, 1), (1, 64, 100), (2, 8, 3), (3, 8, 257), (5, 1, 7), (64, 72, 300),
         (65, 128, 511), (127, 200, 1000), (130, 64, 4097), (257, 320, 2050), (300, 1001, 777),
         (33, 2048, 5000), (64, 136, 33000), (700, 136, 9001)]
BIG = (2061, 136, 8269)     # as many 256x256 tiles as the chip has compute units


def draw(tokens, d, vocab, seed=0, masked=0.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 1000 * tokens + 10 * d + vocab)
    w = (torch.randn((vocab, d), generator=g, device=DEV) * d ** -0.5).bfloat16()
    y = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    h = (torch.randn((tokens, d), generator=g, device=DEV)
         + 8 * torch.rand((tokens, 1), generator=g, device=DEV) * w[y].float()).bfloat16()
    if masked:
        y[torch.rand(tokens, generator=g, device=DEV) < masked] = -100
    dloss = (0.5 + torch.rand(tokens, generator=g, device=DEV)) / tokens
    dlse = torch.randn(tokens, generator=g, device=DEV) / tokens
    return h, w, y, dloss, dlse


def within(got, want, bound, what):
    bad = (got.double() - want).abs() > bound
    assert not bool(bad.any()), "%s: %d of %d, worst %.3g of its bound" % (
        what, int(bad.sum()), bad.numel(),
        float(((got.double() - want).abs() / bound.clamp_min(1e-300)).max()))


def check_fwd(out, h, w, y):
    loss, lse, bl, be = head_ref.xent_fwd(h, w, y)
    within(out[1], lse, be, "lse")
    within(out[0], loss, bl, "loss")


def check_bwd(out, h, w, y, lse, dloss, dlse, before=None):
    dh, dw, bh, bw = head_ref.xent_bwd(h, w, y, lse, dloss, dlse, before)
    if out[0] is not None:
        within(out[0], dh, bh, "dh")
    if out[1] is not None:
        if out[1].dtype == torch.bfloat16:
            bw = bw + 2.0 ** -8 * (dw.abs() + bw)
        within(out[1], dw, bw, "dw")


def saved_lse(h, w, y):
    return head_ref.xent_fwd(h, w, y)[1].float()


@pytest.mark.parametrize("size", SIZES + [BIG], ids=str)
def test_forward(puro, size):
    h, w, y, _, _ = draw(*size)
    check_fwd(puro.puro_linear_xent_fwd(h, w, y), h, w, y)


@pytest.mark.parametrize("dw_dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("size", SIZES + [BIG], ids=str)
def test_backward(puro, size, dw_dtype):
    h, w, y, dloss, dlse = draw(*size)
    lse = saved_lse(h, w, y)
    out = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse, dw_dtype=dw_dtype)
    assert out[1].dtype == dw_dtype
    check_bwd(out, h, w, y, lse, dloss, dlse)


@pytest.mark.parametrize("size", [(70001, 64, 9000), (70001, 24, 4097)], ids=str)
def test_several_pieces(puro, size):
    """More tokens than one piece of the vocabulary holds; the last piece is short."""
    h, w, y, dloss, dlse = draw(*size, masked=0.1)
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    check_fwd((loss, lse), h, w, y)
    check_bwd(puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse), h, w, y, lse, dloss, dlse)


@pytest.mark.parametrize("size", [(3, 8, 257), (65, 128, 511), (300, 72, 777)], ids=str)
def test_backward_without_the_log_sum_exps_gradient(puro, size):
    h, w, y, dloss, _ = draw(*size, masked=0.5)
    lse = saved_lse(h, w, y)
    check_bwd(puro.puro_linear_xent_bwd(h, w, y, lse, dloss), h, w, y, lse, dloss, None)


@pytest.mark.parametrize("size", [(65, 128, 511), (64, 72, 300), BIG], ids=str)
def test_one_gradient_alone(puro, size):
    h, w, y, dloss, dlse = draw(*size)
    lse = saved_lse(h, w, y)
    both = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse)
    dh, none = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse, want_dw=False)
    assert none is None and torch.equal(dh, both[0])
    none, dw = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse, want_dh=False)
    assert none is None and torch.equal(dw, both[1])


@pytest.mark.parametrize("size", [(65, 128, 511), (30, 37, 45), BIG], ids=str)
def test_accumulated_dw(puro, size):
    h, w, y, dloss, dlse = draw(*size)
    lse = saved_lse(h, w, y)
    dw = torch.randn((size[2], size[1]), device=DEV) * 0.01
    before = dw.clone()
    out = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse, dw=dw, accumulate=True)
    assert out[1] is dw
    check_bwd(out, h, w, y, lse, dloss, dlse, before)


@pytest.mark.parametrize("size", [(5, 8, 40), (130, 64, 300), (300, 33, 777), BIG], ids=str)
def test_tokens_without_target(puro, size):
    """Any target outside the vocabulary is none, and nothing in such a token's row matters."""
    tokens, d, vocab = size
    h, w, y, dloss, dlse = draw(*size)
    for k, t in enumerate((-1, -100, vocab, vocab + 5, 2 ** 62, -2 ** 62)):
        y[k::17] = t
    off = (y < 0) | (y >= vocab)
    h[off] = float("nan")
    h[off.nonzero()[0]] = float("inf")
    dloss[off] = float("nan")
    dlse[off] = float("inf")
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    assert bool((loss[off] == 0).all()) and bool((lse[off] == 0).all())
    clean = torch.where(off[:, None], torch.zeros_like(h), h)
    check_fwd((loss, lse), clean, w, y)
    lse[off] = float("nan")
    dh, dw = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse)
    assert bool((dh[off] == 0).all())
    check_bwd((dh, dw), clean, w, y, lse, dloss, dlse)


@pytest.mark.parametrize("size", [(1, 8, 9), (70, 64, 300), BIG], ids=str)
def test_no_token_has_a_target(puro, size):
    h, w, y, dloss, dlse = draw(*size)
    y.fill_(-100)
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    assert not bool(loss.any()) and not bool(lse.any())
    dh, dw = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse)
    assert not bool(dh.any()) and not bool(dw.any())


def test_without_tokens(puro):
    h = torch.empty((0, 24), dtype=torch.bfloat16, device=DEV)
    w = torch.ones((5, 24), dtype=torch.bfloat16, device=DEV)
    y = torch.empty(0, dtype=torch.int64, device=DEV)
    f = torch.empty(0, device=DEV)
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    assert loss.shape == (0,) and lse.shape == (0,)
    for dtype in (torch.bfloat16, torch.float32):
        for d in (24, 1, 3):
            dw = torch.ones((5, d), dtype=dtype, device=DEV)
            dh, out = puro.puro_linear_xent_bwd(h[:, :d], w[:, :d], y, f, f, dw=dw)
            assert dh.shape == (0, d) and out is dw and not bool(dw.any())
    dw = torch.ones((5, 24), device=DEV)
    puro.puro_linear_xent_bwd(h, w, y, f, f, dw=dw, accumulate=True)
    assert bool((dw == 1).all())


LAYOUTS = {"stride": (136, 0), "odd stride": (131, 0), "offset 8": (136, 8), "offset 1": (136, 1)}


@pytest.mark.parametrize("hl", LAYOUTS)
@pytest.mark.parametrize("wl", LAYOUTS)
def test_strided_rows(puro, hl, wl):
    """Rows of wider matrices, with NaN between them, at addresses and strides that are read as they
    lie and that are not: the same results as from dense ones."""
    def lay(x, kind):
        ld, off = LAYOUTS[kind]
        wide = torch.full((x.shape[0], ld + 8), float("nan"), dtype=x.dtype, device=DEV)
        flat = wide.view(-1)[:x.shape[0] * ld + 8].as_strided((x.shape[0], x.shape[1]), (ld, 1), off)
        flat.copy_(x)
        return flat

    h, w, y, dloss, dlse = draw(77, 120, 301)
    lse = saved_lse(h, w, y)
    hs, ws = lay(h, hl), lay(w, wl)
    for a, b in zip(puro.puro_linear_xent_fwd(hs, ws, y), puro.puro_linear_xent_fwd(h, w, y)):
        assert torch.equal(a, b)
    for a, b in zip(puro.puro_linear_xent_bwd(hs, ws, y, lse, dloss, dlse),
                    puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse)):
        assert torch.equal(a, b)


def test_infinite_and_nan_logits(puro):
    h, w, y, dloss, _ = draw(70, 16, 600)
    w[:, 0] = 0
    w[7, 0] = 3e38                 # one vocabulary entry that overflows where h's first entry is large
    h[:, 0] = 0
    h[3, 0] = 3e38                 # +inf: the sum is infinite over infinite
    h[4, 0] = -3e38                # -inf: the entry drops out
    h[5, 1] = float("nan")
    y[3:6] = 2
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    l = h.float() @ w.float().t()
    assert bool(l[3, 7] == float("inf")) and bool(l[4, 7] == -float("inf"))
    assert bool(loss[3].isnan()) and bool(lse[3].isnan() | lse[3].isinf())
    assert bool(loss[5].isnan()) and bool(lse[5].isnan())
    want = torch.logsumexp(l[4].double(), 0)
    assert abs(float(lse[4]) - float(want)) < 1e-4
    keep = [i for i in range(70) if i not in (3, 4, 5)]
    check_fwd((loss[keep], lse[keep]), h[keep], w, y[keep])
    # backward: those tokens' rows are NaN or whole, the others' stay theirs
    y[3] = y[5] = -1
    lse = torch.where(y >= 0, torch.logsumexp(l, 1), torch.zeros(70, device=DEV))
    dh, dw = puro.puro_linear_xent_bwd(h, w, y, lse, dloss)
    assert bool(dh.isfinite()[keep].all())
    _, _, bh, _ = head_ref.xent_bwd(h[keep], w, y[keep], lse[keep], dloss[keep], None)
    want = head_ref.xent_bwd(h[keep], w, y[keep], lse[keep], dloss[keep], None)[0]
    within(dh[keep], want, bh, "dh")


def test_outputs_stay_in_their_place(puro):
    """Outputs in the middle of larger buffers: what lies around them stays."""
    for size in [(5, 8, 40), (130, 33, 301), (64, 72, 300)]:
        tokens, d, vocab = size
        h, w, y, dloss, dlse = draw(*size)
        lse0 = saved_lse(h, w, y)

        def inside(shape, dtype):
            n = 1
            for k in shape:
                n *= k
            buf = torch.full((n + 4096,), 7.0, dtype=dtype, device=DEV)
            return buf, buf[2048:2048 + n].view(shape)

        loss, lse = inside((tokens,), torch.float32), inside((tokens,), torch.float32)
        puro.puro_linear_xent_fwd(h, w, y, loss=loss[1], lse=lse[1])
        for dtype in (torch.bfloat16, torch.float32):
            dh, dw = inside((tokens, d), torch.bfloat16), inside((vocab, d), dtype)
            puro.puro_linear_xent_bwd(h, w, y, lse0, dloss, dlse, dh=dh[1], dw=dw[1])
            for buf, view in (loss, lse, dh, dw):
                n = view.numel()
                assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + n:] == 7).all())


def test_workspace_of_the_callers(puro):
    """A workspace of exactly the bytes that are asked for, full of NaN, used twice."""
    import ctypes
    from blockwise_fp8_gemm_x128_amd._lib import PuroLinearXent, PuroLinearXentGrad
    h, w, y, dloss, dlse = draw(90, 30, 400)
    lse = saved_lse(h, w, y)
    p = [t.data_ptr() for t in (h, w, y, lse, dloss)]
    n1 = puro.lib().puro_linear_xent_fwd_workspace(ctypes.byref(
        PuroLinearXent(90, 30, 400, 30, 30, p[0], p[1], p[2], p[3], p[3])))
    n2 = puro.lib().puro_linear_xent_bwd_workspace(ctypes.byref(
        PuroLinearXentGrad(90, 30, 400, 30, 30, 0, 0, p[0], p[1], p[2], p[3], p[4], None, p[0],
                           p[1])))
    for n, call in ((n1, lambda ws: puro.puro_linear_xent_fwd(h, w, y, workspace=ws)),
                    (n2, lambda ws: puro.puro_linear_xent_bwd(h, w, y, lse, dloss, workspace=ws))):
        buf = torch.full((n + 512,), 255, dtype=torch.uint8, device=DEV)
        want = call(None)
        for _ in range(2):
            for a, b in zip(call(buf[256:256 + n]), want):
                assert torch.equal(a, b)
        assert bool((buf[:256] == 255).all()) and bool((buf[256 + n:] == 255).all())
        with pytest.raises(Exception, match="workspace"):
            call(buf[256:256 + n - 1])


@pytest.mark.parametrize("size", [(64, 72, 300), (300, 72, 777), BIG], ids=str)
def test_repeats_exactly(puro, size):
    h, w, y, dloss, dlse = draw(*size, masked=0.1)
    first = [*puro.puro_linear_xent_fwd(h, w, y)]
    first += puro.puro_linear_xent_bwd(h, w, y, first[1], dloss, dlse)
    for _ in range(3):
        again = [*puro.puro_linear_xent_fwd(h, w, y)]
        again += puro.puro_linear_xent_bwd(h, w, y, again[1], dloss, dlse)
        assert all(torch.equal(a, b) for a, b in zip(first, again))


def test_two_streams_at_once(puro):
    sets = [draw(300, 72, 777, seed=k) for k in range(2)]
    lses = [saved_lse(*s[:3]) for s in sets]
    want = [puro.puro_linear_xent_bwd(*s[:3], l, *s[3:]) for s, l in zip(sets, lses)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    outs = []
    for _ in range(5):
        for s, l, st in zip(sets, lses, streams):
            with torch.cuda.stream(st):
                outs.append(puro.puro_linear_xent_bwd(*s[:3], l, *s[3:]))
    torch.cuda.synchronize()
    for k, o in enumerate(outs):
        assert torch.equal(o[0], want[k % 2][0]) and torch.equal(o[1], want[k % 2][1])


def test_captured_and_replayed(puro):
    h, w, y, dloss, dlse = draw(300, 72, 777, masked=0.2)
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    dh, dw = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        puro.puro_linear_xent_fwd(h, w, y, loss=loss, lse=lse)
        puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse, dh=dh, dw=dw)
    for k in range(4):
        other = draw(300, 72, 777, seed=k + 1, masked=0.2)
        for a, b in zip((h, w, y, dloss, dlse), other):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        want = [*puro.puro_linear_xent_fwd(h, w, y)]
        want += puro.puro_linear_xent_bwd(h, w, y, want[1], dloss, dlse)
        for a, b in zip((loss, lse, dh, dw), want):
            assert torch.equal(a, b)


def test_refusals_of_the_binding(puro):
    h, w, y, dloss, dlse = draw(9, 16, 40)
    lse = saved_lse(h, w, y)
    bad = [lambda: puro.puro_linear_xent_fwd(h.float(), w, y),
           lambda: puro.puro_linear_xent_fwd(h, w.float(), y),
           lambda: puro.puro_linear_xent_fwd(h, w[:, :8], y),
           lambda: puro.puro_linear_xent_fwd(h, w, y.int()),
           lambda: puro.puro_linear_xent_fwd(h, w, y[:-1]),
           lambda: puro.puro_linear_xent_fwd(h.t(), w, y),
           lambda: puro.puro_linear_xent_fwd(h[0], w, y),
           lambda: puro.puro_linear_xent_fwd(h, w[:0], y),
           lambda: puro.puro_linear_xent_fwd(h, w, y, loss=torch.empty(9)),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse.double(), dloss),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse, dloss[:-1]),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse.half()),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse, dloss, accumulate=True),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dw_dtype=torch.float16),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse, dloss, accumulate=True,
                                             dw=torch.zeros_like(w)),
           lambda: puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dh=torch.zeros_like(h).float())]
    for call in bad:
        with pytest.raises(puro.PuroError):
            call()


# weights past 2^32 bytes, and a piece of P past them
@pytest.mark.parametrize("size", [(3, 2048, 1100003), (540001, 64, 4100)], ids=str)
def test_offsets_past_32_bits(puro, size):
    h, w, y, dloss, dlse = draw(*size)
    y[-1] = size[2] - 1
    loss, lse = puro.puro_linear_xent_fwd(h, w, y)
    check_fwd((loss, lse), h, w, y)
    out = puro.puro_linear_xent_bwd(h, w, y, lse, dloss, dlse)
    check_bwd(out, h, w, y, lse, dloss, dlse)
