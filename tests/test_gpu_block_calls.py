"""GPU tests of how the binding makes its calls: what it refuses, which stream and which types it
takes where the arguments leave them open."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16


def rnd(shape, seed, dtype=F32, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).to(DEV)


@pytest.mark.parametrize("make", [
    lambda n: torch.empty(n - 1, dtype=torch.uint8, device=DEV),
    lambda n: torch.empty(1, dtype=torch.uint8, device=DEV).expand(n),
    lambda n: torch.empty(2 * n, dtype=torch.uint8, device=DEV)[::2],
    lambda n: torch.empty(n, dtype=torch.uint8),
    lambda n: bytearray(n),
])
def test_norm_bwd_workspace_views_are_refused(puro, make):
    """Scratch memory that has fewer bytes behind its address than the kernels write."""
    from blockwise_fp8_gemm_x128_amd import PuroError
    rows, cols = 64, 512
    x, w, rstd = rnd((rows, cols), 1, BF16), rnd((cols,), 2), torch.ones(rows, device=DEV)
    need = puro.lib().puro_block_norm_workspace(rows, cols)
    assert need >= 2 * cols * 4
    args = (x, x, x, x, rstd, rstd, w, w)
    with pytest.raises(PuroError, match="workspace"):
        puro.puro_block_norm_bwd(*args, workspace=make(need))
    a = puro.puro_block_norm_bwd(*args)
    b = puro.puro_block_norm_bwd(*args, workspace=torch.empty(need // 4, device=DEV))
    assert all(torch.equal(x, y) for x, y in zip(a, b) if x is not None)


def test_optimizer_workspace_is_checked(puro):
    from blockwise_fp8_gemm_x128_amd import PuroError
    w = rnd((64, 64), 3)
    whole = puro.optim_workspace(DEV)
    norm = puro.puro_frobenius_norm(w, workspace=whole)
    assert torch.equal(norm, puro.puro_frobenius_norm(w))
    u, radius = rnd((64, 64), 4), norm.clone()
    before = w.clone()
    for bad in (whole[:-1], whole[:1].expand(whole.numel()), whole.cpu(), bytearray(whole.numel())):
        with pytest.raises(PuroError, match="workspace"):
            puro.puro_frobenius_norm(w, workspace=bad)
        with pytest.raises(PuroError, match="workspace"):
            puro.puro_hyperball_step(w, u, 0.1, radius, workspace=bad)
    assert torch.equal(w, before)
    puro.puro_hyperball_step(w, u, 0.1, radius, workspace=whole)
    puro.puro_hyperball_step(before, u, 0.1, radius)
    assert torch.equal(w, before)


def test_prepared_group_call_without_a_tensor(puro):
    """prepare() of a call whose tensors are inside a ctypes array, on the current stream."""
    ws = [rnd((128, 256), 5, BF16), rnd((256, 128), 6, BF16)]
    want_q, want_s = puro.puro_quant_w_128x128_group(ws)
    qs, ss = [torch.zeros_like(q) for q in want_q], [torch.zeros_like(s) for s in want_s]
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    for stream in (torch.cuda.current_stream(), st):
        with torch.cuda.stream(stream):
            call = puro.prepare("puro_quant_w_128x128_group", puro.w_group_items(ws, qs, ss), 2)
            for t in (*qs, *ss):
                t.zero_()
            call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((*qs, *ss), (*want_q, *want_s)))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_residual_type_of_the_last_boundary(puro, dtype):
    """From checkpoints and without a gradient of the stream nothing says the stream's type: it is
    asked for, and dr has it. Its values are those with a gradient of zeros, and fp32 ones are
    not rounded to bf16: against 64 bits within the bound that block_ref derives."""
    import block_ref as ref
    from blockwise_fp8_gemm_x128_amd import PuroError
    rows, cols = 40, 384
    y, r = rnd((rows, cols), 7, BF16), rnd((rows, cols), 8, dtype)
    wo, wp, dn = rnd((cols,), 9), rnd((cols,), 10), rnd((rows, cols), 11, BF16, 1e-3)
    o = puro.puro_block_norm_fwd(y, r, wo, wp)
    saved = ((o.yq, o.ys), (o.rq, o.rs), o.rstd_y, o.rstd_r, wo, wp)
    with pytest.raises(PuroError, match="residual_dtype"):
        puro.puro_block_norm_bwd(None, dn, *saved)
    with pytest.raises(PuroError, match="residual_dtype"):
        puro.puro_block_norm_bwd(None, dn, *saved, residual_dtype=torch.float16)
    with pytest.raises(PuroError, match="residual_dtype"):
        puro.puro_block_norm_bwd(torch.zeros_like(r), dn, *saved,
                                 residual_dtype=F32 if dtype is BF16 else BF16)
    a = puro.puro_block_norm_bwd(None, dn, *saved, residual_dtype=dtype)
    b = puro.puro_block_norm_bwd(torch.zeros_like(r), dn, *saved)
    assert a.dr.dtype == b.dr.dtype == dtype
    assert all(torch.equal(x, z) for x, z in zip(a[:4], b[:4]))
    c = puro.puro_block_norm_bwd(None, dn, *saved, out=b, residual_dtype=dtype)
    assert c.dr is b.dr and torch.equal(c.dr, a.dr)
    with pytest.raises(PuroError, match="residual_dtype"):
        puro.puro_block_norm_bwd(None, dn, *saved, out=b,
                                 residual_dtype=F32 if dtype is BF16 else BF16)
    v, e = ref.norm_bwd(None, ref.f64(dn), ref.f64(ref.decode32(o.yq, o.ys)),
                        ref.f64(ref.decode32(o.rq, o.rs)), ref.f64(o.rstd_y), ref.f64(o.rstd_r),
                        ref.f64(wo), ref.f64(wp), ref.gate64(None), 1.0, 1.0, None)
    ref.close(a.dr, v["dr"], e["dr"] + ref.out_err(v["dr"], dtype) * 1.01, "dr")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_stack_keeps_the_streams_type(puro, dtype):
    """The gradient of an fp32 residual stream stays in fp32 through every boundary: it has bits
    that bf16 has not."""
    from blockwise_fp8_gemm_x128_amd.mlp_stack import MlpStack
    stack = MlpStack(2, 256, 128, seed=3)
    n, kept = stack.forward(rnd((128, 256), 12, dtype))
    dr, _, _ = stack.backward(rnd((128, 256), 13, BF16), kept)
    assert n.dtype == BF16 and dr.dtype == dtype
    if dtype == F32:
        assert not torch.equal(dr, dr.to(BF16).float())


def test_gate_per_token_without_columns(puro):
    """A sum over no columns: zero, and not what the memory held."""
    e, rstd = torch.empty((5, 0), dtype=BF16, device=DEV), torch.ones(5, device=DEV)
    w, gate = torch.empty(0, device=DEV), torch.ones((5, 1), device=DEV)
    out = puro.BlockNormGrads(torch.empty_like(e), torch.empty_like(e), torch.empty_like(w),
                              torch.empty_like(w), torch.full((5, 1), 7.0, device=DEV))
    g = puro.puro_block_norm_bwd(e, e, e, e, rstd, rstd, w, w, gate, out=out)
    assert torch.all(g.dgate == 0)
    for other in (None, w, e):                              # no gate, one per column, per element
        o = puro.puro_block_norm_fwd(e, e, w, w, other)
        assert o.r_out.shape == (5, 0)
        g = puro.puro_block_norm_bwd(e, e, e, e, rstd, rstd, w, w, other)
        assert g.dr.shape == (5, 0) and g.dw_pre.shape == (0,)
    big = puro.BlockNormGrads(None, torch.empty((300000, 0), dtype=BF16, device=DEV), None, None,
                              torch.full((300001, 1), 7.0, device=DEV)[:300000])
    e = torch.empty((300000, 0), dtype=BF16, device=DEV)
    rstd, gate = torch.ones(300000, device=DEV), torch.ones((300000, 1), device=DEV)
    puro.puro_block_norm_bwd(e, e, (e.view(torch.uint8), torch.empty((0, 300000), device=DEV)),
                             (e.view(torch.uint8), torch.empty((0, 300000), device=DEV)), rstd,
                             rstd, w, w, gate, out=big)
    assert torch.all(big.dgate == 0)


@pytest.mark.parametrize("pow2", [False, True])
def test_operators_write_the_quantisers_bytes(puro, pow2):
    """Where the input of a code is exact, its bytes are the quantisers': the activation's checkpoint
    and the norm's of its input against the activation quantiser; a forward operand that stands
    for a matrix exactly, requantised along its rows, against the transposing quantiser of that
    matrix."""
    sfx = "_pow2" if pow2 else ""
    act, turn = (getattr(puro, n + sfx) for n in ("puro_quant_act_1x128", "puro_quant_transpose"))
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731
    rows, f = 384, 640
    gu = rnd((rows, 2 * f), 14, BF16, 3.0)
    gu[5] = 0.0
    o = puro.puro_swiglu_fwd(gu, pow2=pow2)
    for i in range(2):
        q, s = act(gu[:, i * f:(i + 1) * f].contiguous())
        assert same(o.guq[:, i * f:(i + 1) * f].contiguous(), q)
        assert same(o.gus[i * f // 128:(i + 1) * f // 128].contiguous(), s)
    y, w = gu[:, :f].contiguous(), rnd((f,), 15)
    n = puro.puro_block_norm_fwd(y, y, w, w, pow2=pow2)
    q, s = act(y)
    assert same(n.yq, q) and same(n.ys, s)
    # E4M3 values times a power of two per row, 448 among them in every group: the scale is that
    # power, under either rule, and every value is what its code stands for
    codes = torch.randint(0, 256, (rows, f), generator=torch.Generator().manual_seed(16))
    codes[(codes & 0x7F) == 0x7F] = 0x38
    codes[:, ::128] = 0x7E
    power = torch.exp2(torch.arange(rows) % 9 - 4.0)[:, None]
    x = (codes.to(torch.uint8).view(torch.float8_e4m3fn).float() * power).to(BF16).to(DEV)
    q, s = act(x)
    assert torch.equal(q.cpu().int(), codes.int())
    assert torch.equal(s.cpu(), power.t().expand(f // 128, rows))
    for a, b in zip(puro.puro_ckpt_transpose(q, s, pow2=pow2), turn(x)):
        assert same(a, b)
