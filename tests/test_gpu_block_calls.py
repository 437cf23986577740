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
