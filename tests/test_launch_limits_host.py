"""Refusal of sizes whose launch would have 2^32 threads or more (no GPU): HIP takes such a launch
and runs only the blocks that are left of the thread count modulo 2^32, so the call would return
PURO_OK with most of its output unwritten. No call here reaches a kernel launch."""
import os

import pytest

SHAPE = 2
P = 0x10000   # never dereferenced: every call below fails validation first
MAX = 1 << 24


@pytest.fixture(scope="module")
def L():
    from blockwise_fp8_gemm_x128_amd import _lib
    from blockwise_fp8_gemm_x128_amd.build import LIB_PATH, build
    if not os.path.exists(LIB_PATH):
        build(verbose=False)
    lib = _lib.lib()
    level = lib.puro_debug_level()   # debug mode would look at the inputs first
    lib.puro_set_debug(0)
    yield lib
    lib.puro_set_debug(level)


# 256 threads for 16 rows x 256 columns: 2^20 row tiles x 16 column tiles are 2^24 blocks, 2^32
# threads; one column more is 17 column tiles, the thread count modulo 2^32 positive. 512 threads
# for 128 x 128: 2^17 x 64 tiles are 2^23 blocks.
@pytest.mark.parametrize("cols", [4096, 4097])
def test_elementwise_calls_past_the_thread_limit(L, cols):
    for kind in (0, 1):
        assert L.puro_ckpt_pack(P, kind, MAX, cols, cols, 0, P, P, None) == SHAPE
        assert L.puro_ckpt_unpack(P, P, MAX, cols, P, kind, cols, None) == SHAPE
    assert L.puro_swiglu_fwd(P, MAX, cols, P, P, P, P, P, 0, None) == SHAPE
    assert L.puro_swiglu_bwd(P, P, None, None, MAX, cols, P, None) == SHAPE
    assert L.puro_swiglu_bwd(P, None, P, P, MAX, cols, P, None) == SHAPE


@pytest.mark.parametrize("cols", [8192, 8192 + 128])
def test_tiled_calls_past_the_thread_limit(L, cols):
    assert L.puro_ckpt_transpose(P, P, MAX, cols, 0, P, P, None) == SHAPE
    assert L.puro_ckpt_transpose(P, P, cols, MAX, 0, P, P, None) == SHAPE
    for gu in ((P, None, None), (None, P, P)):
        assert L.puro_swiglu_bwd_fp8(P, *gu, MAX, cols, 0, *((P,) * 6), None) == SHAPE
        assert L.puro_swiglu_bwd_fp8(P, *gu, cols, MAX, 0, *((P,) * 6), None) == SHAPE


@pytest.mark.parametrize("sfx", ["", "_pow2"])
def test_quantisers_past_the_thread_limit(L, sfx):
    """256 threads for 64 x 128 (activations) and 128 x 128 (weights), 512 for 128 x 128 (column
    groups)."""
    from blockwise_fp8_gemm_x128_amd._lib import PuroWItem
    call = lambda name: getattr(L, name + sfx)  # noqa: E731
    for n in (1 << 13, (1 << 13) + 128):
        assert call("puro_quant_act_1x128")(P, MAX, n, P, P, None) == SHAPE
        assert call("puro_quant_transpose")(P, MAX, n, P, P, None) == SHAPE
        assert call("puro_quant_dual_1x128")(P, MAX, n, P, P, P, P, None) == SHAPE
        assert call("puro_quant_w_128x128")(P, MAX, 2 * n, P, P, None) == SHAPE
        items = (PuroWItem * 2)(*(PuroWItem(P, MAX, n, P, P) for _ in range(2)))
        assert call("puro_quant_w_128x128_group")(items, 2, None) == SHAPE


@pytest.mark.parametrize("sfx", ["", "_pow2"])
def test_gemms_past_the_thread_limit(L, sfx):
    """2^24 x 2^17 outputs are 2^25 tiles of 256 x 256, the largest, of 256 threads or more."""
    n = 1 << 17
    assert getattr(L, "puro_fp8_gemm_fwd" + sfx)(P, P, P, P, P, MAX, n, 128, None) == SHAPE
    assert getattr(L, "puro_fp8_gemm_dgrad" + sfx)(P, P, P, P, P, MAX, 128, n, None) == SHAPE
    assert getattr(L, "puro_fp8_gemm_wgrad" + sfx)(P, P, P, P, P, 128, MAX, n, 0, None) == SHAPE


def test_norm_without_columns(L):
    """Empty tensors may have no address: that of the weight after the block does not say that its
    half was left out."""
    import ctypes

    from blockwise_fp8_gemm_x128_amd._lib import PuroBlockNorm, PuroBlockNormGrad
    for kind in range(4):
        sizes = dict(rows=8, cols=0, gate_kind=kind, alpha=1.0, beta=1.0, gate=P)
        d = PuroBlockNorm(eps=1e-6, rstd_y=P, rstd_r=P, **sizes)
        assert L.puro_block_norm_fwd(ctypes.byref(d), None) == 0
        if kind != 2:
            assert L.puro_block_norm_bwd(ctypes.byref(PuroBlockNormGrad(**sizes)), None, None) == 0


def test_gate_per_token_without_columns(L):
    """Its gradient, a sum over no columns, is zero and has to be written: its address is checked."""
    import ctypes

    from blockwise_fp8_gemm_x128_amd._lib import PuroBlockNormGrad
    for status, dgate in ((1, None), (3, P + 1)):
        d = PuroBlockNormGrad(rows=8, cols=0, gate_kind=2, alpha=1.0, beta=1.0, w_post=P, gate=P,
                              dgate=dgate)
        assert L.puro_block_norm_bwd(ctypes.byref(d), P, None) == status
