"""Which type the block norm's backward call takes the residual stream to have (no GPU)."""
import pytest
import torch

F32, BF16 = torch.float32, torch.bfloat16


def test_residual_type():
    from blockwise_fp8_gemm_x128_amd import PuroError
    from blockwise_fp8_gemm_x128_amd import binding
    full, half = torch.zeros((2, 2)), torch.zeros((2, 2), dtype=BF16)
    pair = (torch.zeros((2, 2), dtype=torch.uint8), torch.ones((1, 2)))
    res = binding._residual
    assert res(full, pair, None) is F32 and res(half, pair, None) is BF16
    assert res(None, full, None) is F32 and res(None, half, None) is BF16
    assert res(None, pair, F32) is F32 and res(None, pair, BF16) is BF16
    assert res(full, pair, F32) is F32
    with pytest.raises(PuroError, match="residual_dtype"):   # nothing says which it is
        res(None, pair, None)
    for args in ((full, pair, BF16), (None, half, F32), (None, pair, torch.float16)):
        with pytest.raises(PuroError, match="residual_dtype"):
            res(*args)
