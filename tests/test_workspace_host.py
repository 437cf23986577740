"""What the binding takes as scratch memory (no GPU): the kernels write the bytes behind the
tensor's address, so a view whose elements share bytes or lie apart is not what its size says."""
import pytest
import torch


@pytest.fixture
def need():
    from blockwise_fp8_gemm_x128_amd import binding
    return lambda t, n: binding._need_workspace(t, n, torch.device("cpu"))


def test_whole_buffers_are_taken(need):
    need(torch.empty(64, dtype=torch.uint8), 64)
    need(torch.empty((4, 4), dtype=torch.float32), 64)
    need(torch.empty(80, dtype=torch.uint8)[16:], 64)
    need(torch.empty(0, dtype=torch.uint8), 0)


@pytest.mark.parametrize("make", [
    lambda: torch.empty(63, dtype=torch.uint8),
    lambda: torch.empty(1, dtype=torch.uint8).expand(64),
    lambda: torch.empty((1, 8), dtype=torch.float32).expand(8, 8),
    lambda: torch.empty(128, dtype=torch.uint8)[::2],
    lambda: torch.empty((8, 8), dtype=torch.float32).t(),
    lambda: torch.empty((8, 8), dtype=torch.float32).to_sparse_csr(),
    lambda: torch.empty(64, dtype=torch.uint8, device="meta"),
    lambda: bytearray(64),
    lambda: 0x10000,
])
def test_views_and_others_are_refused(need, make):
    from blockwise_fp8_gemm_x128_amd import PuroError
    with pytest.raises(PuroError, match="workspace"):
        need(make(), 64)
