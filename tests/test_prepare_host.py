"""The binding's pre-marshalled calls (no GPU): which stream they are bound to."""
import types

import torch


def test_prepare_without_a_tensor_takes_the_current_stream(monkeypatch):
    """A call whose tensors are all inside a ctypes array names no device: the current device's
    current stream is the one it runs on."""
    from blockwise_fp8_gemm_x128_amd import binding
    got = []
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(
        cuda_stream=0x1230 if dev is None else 0))
    monkeypatch.setattr(binding, "lib", lambda: types.SimpleNamespace(
        puro_quant_w_128x128_group=lambda *a: got.append(a) or 0))
    items = binding.w_group_items([], [], [])
    binding.prepare("puro_quant_w_128x128_group", items, 0)()
    assert got == [(items, 0, 0x1230)]
