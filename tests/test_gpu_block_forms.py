"""The block norm in the combinations of stream type, stored form, gate and row layout that
test_gpu_block.py leaves out, each of which is a kernel or a path of its own: an fp32 stream from
checkpoints, a bf16 stream from stored activations, and every gate in every layout of a row over
lanes (16, 32 or 64 of a wave, one, groups of 16, whole waves, two vectors per lane)."""
import pytest
import torch

import test_gpu_block as block

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16

# rows, columns: one lane; 16, 32 and 64 lanes; groups; waves; waves with two vectors (forward from
# 6144 columns, backward from 8192), whole and ragged, several rows to a block
LAYOUTS = [(37, 5), (40, 100), (33, 256), (9, 500), (1303, 384), (1111, 1603), (17, 1000),
           (300, 2048), (6, 5123), (600, 7100), (3, 8203), (280, 9216)]


@pytest.mark.parametrize("rows,cols", LAYOUTS)
@pytest.mark.parametrize("res,saved", [(F32, "fp8"), (BF16, "asis")])
def test_backward_stored_forms(puro, rows, cols, res, saved):
    block.say("norm bwd", rows, cols, res, saved)
    d = block.bwd_inputs(puro, rows, cols, res, "channel", saved)
    v, e = block.bwd_ref(d, "channel", 0.75, 0.9375)
    block.check_bwd(block.bwd_call(puro, d, 0.75, 0.9375), v, e, res, "channel")


@pytest.mark.parametrize("rows,cols", LAYOUTS)
@pytest.mark.parametrize("kind", ["none", "token", "full"])
@pytest.mark.parametrize("res,saved", [(F32, "fp8"), (BF16, "asis")])
def test_backward_gates(puro, rows, cols, kind, res, saved):
    block.say("norm bwd", rows, cols, res, saved, kind)
    d = block.bwd_inputs(puro, rows, cols, res, kind, saved)
    v, e = block.bwd_ref(d, kind, 0.75, 0.9375)
    block.check_bwd(block.bwd_call(puro, d, 0.75, 0.9375), v, e, res, kind)


@pytest.mark.parametrize("rows,cols", LAYOUTS)
@pytest.mark.parametrize("half", ["post", "pre"])
@pytest.mark.parametrize("res,saved", [(F32, "fp8"), (BF16, "asis")])
def test_backward_halves(puro, rows, cols, half, res, saved):
    block.say("norm bwd", rows, cols, res, saved, half)
    d = block.bwd_inputs(puro, rows, cols, res, "full", saved, half)
    v, e = block.bwd_ref(d, "full", 1.5, 1.0)
    block.check_bwd(block.bwd_call(puro, d, 1.5, 1.0), v, e, res, "full")


@pytest.mark.parametrize("rows,cols", LAYOUTS)
@pytest.mark.parametrize("kind", ["none", "token", "full"])
@pytest.mark.parametrize("res", [BF16, F32])
def test_forward_gates(puro, rows, cols, kind, res):
    block.check_fwd(puro, rows, cols, res, kind, "both", True, kind == "token")


@pytest.mark.parametrize("rows,cols", LAYOUTS)
@pytest.mark.parametrize("half", ["post", "pre"])
def test_forward_halves(puro, rows, cols, half):
    block.check_fwd(puro, rows, cols, F32, "full", "both", True, False, half)
    block.check_fwd(puro, rows, cols, BF16, "token", "bf16", False, False, half)
