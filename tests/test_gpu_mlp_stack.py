"""The stack of MLP blocks that runs the operators between the GEMMs together with the GEMMs: its
output and every gradient against the same network in float64 autograd on the CPU, and that it
learns.

Tolerance: each FP8 rounding on a path is a relative error of at most 2^-4 and, over the roughly
uniform positions between two codes, 2^-4/sqrt(3) = 0.036 in the mean square. A gradient of the
two-block stack passes, through its forward and backward pass, at most 8 roundings per block (n, the
weight, h, y and r as stored, gu as stored, dy, dgu) and as many again in the blocks between it and
the loss: rounding errors that are independent add to 0.036 sqrt(16) = 0.15 of the tensor's norm.
0.2 leaves a third for their being correlated. The output passes the forward half only: 0.1."""
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def rms_norm(x, w, eps):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + eps) * w


def reference(stack, r):
    """Output and gradients of sum(n * t) for a fixed t, in float64 autograd."""
    leaf = lambda x: x.detach().double().cpu().requires_grad_()  # noqa: E731
    r0, w0 = leaf(r), leaf(stack.w_first)
    params = [[leaf(x) for x in (p.wgu16, p.wd16, p.w_post, p.gate, p.w_pre)]
              for p in stack.layers]
    x, n = r0, rms_norm(r0, w0, stack.eps)
    for wgu, wd, w_post, gate, w_pre in params:
        g, u = (n @ wgu.t()).chunk(2, 1)
        y = (torch.nn.functional.silu(g) * u) @ wd.t()
        x = stack.beta * x + stack.alpha * gate * rms_norm(y, w_post, stack.eps)
        n = rms_norm(x, w_pre, stack.eps)
    return r0, w0, params, n


def test_stack_against_float64_autograd(puro):
    from blockwise_fp8_gemm_x128_amd.mlp_stack import MlpStack
    stack = MlpStack(2, 256, 384, seed=3, alpha=0.75, beta=0.9375)
    g = torch.Generator().manual_seed(5)
    r = torch.randn((256, 256), generator=g).bfloat16().cuda()
    t = torch.randn((256, 256), generator=g).bfloat16().cuda()
    n, kept = stack.forward(r)
    dr, dw_first, grads = stack.backward(t, kept)
    r0, w0, params, want = reference(stack, r)
    (want * t.double().cpu()).sum().backward()

    def rel(got, ref):
        ref = ref.detach()
        return float((got.double().cpu() - ref).norm() / ref.norm())

    assert rel(n, want) <= 0.1
    pairs = [("dr", dr, r0), ("dw_first", dw_first, w0)]
    for i, (got, leaves) in enumerate(zip(grads, params)):
        pairs += [(f"{name} of block {i}", x, y) for name, x, y in
                  zip(("wgu", "wd", "w_post", "gate", "w_pre"), got, leaves)]
    for name, got, leaf in pairs:
        e = rel(got, leaf.grad)
        say(name, "relative error", round(e, 4))
        assert e <= 0.2, (name, e)


def test_stack_learns(puro):
    from blockwise_fp8_gemm_x128_amd.mlp_stack import train
    losses = train(steps=30, say=say)
    assert all(x == x for x in losses)
    assert losses[-1] < 0.8 * losses[0], losses
