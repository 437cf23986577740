"""A stack of MLP blocks trained end to end on the library's operators: every step between two FP8
GEMMs is one of its kernels, and what the forward pass keeps for the backward pass is 8 bits wide.

    boundary 0      n_0 = norm(r_0) w_pre_0                                   (norm before a block)
    block i         gu = n_i Wgu_i^T,  h = silu(g) u,  y_i = h Wd_i^T
    boundary i + 1  r_{i+1} = beta r_i + alpha gate_i norm(y_i) w_post_i,
                    n_{i+1} = norm(r_{i+1}) w_pre_{i+1}                       (both norms, one pass)

The boundaries and the activation hand the GEMMs their FP8 operands directly. Kept per block and
token: n (its GEMM operand, 1 byte a value), gu and y, r (checkpoints, 1 byte a value): 2 f + 3 d
bytes instead of 4 f + 6 d in bf16. In the backward pass the block norm reads y and r from their
checkpoints, the activation's gradient goes straight to the operands of the two GEMMs behind it, and
the weight gradients' transposed operands are made from the kept ones (n: puro_ckpt_transpose; h:
from the checkpoint of gu).

``python -m blockwise_fp8_gemm_x128_amd.mlp_stack`` trains a small stack to imitate another one:
matrices by the projected step, vectors by AdamW.
"""
from __future__ import annotations

from typing import List, NamedTuple

import torch

from . import binding as puro


class Layer(NamedTuple):
    """Parameters of one block and of the boundary behind it. Masters fp32, matrices also as the
    bf16 copies the quantiser reads."""
    wgu: torch.Tensor     # fp32 [2f, d]
    wd: torch.Tensor      # fp32 [d, f]
    wgu16: torch.Tensor
    wd16: torch.Tensor
    w_post: torch.Tensor  # fp32 [d]
    gate: torch.Tensor    # fp32 [d]
    w_pre: torch.Tensor   # fp32 [d]: the norm behind this boundary (the next block's, or the last)


class Kept(NamedTuple):
    """What one block's forward pass leaves for its backward pass."""
    n: tuple              # operand of the gate_up GEMM: (codes, scales)
    gu: tuple             # checkpoint
    wgu: tuple            # FP8 weights: (codes, scales)
    wd: tuple
    norm: puro.BlockNorm  # the boundary behind the block


class MlpStack:
    """`layers` blocks of width d and MLP width f (multiples of 128) for batches whose token count
    is a multiple of 128."""

    def __init__(self, layers: int, d: int, f: int, seed: int = 0, alpha: float = 1.0,
                 beta: float = 1.0, eps: float = 1e-6, device="cuda:0"):
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)

        def matrix(rows, cols):
            return torch.randn((rows, cols), generator=gen, device=device) * cols ** -0.5

        def vector(value):
            return torch.full((d,), value, device=device)

        self.alpha, self.beta, self.eps = alpha, beta, eps
        self.w_first = vector(1.0)
        self.layers: List[Layer] = []
        for _ in range(layers):
            wgu, wd = matrix(2 * f, d), matrix(d, f)
            self.layers.append(Layer(wgu, wd, wgu.bfloat16(), wd.bfloat16(), vector(1.0),
                                     vector(0.5), vector(1.0)))

    def forward(self, r):
        """r: the residual stream, bf16 or fp32 [tokens, d] -> (n bf16 [tokens, d], kept)."""
        first = puro.puro_block_norm_fwd(None, r, None, self.w_first, eps=self.eps)
        kept, n, last = [], (first.nq, first.ns), len(self.layers) - 1
        for i, p in enumerate(self.layers):
            (wguq, wdq), (wgus, wds) = puro.puro_quant_w_128x128_group([p.wgu16, p.wd16])
            gu = puro.puro_fp8_gemm_fwd(*n, wguq, wgus)
            act = puro.puro_swiglu_fwd(gu)
            y = puro.puro_fp8_gemm_fwd(act.hq, act.hs, wdq, wds)
            norm = puro.puro_block_norm_fwd(y, r, p.w_post, p.w_pre, p.gate, alpha=self.alpha,
                                            beta=self.beta, eps=self.eps,
                                            n="bf16" if i == last else "fp8")
            kept.append(Kept(n, (act.guq, act.gus), (wguq, wgus), (wdq, wds),
                             norm._replace(r_out=None)))
            r, n = norm.r_out, (norm.nq, norm.ns)
        return norm.n, (first, kept, r.dtype)

    def backward(self, dn, kept):
        """dn: the gradient of forward's n, bf16 -> (dr in the residual stream's type, dw_first,
        [gradients of each layer's wgu, wd, w_post, gate, w_pre])."""
        first, kept, stream = kept
        grads, dr = [], None
        for p, k in zip(reversed(self.layers), reversed(kept)):
            o = puro.puro_block_norm_bwd(dr, dn, (k.norm.yq, k.norm.ys), (k.norm.rq, k.norm.rs),
                                         k.norm.rstd_y, k.norm.rstd_r, p.w_post, p.w_pre, p.gate,
                                         alpha=self.alpha, beta=self.beta, residual_dtype=stream)
            dyq, dys, dytq, dyts = puro.puro_quant_dual_1x128(o.dy)
            dh = puro.puro_fp8_gemm_dgrad(dyq, dys, *k.wd)
            a = puro.puro_swiglu_bwd_fp8(dh, k.gu)
            dwd = puro.puro_fp8_gemm_wgrad(dytq, dyts, a.htq, a.hts)
            dn = puro.puro_fp8_gemm_dgrad(a.dguq, a.dgus, *k.wgu)
            dwgu = puro.puro_fp8_gemm_wgrad(a.dgutq, a.dguts, *puro.puro_ckpt_transpose(*k.n))
            grads.append((dwgu, dwd, o.dw_post, o.dgate, o.dw_pre))
            dr = o.dr
        o = puro.puro_block_norm_bwd(dr, dn, None, (first.rq, first.rs), None, first.rstd_r, None,
                                     self.w_first, residual_dtype=stream)
        return o.dr, o.dw_pre, grads[::-1]


class Trainer:
    """Projected steps of the matrices along their gradients, scaled to the matrix's radius; AdamW
    for the vectors."""

    def __init__(self, stack: MlpStack, lr: float):
        self.stack, self.lr, self.step = stack, lr, 0
        self.radii = [(puro.puro_frobenius_norm(p.wgu), puro.puro_frobenius_norm(p.wd))
                      for p in stack.layers]
        vectors = [stack.w_first, *(v for p in stack.layers for v in (p.w_post, p.gate, p.w_pre))]
        self.state = [(v, torch.zeros_like(v), torch.zeros_like(v)) for v in vectors]

    def update(self, dw_first, grads):
        self.step += 1
        for p, radii, (dwgu, dwd, *_) in zip(self.stack.layers, self.radii, grads):
            for w, w16, g, r in ((p.wgu, p.wgu16, dwgu, radii[0]), (p.wd, p.wd16, dwd, radii[1])):
                g.mul_(r / puro.puro_frobenius_norm(g).clamp_min(1e-30))
                puro.puro_hyperball_step(w, g, self.lr, r, w_bf16=w16)
        flat = [dw_first, *(v for g in grads for v in g[2:])]
        for (v, m, s), g in zip(self.state, flat):
            puro.puro_adamw_step(v, g, m, s, 0.1 * self.lr, 0.9, 0.95, 1e-8, 0.0, self.step)


def train(layers=2, d=256, f=512, tokens=1024, steps=30, lr=0.05, seed=0, say=print):
    """Trains a stack on the outputs of another one; returns the loss of every step."""
    teacher, student = MlpStack(layers, d, f, seed + 1), MlpStack(layers, d, f, seed + 2)
    trainer = Trainer(student, lr)
    gen = torch.Generator(device="cuda:0")
    gen.manual_seed(seed)
    losses = []
    for step in range(steps):
        r = torch.randn((tokens, d), generator=gen, device="cuda:0").bfloat16()
        target, _ = teacher.forward(r)
        n, kept = student.forward(r)
        diff = n.float() - target.float()
        losses.append(float(diff.square().mean()))
        _, dw_first, grads = student.backward((2.0 / diff.numel() * diff).bfloat16(), kept)
        trainer.update(dw_first, grads)
        if say and (step % 5 == 0 or step == steps - 1):
            say("step %3d  loss %.4f" % (step, losses[-1]))
    return losses


def main(argv=None):
    import argparse
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--d", type=int, default=256)
    ap.add_argument("--f", type=int, default=512)
    ap.add_argument("--tokens", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=30)
    ap.add_argument("--lr", type=float, default=0.05)
    a = ap.parse_args(argv)
    train(a.layers, a.d, a.f, a.tokens, a.steps, a.lr)


if __name__ == "__main__":
    main()
