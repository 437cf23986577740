"""The token model that runs the output head's cross entropy, the blocks, the orthogonalised momentum
and the projected step together: its loss and the head's gradients against the definitions in 64 bits
at the model's own hidden states (tests/head_ref.py), every other gradient against float64 autograd
of the whole network, and an optimizer step against its parts.

Tolerance of the gradients behind the head: as for the stack itself (tests/test_gpu_mlp_stack.py: 0.2
of the tensor's norm for at most 16 independent FP8 roundings of 0.036 each); the gradient that
enters the stack differs from the exact network's by what the hidden states differ, at most
0.1 of their norm on the forward half of that path, which those 16 roundings count already. The
embedding's gradient is the stack's input gradient, added up over the tokens."""
import pytest
import torch

import head_ref
from test_gpu_mlp_stack import reference
from test_gpu_ortho import check_momentum
from test_gpu_xent import check_bwd, check_fwd

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def batch(vocab, tokens, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    x = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    y = torch.randint(0, vocab, (tokens,), generator=g, device=DEV)
    y[::9] = -100
    has = y >= 0
    return x, y, has.float() / has.sum()


def test_gradients(puro):
    from blockwise_fp8_gemm_x128_amd.mlp_stack import TokenModel
    model = TokenModel(1000, 2, 256, 384, seed=3)
    x, y, dloss = batch(1000, 256, 5)
    loss, kept = model.forward(x, y)
    n, lse = kept[2], kept[3]
    check_fwd((loss, lse), n, model.head16, y)
    demb, dhead, dw_first, grads = model.backward(dloss, kept)
    check_bwd((None, dhead), n, model.head16, y, lse, dloss, None)
    # the whole network
    r0, w0, params, out = reference(model.stack, model.embedding16[x])
    keep = (y >= 0).cpu()
    logits = out @ model.head16.double().cpu().t()
    total = torch.nn.functional.cross_entropy(logits[keep], y.cpu()[keep], reduction="mean")
    total.backward()

    def rel(got, ref):
        return float((got.double().cpu() - ref).norm() / ref.norm())

    want = torch.zeros_like(model.embedding, dtype=torch.float64).cpu()
    want.index_add_(0, x.cpu(), r0.grad)
    pairs = [("embedding", demb, want), ("w_first", dw_first, w0.grad)]
    for i, (got, leaves) in enumerate(zip(grads, params)):
        pairs += [(f"{name} of block {i}", a, b.grad) for name, a, b in
                  zip(("wgu", "wd", "w_post", "gate", "w_pre"), got, leaves)]
    for name, got, ref in pairs:
        assert rel(got, ref) <= 0.2, (name, rel(got, ref))


def test_optimizer_step(puro):
    """Two steps of every matrix: momentum, its direction, and the projection, each from what the one
    before it left."""
    from blockwise_fp8_gemm_x128_amd.mlp_stack import TokenModel, TokenTrainer
    model = TokenModel(512, 2, 128, 256, seed=1)
    trainer = TokenTrainer(model, 0.05, beta=0.9)
    for step in range(2):
        x, y, dloss = batch(512, 128, step)
        _, kept = model.forward(x, y)
        parts = model.backward(dloss, kept)
        grads = parts[3]
        before = [[(w.clone(), m.clone()) for w, m in zip(ws, ms)]
                  for ws, ms in zip(trainer._matrices(), trainer.momenta)]
        tables = [w.clone() for w in (model.embedding, model.head)]
        trainer.update_all(*parts)
        for i, (ws, ms) in enumerate(zip(trainer._matrices(), trainer.momenta)):
            rows, cols = ws[0].shape
            scale = (rows / min(rows, cols)) ** 0.5
            for (w0, m0), w, m, g, radii in zip(before[i], ws, ms, grads, trainer.radii):
                v = check_momentum(m, g[i], m0, 0.9, True)
                want = w0.double() - 0.05 * scale * head_ref.ortho(v)
                want *= float(radii[i]) / want.norm()
                # u's error is at most 5e-3 of it (its rounding and that of the steps), lr 0.05 of the
                # radius, so 2.5e-4 of w; and again through the projection
                assert float((w.double() - want).norm()) <= 1e-3 * float(radii[i])
                assert abs(float(w.double().norm()) / float(radii[i]) - 1) <= 1e-6
        for p in model.stack.layers:
            assert torch.equal(p.wgu16, p.wgu.bfloat16()) and torch.equal(p.wd16, p.wd.bfloat16())
        for w, w16, old in ((model.embedding, model.embedding16, tables[0]),
                            (model.head, model.head16, tables[1])):
            assert torch.equal(w16, w.bfloat16()) and not torch.equal(w, old)


def test_training_runs(puro):
    from blockwise_fp8_gemm_x128_amd.mlp_stack import main, train_tokens
    losses = train_tokens(vocab=500, layers=1, d=128, f=128, tokens=128, steps=3, say=None)
    assert len(losses) == 3 and all(x == x for x in losses)
    main(["--vocab", "500", "--layers", "1", "--d", "128", "--f", "128", "--tokens", "128",
          "--steps", "1"])
