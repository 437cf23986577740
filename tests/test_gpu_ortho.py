"""The orthogonalised momentum and the projected step that takes it, on the GPU, against the
definitions in 64 bits (tests/head_ref.py, which says what bounds them)."""
import pytest
import torch

import head_ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"

# (count, rows, cols): single elements, rows and columns, sizes that end inside a tile or a chunk, wide
# and tall, both tile shapes
SIZES = [(1, 1, 1), (2, 1, 7), (2, 7, 1), (1, 5, 300), (1, 300, 5), (2, 5, 3), (3, 64, 64),
         (3, 33, 35), (2, 65, 130), (2, 130, 65), (2, 257, 300), (1, 128, 512), (1, 600, 257),
         (1, 1100, 90), (1, 1024, 1024), (64, 300, 520), (64, 520, 300), (43, 520, 520),
         # short sides around the small matrix's sizes, with long reductions
         (2, 16, 200), (1, 17, 3001), (28, 32, 77), (1, 33, 5000), (2, 5000, 48), (1, 64, 64),
         (3, 100, 1000), (1, 4097, 128), (64, 128, 130),
         # just above: few tiles, whose long reductions are split
         (1, 129, 3000), (1, 3000, 129), (2, 200, 1500), (1, 140, 150), (1, 150, 12000)]


def draw(count, rows, cols, seed=0, low_rank=True):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed + 100000 * count + 300 * rows + cols)

    def one():
        x = 0.5 * torch.randn((count, rows, cols), generator=g, device=DEV)
        if low_rank:
            rank = max(1, min(rows, cols) // 8)
            left = torch.randn((count, rows, rank), generator=g, device=DEV)
            x += torch.bmm(left, torch.randn((count, rank, cols), generator=g, device=DEV))
        return 1e-3 * x

    return one(), one()


def check(u, v, scale=1.0, **kw):
    """One matrix's direction: at most half a step of bf16 off the exact steps (2^-8), plus, over the
    matrix, twice what the rounded operands cost in 64 bits, and in no element 24 times the root mean
    square of that.

    24 = 2 x 12: where an error lies along one singular direction (many steps of coefficients that
    do not converge amplify a few directions by their slope, -1 to 4 a step) its elements are
    products of two components of unit vectors, x y for x, y about normal. |x y| exceeds t with
    probability sqrt(2 / (pi t)) exp(-t): 1.4e-6 for t = 12 (1 % over the 8450 elements of 65 x 130),
    but 1.1e-5 for t = 10 (10 %), before the factor 2 between two roundings' errors. Errors along
    many directions are about normal and stay far below."""
    want = scale * head_ref.ortho(v, **kw)
    ways = [False, True] if kw.get("steps", 5) >= 3 else [False]
    rms = max(float((scale * head_ref.ortho_rounded(v, grouped=g, **kw) - want).square().mean().sqrt())
              for g in ways) + 2.0 ** -14 * float(want.square().mean().sqrt())
    off = (u.double() - want)
    assert float(off.norm()) <= 2.0 ** -8 * float(want.norm()) + 2 * rms * want.numel() ** 0.5
    assert bool((off.abs() <= 2.0 ** -8 * (want.abs() + 24 * rms) + 24 * rms).all())


def check_momentum(got, g, m, beta, nesterov):
    want, v = head_ref.momentum(g, m, beta, nesterov)
    bound = 2.0 ** -23 * (m.double().abs() + g.double().abs())
    assert bool(((got.double() - want).abs() <= bound).all())
    return v


@pytest.mark.parametrize("size", SIZES, ids=str)
def test_gradient_alone(puro, size):
    g, _ = draw(*size)
    us = puro.puro_newton_schulz(g.unbind(0))
    assert len(us) == size[0]
    for x, u in list(zip(g, us))[::7]:
        assert u.dtype == torch.bfloat16 and u.shape == x.shape
        check(u, x.double())


@pytest.mark.parametrize("nesterov", [True, False], ids=["nesterov", "plain"])
@pytest.mark.parametrize("size", SIZES[::2], ids=str)
def test_momentum(puro, size, nesterov):
    g, m = draw(*size)
    before = m.clone()
    us = puro.puro_newton_schulz(g.unbind(0), m.unbind(0), beta=0.9, nesterov=nesterov, scale=0.25)
    for x, old, new, u in list(zip(g, before, m, us))[::7]:
        v = check_momentum(new, x, old, 0.9, nesterov)
        check(u, v, scale=0.25)


def test_new_momentum_elsewhere(puro):
    g, m = draw(3, 33, 35)
    before, out = m.clone(), torch.empty_like(m)
    us = puro.puro_newton_schulz(g.unbind(0), m.unbind(0), ms_out=out.unbind(0))
    assert torch.equal(m, before)
    again = puro.puro_newton_schulz(g.unbind(0), m.unbind(0))
    assert torch.equal(m, out) and all(torch.equal(a, b) for a, b in zip(us, again))


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 16])
@pytest.mark.parametrize("size", [(2, 65, 130), (2, 130, 65), (2, 150, 170), (2, 150, 230),
                                  (2, 230, 150)], ids=str)
def test_steps(puro, size, steps):
    g, _ = draw(*size)
    for x, u in zip(g, puro.puro_newton_schulz(g.unbind(0), steps=steps)):
        check(u, x.double(), steps=steps)


def test_other_coefficients(puro):
    """The cubic iteration that converges to the orthogonal factor itself."""
    k = (1.5, -0.5, 0.0)
    for side, other in ((40, 70), (150, 400), (150, 170)):
        g, _ = draw(2, side, other, low_rank=False)
        for x, u in zip(g, puro.puro_newton_schulz(g.unbind(0), steps=16, coefficients=k)):
            check(u, x.double(), steps=16, coefficients=k)
            off = u.double() @ u.double().t() - torch.eye(side, device=DEV)
            assert float(off.abs().max()) < 0.1


@pytest.mark.parametrize("factor", [1e-30, 1e-6, 1e30], ids=str)
def test_any_magnitude(puro, factor):
    g, _ = draw(2, 65, 130)
    for x, u in zip(g * factor, puro.puro_newton_schulz((g * factor).unbind(0))):
        check(u, x.double())


def test_singular_values_come_out_near_one(puro):
    g, _ = draw(2, 256, 512)
    for u in puro.puro_newton_schulz(g.unbind(0)):
        s = torch.linalg.svdvals(u.double().cpu())
        assert float(s.min()) > 0.6 and float(s.max()) < 1.3


def test_zero_infinite_and_nan_matrices_keep_to_themselves(puro):
    g, _ = draw(5, 70, 140)
    g[1] = 0
    g[2, 3, 4] = float("nan")
    g[3, 69, 139] = float("inf")
    us = puro.puro_newton_schulz(g.unbind(0))
    assert not bool(us[1].any())
    assert bool(us[2].isnan().all()) and bool(us[3].isnan().all())
    for k in (0, 4):
        check(us[k], g[k].double())


def test_addresses_of_any_alignment(puro):
    """Slices of a flat buffer, each one element further: the same directions as from aligned ones."""
    g, m = draw(3, 36, 68)
    want = puro.puro_newton_schulz(g.unbind(0), m.clone().unbind(0))
    n = 36 * 68

    def shifted(x, dtype):
        buf = torch.full((3 * (n + 1) + 8,), 7.0, dtype=dtype, device=DEV)
        views = [buf[k * (n + 1) + 1:k * (n + 1) + 1 + n].view(36, 68) for k in range(3)]
        for v, t in zip(views, x):
            v.copy_(t)
        return buf, views

    (_, gs), (mb, ms), (ub, us) = (shifted(x, t) for x, t in
                                   ((g, torch.float32), (m, torch.float32), (want, torch.bfloat16)))
    for u in us:
        u.zero_()
    puro.puro_newton_schulz(gs, ms, us=us)
    # the sum of squares runs in another order: not bit for bit
    for a, b in zip(us, want):
        assert float((a.double() - b.double()).abs().max()) <= 2.0 ** -6 * float(b.abs().max())
    for buf in (mb, ub):
        assert all(float(buf[k * (n + 1)]) == 7 for k in range(4))


def test_outputs_and_workspace_stay_in_their_place(puro):
    for size in [(2, 33, 35), (2, 130, 65), (1, 64, 256)]:
        g, _ = draw(*size)
        n = size[1] * size[2]
        need = puro.lib().puro_newton_schulz_workspace(*size)
        ws = torch.full((need + 512,), 255, dtype=torch.uint8, device=DEV)
        buf = torch.full((size[0] * n + 4096,), 7.0, dtype=torch.bfloat16, device=DEV)
        us = buf[2048:2048 + size[0] * n].view(size)
        want = puro.puro_newton_schulz(g.unbind(0))
        puro.puro_newton_schulz(g.unbind(0), us=us.unbind(0), workspace=ws[256:256 + need])
        assert all(torch.equal(a, b) for a, b in zip(us, want))
        assert bool((buf[:2048] == 7).all()) and bool((buf[2048 + size[0] * n:] == 7).all())
        assert bool((ws[:256] == 255).all()) and bool((ws[256 + need:] == 255).all())
        with pytest.raises(puro.PuroError, match="workspace"):
            puro.puro_newton_schulz(g.unbind(0), workspace=ws[:need - 1])


@pytest.mark.parametrize("size", [(2, 130, 65), (43, 520, 520)], ids=str)
def test_repeats_exactly_and_alone_as_in_a_group(puro, size):
    g, _ = draw(*size)
    first = puro.puro_newton_schulz(g.unbind(0))
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(first, puro.puro_newton_schulz(g.unbind(0))))


def test_captured_and_replayed(puro):
    g, m = draw(2, 130, 200)
    us = puro.puro_newton_schulz(g.unbind(0), m.clone().unbind(0))
    torch.cuda.synchronize()
    start = m.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        puro.puro_newton_schulz(g.unbind(0), m.unbind(0), us=us)
    state = start.clone()
    m.copy_(start)
    for k in range(4):
        g.copy_(draw(2, 130, 200, seed=k + 1)[0])
        graph.replay()
        torch.cuda.synchronize()
        want = puro.puro_newton_schulz(g.unbind(0), state.unbind(0))
        assert torch.equal(m, state) and all(torch.equal(a, b) for a, b in zip(us, want))


def test_another_stream(puro):
    g, _ = draw(2, 130, 200)
    want = puro.puro_newton_schulz(g.unbind(0))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        outs = [puro.puro_newton_schulz(g.unbind(0)) for _ in range(4)]
    outs += [puro.puro_newton_schulz(g.unbind(0)) for _ in range(4)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in outs for a, b in zip(o, want))


@pytest.mark.parametrize("shape", [(8, 8), (100, 36), (2048, 2048)], ids=str)
def test_projected_step_with_a_bf16_direction(puro, shape):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    w = torch.randn(shape, generator=gen, device=DEV)
    u = torch.randn(shape, generator=gen, device=DEV).bfloat16()
    r = puro.puro_frobenius_norm(w)
    a, b = w.clone(), w.clone()
    a16 = puro.puro_hyperball_step_u16(a, u, 0.1, r)
    b16 = puro.puro_hyperball_step(b, u.float(), 0.1, r)
    assert torch.equal(a, b) and torch.equal(a16, b16)


def test_refusals_of_the_binding(puro):
    g, m = draw(2, 8, 12)
    gs, ms = list(g), list(m)
    bad = [lambda: puro.puro_newton_schulz(gs, ms[:1]),
           lambda: puro.puro_newton_schulz(gs, ms_out=ms),
           lambda: puro.puro_newton_schulz([g[0], g[1].t().contiguous()]),
           lambda: puro.puro_newton_schulz([g[0].t()]),
           lambda: puro.puro_newton_schulz([g[0].double()]),
           lambda: puro.puro_newton_schulz([g[0].reshape(-1)]),
           lambda: puro.puro_newton_schulz(gs, us=[torch.empty_like(x) for x in gs]),
           lambda: puro.puro_newton_schulz(gs, [x.half() for x in ms]),
           lambda: puro.puro_newton_schulz(gs * 33),
           lambda: puro.puro_newton_schulz(gs, steps=0),
           lambda: puro.puro_newton_schulz(gs, coefficients=(3.0, 0.0, 0.0))]
    for call in bad:
        with pytest.raises(puro.PuroError):
            call()
    w = torch.zeros((8, 8), device=DEV)
    with pytest.raises(puro.PuroError):
        puro.puro_hyperball_step_u16(w, w, 0.1, torch.ones(1, device=DEV))


@pytest.mark.parametrize("size", [(1, 2 ** 20, 90), (1, 160, 2 ** 20)], ids=str)
def test_longest_sides(puro, size):
    g = draw(*size)[0]
    check(puro.puro_newton_schulz([g[0]])[0], g[0])


def test_offsets_past_32_bits(puro):
    """A group of 2^31 elements and more, its last matrix another one than the rest."""
    g = [draw(1, 2050, 16400, seed=k)[0][0] for k in range(2)]
    us = puro.puro_newton_schulz([g[0]] * 63 + [g[1]])
    check(us[0], g[0])
    check(us[63], g[1])
    assert all(torch.equal(u, us[0]) for u in us[1:63])


# tiles of 128x128 between half of the chip's compute units and all of them, for one symmetric product, for
# two in a launch, and for the products with X; wide and tall
@pytest.mark.parametrize("size", [(9, 520, 520), (14, 520, 600), (14, 600, 520), (5, 520, 800),
                                  (5, 800, 520)], ids=str)
def test_a_tile_for_most_compute_units(puro, size):
    g, m = draw(*size)
    ms = [x.clone() for x in m.unbind(0)]
    us = puro.puro_newton_schulz(g.unbind(0), ms)
    for k in range(size[0]):
        check(us[k], check_momentum(ms[k], g[k], m[k], 0.95, True))
