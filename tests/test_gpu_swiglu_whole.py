"""Values of the activation's gradient straight to FP8 operands at batches of 86 tiles of 128 x 128
and more, which one kernel works out whole (smaller ones are split by tensor), and where its codes
go past the caches. The reference is the 64-bit form of block_ref, which derives the bounds; a large
batch is checked in bands of rows, columns and tiles, each against the reference of its own."""
import numpy as np
import pytest
import torch

import block_ref as ref

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16 = torch.bfloat16


def gaussian(shape, seed, std):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, device=DEV) * std


def inputs(rows, f):
    """Gaussian, with large channels, zero rows and groups and the ends of the sigmoid."""
    gu = gaussian((rows, 2 * f), rows + f, 2.0)
    gu[:, f // 3] *= 30.0
    gu[:, f + f // 5] *= 30.0
    gu[rows // 2] = 0.0
    gu[3, :128] = 0.0
    gu[rows - 1, 0], gu[0, f - 1] = 120.0, -120.0
    dh = gaussian((rows, f), rows + f + 1, 1e-3)
    dh[:, f // 4] *= 30.0
    dh[rows // 3] = 0.0
    dh[128:256, 7] = 0.0                        # a column group of zeros
    return gu.to(BF16), dh.to(BF16)


def values(src, rows, cols, f):
    """(g, u) in float64 of the rows and of the columns (slices of one half)."""
    if isinstance(src, torch.Tensor):
        return ref.f64(src[rows, cols]), ref.f64(src[rows, f + cols.start:f + cols.stop])
    q, s = src
    k, c0, c1 = f // 128, cols.start // 128, cols.stop // 128
    return tuple(ref.f64(ref.decode32(q[rows, o + cols.start:o + cols.stop],
                                      s[b + c0:b + c1, rows]))
                 for o, b in ((0, 0), (f, k)))


def check_part(o, src, dh, rows, cols, f, pow2):
    """All six outputs at these rows and columns, whose ends are multiples of 128."""
    g, u = values(src, rows, cols, f)
    dg, du, eg, eu = ref.swiglu_bwd(ref.f64(dh[rows, cols]), g, u)
    h, eh = ref.swiglu(g, u)
    r, c = slice(rows.start // 128, rows.stop // 128), (cols.start // 128, cols.stop // 128)
    for half, want, err in ((0, dg, eg), (1, du, eu)):
        at = slice(half * f + cols.start, half * f + cols.stop)
        k = half * f // 128
        ref.check_codes(o.dguq[rows, at], o.dgus[k + c[0]:k + c[1], rows], want, err, pow2,
                        ("dg", "du")[half])
        ref.check_codes(o.dgutq[at, rows], o.dguts[r, at], np.ascontiguousarray(want.T),
                        np.ascontiguousarray(err.T), pow2, ("dg", "du")[half] + " transposed")
    ref.check_codes(o.htq[cols, rows], o.hts[r, cols], np.ascontiguousarray(h.T),
                    np.ascontiguousarray(eh.T), pow2, "h transposed")


def saved_of(puro, gu, saved, pow2):
    if saved == "asis":
        return gu
    o = puro.puro_swiglu_fwd(gu, fp8=False, pow2=pow2)
    return o.guq, o.gus


def guarded(rows, f):
    """The six outputs, filled with a code and a scale that no input here gives."""
    codes = lambda *s: torch.full(s, 0x55, dtype=torch.uint8, device=DEV)  # noqa: E731
    scales = lambda *s: torch.full(s, -1.0, device=DEV)  # noqa: E731
    return (codes(rows, 2 * f), scales(2 * f // 128, rows), codes(2 * f, rows),
            scales(rows // 128, 2 * f), codes(f, rows), scales(rows // 128, f))


# 86 tiles, the fewest; 104 and 130; one column and one row of tiles
@pytest.mark.parametrize("rows,f", [(128 * 43, 256), (1664, 1024), (1280, 1664),
                                    (128 * 86, 128), (128, 128 * 87)])
@pytest.mark.parametrize("saved", ["fp8", "asis"])
@pytest.mark.parametrize("pow2", [False, True])
def test_whole_tiles(puro, rows, f, saved, pow2):
    assert rows * f // 128 ** 2 >= 86
    gu, dh = inputs(rows, f)
    src = saved_of(puro, gu, saved, pow2)
    o = puro.puro_swiglu_bwd_fp8(dh, src, pow2=pow2, out=guarded(rows, f))
    assert not any(torch.any(s == -1.0) for s in (o.dgus, o.dguts, o.hts))
    check_part(o, src, dh, slice(0, rows), slice(0, f), f, pow2)


@pytest.mark.parametrize("saved", ["fp8", "asis"])
@pytest.mark.parametrize("pow2", [False, True])
def test_codes_past_the_caches(puro, saved, pow2):
    """More than 256 MiB of codes (69 x 48 tiles, 5 bytes an element of h). Tile by tile its outputs
    are those of the same tile's rows in a batch of one column of tiles; bands are compared with
    the reference."""
    rows, f = 128 * 69, 6144
    assert 5 * rows * f > 256 << 20
    gu, dh = inputs(rows, f)
    src = saved_of(puro, gu, saved, pow2)
    o = puro.puro_swiglu_bwd_fp8(dh, src, pow2=pow2, out=guarded(rows, f))
    assert not any(torch.any(s == -1.0) for s in (o.dgus, o.dguts, o.hts))
    for rs, cs in ((slice(0, 256), slice(0, 256)), (slice(rows - 256, rows), slice(f - 256, f)),
                   (slice(2944, 3072), slice(0, f)), (slice(0, rows), slice(1920, 2048))):
        check_part(o, src, dh, rs, cs, f, pow2)
    # every other place: the same rows in batches of 20 bands and 512 columns (80 tiles: the split
    # kernel), whose scales and codes have to be the same bytes
    k = f // 128
    for r0 in range(0, rows, 2560):
        r1 = min(rows, r0 + 2560)
        for c0 in range(0, f, 512):
            cols = torch.cat([torch.arange(c0, c0 + 512), torch.arange(f + c0, f + c0 + 512)]).to(DEV)
            if saved == "asis":
                part = gu[r0:r1, cols].contiguous()
            else:
                groups = torch.cat([torch.arange(c0 // 128, c0 // 128 + 4),
                                    torch.arange(k + c0 // 128, k + c0 // 128 + 4)]).to(DEV)
                part = (src[0][r0:r1, cols].contiguous(), src[1][groups, r0:r1].contiguous())
            p = puro.puro_swiglu_bwd_fp8(dh[r0:r1, c0:c0 + 512].contiguous(), part, pow2=pow2)
            t0, t1 = r0 // 128, r1 // 128
            g = torch.cat([torch.arange(c0 // 128, c0 // 128 + 4),
                           torch.arange(k + c0 // 128, k + c0 // 128 + 4)]).to(DEV)
            for name, a, b in (("dguq", o.dguq[r0:r1, cols], p.dguq),
                               ("dgus", o.dgus[g, r0:r1], p.dgus),
                               ("dgutq", o.dgutq[cols, r0:r1], p.dgutq),
                               ("dguts", o.dguts[t0:t1, cols], p.dguts),
                               ("htq", o.htq[c0:c0 + 512, r0:r1], p.htq),
                               ("hts", o.hts[t0:t1, c0:c0 + 512], p.hts)):
                assert torch.equal(a, b), (name, r0, c0)
