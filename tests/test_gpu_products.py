"""The products over segments, matmul and outer (GPU only), against 64-bit
forms: types, layouts, odd widths, segments from none to many rows, gathered
rows, NaN in rows that take no part, and rows left as they were."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

LENGTHS = {
    "mixed": [0, 5, 1, 130, 17, 0, 300, 64],
    "single-tokens": [1] * 20 + [3, 0, 2],
    "tens": [40, 33, 0, 90, 64],
    "long": [700, 0, 1033, 513],
    "one": [1],
    "empty": [0, 0],
}
WIDTHS = [(64, 128), (200, 72), (8, 8), (33, 45), (1, 1), (512, 264), (130, 300)]


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_matmul(kind, lengths):
    t, ls = ru.TYPES[kind], LENGTHS[lengths]
    for i, (k, m) in enumerate(WIDTHS):
        g = ru.gen(100 * i + len(ls))
        off = ru.offsets(ls, base=3)
        n, pool = int(off[-1]) + 4, 50
        x = ru.randn(g, pool, k, dtype=t)
        full = ru.randn(g, n, k, dtype=t)
        rows = torch.randint(0, pool, (n,), generator=g)
        for transpose in (False, True):
            w = ru.randn(g, len(ls), *((m, k) if transpose else (k, m)), dtype=t)
            for values, idx in ((x, rows), (full, None)):
                ru.say(f"matmul {kind} {lengths} k={k} m={m} transpose={transpose} gathered={idx is not None}")
                out = torch.full((n, m), 7.0, dtype=t, device="cuda")
                got = sr().matmul(values.cuda(), w.cuda(), off.cuda(), transpose=transpose,
                                  rows=None if idx is None else idx.cuda(), out=out)
                torch.cuda.synchronize()
                assert got is out
                ref, mag = ru.matmul(values, w, off, transpose, idx, fill=7.0)
                ru.assert_close(out, ref, mag, k, "matmul")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_outer(kind, lengths):
    t, ls = ru.TYPES[kind], LENGTHS[lengths]
    for i, (k, m) in enumerate(WIDTHS):
        g = ru.gen(100 * i + len(ls))
        off = ru.offsets(ls, base=3)
        n, pool = int(off[-1]) + 4, 50
        left, right = ru.randn(g, n, k, dtype=t), ru.randn(g, pool, m, dtype=t)
        rows = torch.randint(0, pool, (n,), generator=g)
        ref, mag = ru.outer(left, right, off, right_rows=rows)
        for odt in {t, torch.float32}:
            ru.say(f"outer {kind} -> {odt} {lengths} k={k} m={m}")
            got = sr().outer(left.cuda(), right.cuda(), off.cuda(), right_rows=rows.cuda(), out_dtype=odt)
            torch.cuda.synchronize()
            ru.assert_close(got, ref, mag, max(ls), "outer")
        ref2, mag2 = ru.outer(right, left, off, left_rows=rows)
        got = sr().outer(right.cuda(), left.cuda(), off.cuda(), left_rows=rows.cuda())
        torch.cuda.synchronize()
        ru.assert_close(got, ref2, mag2, max(ls), "outer, left gathered")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("segments,rows", [(1, 20000), (3, 9001), (5, 40003)])
def test_outer_long_segments(kind, segments, rows):
    """Segments long enough to be cut into pieces that are added afterwards."""
    t = ru.TYPES[kind]
    g = ru.gen(rows)
    cuts = torch.randint(0, rows + 1, (segments - 1,), generator=g).sort().values.tolist()
    off = torch.tensor([0, *cuts, rows])
    for k, m in ((64, 96), (24, 40), (17, 5)):
        left, right = ru.randn(g, rows, k, dtype=t), ru.randn(g, rows, m, dtype=t)
        ru.say(f"outer long {kind} S={segments} N={rows} k={k} m={m}")
        a = sr().outer(left.cuda(), right.cuda(), off.cuda(), out_dtype=torch.float32)
        b = sr().outer(left.cuda(), right.cuda(), off.cuda(), out_dtype=torch.float32)
        torch.cuda.synchronize()
        assert torch.equal(a, b)
        ref, mag = ru.outer(left, right, off)
        ru.assert_close(a, ref, mag, rows, "outer")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("k,m", [(64, 64), (30, 50)])
def test_rows_of_no_segment_take_no_part(kind, k, m):
    """NaN and infinity in rows outside the segments, and gather entries outside the values."""
    t = ru.TYPES[kind]
    for ls in ([5, 0, 3], [300, 40], [900]):
        g = ru.gen(sum(ls))
        off = ru.offsets(ls, base=2)
        n = int(off[-1]) + 3
        x, y = ru.randn(g, n, k, dtype=t), ru.randn(g, n, m, dtype=t)
        for z in (x, y):
            z[:2], z[-3:] = float("nan"), float("inf")
        w = ru.randn(g, len(ls), k, m, dtype=t)
        rows = torch.arange(n)
        rows[3], rows[4] = -1, n  # zero rows
        ru.say(f"outside rows {kind} {ls} {k}x{m}")
        out = torch.full((n, m), 7.0, dtype=t, device="cuda")
        sr().matmul(x.cuda(), w.cuda(), off.cuda(), rows=rows.cuda(), out=out)
        dw = sr().outer(x.cuda(), y.cuda(), off.cuda())
        torch.cuda.synchronize()
        clean = x.clone()
        clean[:2], clean[-3:] = 0, 0
        ref, mag = ru.matmul(clean, w, off, rows=rows, fill=7.0)
        ru.assert_close(out, ref, mag, k, "matmul")
        assert (out[3:5].cpu() == 0).all()
        cy = y.clone()
        cy[:2], cy[-3:] = 0, 0
        ref, mag = ru.outer(clean, cy, off)
        ru.assert_close(dw, ref, mag, max(ls), "outer")


def test_infinity_and_nan_of_a_row_stay_in_it():
    g = ru.gen(5)
    off = ru.offsets([4, 60, 200])
    n = int(off[-1])
    for kind in ("bf16", "f16", "f32"):
        x, w = ru.randn(g, n, 96, dtype=ru.TYPES[kind]), ru.randn(g, 3, 96, 40, dtype=ru.TYPES[kind])
        x[10, 5], x[70, 95] = float("nan"), float("inf")
        ru.say(f"nan row {kind}")
        out = sr().matmul(x.cuda(), w.cuda(), off.cuda()).cpu()
        bad = ~torch.isfinite(out)
        assert out[10].isnan().all() and bad[70].all()
        bad[10], bad[70] = False, False
        assert not bad.any()


def _same_specials(got, ref, mag, n, what, lost):
    """NaN and infinities where the 64-bit form has them, the rest within the
    bound.  Where the terms' magnitudes pass float's range, a float sum may
    pass it on the way, in any order of its own: nothing is asked there.
    `lost`: the parts that a value is split into (x = h + m + l) count as zero
    below 2^-126, the smallest normal bf16, so that a term x w is off by less
    than 2^-125 (|x| + |w|): the sum of |x| + |w| over the terms."""
    within = ~(mag > torch.finfo(torch.float32).max) | ~torch.isfinite(ref)
    got, ref, mag, lost = got.cpu()[within], ref[within], mag[within], lost[within]
    assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
    inf = torch.isinf(ref)
    assert torch.equal(torch.isinf(got), inf) and torch.equal(got[inf].double(), ref[inf]), what
    fine = torch.isfinite(ref)
    ru.assert_close(got[fine], ref[fine], mag[fine], n, what, more=2.0 ** -125 * lost[fine])


@pytest.mark.parametrize("m", [512, 500])
def test_float_specials_in_large_calls(m):
    """float32 products made of bf16 parts: infinities, NaN, the largest and
    the smallest values come out as float arithmetic gives them."""
    g = ru.gen(m)
    off = ru.offsets([700, 0, 500, 900, 300, 600, 512, 488])
    n, k = int(off[-1]), 96
    x, w = ru.randn(g, n, k), ru.randn(g, 8, k, m)
    x[5, 3], x[800, 90], x[1500, 0] = float("inf"), float("nan"), float("-inf")
    w[6, 7, 11] = float("inf")
    x[2000] = x[2200] = torch.finfo(torch.float32).max
    w[4] *= 1e-30  # segment 4 has row 2200: large times small
    x[2500] *= 1e-30
    x[2501] *= 1e-38
    ru.say(f"float specials m={m}")
    out = sr().matmul(x.cuda(), w.cuda(), off.cuda())
    ref, mag = ru.matmul(x, w, off)
    lost = ru.matmul(x, torch.ones_like(w), off)[1] + ru.matmul(torch.ones_like(x), w, off)[1]
    _same_specials(out, ref, mag, k, "matmul", lost)
    out = sr().matmul(x.cuda(), w.transpose(1, 2).contiguous().cuda(), off.cuda(), transpose=True)
    _same_specials(out, ref, mag, k, "matmul transposed", lost)
    y = ru.randn(g, n, m)
    y[5, 8] = float("nan")
    x[2000] = x[2200] = 1.0
    dw = sr().outer(x.cuda(), y.cuda(), off.cuda())
    ref, mag = ru.outer(x, y, off)
    lost = ru.outer(x, torch.ones_like(y), off)[1] + ru.outer(torch.ones_like(x), y, off)[1]
    _same_specials(dw, ref, mag, 900, "outer", lost)
    dw = sr().outer(x[:, :24].contiguous().cuda(), y[:, :40].contiguous().cuda(), off.cuda())
    ref, mag = ru.outer(x[:, :24], y[:, :40], off)
    _same_specials(dw, ref, mag, 900, "outer, in pieces", lost[:, :24, :40])


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,segments,k,m", [(3000, 4, 320, 512), (3000, 4, 331, 515), (6000, 3, 264, 1024),
                                               (1500, 40, 128, 640), (2100, 70, 72, 136), (5000, 12, 520, 1032)])
def test_larger_calls(kind, rows, segments, k, m):
    """Sizes at which the larger tiles are taken, both layouts, gathered and not, against 64 bits on the GPU."""
    t, g = ru.TYPES[kind], ru.gen(rows + k)
    cuts = torch.randint(0, rows + 1, (segments - 1,), generator=g).sort().values.tolist()
    off = torch.tensor([0, *cuts, rows])
    x, y = ru.randn(g, rows, k, dtype=t), ru.randn(g, rows, m, dtype=t)
    w = ru.randn(g, segments, k, m, dtype=t)
    idx = torch.randint(0, rows, (rows,), generator=g)
    ru.say(f"larger {kind} N={rows} S={segments} k={k} m={m}")
    s = sr()
    for rows_t in (None, idx):
        ref, mag = ru.matmul(x.cuda(), w.cuda(), off, rows=None if rows_t is None else rows_t.cuda())
        ref, mag = ref.cpu(), mag.cpu()
        cuda_idx = None if rows_t is None else rows_t.cuda()
        ru.assert_close(s.matmul(x.cuda(), w.cuda(), off.cuda(), rows=cuda_idx), ref, mag, k, "matmul")
        wt = w.transpose(1, 2).contiguous().cuda()
        ru.assert_close(s.matmul(x.cuda(), wt, off.cuda(), rows=cuda_idx, transpose=True), ref, mag, k, "transposed")
    longest = int((off[1:] - off[:-1]).max())
    ref, mag = ru.outer(x.cuda(), y.cuda(), off, left_rows=idx.cuda())
    ru.assert_close(s.outer(x.cuda(), y.cuda(), off.cuda(), left_rows=idx.cuda()), ref.cpu(), mag.cpu(), longest, "outer")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_unaligned_bases(kind):
    """Inputs and output that start off a 16-byte boundary give the same results."""
    t = ru.TYPES[kind]
    g = ru.gen(9)
    off = ru.offsets([70, 3, 0, 40])
    n, k, m = int(off[-1]), 64, 80

    def shifted(x):
        flat = torch.empty(x.numel() + 1, dtype=t, device="cuda")
        v = flat[1:].view(x.shape)
        v.copy_(x)
        return v

    x, w = ru.randn(g, n, k, dtype=t), ru.randn(g, 4, k, m, dtype=t)
    ru.say(f"unaligned {kind}")
    out = shifted(torch.zeros(n, m))
    sr().matmul(shifted(x), shifted(w), off.cuda(), out=out)
    ref, mag = ru.matmul(x, w, off)
    ru.assert_close(out, ref, mag, k, "matmul")
    y = ru.randn(g, n, m, dtype=t)
    dw = sr().outer(shifted(x), shifted(y), off.cuda())
    ref, mag = ru.outer(x, y, off)
    ru.assert_close(dw, ref, mag, 70, "outer")


def test_many_segments():
    """More segments than one round of 64 probes finds, most of them empty or of one row."""
    g = ru.gen(11)
    ls = torch.randint(0, 3, (5000,), generator=g).tolist()
    off = ru.offsets(ls)
    x, w = ru.randn(g, int(off[-1]), 16, dtype=torch.bfloat16), ru.randn(g, 5000, 16, 24, dtype=torch.bfloat16)
    ru.say("many segments")
    out = sr().matmul(x.cuda(), w.cuda(), off.cuda())
    ref, mag = ru.matmul(x, w, off)
    ru.assert_close(out, ref, mag, 16, "matmul")
    y = ru.randn(g, int(off[-1]), 24, dtype=torch.bfloat16)
    dw = sr().outer(x.cuda(), y.cuda(), off.cuda())
    ref, mag = ru.outer(x, y, off)
    ru.assert_close(dw, ref, mag, 2, "outer")


def test_gradients_against_differences():
    """d/dx and d/dw of a loss <g, x W> by the calls' own forms: the loss is
    linear in each, so a difference of any size is exact up to rounding."""
    g = ru.gen(21)
    off = ru.offsets([9, 0, 40, 1])
    n, k, m = int(off[-1]), 24, 36
    x, w, c = ru.randn(g, n, k), ru.randn(g, 4, k, m), ru.randn(g, n, m)
    dx_dir, dw_dir = ru.randn(g, n, k), ru.randn(g, 4, k, m)
    ru.say("gradients of matmul")
    s = sr()
    loss = lambda a, b: (s.matmul(a.cuda(), b.cuda(), off.cuda()).double().cpu() * c.double()).sum()  # noqa: E731
    dx = s.matmul(c.cuda(), w.cuda(), off.cuda(), transpose=True).cpu().double()
    dw = s.outer(x.cuda(), c.cuda(), off.cuda()).cpu().double()
    # 2 losses of n * m terms, each a sum of k products rounded in 32 bits
    scale = float((x.abs().double().sum() + dx_dir.abs().double().sum()) * w.abs().max() * c.abs().max() * m)
    assert abs((loss(x + dx_dir, w) - loss(x, w)) - (dx * dx_dir.double()).sum()) <= 4 * (k + 8) * 2.0 ** -23 * scale
    scale = float(x.abs().double().sum() * (w.abs().max() + dw_dir.abs().max()) * c.abs().max() * m)
    assert abs((loss(x, w + dw_dir) - loss(x, w)) - (dw * dw_dir.double()).sum()) <= 4 * (k + 8) * 2.0 ** -23 * scale


def test_refusals():
    s = sr()
    x = torch.zeros(4, 8, device="cuda")
    w = torch.zeros(2, 8, 6, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    for bad in (
        lambda: s.matmul(x.cpu(), w, off), lambda: s.matmul(x, w.cpu(), off), lambda: s.matmul(x.t(), w, off),
        lambda: s.matmul(x, w, off, transpose=True), lambda: s.matmul(x, w[:1], off),
        lambda: s.matmul(x, w, off.int()), lambda: s.matmul(x, w, off, rows=torch.zeros(4, 1, device="cuda").long()),
        lambda: s.matmul(x, w, off, out=torch.zeros(4, 5, device="cuda")),
        lambda: s.matmul(x, w.transpose(1, 2), off, transpose=True),
        lambda: s.outer(x, torch.zeros(3, 6, device="cuda"), off), lambda: s.outer(x, x.t(), off),
        lambda: s.outer(x, x, off, out=torch.zeros(2, 8, 7, device="cuda")),
    ):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: s.matmul(x.int(), w, off), lambda: s.matmul(x, w.bfloat16(), off),
                lambda: s.outer(x, x.half(), off), lambda: s.outer(x, x, off, out_dtype=torch.bfloat16),
                lambda: s.outer(x.double(), x.double(), off)):
        with pytest.raises(TypeError):
            bad()
