"""Sums of outer products with a 16-bit and a float32 side, and the gradients
of 16-bit adapters' factors made from float32 low-rank rows (GPU only).

The 16-bit side enters exactly.  Of a product with the float32 side, in bf16
parts, less than 2^-22 is left out, under two of the units (2^-23) that each
term has in the bound of a 32-bit sum, whose eight spare ones hold that.
"""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

LENGTHS = {
    "mixed": [0, 5, 1, 130, 17, 0, 300, 64],
    "single": [1] * 20 + [3, 0, 2],
    "long": [700, 0, 1033, 513],
    "pieces": [9001, 20000],
    "empty": [0, 0],
}
WIDTHS = [(64, 128), (200, 72), (33, 45), (1, 1), (264, 8), (40, 300)]


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("wide_left", [False, True])
@pytest.mark.parametrize("lengths", LENGTHS)
def test_outer_of_two_types(kind, wide_left, lengths):
    short, ls = ru.TYPES[kind], LENGTHS[lengths]
    for i, (k, m) in enumerate(WIDTHS):
        g = ru.gen(100 * i + len(ls))
        off = ru.offsets(ls, base=3)
        n, pool = int(off[-1]) + 4, 50
        lt, rt = (torch.float32, short) if wide_left else (short, torch.float32)
        left, right = ru.randn(g, n, k, dtype=lt), ru.randn(g, pool, m, dtype=rt)
        rows = torch.randint(0, pool, (n,), generator=g)
        ref, mag = ru.outer(left, right, off, right_rows=rows)
        for odt in (short, torch.float32):
            ru.say(f"outer {lt} {rt} -> {odt} {lengths} k={k} m={m}")
            got = sr().outer(left.cuda(), right.cuda(), off.cuda(), right_rows=rows.cuda(), out_dtype=odt)
            torch.cuda.synchronize()
            assert got.dtype == odt
            ru.assert_close(got, ref, mag, max(ls), "outer")
        out = torch.full((len(ls), m, k), 7.0, dtype=short, device="cuda")
        sr().outer(right.cuda(), left.cuda(), off.cuda(), left_rows=rows.cuda(), out=out)
        torch.cuda.synchronize()
        ru.assert_close(out, ref.transpose(1, 2), mag.transpose(1, 2), max(ls), "outer, left gathered")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k,m", [(64, 128), (33, 45)])
def test_single_products_keep_their_bits(kind, k, m):
    """One row a segment: a product alone, off by its parts left out (2^-22) and
    two roundings to float32 (2^-24 each).  Without the third part of a float
    it would be off by up to 2^-17."""
    g = ru.gen(k)
    t = ru.TYPES[kind]
    x, y = ru.randn(g, 300, k, dtype=t), ru.randn(g, 300, m)
    off = torch.arange(301)
    ref = x.double()[:, :, None] * y.double()[:, None, :]
    ru.say(f"single products {kind} {k}x{m}")
    for got, want in ((sr().outer(x.cuda(), y.cuda(), off.cuda(), out_dtype=torch.float32), ref),
                      (sr().outer(y.cuda(), x.cuda(), off.cuda(), out_dtype=torch.float32), ref.transpose(1, 2))):
        err = (got.cpu().double() - want).abs()
        assert bool((err <= (2.0 ** -22 + 2.0 ** -23) * want.abs() + 2.0 ** -125).all())


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("k,m", [(64, 128), (130, 45)])
def test_specials_of_either_side(kind, k, m):
    """Infinities and NaN come out where 64 bits put them, whichever side has them."""
    g = ru.gen(k + m)
    off = ru.offsets([30, 400, 0, 7, 90])
    n = int(off[-1])
    x, y = ru.randn(g, n, k, dtype=ru.TYPES[kind]), ru.randn(g, n, m)
    x[5, 3], x[100, k - 1], y[200, 7], y[435, m - 1] = float("inf"), float("nan"), -float("inf"), float("nan")
    ru.say(f"specials of two types {kind} {k}x{m}")
    for turn in (False, True):
        got = sr().outer(*((y.cuda(), x.cuda()) if turn else (x.cuda(), y.cuda())), off.cuda(), out_dtype=torch.float32)
        ref, mag = ru.outer(y, x, off) if turn else ru.outer(x, y, off)
        got = got.cpu()
        assert torch.equal(got.isnan(), ref.isnan()) and torch.equal(got.isinf(), ref.isinf())
        inf = ref.isinf()
        assert torch.equal(got[inf].double(), ref[inf])
        ok = ref.isfinite()
        ru.assert_close(got[ok], ref[ok], mag[ok], 400, "the others")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("k,m,r", [(48, 80, 8), (520, 264, 40), (61, 99, 5)])
def test_gradients_of_factors_are_rounded_once(kind, k, m, r):
    """A training step of adapters that own several segments: output, input
    gradient, and both factors' gradients, each off by half a step of its type
    and its 32-bit sums alone."""
    s = sr()
    t, g = ru.TYPES[kind], ru.gen(k + r)
    ls, which, count = [30, 0, 170, 64, 5, 333], torch.tensor([1, 0, 0, 1, 2, -1]), 4
    off = ru.offsets(ls)
    n = int(off[-1])
    x, c = ru.randn(g, n, k, dtype=t), ru.randn(g, n, m, dtype=t)
    w = ru.randn(g, m, k, dtype=t, std=k ** -0.5)
    down, up = ru.randn(g, count, r, k, dtype=t, std=k ** -0.5), ru.randn(g, count, m, r, dtype=t, std=r ** -0.5)
    scale = torch.rand(count, generator=g) + 0.5
    row_which = which.repeat_interleave(torch.tensor(ls))
    ru.say(f"adapter gradients {kind} k={k} m={m} r={r}")
    args = (w.cuda(), off.cuda(), which.cuda(), down.cuda(), up.cuda())
    out, low = s.adapter(x.cuda(), *args, scale=scale.cuda(), want_low=torch.float32)
    dx, glow = s.adapter(c.cuda(), *args, scale=scale.cuda(), transpose=True, want_low=torch.float32)
    order, _, bounds = s.group(row_which.cuda(), count)
    dup = s.outer(c.cuda(), low, bounds, left_rows=order, right_rows=order, out_dtype=t)
    ddown = s.outer(glow, x.cuda(), bounds, left_rows=order, right_rows=order, out_dtype=t)
    torch.cuda.synchronize()
    assert low.dtype == glow.dtype == torch.float32 and dup.dtype == ddown.dtype == t
    more = 0.0 if kind == "f32" else 2.0 ** -16  # the low-rank rows enter the second product as two bf16
    ref, mag, part, rlow, mlow = ru.adapter(x, w, off, which, down, up, scale)
    ru.assert_close(out, ref, mag, 2 * k + r, "out", more=more * part)
    ru.assert_close(low, rlow, mlow, k, "low")
    gref, gmag, gpart, rglow, mglow = ru.adapter(c, w, off, which, down, up, scale, transpose=True)
    ru.assert_close(dx, gref, gmag, 2 * m + r, "grad of x", more=more * gpart)
    ru.assert_close(glow, rglow, mglow, m, "low of the gradient")
    # the formula's: d/dU of <c, low U^T>, and of D from the gradient's low-rank rows
    rows = [row_which == j for j in range(count)]
    for name, got, a, b, ma, mb, terms in (
            ("grad of up", dup, c.double(), rlow, c.double().abs(), mlow, n + k),
            ("grad of down", ddown, rglow, x.double(), mglow, x.double().abs(), n + m)):
        ref = torch.stack([a[i].t() @ b[i] for i in rows])
        mag = torch.stack([ma[i].t() @ mb[i] for i in rows])
        ru.assert_close(got, ref, mag, terms, name)
    assert (dup[3].cpu() == 0).all() and (ddown[3].cpu() == 0).all()
    # against differences: <c, out> is linear in up
    if kind == "f32":
        step = ru.randn(g, count, m, r)
        moved = s.adapter(x.cuda(), w.cuda(), off.cuda(), which.cuda(), down.cuda(), (up + step).cuda(), scale=scale.cuda())
        diff = ((moved.cpu().double() - out.cpu().double()) * c.double()).sum()
        bound = 4 * (2 * k + r + 8) * 2.0 ** -23 * float((c.double().abs() * (mag_of(x, w, off, which, down, up, scale)
                                                         + mag_of(x, w, off, which, down, step, scale))).sum())
        assert abs(diff - (dup.cpu().double() * step.double()).sum()) <= bound


def mag_of(x, w, off, which, down, up, scale):
    return ru.adapter(x, w, off, which, down, up, scale)[1]


def test_low_rank_rows_of_a_16_bit_call_as_asked():
    """True: of the values' type, the float32 rows rounded; zeros without an adapter in both."""
    g = ru.gen(4)
    for kind in ("bf16", "f16"):
        t = ru.TYPES[kind]
        x, w = ru.randn(g, 90, 64, dtype=t), ru.randn(g, 72, 64, dtype=t)
        down, up = ru.randn(g, 2, 12, 64, dtype=t), ru.randn(g, 2, 72, 12, dtype=t)
        off, which = ru.offsets([40, 0, 30, 20]), torch.tensor([1, 0, -1, 0])
        args = [v.cuda() for v in (x, w, off, which, down, up)]
        ru.say(f"low-rank rows {kind}")
        out, low = sr().adapter(*args, want_low=True)
        same, wide = sr().adapter(*args, want_low=torch.float32)
        named = sr().adapter(*args, want_low=t)[1]
        assert low.dtype == t and torch.equal(out, same) and torch.equal(low, wide.to(t)) and torch.equal(low, named)
        assert torch.equal(sr().adapter(*args, want_low=1)[1], low) and torch.equal(sr().adapter(*args, want_low=0), out)
        assert not wide[40:70].any() and not low[40:70].any()


def test_refusals():
    x, y = torch.zeros(4, 8, device="cuda"), torch.zeros(4, 6, device="cuda")
    off = torch.tensor([0, 2, 4], device="cuda")
    for bad in (lambda: sr().outer(x.half(), y, off), lambda: sr().outer(x, y.bfloat16(), off),
                lambda: sr().outer(x.half(), y.bfloat16(), off, out_dtype=torch.float32),
                lambda: sr().outer(x.half(), y, off, out_dtype=torch.bfloat16),
                lambda: sr().outer(x, y, off, out_dtype=torch.float16)):
        with pytest.raises(TypeError):
            bad()
    w, d, u = torch.zeros(6, 8, device="cuda"), torch.zeros(3, 2, 8, device="cuda"), torch.zeros(3, 6, 2, device="cuda")
    which = torch.tensor([0, 1], device="cuda")
    for low in (torch.float16, torch.int32):
        with pytest.raises(TypeError):
            sr().adapter(x, w, off, which, d, u, want_low=low)
