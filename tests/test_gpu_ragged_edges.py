"""Products, adapters and joins over ragged groups at their edges (GPU only):
rows that do not exist, rows named twice, element offsets past 32 bits, many
long requests.  Inputs are compared with plain 64-bit forms."""
import pytest
import torch

from tests import ragged_util as ru
from tests.test_gpu_adapter import _check

pytestmark = pytest.mark.gpu


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("r", [40, 33])
def test_long_requests_of_higher_rank(kind, transpose, r):
    """Enough rows and ranks for the taller tiles of the low-rank rows; requests end inside them."""
    _check(kind, [700, 1, 1300, 0, 63, 1500, 65, 1400, 128], 136, 264, r, transpose, count=4, seed=r)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("segments,mean,k,m", [(64, 90, 256, 256), (3, 2000, 72, 136), (2, 700, 48, 64), (260, 9, 64, 40),
                                               (2, 700, 47, 61)])
def test_outer_of_rows_that_may_not_exist(kind, segments, mean, k, m):
    """Both operands gathered; a row outside the operand counts as zeros, one named twice counts twice."""
    t, g = ru.TYPES[kind], ru.gen(segments + k)
    lengths = torch.randint(0, 2 * mean + 1, (segments,), generator=g)
    lengths[0] = 0
    off = ru.offsets(lengths.tolist(), base=5)
    n, pool = int(off[-1]) + 3, 300
    left, right = ru.randn(g, pool, k, dtype=t), ru.randn(g, pool + 1, m, dtype=t)
    li, ri = torch.randint(0, pool, (n,), generator=g), torch.randint(0, pool + 1, (n,), generator=g)
    li[::13], li[1::29], ri[2::17] = -1, 2 ** 40, pool + 1
    li[3::31], ri[5::37] = -2 ** 62, 2 ** 32
    ru.say(f"outer, missing rows {kind} S={segments} N={n} k={k} m={m}")
    got = sr().outer(left.cuda(), right.cuda(), off.cuda(), left_rows=li.cuda(), right_rows=ri.cuda())
    torch.cuda.synchronize()

    def rows(v, i):
        ok = (i >= 0) & (i < v.shape[0])
        return torch.where(ok[:, None], v[i.clamp(0, v.shape[0] - 1)], 0.0)

    ref, mag = ru.outer(rows(left.double(), li), rows(right.double(), ri), off)
    ru.assert_close(got, ref, mag, int(lengths.max()), "outer")


def test_outer_of_a_tensor_with_itself():
    g = ru.gen(3)
    x = ru.randn(g, 1000, 160, dtype=torch.bfloat16)
    off = ru.offsets([400, 0, 600])
    ru.say("outer of one tensor")
    xc = x.cuda()
    got = sr().outer(xc, xc, off.cuda())
    ref, mag = ru.outer(x, x, off)
    ru.assert_close(got, ref, mag, 600, "outer")
    assert torch.equal(got, got.transpose(1, 2)), "each cell and its mirror sum the same products in the same order"


@pytest.mark.parametrize("kind,k", [("bf16", 2048), ("f32", 1030)])
def test_inputs_past_32_bits(kind, k):
    """Operands of more than 2^31 elements, of which the last rows are used."""
    t, g = ru.TYPES[kind], ru.gen(k)
    n, last, m = 2 ** 31 // k + 5000, 200, 72
    off = ru.offsets([90, 0, 110])
    tail = ru.randn(g, last, k, dtype=t)
    w, y = ru.randn(g, 3, m, k, dtype=t), ru.randn(g, last, m, dtype=t)
    ru.say(f"inputs past 32 bits {kind} {n} x {k}")
    x = torch.zeros(n, k, dtype=t, device="cuda")
    x[n - last:] = tail.cuda()
    rows = torch.arange(n - last, n, device="cuda").flip(0)
    flip = tail.flip(0)
    ref, mag = ru.matmul(flip, w, off, True)
    ru.assert_close(sr().matmul(x, w.cuda(), off.cuda(), transpose=True, rows=rows), ref, mag, k, "matmul")
    ref, mag = ru.outer(flip, y, off)
    ru.assert_close(sr().outer(x, y.cuda(), off.cuda(), left_rows=rows), ref, mag, 110, "outer")
    # segments that begin and end at the far rows, not gathered
    far = off + (n - last)
    ref, mag = ru.outer(tail, y, off)
    wide = torch.zeros(n, m, dtype=t, device="cuda")
    wide[n - last:] = y.cuda()
    ru.assert_close(sr().outer(x, wide, far.cuda()), ref, mag, 110, "outer of far rows")
    weights = torch.rand(last // 2, 2, generator=g)
    position = torch.arange(n - last, n).view(-1, 2)
    out = sr().combine(x, position.cuda(), weights.cuda())
    two = tail.double().view(-1, 2, k) * weights.double()[:, :, None]
    ru.assert_close(out, two.sum(1), two.abs().sum(1), 2, "combine")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_outputs_past_32_bits(kind):
    t, g = ru.TYPES[kind], ru.gen(8)
    n, k, m, r = 66000, 24, 32768, 8
    ru.say(f"outputs past 32 bits {kind} {n} x {m}")
    x, w = ru.randn(g, n, k, dtype=t), ru.randn(g, 2, k, m, dtype=t)
    off = torch.tensor([0, 33000, n])
    out = sr().matmul(x.cuda(), w.cuda(), off.cuda())[-100:].clone()
    ref, mag = ru.matmul(x[-100:], w[1:], torch.tensor([0, 100]))
    ru.assert_close(out, ref, mag, k, "matmul")
    down, up = ru.randn(g, 1, r, k, dtype=t), ru.randn(g, 1, m, r, dtype=t)
    base = w[0].t().contiguous()
    which = torch.tensor([-1, 0])
    got = sr().adapter(x.cuda(), base.cuda(), off.cuda(), which.cuda(), down.cuda(), up.cuda())[-100:].clone()
    ref, mag, part, _, _ = ru.adapter(x[-100:], base, torch.tensor([0, 100]), which[1:], down, up, None, False)
    ru.assert_close(got, ref, mag, 2 * k + r, "adapter", more=0.0 if kind == "f32" else 2.0 ** -16 * part)


@pytest.mark.parametrize("entries,groups", [(262144, 30000), (262145, 30000), (1200000, 700), (1200000, 5000000)])
def test_group_of_many(entries, groups):
    g = ru.gen(entries + groups)
    index = torch.randint(-3, groups + 3, (entries,), generator=g)
    ru.say(f"group entries={entries} groups={groups}")
    got = sr().group(index.cuda(), groups)
    torch.cuda.synchronize()
    for a, b, name in zip(got, ru.group(index, groups), ("order", "position", "offsets")):
        assert torch.equal(a.cpu(), b), name


def test_gathered_calls_replayed():
    """Gathered products and outer sums of more than one step, captured and replayed with other rows each time."""
    g = ru.gen(12)
    s = sr()
    pool, n, k, m = 500, 3000, 256, 264
    off = ru.offsets([900, 0, 1400, 700])
    x, y = ru.randn(g, pool, k, dtype=torch.bfloat16), ru.randn(g, pool, m, dtype=torch.bfloat16)
    w = ru.randn(g, 4, k, m, dtype=torch.bfloat16)
    dev = [v.cuda() for v in (x, y, w, off)]
    rows = torch.zeros(n, dtype=torch.int64, device="cuda")
    ru.say("gathered calls replayed")

    def work():
        return (s.matmul(dev[0], dev[2], dev[3], rows=rows), s.outer(dev[0], dev[1], dev[3], left_rows=rows, right_rows=rows))

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = work()
    for rep in range(4):
        rows.copy_(torch.randint(-2, pool + 2, (n,), generator=g))
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, work()):
            assert torch.equal(a, b), rep
        torch.cuda.synchronize()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("k,m", [(64, 128), (13, 7)])
def test_no_source_rows_at_all(kind, k, m):
    """An operand without a row, of which every row that is named is missing."""
    t = ru.TYPES[kind]
    s = sr()
    none = torch.empty(0, k, dtype=t, device="cuda")
    rows = torch.tensor([0, -1, 5], device="cuda")
    off = torch.tensor([0, 1, 3], device="cuda")
    ru.say(f"no source rows {kind} k={k} m={m}")
    out = s.matmul(none, torch.ones(2, k, m, dtype=t, device="cuda"), off, rows=rows)
    assert out.shape == (3, m) and not out.any()
    right = torch.ones(3, m, dtype=t, device="cuda")
    assert not s.outer(none, right, off, left_rows=rows).any()
    assert not s.outer(right, none, off, right_rows=rows).any()
    assert not s.combine(none, rows.view(3, 1), torch.ones(3, 1, device="cuda")).any()
    values = torch.empty(0, m, dtype=t, device="cuda")
    grad, part = s.combine_grad(right, values, rows.view(3, 1), torch.ones(3, 1, device="cuda"))
    assert grad.shape == (0, m) and not part.any()
    # an adapter call without an adapter, and one whose segments hold no row
    x, w = torch.ones(3, k, dtype=t, device="cuda"), torch.ones(m, k, dtype=t, device="cuda")
    down, up = torch.empty(0, 4, k, dtype=t, device="cuda"), torch.empty(0, m, 4, dtype=t, device="cuda")
    which = torch.tensor([0, 7], device="cuda")
    assert torch.equal(s.adapter(x, w, off, which, down, up), torch.full((3, m), float(k), dtype=t, device="cuda"))


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k,m,r", [(640, 648, 8), (641, 643, 33), (712, 640, 64)])
def test_large_float_adapters(k, m, r, transpose):
    """Enough tiles for float products in bf16 parts, whole units and odd widths."""
    _check("f32", [700, 1, 1300, 0, 63, 1500, 65, 1400, 128], k, m, r, transpose, count=4, seed=5)


@pytest.mark.parametrize("transpose", [False, True])
def test_infinity_and_nan_in_large_float_adapters(transpose):
    """They come out where 64 bits put them, and nowhere else; the other rows keep their accuracy."""
    g = ru.gen(6)
    k, m, r, n = 640, 648, 8, 5000
    off, which = torch.tensor([0, 2000, 2100, n]), torch.tensor([1, -1, 0])
    have = m if transpose else k
    x, w = ru.randn(g, n, have), ru.randn(g, m, k, std=have ** -0.5)
    down, up = ru.randn(g, 2, r, k, std=k ** -0.5), ru.randn(g, 2, m, r, std=r ** -0.5)
    x[3, 5], x[2050, 0], x[4999, 17], x[1000, 3] = float("nan"), float("inf"), -float("inf"), 3e38
    x[1000, 4] = -3e38
    ru.say(f"large float adapter with specials transpose={transpose}")
    got = sr().adapter(*(v.cuda() for v in (x, w, off, which, down, up)), transpose=transpose).cpu()
    ref, mag, _, _, _ = ru.adapter(x, w, off, which, down, up, None, transpose)
    assert torch.equal(got.isnan(), ref.isnan())
    assert torch.equal(got[2050].double(), ref[2050]) and bool((got[2050].abs() == float("inf")).all())
    plain = torch.ones(n, dtype=torch.bool)
    plain[[3, 2050, 4999, 1000]] = False
    ru.assert_close(got[plain], ref[plain], mag[plain], 2 * have + r, "other rows")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,k,m,r", [(90, 64, 96, 8), (700, 64, 96, 40), (700, 61, 99, 5), (5000, 648, 640, 8), (6100, 136, 2048, 33)])
def test_specials_of_an_adapter_stay_with_its_rows(kind, transpose, rows, k, m, r):
    """Infinities and NaN in the second factor of two adapters; requests of others share their tiles."""
    t, g = ru.TYPES[kind], ru.gen(rows + r)
    cuts = torch.randint(0, rows + 1, (23,), generator=g).sort().values.tolist()
    off, which = torch.tensor([0, *cuts, rows]), torch.arange(24) % 5 - 1
    have = m if transpose else k
    x, w = ru.randn(g, rows, have, dtype=t), ru.randn(g, m, k, dtype=t, std=have ** -0.5)
    down, up = ru.randn(g, 4, r, k, dtype=t, std=k ** -0.5), ru.randn(g, 4, m, r, dtype=t, std=r ** -0.5)
    second = down.transpose(1, 2) if transpose else up  # [4, outputs, r]
    second[1, 7, r - 1], second[1, 50, 0], second[3, 40, 2] = float("nan"), float("inf"), -float("inf")
    ru.say(f"specials of an adapter {kind} N={rows} k={k} m={m} r={r} transpose={transpose}")
    got = sr().adapter(*(v.cuda() for v in (x, w, off, which, down.contiguous(), up)), transpose=transpose).cpu()
    ref, mag, part, _, _ = ru.adapter(x, w, off, which, down, up, None, transpose)
    assert torch.equal(got.isfinite(), ref.isfinite())
    if kind == "f32":
        assert torch.equal(got.isnan(), ref.isnan())
    ok = ref.isfinite()
    zero = torch.zeros((), dtype=torch.float64)
    mag, part = torch.where(ok, mag, zero), torch.where(ok, part, zero)
    ru.assert_close(torch.where(ok, got, torch.zeros((), dtype=t)), torch.where(ok, ref, zero), mag, 2 * have + r, "the others",
                    more=0.0 if kind == "f32" else 2.0 ** -16 * part)
