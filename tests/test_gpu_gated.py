"""segred_gated and its gradient (GPU only) against 64-bit forms: every kernel of
the dispatch, ragged and empty segments, gathered and missing rows, odd sizes, all
activations."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh", "relu"]


def _case(t, lengths, k, m, base=0, extra=0, gather=None, seed=0, std=1.0):
    g = A.gen(seed + k * 31 + m)
    off = A.offsets(lengths, base)
    n = int(off[-1]) + extra
    src = n if gather is None else gather
    x = A.randn(g, src, k, dtype=A.TYPES[t])
    w = A.randn(g, len(lengths), 2 * m, k, dtype=A.TYPES[t], std=std * k ** -0.5)
    d = A.randn(g, n, m, dtype=A.TYPES[t])
    rows = torch.randint(-1, src + 1, (n,), generator=g) if gather is not None else None
    return [v.cuda() if v is not None else None for v in (x, w, off, d, rows)]


def _check(x, w, off, d, rows, act, what):
    A.say(what)
    n, m = d.shape
    out, pair = torch.full((n, m), 7.0, dtype=x.dtype, device="cuda"), torch.full((n, 2 * m), 7.0, dtype=x.dtype, device="cuda")
    assert sr.gated(x, w, off, activation=act, rows=rows, out=out) is out
    torch.cuda.synchronize()
    ref, err = A.gated(x, w, off, act, rows, fill=7.0)
    A.check(out, ref, err, f"{what} out")
    if act == "relu":  # a sum within its error of 0 has either slope
        z = A.gated(x, w, off, act, rows, fill=7.0)[0] != 0
        d = torch.where(z, d, 0)
    assert sr.gated_grad(d, x, w, off, activation=act, rows=rows, out=pair) is pair
    torch.cuda.synchronize()
    ref, err = A.gated(x, w, off, act, rows, grad=d, fill=7.0)
    if act == "relu":
        keep = torch.cat([z, z], 1)
        ref, err, pair = torch.where(keep, ref, 0.0), torch.where(keep, err, 0.0), torch.where(keep, pair, 0)
        # and one that is not 0 but near it
        near = err > 0.01 * ref.abs()
        ref, pair = torch.where(near, 0.0, ref), torch.where(near, 0, pair)
    A.check(pair, ref, err, f"{what} grad")
    inside = torch.zeros(n, dtype=torch.bool, device="cuda")
    inside[int(off[0]):int(off[-1])] = True
    assert (out[~inside] == 7).all() and (act == "relu" or (pair[~inside] == 7).all())


SHAPES = [([3, 0, 1, 9], 64, 32), ([5], 1, 1), ([17, 2, 0, 40], 100, 50), ([1] * 20, 128, 96), ([33, 0, 0, 7], 33, 17),
          ([70, 130, 0, 64], 256, 64), ([16, 15, 17], 520, 24), ([128], 72, 200), ([40, 60], 63, 130)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lengths,k,m", SHAPES)
def test_shapes(t, lengths, k, m):
    for i, act in enumerate(ACTS):
        gather = 11 if i % 2 else None
        _check(*_case(t, lengths, k, m, base=i % 3, extra=i, gather=gather, seed=i), act, f"gated {t} {lengths} {k}x{m} {act}")


# mean rows and tiles on both sides of the rule's limits, for each kernel
KERNELS = [("bf16", [8] * 40, 256, 128), ("bf16", [60, 20, 0, 44, 30, 26], 512, 192), ("bf16", [300, 0, 4500, 1360], 256, 1024),
           ("f16", [4096, 2000, 16, 0, 3000], 320, 1088), ("f16", [129] * 60, 256, 1000), ("bf16", [700, 300, 24], 192, 512),
           ("f32", [6] * 30, 128, 64), ("f32", [20] * 8, 136, 72), ("f32", [500, 0, 301], 128, 300), ("f32", [300, 41], 65, 130),
           ("f32", [2000, 1000], 96, 130), ("bf16", [200, 111], 99, 65)]


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("lengths,k,m", [([1], 1, 1), ([3, 16, 0, 1], 31, 5), ([17, 2], 33, 40), ([8] * 12, 257, 100),
                                         ([8] * 40, 257, 200), ([16], 1023, 515)])
def test_few_rows_that_are_no_whole_units(t, lengths, k, m):
    _check(*_case(t, lengths, k, m, base=1, extra=2, gather=9), "gelu", f"gated {t} {lengths} {k}x{m}")


@pytest.mark.parametrize("t,lengths,k,m", KERNELS)
def test_kernels(t, lengths, k, m):
    n = sum(lengths)
    _check(*_case(t, lengths, k, m), "silu", f"gated {t} n={n} {k}x{m}")
    _check(*_case(t, lengths, k, m, gather=n // 2, seed=1), "gelu", f"gated {t} n={n} {k}x{m} gathered")


@pytest.mark.parametrize("act", ACTS)
def test_far_from_zero(act):
    """Pre-activations to +-1000: where exponentials leave float's range."""
    for t in ("f32", "bf16"):
        _check(*_case(t, [40, 30], 64, 40, std=200.0), act, f"gated {t} {act} large")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_bad_rows_stay_alone(t):
    """Infinities and NaN of a row reach that row alone, those of a segment's weights its rows alone."""
    x, w, off, d, _ = _case(t, [70, 200, 30], 256, 136)
    want, pair = sr.gated(x, w, off), sr.gated_grad(d, x, w, off)
    y, v = x.clone(), w.clone()
    y[5, 3], y[100, 255] = float("nan"), float("inf")
    v[2, 7, 9] = float("nan")
    out, grad = sr.gated(y, v, off), sr.gated_grad(d, y, v, off)
    good = torch.ones(300, dtype=torch.bool, device="cuda")
    good[[5, 100]] = False
    good[270:] = False
    # (float tiles that meet such a value are computed again, with other last bits)
    for a, b in ((out, want), (grad, pair)):
        if t == "f32":
            assert (a[good] - b[good]).abs().max() <= 1e-4 * b.abs().max()
        else:
            assert torch.equal(a[good], b[good])
    assert out[5].isnan().all() and out[270:, 7].isnan().all()
    keep = [i for i in range(136) if i != 7]
    assert out[270:, keep].isfinite().all()


def test_float_range():
    """Sums whose bf16 parts overflow but that float holds."""
    x = torch.zeros(3, 32, device="cuda")
    w = torch.zeros(1, 160, 32, device="cuda")
    x[:, 0], w[0, :80, 0], w[0, 80:, 1] = 3e38, 1.0, 1.0
    x[:, 1] = 1.0
    out = sr.gated(x.repeat(100, 1), w, torch.tensor([0, 300], device="cuda"), activation="relu")
    assert (out == 3e38).all()


def test_rows_behind_the_last():
    x, w, off, d, _ = _case("bf16", [10, 20], 64, 32, extra=40)
    off = torch.tensor([0, 10, 90], device="cuda")  # reaches past the 70 rows: those are not touched
    out = sr.gated(x, w, off)
    ref, err = A.gated(x, w, torch.tensor([0, 10, 70]), "silu")
    A.check(out, ref, err, "an end past the rows")


def test_no_rows_and_no_segments():
    w = torch.zeros(2, 64, 16, device="cuda")
    assert sr.gated(torch.empty(0, 16, device="cuda"), w, torch.zeros(3, dtype=torch.int64, device="cuda")).shape == (0, 32)
    out = torch.full((5, 32), 3.0, device="cuda")
    sr.gated(torch.zeros(5, 16, device="cuda"), w[:0], torch.zeros(1, dtype=torch.int64, device="cuda"), out=out)
    assert (out == 3).all()


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("k,m", [(64, 128), (13, 7)])
def test_no_source_rows_at_all(t, k, m):
    """Operands without a row, of which every row that is named is missing: act(0) * 0."""
    none, w = torch.empty(0, k, dtype=A.TYPES[t], device="cuda"), torch.ones(2, 2 * m, k, dtype=A.TYPES[t], device="cuda")
    rows, off = torch.tensor([0, -1, 5], device="cuda"), torch.tensor([0, 1, 3], device="cuda")
    assert not sr.gated(none, w, off, rows=rows).any()
    assert not sr.gated_grad(torch.ones(3, m, dtype=A.TYPES[t], device="cuda"), none, w, off, rows=rows).any()


def test_refusals():
    x, w = torch.zeros(4, 16, device="cuda"), torch.zeros(2, 64, 16, device="cuda")
    off, d = torch.tensor([0, 2, 4], device="cuda"), torch.zeros(4, 32, device="cuda")
    for bad in (dict(activation="tanh"), dict(weights=torch.zeros(2, 63, 16, device="cuda")), dict(weights=w[0]),
                dict(weights=w[:1]), dict(weights=torch.zeros(2, 64, 15, device="cuda")), dict(offsets=off.int()),
                dict(offsets=off.cpu()), dict(rows=torch.zeros(4, device="cuda")), dict(values=x.cpu()), dict(out=d[:, :31])):
        with pytest.raises(ValueError):
            sr.gated(**{"values": x, "weights": w, "offsets": off, **bad})
    with pytest.raises(TypeError):
        sr.gated(x, w.half(), off)
    with pytest.raises(ValueError):
        sr.gated_grad(d[:3], x, w, off)
    with pytest.raises(ValueError):
        sr.gated_grad(d.half(), x, w, off)
