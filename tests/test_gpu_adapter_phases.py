"""Adapters beside large 16-bit projections (GPU only): sizes at which the tiles
of 128 or 256 rows by 256 columns are taken, which needs 256 columns and 128
tiles of 128 rows, in both directions, and what an infinity or a NaN does there."""
import pytest
import torch

from tests import ragged_util as ru
from tests.test_gpu_adapter import _check

pytestmark = pytest.mark.gpu


def cuts(rows, segments, seed):
    """Uneven segments of `rows` in all, an empty one and one of a single row among them."""
    at = torch.randint(0, rows + 1, (segments - 4,), generator=ru.gen(seed)).sort().values.tolist()
    at = sorted([*at, rows // 2, rows // 2, rows // 2 + 1])
    return [b - a for a, b in zip([0, *at], [*at, rows])]


# (rows, k, m): 44 * 3 tiles of 128 rows in either direction; 17 * 8; and 48 * 8 forwards, where 256 rows save a round
SIZES = [(5600, 648, 640), (2100, 1800, 2048), (6100, 264, 2048)]


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,k,m", SIZES)
@pytest.mark.parametrize("r", [33, 40])
def test_large_tiles(kind, transpose, rows, k, m, r):
    """Requests that end inside tiles, some without an adapter, ranks of more than one step, the low-rank rows too."""
    _check(kind, cuts(rows, 15, rows), k, m, r, transpose, count=4, which=torch.arange(15) % 6 - 1, seed=r)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("transpose", [False, True])
def test_one_adapter_for_all_and_none(kind, transpose):
    _check(kind, [5700], 648, 640, 16, transpose, which=torch.tensor([2]))
    _check(kind, [2000, 3700], 648, 640, 16, transpose, which=torch.tensor([-1, 7]))


def specials(kind, transpose, rows, k, m, r, seed):
    t, g = ru.TYPES[kind], ru.gen(seed)
    off, which = ru.offsets(cuts(rows, 24, seed)), torch.arange(24) % 5 - 1
    have = m if transpose else k
    x, w = ru.randn(g, rows, have, dtype=t), ru.randn(g, m, k, dtype=t, std=have ** -0.5)
    down, up = ru.randn(g, 4, r, k, dtype=t, std=k ** -0.5), ru.randn(g, 4, m, r, dtype=t, std=r ** -0.5)
    return off, which, x, w, down, up, have


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("rows,k,m", SIZES)
def test_specials_stay_with_their_rows(kind, transpose, rows, k, m):
    import segmented_reduction_amd as sr
    r = 33
    off, which, x, w, down, up, have = specials(kind, transpose, rows, k, m, r, 7)
    x[rows // 3, 4], x[rows // 2, 9], x[5, 0] = float("nan"), float("inf"), -float("inf")
    second = down.transpose(1, 2) if transpose else up  # [4, outputs, r]
    second[1, 7, r - 1], second[1, 260, 0], second[3, 40, 2] = float("nan"), float("inf"), -float("inf")
    second[2] = float("nan")
    ru.say(f"specials in large tiles {kind} N={rows} k={k} m={m} transpose={transpose}")
    got = sr.adapter(*(v.cuda() for v in (x, w, off, which, down, up)), transpose=transpose).cpu()
    ref, mag, part, _, _ = ru.adapter(x, w, off, which, down, up, None, transpose)
    assert torch.equal(got.isfinite(), ref.isfinite())
    ok = ref.isfinite()
    assert ok.any()
    zero = torch.zeros((), dtype=torch.float64)
    mag, part = torch.where(ok, mag, zero), torch.where(ok, part, zero)
    ru.assert_close(torch.where(ok, got, torch.zeros((), dtype=x.dtype)), torch.where(ok, ref, zero), mag, 2 * have + r,
                    "the others", more=2.0 ** -16 * part)


@pytest.mark.parametrize("transpose", [False, True])
def test_a_bad_adapter_does_not_hold_up_the_others(transpose):
    """Requests of an adapter of NaN among others: tiles that hold both are
    computed a second time in smaller ones, so the call takes a few times as
    long (and took 300 to 500 times as long with a walk per element)."""
    import segmented_reduction_amd as sr
    off, which, x, w, down, up, _ = specials("bf16", transpose, 6000, 2048, 2048, 32, 8)
    dev = [v.cuda() for v in (x, w, off, which, down, up)]
    ru.say(f"time beside a bad adapter transpose={transpose}")

    def best():
        times = []
        for _ in range(12):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            sr.adapter(*dev, transpose=transpose)
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    good = best()
    dev[4 if transpose else 5][1] = float("nan")
    assert best() < 20 * good
