"""Float products of finite values that leave float's range (GPU only): the
calls that make them of bf16 parts give the infinity that float arithmetic
gives.  All terms of a sum share a sign, so that any order of adding passes the
range, or does not, with the sum itself."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

MOST = torch.finfo(torch.float32).max


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


def scaled(g, rows, cols, by_row, low, high, signs):
    """Values of 1 to 2 times a power of ten per row (or column), 10^low .. 10^high, of one sign each if `signs`."""
    n = rows if by_row else cols
    s = 10.0 ** (low + (high - low) * torch.rand(n, generator=g, dtype=torch.float64))
    if signs:
        s = s * (torch.randint(0, 2, (n,), generator=g) * 2 - 1)
    return ((1 + torch.rand(rows, cols, generator=g, dtype=torch.float64)) * (s[:, None] if by_row else s)).float()


def check(got, ref, mag, n, what):
    got = got.cpu()
    over, under = ref.abs() > MOST * (1 + 2.0 ** -10), ref.abs() < MOST * (1 - 2.0 ** -10)
    assert over.any() and under.any()
    assert not got[over | under].isnan().any(), (what, int(got[over | under].isnan().sum()))
    want = torch.where(ref > 0, float("inf"), -float("inf"))
    assert bool((got[over].double() == want[over]).all()), what
    ru.assert_close(got[under], ref[under], mag[under], n, what)


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k,m", [(256, 512), (131, 333)])
def test_matmul(transpose, k, m):
    g = ru.gen(k)
    off = ru.offsets([900, 0, 700, 1200, 1300])
    x = scaled(g, 4100, k, True, 0, 30, False)
    w = torch.stack([scaled(g, k, m, False, 0, 30, True) for _ in range(5)])
    ref, mag = ru.matmul(x, w, off)
    ru.say(f"overflow matmul k={k} m={m} transpose={transpose}")
    given = w.transpose(1, 2).contiguous() if transpose else w
    check(sr().matmul(x.cuda(), given.cuda(), off.cuda(), transpose=transpose), ref, mag, k, "matmul")


@pytest.mark.parametrize("k,m,lengths", [(256, 512, [500] * 16 + [0]), (64, 96, [3000, 0, 2000]), (33, 45, [700, 2300]),
                                         (200, 130, [60, 0, 80])])
def test_outer(k, m, lengths):
    """Whole segments, and pieces that are added afterwards."""
    g = ru.gen(k + m)
    off = ru.offsets(lengths)
    n = int(off[-1])
    x, y = scaled(g, n, k, False, 0, 30, True), scaled(g, n, m, False, 0, 30, True)
    ref, mag = ru.outer(x, y, off)
    ru.say(f"overflow outer k={k} m={m}")
    check(sr().outer(x.cuda(), y.cuda(), off.cuda()), ref, mag, max(lengths), "outer")
    short = x.bfloat16()
    ref, mag = ru.outer(short, y, off)
    check(sr().outer(short.cuda(), y.cuda(), off.cuda(), out_dtype=torch.float32), ref, mag, max(lengths), "bf16 and f32")
    got = sr().outer(y.cuda(), short.cuda(), off.cuda(), out_dtype=torch.float32)
    check(got, ref.transpose(1, 2), mag.transpose(1, 2), max(lengths), "f32 and bf16")


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k,m", [(640, 648), (643, 645)])
def test_adapter(transpose, k, m):
    g = ru.gen(m)
    off, which = ru.offsets([700, 1, 1300, 0, 1500, 1600]), torch.tensor([0, 1, -1, 0, 1, 0])
    have, give = (m, k) if transpose else (k, m)
    x, w = scaled(g, 5101, have, True, 0, 30, False), scaled(g, have, give, False, 0, 30, True)
    w = w if transpose else w.t().contiguous()
    down, up = torch.zeros(2, 8, k), torch.zeros(2, m, 8)
    ref, mag, _, _, _ = ru.adapter(x, w, off, which, down, up, None, transpose)
    ru.say(f"overflow adapter k={k} m={m} transpose={transpose}")
    got = sr().adapter(*(v.cuda() for v in (x, w, off, which, down, up)), transpose=transpose)
    check(got, ref, mag, have, "adapter")
