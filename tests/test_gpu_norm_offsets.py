"""segred_norm and its gradient (GPU only) for rows far from zero: a row's mean is no
part of the result, so what is lost is measured by the row's spread alone."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu

# both sides of every kernel's limits, and widths w for which w * fl(1 / w) is not 1 in float32
WIDTHS = [1, 2, 41, 55, 97, 128, 129, 333, 512, 615, 1000, 1023, 1763, 2048, 2745, 4096, 5125, 8192, 12005, 16384, 16405, 20011]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k", WIDTHS)
def test_constant_rows(t, k):
    """x - mean is 0 whatever the constant is: the bias stays, and 0 / 0 with eps = 0."""
    c = torch.tensor([1.0, 3.0, -1000.0, 999.9, 0.1, 31000.0, -7.7, 12345.6], device="cuda").to(A.TYPES[t])
    x = c[:, None].repeat(1, k).contiguous()
    g = A.gen(k)
    w, b = (A.randn(g, k) + 1).cuda(), A.randn(g, k).cuda()
    d = A.randn(g, 8, k, dtype=A.TYPES[t]).cuda()
    A.say(f"constant rows {t} {k}")
    out, dx = sr.norm(x, w, b), sr.norm_grad(d, x, w)[0]
    none, none_dx = sr.norm(x, w, b, eps=0.0), sr.norm_grad(d, x, w, eps=0.0)[0]
    torch.cuda.synchronize()
    assert torch.equal(out, b.to(x.dtype).expand(8, k))
    assert none.isnan().all() and none_dx.isnan().all()
    flat = torch.zeros(8, k, dtype=torch.float64, device="cuda")
    refs, errs = A.norm_grad(d, flat, w, 1e-5, True)
    A.check(dx, refs[0], errs[0], f"constant rows {t} {k} dx")


@pytest.mark.parametrize("t,level,spread", [("f32", 1e3, 2.0 ** -10), ("f32", 3e4, 2.0 ** -12), ("f32", -4e5, 2.0 ** -10),
                                            ("bf16", 200.0, 2.0 ** -6), ("f16", 3e3, 2.0 ** -8)])
@pytest.mark.parametrize("k", WIDTHS[1:])
def test_rows_far_from_zero(t, level, spread, k):
    """The bounds of rows around zero hold for the same rows beside any level.

    The row is taken around a number near its mean (exactly, or to half a step of the
    difference), and what that misses the mean by is found from the differences, so no
    error is in proportion to the mean but of second order: depth u of half a step of it."""
    g = A.gen(k)
    n = 7
    x = (level * (1 + 0.01 * torch.rand(n, 1, generator=g)) + torch.randn(n, k, generator=g) * abs(level) * spread).to(A.TYPES[t])
    w, b = (A.randn(g, k, std=0.3) + 1).cuda(), A.randn(g, k, std=0.3).cuda()
    d = A.randn(g, n, k, dtype=A.TYPES[t]).cuda()
    x = x.cuda()
    A.say(f"norm {t} {n}x{k} around {level}")
    out = sr.norm(x, w, b)
    dx, dw, db = sr.norm_grad(d, x, w, want_bias=True)
    torch.cuda.synchronize()
    mean = x.double().mean(1, keepdim=True)
    apart = x.double() - mean
    second = (A.depth(k) + 8) * A.U * 2 * A.U * mean.abs()  # of x - mean
    ref, err, unit, r, _, _ = A.norm(apart, w, b, 1e-5, True)
    A.check(out, ref, err + 2 * second * r * w.double().abs(), "out")
    refs, errs = A.norm_grad(d, apart, w, 1e-5, True)
    gw = d.double().abs() * w.double().abs()
    more = r * 2 * second * r * (gw.mean(1, keepdim=True) * (1 + 2 * unit.abs()) + unit.abs() * (gw * unit.abs()).mean(1, keepdim=True))
    A.check(dx, refs[0], errs[0] + more, "dx")
    A.check(dw, refs[1], errs[1] + (d.double().abs() * 2 * second * r).sum(0), "dw")
    A.check(db, refs[2], errs[2], "db")


def test_an_outlier_in_front():
    """The first element is far from all others."""
    for t in ("f32", "bf16"):
        for k in (100, 700, 3000, 9000, 17000):
            g = A.gen(k)
            x = torch.randn(5, k, generator=g)
            x[:, 0] = 1e4
            x, w, d = x.to(A.TYPES[t]).cuda(), (A.randn(g, k, std=0.3) + 1).cuda(), A.randn(g, 5, k, dtype=A.TYPES[t]).cuda()
            A.say(f"norm {t} outlier {k}")
            out = sr.norm(x, w)
            dx, dw, _ = sr.norm_grad(d, x, w)
            torch.cuda.synchronize()
            ref, err, *_ = A.norm(x, w, None, 1e-5, True)
            A.check(out, ref, err, f"outlier {t} {k} out")
            refs, errs = A.norm_grad(d, x, w, 1e-5, True)
            A.check(dx, refs[0], errs[0], f"outlier {t} {k} dx")
            A.check(dw, refs[1], errs[1], f"outlier {t} {k} dw")
