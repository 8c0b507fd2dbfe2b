"""A shared projection with a low-rank adapter per segment (GPU only).

Beside the bound of a 32-bit sum, the 16-bit calls hold the low-rank rows as
two bf16, which is off by 2^-17 relative at most (and float16's second factor
is split the same way): 2^-16 of the magnitude of the adapters' part in all.
"""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

LENGTHS = {
    "mixed": [0, 5, 1, 130, 17, 0, 300, 64],
    "single-tokens": [1] * 48,
    "one-token": [1],
    "hundreds": [100, 0, 133, 90, 1],
    "long": [700, 0, 1033, 513],
    "empty": [0, 0],
}
WIDTHS = [(64, 128, 16), (200, 72, 8), (33, 45, 5), (512, 264, 64), (256, 512, 4), (520, 512, 40), (128, 64, 100)]


def _check(kind, ls, k, m, r, transpose, count=3, scaled=True, which=None, seed=0, base=2):
    import segmented_reduction_amd as sr
    t, g = ru.TYPES[kind], ru.gen(seed + k + r)
    off = ru.offsets(ls, base=base)
    n = int(off[-1]) + 3
    have, give = (m, k) if transpose else (k, m)
    x = ru.randn(g, n, have, dtype=t)
    w = ru.randn(g, m, k, dtype=t, std=have ** -0.5)
    down, up = ru.randn(g, count, r, k, dtype=t, std=k ** -0.5), ru.randn(g, count, m, r, dtype=t, std=r ** -0.5)
    scale = torch.rand(count, generator=g) + 0.5 if scaled else None
    if which is None:
        which = torch.randint(-1, count + 1, (len(ls),), generator=g)
    ru.say(f"adapter {kind} S={len(ls)} N={n} k={k} m={m} r={r} transpose={transpose} scaled={scaled}")
    out = torch.full((n, give), 7.0, dtype=t, device="cuda")
    cuda = lambda v: None if v is None else v.cuda()  # noqa: E731
    got, low = sr.adapter(x.cuda(), w.cuda(), off.cuda(), which.cuda(), down.cuda(), up.cuda(), scale=cuda(scale),
                          transpose=transpose, want_low=True, out=out)
    torch.cuda.synchronize()
    assert got is out and low.shape == (n, r)
    ref, mag, part, rlow, mlow = ru.adapter(x, w, off, which, down, up, scale, transpose, fill=7.0)
    # the error of the 32-bit low-rank rows passes through the second factor: its terms are in mag
    ru.assert_close(out, ref, mag, 2 * have + r, "out", more=0.0 if kind == "f32" else 2.0 ** -16 * part)
    a, b = int(off[0]), int(off[-1])
    ru.assert_close(low[a:b], rlow[a:b], mlow[a:b], have, "low")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lengths", LENGTHS)
@pytest.mark.parametrize("transpose", [False, True])
def test_adapter(kind, lengths, transpose):
    for k, m, r in WIDTHS:
        _check(kind, LENGTHS[lengths], k, m, r, transpose)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("segments", [1, 16, 17, 40, 64, 65, 100])
def test_single_tokens_of_many_adapters(kind, segments):
    which = torch.randperm(128, generator=ru.gen(segments))[:segments]
    for transpose in (False, True):
        _check(kind, [1] * segments, 1024, 256, 16, transpose, count=128, which=which, base=0)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_adapters_that_alternate_and_none_at_all(kind):
    ls = [3] * 40
    _check(kind, ls, 96, 160, 8, False, count=2, which=torch.arange(40) % 2)
    _check(kind, ls, 96, 160, 8, True, count=2, which=torch.arange(40) % 2, scaled=False)
    _check(kind, ls, 96, 160, 8, False, count=2, which=torch.full((40,), -1))
    _check(kind, ls, 96, 160, 8, False, count=0, which=torch.zeros(40, dtype=torch.int64))


def test_low_rank_rows_past_float16():
    """Low-rank rows beyond float16's range are held; only the result has to fit."""
    import segmented_reduction_amd as sr
    x = torch.full((3, 64), 64.0, dtype=torch.float16)
    w = torch.zeros(32, 64, dtype=torch.float16)
    down = torch.full((1, 8, 64), 64.0, dtype=torch.float16)  # low = 64 * 64 * 64 = 262144
    up = torch.full((1, 32, 8), 2.0 ** -12, dtype=torch.float16)
    ru.say("adapter past float16")
    out = sr.adapter(x.cuda(), w.cuda(), torch.tensor([0, 3]).cuda(), torch.tensor([0]).cuda(), down.cuda(), up.cuda())
    assert (out.cpu() == 8 * 64.0).all()


def test_nan_of_a_request_stays_in_it():
    import segmented_reduction_amd as sr
    for kind in ("bf16", "f16", "f32"):
        t, g = ru.TYPES[kind], ru.gen(2)
        x, w = ru.randn(g, 40, 64, dtype=t), ru.randn(g, 96, 64, dtype=t, std=0.1)
        down, up = ru.randn(g, 3, 8, 64, dtype=t), ru.randn(g, 3, 96, 8, dtype=t)
        off, which = ru.offsets([10] * 4), torch.tensor([0, 1, 2, 0])
        down[1] = float("nan")  # the adapter of rows 10..19 only
        x[33, 4] = float("inf")
        ru.say(f"adapter nan {kind}")
        out = sr.adapter(x.cuda(), w.cuda(), off.cuda(), which.cuda(), down.cuda(), up.cuda()).cpu()
        assert out[10:20].isnan().all() and not torch.isfinite(out[33]).any()
        rest = [r for r in range(40) if not 10 <= r < 20 and r != 33]
        assert torch.isfinite(out[rest]).all()


def test_gradients_of_both_factors():
    """Output, input gradient and the factors' gradients of a step over adapters that own several segments."""
    import segmented_reduction_amd as sr
    g = ru.gen(12)
    ls, which = [30, 0, 17, 64, 5], torch.tensor([1, 0, 0, 1, 2])
    off = ru.offsets(ls)
    n, k, m, r, count = int(off[-1]), 48, 80, 8, 4
    x, w = ru.randn(g, n, k), ru.randn(g, m, k, std=k ** -0.5)
    down, up, scale = ru.randn(g, count, r, k, std=k ** -0.5), ru.randn(g, count, m, r), torch.rand(count, generator=g)
    c = ru.randn(g, n, m)
    row_which = which.repeat_interleave(torch.tensor(ls))
    ru.say("adapter gradients")
    args = (w.cuda(), off.cuda(), which.cuda(), down.cuda(), up.cuda())
    _, low = sr.adapter(x.cuda(), *args, scale=scale.cuda(), want_low=True)
    dx, glow = sr.adapter(c.cuda(), *args, scale=scale.cuda(), transpose=True, want_low=True)
    order, _, bounds = sr.group(row_which.cuda(), count)
    dup = sr.outer(c.cuda(), low, bounds, left_rows=order, right_rows=order)
    ddown = sr.outer(glow, x.cuda(), bounds, left_rows=order, right_rows=order)
    torch.cuda.synchronize()
    leaves = [v.double().requires_grad_() for v in (x, down, up)]
    xd, dd, ud = leaves
    out = xd @ w.double().t()
    lowd = scale.double()[row_which, None] * torch.einsum("nk,nrk->nr", xd, dd[row_which])
    out = out + torch.einsum("nr,nmr->nm", lowd, ud[row_which])
    (out * c.double()).sum().backward()
    with torch.no_grad():
        _, mag, _, _, _ = ru.adapter(c, w, off, which, down, up, scale, transpose=True)
        ru.assert_close(dx, xd.grad, mag, 2 * m + r, "grad of x")
        mlow = scale.double()[row_which, None] * torch.einsum("nk,nrk->nr", x.double().abs(), down.double().abs()[row_which])
        mg = scale.double()[row_which, None] * torch.einsum("nm,nmr->nr", c.double().abs(), up.double().abs()[row_which])
        mup = torch.zeros(count, m, r, dtype=torch.float64).index_add_(
            0, row_which, c.double().abs()[:, :, None] * mlow[:, None, :])
        mdown = torch.zeros(count, r, k, dtype=torch.float64).index_add_(
            0, row_which, mg[:, :, None] * x.double().abs()[:, None, :])
        ru.assert_close(dup, ud.grad, mup, n + k, "grad of up")
        ru.assert_close(ddown, dd.grad, mdown, n + m, "grad of down")
    assert (dup[3].cpu() == 0).all() and (ddown[3].cpu() == 0).all()


def test_refusals():
    import segmented_reduction_amd as sr
    z = lambda *s: torch.zeros(*s, device="cuda")  # noqa: E731
    x, w, d, u = z(4, 8), z(6, 8), z(3, 2, 8), z(3, 6, 2)
    off, which = torch.tensor([0, 2, 4], device="cuda"), torch.tensor([0, 1], device="cuda")
    for bad in (lambda: sr.adapter(x.cpu(), w, off, which, d, u), lambda: sr.adapter(x, w, off, which.cpu(), d, u),
                lambda: sr.adapter(x, w, off, which[:1], d, u), lambda: sr.adapter(x, w, off, which.int(), d, u),
                lambda: sr.adapter(x, w, off, which, d, u, transpose=True), lambda: sr.adapter(x, w, off, which, u, d),
                lambda: sr.adapter(x, w, off, which, d, u[:2]), lambda: sr.adapter(x, w.t(), off, which, d, u),
                lambda: sr.adapter(x, w, off, which, d, u, scale=z(2)),
                lambda: sr.adapter(x, w, off, which, d, u, scale=z(3).half()),
                lambda: sr.adapter(x, w, off, which, d, u, out=z(4, 7))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: sr.adapter(x.int(), w, off, which, d, u), lambda: sr.adapter(x, w.half(), off, which, d, u)):
        with pytest.raises(TypeError):
            bad()
