"""The weighted join of a token's rows and its gradient (GPU only)."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1, 8), (5, 3, 33), (40, 8, 2048), (33, 6, 200), (3, 1, 1), (64, 9, 512), (2, 17, 1000)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,fanout,m", SHAPES)
def test_combine_and_gradient(kind, tokens, fanout, m):
    import segmented_reduction_amd as sr
    t, g = ru.TYPES[kind], ru.gen(tokens * m)
    n = tokens * fanout + 3
    y, c = ru.randn(g, n, m, dtype=t), ru.randn(g, tokens, m, dtype=t)
    position = torch.randperm(n, generator=g)[: tokens * fanout].view(tokens, fanout)
    position[0, 0] = -1
    position[-1, -1] = n
    w = torch.rand(tokens, fanout, generator=g) - 0.3
    ru.say(f"combine {kind} {tokens}x{fanout}x{m}")
    out = sr.combine(y.cuda(), position.cuda(), w.cuda())
    dv = torch.full((n, m), 5.0, dtype=t, device="cuda")
    got, dw = sr.combine_grad(c.cuda(), y.cuda(), position.cuda(), w.cuda(), out=dv)
    torch.cuda.synchronize()
    assert got is dv and dw.dtype == torch.float32
    ref, mag = ru.combine(y, position, w)
    ru.assert_close(out, ref, mag, fanout, "combine")
    ok = (position >= 0) & (position < n)
    rv = torch.full((n, m), 5.0, dtype=torch.float64)
    rv[position[ok]] = (w.double()[..., None] * c.double()[:, None, :])[ok]
    ru.assert_close(dv, rv, rv.abs(), 1, "grad of values")
    rows = y.double()[position.clamp(0, n - 1)]
    terms = torch.where(ok[..., None], c.double()[:, None, :] * rows, 0.0)
    ru.assert_close(dw, terms.sum(-1), terms.abs().sum(-1), m, "grad of weights")
    assert (dw.cpu()[~ok] == 0).all()


def test_a_token_of_no_rows_gets_zeros():
    import segmented_reduction_amd as sr
    y = torch.full((4, 24), float("nan"), device="cuda")
    ru.say("combine without rows")
    out = sr.combine(y, torch.full((3, 2), -1, device="cuda"), torch.ones(3, 2, device="cuda"))
    assert (out.cpu() == 0).all()
    out = sr.combine(y, torch.empty(3, 0, dtype=torch.int64, device="cuda"), torch.empty(3, 0, device="cuda"))
    assert (out.cpu() == 0).all()
    assert sr.combine(y[:0], torch.zeros(2, 1, dtype=torch.int64, device="cuda"),
                      torch.ones(2, 1, device="cuda")).cpu().abs().max() == 0
    assert sr.combine(y, torch.empty(0, 2, dtype=torch.int64, device="cuda"), torch.empty(0, 2, device="cuda")).shape == (0, 24)


def test_combine_reads_a_row_as_often_as_it_is_named():
    import segmented_reduction_amd as sr
    g = ru.gen(8)
    y = ru.randn(g, 6, 40)
    position = torch.tensor([[1, 1, 1], [1, 2, 1]])
    w = torch.rand(2, 3, generator=g)
    ru.say("combine repeated rows")
    out = sr.combine(y.cuda(), position.cuda(), w.cuda())
    ref, mag = ru.combine(y, position, w)
    ru.assert_close(out, ref, mag, 3, "combine")


def test_gradient_against_differences():
    """<c, combine> is linear in the rows and in the weights."""
    import segmented_reduction_amd as sr
    g = ru.gen(4)
    n, t, k, m = 12, 4, 3, 20
    y, dy, c = ru.randn(g, n, m), ru.randn(g, n, m), ru.randn(g, t, m)
    position = torch.randperm(n, generator=g).view(t, k)
    w, dw_dir = torch.rand(t, k, generator=g), ru.randn(g, t, k)
    ru.say("combine differences")
    loss = lambda a, b: (sr.combine(a.cuda(), position.cuda(), b.cuda()).cpu().double() * c.double()).sum()  # noqa: E731
    dv, dw = sr.combine_grad(c.cuda(), y.cuda(), position.cuda(), w.cuda())
    bound = 4 * (k + 8) * 2.0 ** -23 * t * k * m * float(c.abs().max()) * float((y.abs().max() + dy.abs().max())
                                                                               * (1 + dw_dir.abs().max()))
    assert abs(loss(y + dy, w) - loss(y, w) - (dv.cpu().double() * dy.double()).sum()) <= bound
    assert abs(loss(y, w + dw_dir) - loss(y, w) - (dw.cpu().double() * dw_dir.double()).sum()) <= bound


def test_refusals():
    import segmented_reduction_amd as sr
    y = torch.zeros(4, 8, device="cuda")
    p = torch.zeros(2, 2, dtype=torch.int64, device="cuda")
    w = torch.zeros(2, 2, device="cuda")
    g = torch.zeros(2, 8, device="cuda")
    for bad in (lambda: sr.combine(y.cpu(), p, w), lambda: sr.combine(y, p.cpu(), w), lambda: sr.combine(y, p.int(), w),
                lambda: sr.combine(y, p.view(-1), w), lambda: sr.combine(y, p, w[:1]), lambda: sr.combine(y, p, w.half()),
                lambda: sr.combine(y.t(), p, w), lambda: sr.combine(y, p, w, out=torch.zeros(2, 9, device="cuda")),
                lambda: sr.combine_grad(g[:1], y, p, w), lambda: sr.combine_grad(g.half(), y, p, w),
                lambda: sr.combine_grad(g, y, p, w, out=g)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        sr.combine(y.int(), p, w)
