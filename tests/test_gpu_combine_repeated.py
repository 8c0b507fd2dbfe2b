"""The gradient of the weighted join where rows are named more than once (GPU only)."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


def inputs(kind, tokens, fanout, n, m, seed):
    t, g = ru.TYPES[kind], ru.gen(seed)
    y, c = ru.randn(g, n, m, dtype=t), ru.randn(g, tokens, m, dtype=t)
    position = torch.randint(-1, n + 1, (tokens, fanout), generator=g)
    if n > 2:
        position[position == 2] = 1  # row 2 is named by none
    return y, c, position, torch.rand(tokens, fanout, generator=g) - 0.3


def check(got, y, c, position, w):
    n, (tokens, fanout) = y.shape[0], position.shape
    at = torch.where((position >= 0) & (position < n), position, n).view(-1)
    terms = (w.double()[..., None] * c.double()[:, None, :]).flatten(0, 1)
    ref = torch.zeros(n + 1, y.shape[1], dtype=torch.float64).index_add_(0, at, terms)[:n]
    mag = torch.zeros(n + 1, y.shape[1], dtype=torch.float64).index_add_(0, at, terms.abs())[:n]
    often = int(torch.bincount(at, minlength=n + 1)[:n].max()) if n else 0
    ru.assert_close(got[0], ref, mag, often, "grad of values")
    ok = (position >= 0) & (position < n)
    rows = torch.cat([y.double(), torch.zeros(1, y.shape[1], dtype=torch.float64)])[at].view(tokens, fanout, -1)
    dots = c.double()[:, None, :] * rows
    ru.assert_close(got[1], dots.sum(-1), dots.abs().sum(-1), y.shape[1], "grad of weights")
    assert not got[1].cpu()[~ok].any()
    if n > 2:
        assert not got[0][2].any()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("tokens,fanout,n,m", [(1, 2, 1, 8), (5, 3, 4, 33), (40, 8, 30, 2048), (700, 6, 9, 200),
                                               (3000, 2, 5000, 72), (64, 9, 3, 1), (2, 17, 1000, 24)])
def test_rows_named_more_than_once(kind, tokens, fanout, n, m):
    y, c, position, w = inputs(kind, tokens, fanout, n, m, tokens + m)
    dev = [v.cuda() for v in (c, y, position, w)]
    ru.say(f"combine gradient, repeated rows {kind} {tokens}x{fanout} rows={n} m={m}")
    out = torch.full((n, m), 5.0, dtype=y.dtype, device="cuda")
    got = sr().combine_grad(*dev, repeated=True, out=out)
    again = sr().combine_grad(*dev, repeated=True)
    torch.cuda.synchronize()
    assert got[0] is out and all(torch.equal(a, b) for a, b in zip(got, again))
    check(got, y, c, position, w)


def test_rows_named_once_are_the_same_either_way():
    g = ru.gen(3)
    y, c = ru.randn(g, 600, 72, dtype=torch.bfloat16), ru.randn(g, 150, 72, dtype=torch.bfloat16)
    position, w = torch.randperm(600, generator=g).view(150, 4), torch.rand(150, 4, generator=g)
    dev = [v.cuda() for v in (c, y, position, w)]
    ru.say("combine gradient, either way")
    for a, b in zip(sr().combine_grad(*dev), sr().combine_grad(*dev, repeated=True)):
        assert torch.equal(a, b)


def test_without_entries_or_rows():
    y, c = torch.ones(4, 24, device="cuda"), torch.ones(3, 24, device="cuda")
    none = torch.empty(3, 0, device="cuda")
    ru.say("combine gradient without entries")
    dv, dw = sr().combine_grad(c, y, none.long(), none, repeated=True)
    assert not dv.any() and dw.shape == (3, 0)
    dv, dw = sr().combine_grad(c[:0], y, none[:0].long(), none[:0], repeated=True)
    assert not dv.any()
    dv, dw = sr().combine_grad(c, y[:0], torch.zeros(3, 2, device="cuda").long(), torch.ones(3, 2, device="cuda"), repeated=True)
    assert dv.shape == (0, 24) and not dw.any()


def test_gradient_against_differences():
    """<c, combine> is linear in the rows."""
    g = ru.gen(4)
    n, t, k, m = 6, 9, 3, 20
    y, dy, c = ru.randn(g, n, m), ru.randn(g, n, m), ru.randn(g, t, m)
    position, w = torch.randint(0, n, (t, k), generator=g), torch.rand(t, k, generator=g)
    ru.say("combine differences, repeated rows")
    loss = lambda a: (sr().combine(a.cuda(), position.cuda(), w.cuda()).cpu().double() * c.double()).sum()  # noqa: E731
    dv = sr().combine_grad(c.cuda(), y.cuda(), position.cuda(), w.cuda(), repeated=True)[0]
    bound = 4 * (t * k + 8) * 2.0 ** -23 * t * k * m * float(c.abs().max()) * float(y.abs().max() + dy.abs().max())
    assert abs(loss(y + dy) - loss(y) - (dv.cpu().double() * dy.double()).sum()) <= bound


def test_captured_and_replayed():
    y, c, position, w = inputs("bf16", 300, 4, 40, 64, 9)
    dev = [v.cuda() for v in (c, y, position, w)]
    ru.say("combine gradient, repeated rows, replayed")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        sr().combine_grad(*dev, repeated=True)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = sr().combine_grad(*dev, repeated=True)
    for rep in range(4):
        position = inputs("bf16", 300, 4, 40, 64, 20 + rep)[2]
        dev[2].copy_(position)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, sr().combine_grad(*dev, repeated=True)):
            assert torch.equal(a, b), rep
        check(outs, y, c, position, w)
