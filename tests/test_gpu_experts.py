"""The operators together, as a layer of experts uses them: group, gathered
products, combine, and the gradients back to tokens, weights and router
weights; on another stream, and captured in a graph (GPU only)."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu


def _layer(sr, x, choice, prob, w1, w2, c):
    """out, and the gradients of <c, out> for x, w1, w2 and prob."""
    order, position, off = sr.group(choice, w1.shape[0])
    h = sr.matmul(x, w1, off, transpose=True, rows=order)
    y = sr.matmul(h, w2, off, transpose=True)
    out = sr.combine(y, position, prob)
    dy, dprob = sr.combine_grad(c, y, position, prob)
    dh = sr.matmul(dy, w2, off)
    dw2 = sr.outer(dy, h, off)
    dx_rows = sr.matmul(dh, w1, off)
    dw1 = sr.outer(dh, x, off, right_rows=order)
    dx = sr.combine(dx_rows, position, torch.ones_like(prob))
    return out, dx, dw1, dw2, dprob


def _inputs(seed, tokens, fanout, experts, k, m):
    g = ru.gen(seed)
    x = ru.randn(g, tokens, k)
    choice = torch.rand(tokens, experts, generator=g).topk(fanout, dim=1).indices
    prob = torch.rand(tokens, fanout, generator=g)
    w1, w2 = ru.randn(g, experts, m, k, std=k ** -0.5), ru.randn(g, experts, k, m, std=m ** -0.5)
    return x, choice, prob, w1, w2, ru.randn(g, tokens, k)


def _check(got, x, choice, prob, w1, w2, c):
    """Relative to the largest value of each result: float32 sums of at most a
    few hundred terms, three products deep, lose well under 2^-16 of it."""
    leaves = [v.double().requires_grad_() for v in (x, w1, w2, prob)]
    xd, a, b, p = leaves
    out = torch.zeros(c.shape, dtype=torch.float64)
    for j in range(choice.shape[1]):
        h = torch.einsum("tk,tmk->tm", xd, a[choice[:, j]])
        out = out + p[:, j, None] * torch.einsum("tm,tkm->tk", h, b[choice[:, j]])
    (out * c.double()).sum().backward()
    for name, u, v in zip(("out", "dx", "dw1", "dw2", "dprob"), got, (out.detach(), *(z.grad for z in leaves))):
        err = float((u.cpu().double() - v).abs().max())
        assert err <= 2.0 ** -16 * float(v.abs().max()), (name, err)


@pytest.mark.parametrize("tokens,fanout,experts,k,m", [(1, 2, 4, 32, 48), (50, 2, 8, 64, 40), (300, 4, 6, 33, 21)])
def test_experts_layer(tokens, fanout, experts, k, m):
    import segmented_reduction_amd as sr
    data = _inputs(tokens, tokens, fanout, experts, k, m)
    ru.say(f"experts {tokens} {fanout} {experts} {k} {m}")
    got = _layer(sr, *(v.cuda() for v in data))
    torch.cuda.synchronize()
    _check(got, *data)


def test_two_streams_at_once():
    import segmented_reduction_amd as sr
    sets = [_inputs(i, 200 + 50 * i, 2, 8, 64, 96) for i in range(3)]
    dev = [[v.cuda() for v in d] for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    ru.say("experts on three streams")
    for _ in range(3):
        got = []
        for s, d in zip(streams, dev):
            with torch.cuda.stream(s):
                got.append(_layer(sr, *d))
    torch.cuda.synchronize()
    for g, d in zip(got, sets):
        _check(g, *d)


def test_two_captured_graphs():
    """Two graphs captured on one stream and replayed at once on two, with eager calls between."""
    import segmented_reduction_amd as sr
    sets = [_inputs(20 + i, 60 + 700 * i, 2, 8, 64, 96) for i in range(2)]
    dev = [[v.cuda() for v in d] for d in sets]
    adapter = [torch.randn(*s, device="cuda") for s in ((64, 64), (96, 64), (4, 8, 64), (4, 96, 8))]
    off, which = torch.tensor([0, 30, 31, 64], device="cuda"), torch.tensor([3, -1, 0], device="cuda")
    long = torch.randn(5000, 16, device="cuda")
    bounds = torch.tensor([0, 100, 5000], device="cuda")
    index = torch.randint(0, 3000, (20000,), device="cuda")

    def work(d):
        return (*_layer(sr, *d), sr.adapter(adapter[0], adapter[1], off, which, adapter[2], adapter[3]),
                sr.outer(long, long, bounds), *sr.group(index, 3000))

    ru.say("captured graphs")
    side = torch.cuda.Stream()
    eager = []
    with torch.cuda.stream(side):
        for d in dev:
            eager.append([v.clone() for v in work(d)])
    side.synchronize()
    graphs, outs = [], []
    for d in dev:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(work(d))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for rep in range(4):
        for o in outs:
            for v in o:
                v.zero_()
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        work(dev[rep % 2])  # eager, meanwhile
        torch.cuda.synchronize()
        for o, e in zip(outs, eager):
            for u, v in zip(o, e):
                assert torch.equal(u, v), rep
