"""A layer of experts in 16-bit types, forwards and back (GPU only).  Each call
is compared with 64 bits on what it was given, so that it may be off by half a
step of its type and its own 32-bit sums alone."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("tokens,fanout,experts,k,m", [(1, 2, 4, 32, 48), (300, 4, 6, 264, 520), (2000, 2, 8, 128, 200),
                                                       (77, 3, 5, 33, 21)])
def test_experts_layer(kind, tokens, fanout, experts, k, m):
    import segmented_reduction_amd as sr
    t, g = ru.TYPES[kind], ru.gen(tokens + k)
    x, c = ru.randn(g, tokens, k, dtype=t), ru.randn(g, tokens, k, dtype=t)
    choice = torch.rand(tokens, experts, generator=g).topk(fanout, dim=1).indices
    prob = torch.rand(tokens, fanout, generator=g)
    w1 = ru.randn(g, experts, m, k, dtype=t, std=k ** -0.5)
    w2 = ru.randn(g, experts, k, m, dtype=t, std=m ** -0.5)
    ru.say(f"experts {kind} {tokens} {fanout} {experts} {k} {m}")
    xd, cd, pd, a, b = (v.cuda() for v in (x, c, prob, w1, w2))
    order, position, off = sr.group(choice.cuda(), experts)
    h = sr.matmul(xd, a, off, transpose=True, rows=order)
    y = sr.matmul(h, b, off, transpose=True)
    out = sr.combine(y, position, pd)
    dy, dprob = sr.combine_grad(cd, y, position, pd)
    dh = sr.matmul(dy, b, off)
    dw2 = sr.outer(dy, h, off)
    dx_rows = sr.matmul(dh, a, off)
    dw1 = sr.outer(dh, xd, off, right_rows=order)
    dx = sr.combine(dx_rows, position, torch.ones_like(pd))
    torch.cuda.synchronize()

    order, position, off = ru.group(choice, experts)
    longest = int((off[1:] - off[:-1]).max())
    H, Y, DY, DH, DX = (v.cpu() for v in (h, y, dy, dh, dx_rows))
    ru.assert_close(h, *ru.matmul(x, w1, off, True, order), k, "hidden rows")
    ru.assert_close(y, *ru.matmul(H, w2, off, True), m, "answers")
    ru.assert_close(out, *ru.combine(Y, position, prob), fanout, "out")
    want = torch.zeros(Y.shape, dtype=torch.float64)
    want[position.view(-1)] = (prob.double()[..., None] * c.double()[:, None, :]).flatten(0, 1)
    ru.assert_close(dy, want, want.abs(), 1, "grad of answers")
    dots = c.double()[:, None, :] * Y.double()[position]
    ru.assert_close(dprob, dots.sum(-1), dots.abs().sum(-1), k, "grad of the router's weights")
    ru.assert_close(dh, *ru.matmul(DY, w2, off), k, "grad of hidden rows")
    ru.assert_close(dx_rows, *ru.matmul(DH, w1, off), m, "grad of rows")
    ru.assert_close(dx, *ru.combine(DX, position, torch.ones_like(prob)), fanout, "grad of tokens")
    ru.assert_close(dw2, *ru.outer(DY, H, off), longest, "grad of the second weights")
    ru.assert_close(dw1, *ru.outer(DH, x, off, right_rows=order), longest, "grad of the first weights")
