"""The 64-bit forms that the GPU tests of the norms, the gated projections and the
cross entropy compare with: their gradients against central differences."""
import pytest
import torch

from tests import around_util as A


def _slope(f, x, way, h=1e-5):
    """The derivative of f along `way`, by differences of the fourth order."""
    return (8 * (f(x + h * way) - f(x - h * way)) - (f(x + 2 * h * way) - f(x - 2 * h * way))) / (12 * h)


def _near(got, want, mag):
    # differences of sums of size mag at h = 1e-5: 2^-52 mag / h, with room for the fourth order's h^4
    assert abs(float(got) - float(want)) <= 1e-9 * (1 + float(mag)), (float(got), float(want))


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("k", [2, 9])
def test_norm_gradients(center, k):
    g = torch.Generator().manual_seed(k)
    x, w, b, d = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((4, k), (k,), (k,), (4, k)))
    f = lambda x, w, b: (A.norm(x, w, b, 1e-2, center)[0] * d).sum()  # noqa: E731
    (dx, dw, db), _ = A.norm_grad(d, x, w, 1e-2, center)
    vx, vw = torch.randn(4, k, generator=g, dtype=torch.float64), torch.randn(k, generator=g, dtype=torch.float64)
    _near(_slope(lambda t: f(t, w, b), x, vx), (dx * vx).sum(), dx.abs().sum() + d.abs().sum())
    _near(_slope(lambda t: f(x, t, b), w, vw), (dw * vw).sum(), d.abs().sum())
    _near(_slope(lambda t: f(x, w, t), b, vw), (db * vw).sum(), d.abs().sum())


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu"])
def test_gated_gradients(act):
    g = torch.Generator().manual_seed(3)
    n, k, m, off = 7, 5, 3, torch.tensor([0, 4, 4, 7])
    x, w = torch.randn(n, k, generator=g, dtype=torch.float64), torch.randn(3, 2 * m, k, generator=g, dtype=torch.float64)
    d, vx, vw = torch.randn(n, m, generator=g, dtype=torch.float64), torch.randn_like(x), torch.randn_like(w)
    f = lambda x, w: (A.gated(x, w, off, act)[0] * d).sum()  # noqa: E731
    pair, _ = A.gated(x, w, off, act, grad=d)
    dx = torch.cat([pair[a:b] @ w[s] for s, (a, b) in enumerate(((0, 4), (4, 4), (4, 7)))])
    dw = torch.stack([pair[a:b].t() @ x[a:b] for a, b in ((0, 4), (4, 4), (4, 7))])
    _near(_slope(lambda t: f(t, w), x, vx, 1e-6), (dx * vx).sum(), 10 * dx.abs().sum())
    _near(_slope(lambda t: f(x, t), w, vw, 1e-6), (dw * vw).sum(), 10 * dw.abs().sum())


@pytest.mark.parametrize("picks", [1, 3])
def test_cross_entropy_gradients(picks):
    g = torch.Generator().manual_seed(picks)
    n, k, v, scale = 6, 5, 11, 0.7
    x, w = torch.randn(n, k, generator=g, dtype=torch.float64), torch.randn(v, k, generator=g, dtype=torch.float64)
    t = torch.randint(-1, v + 1, (n, picks), generator=g)
    t[0] = -100
    probs = torch.rand(n, picks, generator=g, dtype=torch.float64)
    d, vx, vw = torch.randn(n, generator=g, dtype=torch.float64), torch.randn_like(x), torch.randn_like(w)
    f = lambda x, w: (A.cross_entropy(x, w, t, probs, scale)[0][0] * d).sum()  # noqa: E731
    (dx, dw), _ = A.cross_entropy_grad(d, x, w, t, torch.float32, probs, scale)
    assert (dx[0] == 0).all()
    _near(_slope(lambda s: f(s, w), x, vx), (dx * vx).sum(), 10 * dx.abs().sum())
    _near(_slope(lambda s: f(x, s), w, vw), (dw * vw).sum(), 10 * dw.abs().sum())
