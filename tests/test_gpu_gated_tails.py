"""The activations' values far below zero (GPU only), relative to themselves: there
they are small, and what multiplies them may be large."""
import math

import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu

K = 32


def _exact(t, n, m, lo, hi):
    """Rows whose gate is x exactly, for n x m numbers x from lo to hi, and whose other projection is 1.

    Row r has x0 = 1 and x1 = a power of two; gate weight j is (g_j, 0), the other's
    (0, 1 / x1): one term each, no rounding."""
    x = torch.zeros(n, K)
    x[:, 0] = 1.0
    x[:, 1] = torch.exp2(torch.arange(n) % 5 - 2.0)
    g = torch.linspace(lo, hi, m).to(A.TYPES[t])
    w = torch.zeros(1, 2 * m, K)
    w[0, :m, 0] = g.float()
    w[0, m:, 1] = 1.0
    up = x[:, 1:2].double()
    return [v.to(A.TYPES[t]).cuda() for v in (x, w)], torch.tensor([0, n], device="cuda"), g.double().cuda(), up.cuda()


def _phi(g):
    return 0.5 * torch.erfc(-g * math.sqrt(0.5))


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [3, 40, 700])
def test_gelu_far_below_zero(t, n):
    """x Phi(x) and its slope from -12 to -2 are as near to themselves as float's exponent
    allows: the exponent x^2 / 2 is rounded twice (x^2 u), 32 bits of a polynomial and
    its products are 12 u, u = 2^-24; then one rounding to the type."""
    (x, w), off, g, up = _exact(t, n, 512, -12.0, -2.0)
    A.say(f"gelu tails {t} {n}")
    out = sr.gated(x, w, off, activation="gelu")
    d = torch.ones(n, 512, dtype=x.dtype, device="cuda")
    pair = sr.gated_grad(d, x, w, off, activation="gelu")
    torch.cuda.synchronize()
    rel = (g * g + 12) * A.U
    tiny = 1e-36  # below float's normal numbers; none of these results gets there but by underflow
    ref = up * (g * _phi(g))
    A.check(out, ref, rel * ref.abs() + tiny, "out")
    A.check(pair[:, 512:], (g * _phi(g)).expand(n, -1), (rel * (g * _phi(g)).abs()).expand(n, -1) + tiny, "the other's gradient")
    # Phi(x) + x phi(x): from -2 on the second is at least 4.6 times the first, no cancellation beyond 2
    dens = torch.exp(-0.5 * g * g) / math.sqrt(2 * math.pi)
    slope = _phi(g) + g * dens
    size = _phi(g) + (g * dens).abs()
    A.check(pair[:, :512], up * slope, up * (rel * size) + tiny, "the gate's gradient")


@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("t", ["f32", "f16"])
def test_the_other_activations_far_below_zero(t, act):
    """The same of x / (1 + exp(-p)), p = x (silu) or 1.6 (x + 0.045 x^3): p is rounded
    three times and the power of two's argument twice (5 |p| u), and 12 u as above."""
    (x, w), off, g, up = _exact(t, 40, 512, -7.0, -2.0)
    A.say(f"{act} tails {t}")
    out = sr.gated(x, w, off, activation=act)
    torch.cuda.synchronize()
    p = g if act == "silu" else 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
    ref = up * (g * torch.sigmoid(p))
    A.check(out, ref, (5 * p.abs() + 12) * A.U * ref.abs(), "out")
