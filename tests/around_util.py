"""Plain 64-bit forms of the row norms, the gated projections and the cross
entropy, with bounds on what 32-bit arithmetic and one rounding may lose.

u = 2^-24 is half a step of float32.  A sum whose partial sums nest d deep errs by
at most d u sum|terms|; lanes add at most 32 elements by themselves, then 6 + 4
levels join lanes and waves (long rows: k / 512 elements by themselves), so depth()
is above what any kernel nests.  Products of matrices count (n + 8) 2 u sum|terms|
for n terms, as the tests of the ragged products do.  A result of type t is rounded
once, by half a step.
"""
from __future__ import annotations

import math

import torch

from tests.ragged_util import gen, offsets, randn, say  # noqa: F401

U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def depth(k):
    return 64 + k / 512


def half_step(t, x):
    return torch.finfo(t).eps / 2 * x.abs() + (2.0 ** -25 if t == torch.float16 else 0.0)


def check(got, ref, err, what):
    """|got - ref| within `err` (of the 32-bit arithmetic) and one rounding to got's type."""
    tol = err + half_step(got.dtype, ref.abs() + err) + 1e-37
    off = (got.detach().to(ref.device).double() - ref).abs()
    bad = ~(off <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((off / tol).nan_to_num(1e30).max()):.3g} of the bound"


# ------------------------------------------------------------------------ norm

def norm(x, w, b, eps, center):
    """(out, its error bound, unit rows, 1 / sigma, bounds of both)."""
    x, k = x.double(), x.shape[1]
    mean = x.mean(1, keepdim=True) if center else torch.zeros_like(x[:, :1])
    d = depth(k)
    # the mean's own error, and of x - mean: one rounding
    em = (d + 4) * U * x.abs().mean(1, keepdim=True) if center else torch.zeros_like(mean)
    var = ((x - mean) ** 2).mean(1, keepdim=True)
    r = 1 / (var + eps).sqrt()
    # squares around a mean that is em off gain em^2, and rounding
    er = (d + 8) * U + 2 * (em * r) ** 2 + 2 * em * r * U
    unit = (x - mean) * r
    eu = em * r + unit.abs() * (er + 4 * U)
    w = torch.ones(k, dtype=torch.float64, device=x.device) if w is None else w.double()
    b = torch.zeros(k, dtype=torch.float64, device=x.device) if b is None else b.double()
    out = unit * w + b
    return out, eu * w.abs() + 2 * U * (out.abs() + (unit * w).abs()), unit, r, eu, er


def norm_grad(g, x, w, eps, center):
    """((dx, dw, db), (their error bounds))."""
    _, _, unit, r, eu, er = norm(x, w, None, eps, center)
    g, k, n = g.double(), x.shape[1], x.shape[0]
    wd = torch.ones(k, dtype=torch.float64, device=x.device) if w is None else w.double()
    gw = g * wd
    d = depth(k)
    level = gw.mean(1, keepdim=True) if center else torch.zeros_like(gw[:, :1])
    along = (gw * unit).mean(1, keepdim=True)
    dx = r * (gw - level - unit * along)
    # the waves' parts take x around means of their own: at most twice the row's
    spread = 2 * unit.abs() + unit.abs().max(1, keepdim=True).values
    e_level = (d + 4) * U * gw.abs().mean(1, keepdim=True)
    e_along = (d + 8) * U * (gw.abs() * spread).mean(1, keepdim=True) + (gw.abs() * eu).mean(1, keepdim=True) + er * along.abs()
    e = r * (4 * U * gw.abs() + e_level + unit.abs() * e_along + eu * along.abs() + 4 * U * (unit * along).abs() + 2 * U * level.abs())
    e = e + (er + 4 * U) * dx.abs()
    rows = (n + 8) * U
    dw, db = (g * unit).sum(0), g.sum(0)
    e_w = (g.abs() * eu).sum(0) + (rows + 2 * U) * (g * unit).abs().sum(0)
    return (dx, dw, db), (e, e_w, rows * g.abs().sum(0))


# ----------------------------------------------------------------------- gated

def bend(x, act):
    """act(x), its slope, and how far either moves per unit of x at most (nearby)."""
    if act == "silu":
        s = torch.sigmoid(x)
        return x * s, s + x * s * (1 - s), 1.2, 0.6
    if act == "gelu":
        phi = 0.5 * torch.erfc(-x * math.sqrt(0.5))
        return x * phi, phi + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi), 1.2, 0.9
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (x + 0.044715 * x ** 3))
        return x * s, s + x * s * (1 - s) * c * (1 + 3 * 0.044715 * x * x), 1.2, 0.9
    return x.clamp(min=0), (x > 0).double(), 1.0, 0.0


def gated(values, weights, off, act, rows=None, grad=None, fill=0.0):
    """(out, bound) or with `grad` (pair, bound); rows of no segment hold `fill` (bound 0)."""
    x = values.double()
    if rows is not None:
        ok = (rows >= 0) & (rows < x.shape[0])
        x = torch.where(ok[:, None], x[rows.clamp(0, max(x.shape[0] - 1, 0))], 0.0)
    m, k = weights.shape[1] // 2, weights.shape[2]
    out = torch.full((x.shape[0], m if grad is None else 2 * m), fill, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(out)
    o = off.tolist()
    for s, (a, b) in enumerate(zip(o[:-1], o[1:])):
        w = weights[s].double()
        pre, mag = x[a:b] @ w.t(), x[a:b].abs() @ w.abs().t()
        e = (k + 8) * 2 * U * mag
        g, u, eg, eu = pre[:, :m], pre[:, m:], e[:, :m], e[:, m:]
        y, slope, most, curve = bend(g, act)
        # exponents up to |g| (1 + 0.07 g^2) round by as much; beyond 90 everything has settled
        own = (16 + 4 * (g.abs() * (1.6 + 0.0714 * g * g)).clamp(max=90)) * U
        ey = most * eg + own * (g.abs().clamp(max=90) * 1.0 + y.abs()) if act != "relu" else eg
        es = curve * eg + own * (1 + g.abs().clamp(max=90)) if act != "relu" else torch.zeros_like(eg)
        if grad is None:
            out[a:b] = y * u
            err[a:b] = ey * (u.abs() + eu) + y.abs() * eu + 4 * U * (y * u).abs()
        else:
            d = grad[a:b].double()
            out[a:b] = torch.cat([d * u * slope, d * y], 1)
            err[a:b] = torch.cat([d.abs() * (es * (u.abs() + eu) + slope.abs() * eu) + 4 * U * (d * u * slope).abs(),
                                  d.abs() * ey + 4 * U * (d * y).abs()], 1)
    return out, err


# --------------------------------------------------------------- cross entropy

def goals(target, probs, v, device):
    """([N, V] probability of each entry, whether a row has any)."""
    t = target.view(target.shape[0], -1)
    ok = (t >= 0) & (t < v)
    p = torch.ones(t.shape, dtype=torch.float64, device=device) if probs is None else probs.view(t.shape).double()
    goal = torch.zeros(t.shape[0], v, dtype=torch.float64, device=device)
    goal.scatter_add_(1, torch.where(ok, t, 0), torch.where(ok, p, 0.0))
    return goal, ok.any(1)


def cross_entropy(x, w, target, probs=None, scale=1.0):
    """(loss, lse, picked), their bounds, and (logits, bound of a logit, goal, live) for the gradient."""
    x, w = x.double(), w.double()
    n, k, v = x.shape[0], x.shape[1], w.shape[0]
    goal, live = goals(target, probs, v, x.device)
    z = scale * (x @ w.t())
    ez = scale * (k + 10) * 2 * U * (x.abs() @ w.abs().t())
    lse = torch.logsumexp(z, 1)
    reach = (z - lse[:, None]).abs().max(1).values + z.abs().max(1).values  # what the exponents are made of
    # terms more than 30 below the largest are below 2^-43 of the sum
    reach = reach.clamp(max=float(z.abs().max()) + 30)
    e_lse = ez.max(1).values + (8 * reach + 64 + v / 2048 + 4 * lse.abs()) * U
    t = target.view(n, -1)
    ok = (t >= 0) & (t < v)
    at = torch.where(ok, t, 0)
    p = torch.ones(t.shape, dtype=torch.float64, device=x.device) if probs is None else probs.view(t.shape).double()
    p = torch.where(ok, p, 0.0)
    picked = torch.where(ok, z.gather(1, at), 0.0)
    e_picked = torch.where(ok, ez.gather(1, at), 0.0)
    share = p.sum(1)
    loss = torch.where(live, share * lse - (p * picked).sum(1), 0.0)
    picks = t.shape[1]
    e_loss = share.abs() * e_lse + (p.abs() * e_picked).sum(1) + (picks + 4) * U * (p.abs().sum(1) * lse.abs() + (p * picked).abs().sum(1))
    e_loss = torch.where(live, e_loss, 0.0)
    return (loss, lse, picked.view(target.shape)), (e_loss, e_lse, e_picked.view(target.shape)), (z, ez, goal, live, share)


def cross_entropy_grad(grad, x, w, target, t, probs=None, scale=1.0):
    """((dx, dw), bounds); t: the type that the logits' gradient is rounded to."""
    (_, lse, _), (_, e_lse, _), (z, ez, goal, live, share) = cross_entropy(x, w, target, probs, scale)
    x, w, g = x.double(), w.double(), grad.double() * scale
    x = torch.where(live[:, None], x, 0.0)
    p = torch.where(live[:, None], (z - lse[:, None]).exp(), 0.0)
    dz = torch.where(live[:, None], g[:, None] * (share[:, None] * p - goal), 0.0)
    # exponents: the logit's and lse's errors, their roundings and that of their difference
    e_p = p * (ez + e_lse[:, None] + 8 * U * (z.abs() + lse[:, None].abs() + 4))
    e = g.abs()[:, None] * (share.abs()[:, None] * e_p + 8 * U * (share[:, None] * p + goal.abs()))
    e = torch.where(live[:, None], e, 0.0)
    size = dz.abs() + e
    if t == torch.float16:  # by a power of two that brings the largest row's bound to 2^13 .. 2^14
        top = (g.abs() * goal.abs().sum(1))[live]
        floor = 2.0 ** -25 * 2.0 ** (math.floor(math.log2(float(top.max()))) - 13) if top.numel() and top.max() > 0 else 0.0
        e = e + torch.finfo(t).eps / 2 * size + floor * live[:, None]
    elif t == torch.bfloat16:
        e = e + torch.finfo(t).eps / 2 * size
    size = dz.abs() + e
    n, v = z.shape
    dx, dw = dz @ w, dz.t() @ x
    e_x = e @ w.abs() + (v + 8) * 2 * U * (size @ w.abs())
    e_w = e.t() @ x.abs() + (n + 8) * 2 * U * (size.t() @ x.abs())
    return (dx, dw), (e_x, e_w)
