"""Inputs of the cross entropy whose logits are exact in float32 in any order of
summation, and 64-bit forms with the bounds that are left then.

Values are small whole numbers and weights small multiples of 1/8, so every partial
sum of a logit is a multiple of 1/8 below 2^21 and none is rounded; `scale` is a power
of two.  What is left are the exponentials, their sums, and roundings to the types, so
that an entry of the vocabulary that is lost, counted twice or read elsewhere is far
outside the bounds once it has a share in the result.  Each row is given an entry that
has nearly all of it (`lead`): values 2 sign(W_e), whose logit is 2 sum|W_e|.
"""
from __future__ import annotations

import math

import torch

from tests.around_util import U, goals


def entries(v, more=()):
    """Entries at which tiles of 64, 128 and 256 begin and end, the vocabulary's ends first."""
    first = [v - 1, (v - 1) // 256 * 256, (v - 1) // 128 * 128, (v - 1) // 64 * 64, 0, *more]
    for b in (64, 128, 256):
        first += [b - 1, b, (v - 1) // b * b - 1, v // 2 // b * b - 1, v // 2 // b * b]
    seen = []
    for e in first:
        if 0 <= e < v and e not in seen:
            seen.append(e)
    return seen


def case(t, n, k, v, picks=1, seed=0, more=(), skip=0):
    """(x, w, target, probs, grad, scale, lead [n]): on the CPU.  `skip`: where in `entries` to begin."""
    g = torch.Generator().manual_seed(seed + n + 31 * k + 7 * v)
    w = torch.randint(-8, 9, (v, k), generator=g).to(t) / 8
    e = torch.tensor(entries(v, more))
    i = torch.arange(n) + skip
    lead = torch.where(i < e.numel(), e[i % e.numel()], (i * 2654435761) % v)
    x = (2 * w[lead].float().sign()).to(t)
    target = torch.randint(0, v, (n, picks), generator=g)
    target[torch.arange(n) % 11 == 5] = -1
    probs = torch.rand(n, picks, generator=g) if picks > 1 else None
    grad = torch.rand(n, generator=g) + 0.5
    scale = 2.0 ** -max(0, round(math.log2(k / 64)))  # the lead's logit: about 68 at any width from 64 on
    return x, w, target.view(-1) if picks == 1 else target, probs, grad, scale, lead


def below_zero(t, n, k, v, seed=0):
    """Rows whose logits are all far below 0 (about -0.56 * 1.5 k scale)."""
    g = torch.Generator().manual_seed(seed + n + 31 * k + 7 * v)
    w = -torch.randint(1, 9, (v, k), generator=g).to(t) / 8
    x = torch.randint(1, 3, (n, k), generator=g).to(t)
    target = torch.randint(0, v, (n,), generator=g)
    scale = 2.0 ** -max(0, round(math.log2(k / 64)))
    return x, w, target, None, torch.rand(n, generator=g) + 0.5, scale


def forward(x, w, target, probs, scale):
    """(loss, lse, picked), their bounds, and (logits, goal, live, share)."""
    z = scale * (x.double() @ w.double().t())
    v = w.shape[0]
    goal, live = goals(target, probs, v, x.device)
    lse = torch.logsumexp(z, 1)
    # exponents: up to 30 below the largest count (2^-43 beyond), each rounded in three places
    # on the way in and two on the way out; the sum nests as the other bounds have it
    e_lse = (8 * (z.abs().max(1).values + 30) + 64 + v / 2048 + 4 * lse.abs()) * U
    t = target.view(x.shape[0], -1)
    ok = (t >= 0) & (t < v)
    p = torch.ones(t.shape, dtype=torch.float64, device=x.device) if probs is None else probs.view(t.shape).double()
    p = torch.where(ok, p, 0.0)
    picked = torch.where(ok, z.gather(1, torch.where(ok, t, 0)), 0.0)
    share = p.sum(1)
    loss = torch.where(live, share * lse - (p * picked).sum(1), 0.0)
    sums = (t.shape[1] + 4) * U * (p.abs().sum(1) * lse.abs() + (p * picked).abs().sum(1))
    e_loss = torch.where(live, share.abs() * e_lse + sums, 0.0)
    return (loss, lse, picked.view(target.shape)), (e_loss, e_lse, torch.zeros_like(picked).view(target.shape)), (z, goal, live, share)


def backward(x, w, target, probs, grad, scale):
    """((dx, dw), bounds); the logits' gradient is rounded to the type of x."""
    (_, lse, _), (_, e_lse, _), (z, goal, live, share) = forward(x, w, target, probs, scale)
    half = 0.0 if x.dtype == torch.float32 else torch.finfo(x.dtype).eps / 2
    n, v = z.shape
    g = torch.where(live, grad.double() * scale, 0.0)[:, None]
    p = (z - lse[:, None]).exp_()
    dz = g * (share[:, None] * p - goal)
    e = g.abs() * (share[:, None] * p * (e_lse[:, None] + 8 * U * (z.abs() + lse[:, None].abs() + 4)) + 8 * U * (p * share[:, None] + goal))
    e = e + half * (dz.abs() + e)
    if x.dtype == torch.float16:  # dz is scaled so that the largest row's bound is at 2^13 .. 2^14
        top = float((g[:, 0].abs() * goal.sum(1)).max())
        e = e + (2.0 ** (-25 - 13 + math.floor(math.log2(top))) * live[:, None] if top > 0 else 0.0)
    x, w, size = x.double(), w.double(), dz.abs() + e
    dx, dw = dz @ w, dz.t() @ x
    e_x = e @ w.abs() + (v + 8) * 2 * U * (size @ w.abs())
    e_w = e.t() @ x.abs() + (n + 8) * 2 * U * (size.t() @ x.abs())
    return (dx, dw), (e_x, e_w)
