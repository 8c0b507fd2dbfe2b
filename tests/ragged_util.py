"""Plain 64-bit forms of the operators over ragged groups of rows, and the
tolerances their tests use.

A result of type t is off by at most half a step of t, eps(t) / 2 relative to
the value (for float16 not less than half its smallest step, 2^-25, near
zero), plus what the 32-bit sum loses before it: each of n additions errs by
at most one unit in the last place of a partial sum, which is at most the sum
of the magnitudes, so n * 2^-23 * sum|terms| in all.
"""
from __future__ import annotations

import sys

import torch

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def say(msg: str):
    """Name the case on stdout before a GPU step."""
    print(f"[gpu-case] {msg}", flush=True)
    sys.stdout.flush()


def gen(seed: int) -> torch.Generator:
    return torch.Generator().manual_seed(seed)


def randn(g, *shape, dtype=torch.float32, std=1.0) -> torch.Tensor:
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def offsets(lengths, base=0) -> torch.Tensor:
    return torch.tensor([base, *lengths], dtype=torch.int64).cumsum(0)


def assert_close(got: torch.Tensor, ref: torch.Tensor, mag: torch.Tensor, n: int, what: str, more=0.0):
    """|got - ref| within half a step of got's type plus n sums in 32 bits of terms of magnitude `mag`."""
    t = got.dtype
    tol = torch.finfo(t).eps / 2 * ref.abs() + (n + 8) * 2.0 ** -23 * mag * (1 + torch.finfo(t).eps) + more
    if t == torch.float16:
        tol = tol + 2.0 ** -25
    err = (got.detach().cpu().double() - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((err / (tol + 1e-300)).max()):.3g} of the bound"


def matmul(values, weights, off, transpose=False, rows=None, fill=0.0):
    """(product, sum of magnitudes) of each segment's rows with its weights; rows of no segment hold `fill`."""
    x = values.double()
    if rows is not None:
        ok = (rows >= 0) & (rows < x.shape[0])
        x = torch.where(ok[:, None], x[rows.clamp(0, max(x.shape[0] - 1, 0))], 0.0)
    w = weights.double()
    w = w.transpose(1, 2) if transpose else w
    out = torch.full((x.shape[0], w.shape[2]), fill, dtype=torch.float64, device=x.device)
    mag = torch.zeros_like(out)
    o = off.tolist()
    for s, (a, b) in enumerate(zip(o[:-1], o[1:])):
        out[a:b] = x[a:b] @ w[s]
        mag[a:b] = x[a:b].abs() @ w[s].abs()
    return out, mag


def outer(left, right, off, left_rows=None, right_rows=None):
    a = left.double() if left_rows is None else left.double()[left_rows]
    b = right.double() if right_rows is None else right.double()[right_rows]
    o = off.tolist()
    spans = list(zip(o[:-1], o[1:]))
    return (torch.stack([a[i:j].t() @ b[i:j] for i, j in spans]),
            torch.stack([a[i:j].abs().t() @ b[i:j].abs() for i, j in spans]))


def group(index, dim):
    """order, position, offsets of a stable sort by group; entries of no group last."""
    flat = index.reshape(-1)
    fanout = index.shape[1] if index.dim() == 2 else 1
    key = torch.where((flat < 0) | (flat >= dim), dim, flat)
    skey, at = key.sort(stable=True)
    position = torch.empty_like(at)
    position[at] = torch.arange(at.numel())
    position = torch.where(key < dim, position, -1).view(index.shape)
    return at // max(fanout, 1), position, torch.searchsorted(skey, torch.arange(dim + 1))


def combine(values, position, weights):
    ok = (position >= 0) & (position < values.shape[0])
    w = torch.where(ok, weights.double(), 0.0)
    rows = torch.where(ok[..., None], values.double()[position.clamp(0, max(values.shape[0] - 1, 0))], 0.0)
    return (w[..., None] * rows).sum(1), (w[..., None] * rows).abs().sum(1)


def adapter(x, weights, off, which, down, up, scale=None, transpose=False, fill=0.0):
    """(out, magnitude of its terms, magnitude of the adapters' part, low, magnitude of low)."""
    x, w, d, u = x.double(), weights.double(), down.double(), up.double()
    w, first, second = (w, u, d) if transpose else (w.t(), d.transpose(1, 2), u.transpose(1, 2))
    n, r = x.shape[0], down.shape[1]
    out = torch.full((n, w.shape[1]), fill, dtype=torch.float64)
    mag, part = torch.zeros_like(out), torch.zeros_like(out)
    low = torch.zeros(n, r, dtype=torch.float64)
    low_mag = torch.zeros_like(low)
    o = off.tolist()
    for s, (a, b) in enumerate(zip(o[:-1], o[1:])):
        out[a:b], mag[a:b] = x[a:b] @ w, x[a:b].abs() @ w.abs()
        j = int(which[s])
        if 0 <= j < down.shape[0]:
            c = 1.0 if scale is None else float(scale[j])
            low[a:b], low_mag[a:b] = c * (x[a:b] @ first[j]), abs(c) * (x[a:b].abs() @ first[j].abs())
            out[a:b] += low[a:b] @ second[j]
            mag[a:b] += low_mag[a:b] @ second[j].abs()
            part[a:b] = low[a:b].abs() @ second[j].abs()
    return out, mag, part, low, low_mag
