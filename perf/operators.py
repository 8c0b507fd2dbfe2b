"""Measured cases of the operators over ragged groups of rows: grouping rows by
an index, the matrix product of each group with its own weights, the sum of
outer products of each group (the gradient of those weights), the weighted
join of the rows a token was sent to (and its gradient), and a projection that
all rows share with a low-rank adapter per request beside it.

``run`` makes the calls of the library where ``own`` is true, and the plain
torch form of the same operator, in 32 bits, where it is false.  ``exact``
states each operator a third time, group by group in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # a serving step of a mixture of experts: 16 tokens pick 8 of 64 experts; latency is all there is
        {"name": "group-tokens", "kind": "group", "rows": 16, "fanout": 8, "groups": 64, "skew": 1.0},
        # an unsorted edge list sorted by destination before a segmented reduction
        {"name": "group-edges", "kind": "group", "rows": 4000000, "fanout": 1, "groups": 250000, "skew": 0.0},
        # the experts' products of one decoding step: nearly every row meets weights of its own
        {"name": "experts-decode", "kind": "matmul", "rows": 8, "fanout": 8, "groups": 64, "k": 2048, "m": 1024,
         "type": "bf16", "transpose": True, "skew": 0.5},
        # the experts' products of a prompt, rows gathered from the tokens, unevenly loaded experts
        {"name": "experts-prompt", "kind": "matmul", "rows": 4096, "fanout": 8, "groups": 64, "k": 2048, "m": 2048,
         "type": "bf16", "transpose": True, "skew": 0.7},
        # a linear layer per edge type of a graph, odd row count, weights applied from the right
        {"name": "relations", "kind": "matmul", "rows": 200003, "fanout": 1, "groups": 7, "k": 64, "m": 96,
         "type": "f32", "transpose": False, "skew": 1.0},
        # the gradient of those layers' weights: few groups, long sums
        {"name": "relations-grad", "kind": "outer", "rows": 300007, "groups": 5, "k": 64, "m": 96, "type": "f32",
         "skew": 1.0},
        # one training step through the experts' products: output, input gradient, weight gradient
        {"name": "experts-train", "kind": "train", "rows": 4096, "fanout": 2, "groups": 8, "k": 1024, "m": 2560,
         "type": "f16", "skew": 0.7},
        # the experts' answers of one decoding step joined per token
        {"name": "combine-tokens", "kind": "combine", "rows": 16, "fanout": 8, "m": 2048, "type": "bf16"},
        # the gradient of that join over a prompt: rows and weights
        {"name": "combine-grad", "kind": "combine_grad", "rows": 8192, "fanout": 4, "m": 2048, "type": "bf16"},
        # one token each for 48 requests over 32 adapters beside one shared projection
        {"name": "adapter-decode", "kind": "adapter", "segments": 48, "mean": 1, "adapters": 32, "rank": 16,
         "k": 4096, "m": 4096, "type": "bf16"},
        # prompts of 12 requests, some without an adapter
        {"name": "adapter-prompt", "kind": "adapter", "segments": 12, "mean": 500, "adapters": 8, "rank": 64,
         "k": 4096, "m": 2048, "type": "f16"},
        # a training step of the adapters: output, input gradient, gradients of both factors
        {"name": "adapter-train", "kind": "adapter_train", "segments": 8, "mean": 512, "adapters": 4, "rank": 32,
         "k": 2048, "m": 2048, "type": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: mostly whole 16-byte units, now and then any number."""
    w = _log(rng, lo, hi)
    return w if rng.random() < 0.25 else max(8, w // 8 * 8)


def draw(rng):
    """One case of the listed ranges, no dearer than the dearest of them."""
    while True:
        c = _draw(rng)
        w = work(c)
        if w["flops"] <= 2.7e11 and w["bytes"] <= 6.8e8:
            return c


def _draw(rng):
    kind = rng.choice(("group", "matmul", "matmul", "outer", "train", "combine", "combine_grad", "adapter", "adapter",
                       "adapter_train"))
    t = rng.choice(("bf16", "f16", "f32"))
    if kind == "group":
        fanout = rng.choice((1, 1, 2, 4, 8))
        return {"kind": kind, "rows": _log(rng, 1, 4000000 // fanout), "fanout": fanout,
                "groups": _log(rng, 8, 250000), "skew": round(rng.uniform(0, 1), 2)}
    if kind in ("combine", "combine_grad"):
        return {"kind": kind, "rows": _log(rng, 1, 8192), "fanout": rng.choice((1, 2, 3, 4, 6, 8)),
                "m": _width(rng, 64, 2560), "type": t}
    if kind in ("adapter", "adapter_train"):
        segments = _log(rng, 1, 64)
        mean = 1 if kind == "adapter" and rng.random() < 0.4 else _log(rng, 1, max(2, 6000 // segments))
        return {"kind": kind, "segments": segments, "mean": mean, "adapters": _log(rng, 1, 32),
                "rank": rng.choice((4, 8, 12, 16, 32, 64)), "k": _width(rng, 256, 4096), "m": _width(rng, 256, 4096),
                "type": t if t != "f32" or segments * mean < 1024 else "bf16"}
    if kind == "outer":
        return {"kind": kind, "rows": _log(rng, 64, 300000), "groups": _log(rng, 1, 64), "k": _width(rng, 16, 256),
                "m": _width(rng, 16, 256), "type": t, "skew": round(rng.uniform(0, 1), 2)}
    fanout = rng.choice((1, 2, 4, 8))
    c = {"kind": kind, "rows": _log(rng, 1, 32768 // fanout), "fanout": fanout, "groups": _log(rng, 8, 64),
         "k": _width(rng, 64, 2048), "m": _width(rng, 64, 2560), "type": t, "skew": round(rng.uniform(0, 1), 2)}
    if kind == "matmul":
        c["transpose"] = rng.random() < 0.5
    return c


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, device="cuda", dtype=dtype, generator=g).mul_(std)


def _choices(g, case):
    """[rows, fanout] distinct groups per row: a router's best, with a bias per group where the load is uneven."""
    rows, fanout, groups = case["rows"], case["fanout"], case["groups"]
    if fanout == 1 and groups > 1024:
        return torch.randint(0, groups, (rows,), device="cuda", generator=g)
    if fanout == 1 or rows * groups > 1 << 26:
        u = torch.rand(rows, fanout, device="cuda", generator=g) ** (1.0 + case["skew"])
        first = (u * groups).long().clamp_(max=groups - 1)
        step = torch.arange(fanout, device="cuda") * max(1, groups // fanout)
        choice = (first[:, :1] + step) % groups
        return choice.view(-1) if fanout == 1 else choice
    score = _randn(g, rows, groups) + case["skew"] * _randn(g, groups)
    return score.topk(fanout, dim=1).indices


def _grouped(choice, groups):
    """order (source row), position (place of each choice), offsets: by a stable sort."""
    flat = choice.reshape(-1)
    _, at = flat.sort(stable=True)
    fanout = 1 if choice.dim() == 1 else choice.shape[1]
    position = torch.empty_like(at)
    position[at] = torch.arange(at.numel(), device=at.device)
    counts = torch.bincount(flat, minlength=groups)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    return at // fanout, position.view(choice.shape), offsets


def _longest(offsets):
    return max(1, int((offsets[1:] - offsets[:-1]).max()))


def _lengths(g, case):
    """Rows of each request: one each, or ragged around the mean with an empty one among four or more."""
    s, mean = case["segments"], case["mean"]
    if mean == 1:
        n = torch.ones(s, device="cuda", dtype=torch.int64)
    else:
        # the total is mean * segments for every seed
        cuts = torch.randint(0, mean * s + 1, (s - 1,), device="cuda", generator=g).sort().values
        edge = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), mean * s)])
        n = edge[1:] - edge[:-1]
        if s >= 4:
            n[1] += n[2]
            n[2] = 0
    return torch.cat([n.new_zeros(1), n.cumsum(0)])


def prepare(case, seed):
    g = _gen(seed)
    kind = case["kind"]
    s = {"case": case}
    if kind == "group":
        s["index"] = _choices(g, case)
        return s
    t = _TYPES[case["type"]]
    if kind in ("combine", "combine_grad"):
        rows, fanout, m = case["rows"], case["fanout"], case["m"]
        s["values"] = _randn(g, rows * fanout, m, dtype=t)
        s["position"] = torch.randperm(rows * fanout, device="cuda", generator=g).view(rows, fanout)
        s["weights"] = torch.rand(rows, fanout, device="cuda", generator=g) + 0.01
        s["weights"] /= s["weights"].sum(1, keepdim=True)
        if kind == "combine_grad":
            s["grad"] = _randn(g, rows, m, dtype=t)
        return s
    k, m = case["k"], case["m"]
    if kind in ("adapter", "adapter_train"):
        r, count = case["rank"], case["adapters"]
        s["offsets"] = _lengths(g, case)
        s["longest"] = _longest(s["offsets"])
        n = case["segments"] * case["mean"]
        lo = 0 if kind == "adapter_train" else -1
        s["which"] = torch.randint(lo, count, (case["segments"],), device="cuda", generator=g)
        s["values"] = _randn(g, n, k, dtype=t)
        s["weights"] = _randn(g, m, k, dtype=t, std=k ** -0.5)
        s["down"] = _randn(g, count, r, k, dtype=t, std=k ** -0.5)
        s["up"] = _randn(g, count, m, r, dtype=t, std=0.3 * r ** -0.5)
        s["scale"] = torch.rand(count, device="cuda", generator=g) + 0.5
        if kind == "adapter_train":
            s["grad"] = _randn(g, n, m, dtype=t)
            length = s["offsets"][1:] - s["offsets"][:-1]
            s["row_which"] = s["which"].repeat_interleave(length)
        return s
    groups = case["groups"]
    if kind == "outer":
        choice = _choices(g, dict(case, fanout=1))
        _, _, s["offsets"] = _grouped(choice, groups)
        s["left"] = _randn(g, case["rows"], k, dtype=t)
        s["right"] = _randn(g, case["rows"], m, dtype=t)
    else:
        choice = _choices(g, case)
        s["order"], _, s["offsets"] = _grouped(choice, groups)
        s["values"] = _randn(g, case["rows"], k, dtype=t)
        shape = (m, k) if case.get("transpose", True) else (k, m)
        s["weights"] = _randn(g, groups, *shape, dtype=t, std=k ** -0.5)
        if kind == "train":
            s["grad"] = _randn(g, case["rows"] * case["fanout"], m, dtype=t)
    s["longest"] = _longest(s["offsets"])
    return s


# -------------------------------------------------------------- plain forms

def _places(offsets, longest):
    """[groups, longest] row numbers of each group and which of them exist."""
    at = offsets[:-1, None] + torch.arange(longest, device=offsets.device)
    there = at < offsets[1:, None]
    return torch.where(there, at, 0), there


def _pad(x, offsets, longest):
    at, there = _places(offsets, longest)
    return torch.where(there[..., None], x[at].float(), 0.0)


def _unpad(y, offsets, n):
    row = torch.arange(n, device=offsets.device)
    group = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    return y[group, row - offsets[group]]


def _plain_group(index, groups):
    fanout = 1 if index.dim() == 1 else index.shape[1]
    flat = index.reshape(-1)
    key, at = flat.sort(stable=True)
    position = torch.empty_like(at)
    position[at] = torch.arange(at.numel(), device=at.device)
    offsets = torch.searchsorted(key, torch.arange(groups + 1, device=at.device))
    return at // fanout, position.view(index.shape), offsets


def _plain_matmul(values, weights, offsets, longest, transpose, rows=None):
    x = values if rows is None else values[rows]
    w = weights.float()
    w = w.transpose(1, 2).contiguous() if transpose else w
    return _unpad(torch.bmm(_pad(x, offsets, longest), w), offsets, x.shape[0]).to(values.dtype)


def _plain_outer(left, right, offsets, longest, right_rows=None):
    right = right if right_rows is None else right[right_rows]
    a = _pad(left, offsets, longest).transpose(1, 2).contiguous()
    return torch.bmm(a, _pad(right, offsets, longest)).to(left.dtype)


def _plain_adapter(x, w, offsets, longest, which, first, second, scale):
    """x w + scale (x first) second, first [., in, rank] and second [., rank, out] of each request's adapter."""
    has = (which >= 0)[:, None, None]
    a = which.clamp(min=0)
    low = torch.bmm(_pad(x, offsets, longest), first[a].float()) * torch.where(has, scale[a][:, None, None], 0.0)
    add = torch.bmm(low, second[a].float())
    n = x.shape[0]
    out = x.float() @ w.float() + _unpad(add, offsets, n)
    return out.to(x.dtype), _unpad(low, offsets, n)


def _plain(s):
    case, kind = s["case"], s["case"]["kind"]
    if kind == "group":
        return _plain_group(s["index"], case["groups"])
    if kind == "combine":
        return (s["weights"][..., None] * s["values"][s["position"]].float()).sum(1).to(s["values"].dtype)
    if kind == "combine_grad":
        g = s["grad"].float()[:, None, :]
        rows = torch.empty_like(s["values"])
        rows[s["position"].view(-1)] = (s["weights"][..., None] * g).to(rows.dtype).flatten(0, 1)
        return rows, (g * s["values"][s["position"]].float()).sum(-1)
    if kind == "matmul":
        return _plain_matmul(s["values"], s["weights"], s["offsets"], s["longest"], case["transpose"], s["order"])
    if kind == "outer":
        return _plain_outer(s["left"], s["right"], s["offsets"], s["longest"])
    if kind == "train":
        out = _plain_matmul(s["values"], s["weights"], s["offsets"], s["longest"], True, s["order"])
        grad_rows = _plain_matmul(s["grad"], s["weights"], s["offsets"], s["longest"], False)
        grad_weights = _plain_outer(s["grad"], s["values"], s["offsets"], s["longest"], s["order"])
        return out, grad_rows, grad_weights
    down, up = s["down"], s["up"]
    out, low = _plain_adapter(s["values"], s["weights"].t(), s["offsets"], s["longest"], s["which"],
                              down.transpose(1, 2), up.transpose(1, 2), s["scale"])
    if kind == "adapter":
        return out
    grad, grad_low = _plain_adapter(s["grad"], s["weights"], s["offsets"], s["longest"], s["which"], up, down,
                                    s["scale"])
    mine = torch.arange(down.shape[0], device=out.device)[:, None] == s["row_which"]  # [adapters, rows]
    g, x = s["grad"].float(), s["values"].float()
    grad_up = torch.matmul(g.t(), torch.where(mine[..., None], low, 0.0)).to(up.dtype)
    grad_down = torch.matmul(torch.where(mine[..., None], grad_low, 0.0).transpose(1, 2), x).to(down.dtype)
    return out, grad, grad_down, grad_up


# ---------------------------------------------------------- the library's calls

def _calls(s):
    import segmented_reduction_amd as sr
    case, kind = s["case"], s["case"]["kind"]
    if kind == "group":
        return sr.group(s["index"], case["groups"])
    if kind == "combine":
        return sr.combine(s["values"], s["position"], s["weights"])
    if kind == "combine_grad":
        return sr.combine_grad(s["grad"], s["values"], s["position"], s["weights"])
    if kind == "matmul":
        return sr.matmul(s["values"], s["weights"], s["offsets"], transpose=case["transpose"], rows=s["order"])
    if kind == "outer":
        return sr.outer(s["left"], s["right"], s["offsets"])
    if kind == "train":
        out = sr.matmul(s["values"], s["weights"], s["offsets"], transpose=True, rows=s["order"])
        grad_rows = sr.matmul(s["grad"], s["weights"], s["offsets"])
        grad_weights = sr.outer(s["grad"], s["values"], s["offsets"], right_rows=s["order"])
        return out, grad_rows, grad_weights
    args = (s["weights"], s["offsets"], s["which"], s["down"], s["up"])
    if kind == "adapter":
        return sr.adapter(s["values"], *args, scale=s["scale"])
    # low-rank rows in float32, so that the factors' gradients are rounded once
    out, low = sr.adapter(s["values"], *args, scale=s["scale"], want_low=torch.float32)
    grad, grad_low = sr.adapter(s["grad"], *args, scale=s["scale"], transpose=True, want_low=torch.float32)
    order, _, bounds = sr.group(s["row_which"], case["adapters"])
    grad_up = sr.outer(s["grad"], low, bounds, left_rows=order, right_rows=order, out_dtype=s["up"].dtype)
    grad_down = sr.outer(grad_low, s["values"], bounds, left_rows=order, right_rows=order, out_dtype=s["down"].dtype)
    return out, grad, grad_down, grad_up


def run(state):
    return _calls(state) if own else _plain(state)


# --------------------------------------------------------------------- work

def work(case):
    kind = case["kind"]
    if kind == "group":
        n = case["rows"] * case["fanout"]
        return {"bytes": 8 * n * 3 + 8 * (case["groups"] + 1), "flops": 0}
    e = 4 if case["type"] == "f32" else 2
    if kind in ("combine", "combine_grad"):
        rows, n, m = case["rows"], case["rows"] * case["fanout"], case["m"]
        if kind == "combine":
            return {"bytes": e * m * (n + rows) + 12 * n, "flops": 2 * n * m}
        return {"bytes": e * m * (2 * n + rows) + 16 * n, "flops": 3 * n * m}
    k, m = case["k"], case["m"]
    if kind in ("adapter", "adapter_train"):
        n, r, segs = case["segments"] * case["mean"], case["rank"], case["segments"]
        # the adapters that at least one request picks, on average
        live = case["adapters"] * (1 - (1 - 1 / (case["adapters"] + 1)) ** segs)
        both = live * r * (k + m)
        one = {"bytes": e * (n * (k + m) + k * m + both), "flops": 2 * n * (k * m + r * (k + m))}
        if kind == "adapter":
            return one
        # forward and input gradient read the same weights; the factors' gradients are written once
        return {"bytes": e * (2 * n * (k + m) + k * m + 2 * both),
                "flops": 2 * one["flops"] + 2 * n * r * (k + m)}
    groups = case["groups"]
    if kind == "outer":
        n = case["rows"]
        return {"bytes": e * (n * (k + m) + groups * k * m) + 8 * groups, "flops": 2 * n * k * m}
    n = case["rows"] * case["fanout"]
    live = groups * (1 - (1 - 1 / groups) ** n)  # groups that have a row, on average
    if kind == "matmul":
        return {"bytes": e * (case["rows"] * k + n * m + live * k * m) + 8 * (n + groups), "flops": 2 * n * k * m}
    return {"bytes": e * (case["rows"] * k + 2 * n * m + n * k + (live + groups) * k * m) + 8 * (n + groups),
            "flops": 6 * n * k * m}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind == "group":
        return None
    d = torch.float64
    if kind == "combine":
        v, w, p = s["values"].to(d), s["weights"].to(d), s["position"]
        out = torch.zeros(case["rows"], case["m"], dtype=d, device="cuda")
        for j in range(case["fanout"]):
            out += w[:, j, None] * v.index_select(0, p[:, j])
        return out
    if kind == "combine_grad":
        v, w, p, g = s["values"].to(d), s["weights"].to(d), s["position"], s["grad"].to(d)
        rows, part = torch.zeros_like(v), torch.zeros_like(w)
        for j in range(case["fanout"]):
            rows.index_copy_(0, p[:, j], w[:, j, None] * g)
            part[:, j] = torch.linalg.vecdot(g, v.index_select(0, p[:, j]))
        return rows, part
    off = s["offsets"].tolist()
    spans = list(enumerate(zip(off[:-1], off[1:])))
    if kind == "outer":
        return torch.stack([s["left"][a:b].to(d).t() @ s["right"][a:b].to(d) for _, (a, b) in spans])
    if kind in ("matmul", "train"):
        x = s["values"].to(d).index_select(0, s["order"])
        turn = case.get("transpose", True)
        out = torch.cat([x[a:b] @ (s["weights"][i].to(d).t() if turn else s["weights"][i].to(d)) for i, (a, b) in spans])
        if kind == "matmul":
            return out
        g = s["grad"].to(d)
        grad_rows = torch.cat([g[a:b] @ s["weights"][i].to(d) for i, (a, b) in spans])
        return out, grad_rows, torch.stack([g[a:b].t() @ x[a:b] for _, (a, b) in spans])
    x, w = s["values"].to(d), s["weights"].to(d)
    out, which, scale = x @ w.t(), s["which"].tolist(), s["scale"].to(d)
    train = kind == "adapter_train"
    if train:
        g = s["grad"].to(d)
        grad = g @ w
        grad_down, grad_up = torch.zeros_like(s["down"], dtype=d), torch.zeros_like(s["up"], dtype=d)
    for i, (a, b) in spans:
        j = which[i]
        if j < 0 or a == b:
            continue
        down, up = s["down"][j].to(d), s["up"][j].to(d)
        out[a:b] += scale[j] * (x[a:b] @ down.t()) @ up.t()
        if train:
            grad[a:b] += scale[j] * (g[a:b] @ up) @ down
            grad_down[j] += scale[j] * (g[a:b] @ up).t() @ x[a:b]
            grad_up[j] += scale[j] * g[a:b].t() @ (x[a:b] @ down.t())
    return (out, grad, grad_down, grad_up) if train else out
