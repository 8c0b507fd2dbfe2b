"""Measured cases of the operators that stand around the products over ragged
groups of rows in a training step: the normalisation of rows in front of them
(and its gradient, with the sums of the weight's), the gated pair of projections
inside them (and its gradient), and behind them the softmax cross entropy of
rows against a large vocabulary, whose logits are never kept (and its gradient).

``run`` makes the calls of the library where ``own`` is true, and the plain
torch form of the same operator, in 32 bits, where it is false.  ``exact``
states each operator a third time in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
_MOST = {"flops": 4.5e12, "bytes": 1.7e9}  # of a drawn case


def listed():
    return [
        # the experts' gated projections of one decoding step: 8 tokens pick 8 of 64 experts
        {"name": "gated-decode", "kind": "gated", "rows": 8, "fanout": 8, "groups": 64, "k": 2048, "m": 1024,
         "type": "bf16", "act": "silu", "skew": 0.5},
        # the same of a prompt, rows gathered from the tokens, unevenly loaded experts
        {"name": "gated-prompt", "kind": "gated", "rows": 4096, "fanout": 8, "groups": 64, "k": 2048, "m": 1024,
         "type": "bf16", "act": "silu", "skew": 0.7},
        # a training step of a few large experts: output, gradients of both projections, of the rows, of the weights
        {"name": "gated-train", "kind": "gated_train", "rows": 4096, "fanout": 2, "groups": 8, "k": 1024, "m": 2560,
         "type": "f16", "act": "gelu_tanh", "skew": 0.7},
        # gated layers per edge type of a graph, odd row count, forward and back
        {"name": "gated-relations", "kind": "gated_train", "rows": 40007, "fanout": 1, "groups": 5, "k": 96, "m": 130,
         "type": "f32", "act": "gelu", "skew": 1.0},
        # the rows of one decoding step; latency is all there is
        {"name": "norm-tokens", "kind": "norm", "rows": 16, "k": 4096, "type": "bf16", "weight": "bf16", "bias": True,
         "center": True},
        # the rows of a long prompt, by their root mean square
        {"name": "norm-prompt", "kind": "norm", "rows": 16384, "k": 4096, "type": "bf16", "weight": "bf16",
         "bias": False, "center": False},
        # a training step over a batch, parameters kept in float32
        {"name": "norm-train", "kind": "norm_train", "rows": 16384, "k": 2048, "type": "bf16", "weight": "f32",
         "bias": True, "center": True},
        # the features of a graph's nodes: odd rows, odd width
        {"name": "norm-nodes", "kind": "norm_train", "rows": 50021, "k": 333, "type": "f32", "weight": "f32",
         "bias": True, "center": True},
        # scoring a handful of continuations
        {"name": "loss-few", "kind": "loss", "rows": 8, "k": 2048, "vocab": 32000, "picks": 1, "type": "bf16"},
        # the perplexity of an evaluation batch
        {"name": "loss-eval", "kind": "loss", "rows": 4096, "k": 2048, "vocab": 65536, "picks": 1, "type": "bf16"},
        # the end of a training step: loss, gradient of the rows and of the vocabulary's weights
        {"name": "loss-train", "kind": "loss_train", "rows": 4096, "k": 2048, "vocab": 65536, "picks": 1,
         "type": "bf16"},
        # learning from a teacher's 32 most likely tokens, odd vocabulary
        {"name": "loss-distil", "kind": "loss_train", "rows": 1500, "k": 1024, "vocab": 32011, "picks": 32,
         "type": "f16"},
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
        if w["flops"] <= _MOST["flops"] and w["bytes"] <= _MOST["bytes"]:
            return c


def _draw(rng):
    kind = rng.choice(("gated", "gated", "gated_train", "norm", "norm_train", "loss", "loss_train"))
    t = rng.choice(("bf16", "f16", "f32"))
    if kind in ("norm", "norm_train"):
        k = _width(rng, 32, 8192)
        return {"kind": kind, "rows": _log(rng, 1, min(65536, (1 << 26) // k)), "k": k, "type": t,
                "weight": rng.choice((t, "f32")), "bias": rng.random() < 0.5, "center": rng.random() < 0.5}
    if kind in ("loss", "loss_train"):
        rows, k, vocab = _log(rng, 1, 4096), _width(rng, 64, 2048), _log(rng, 500, 65536)
        if t == "f32" and rows * k * vocab > 1 << 37:
            t = "bf16"
        return {"kind": kind, "rows": rows, "k": k, "vocab": vocab, "picks": rng.choice((1, 1, 1, 4, 16, 32)),
                "type": t}
    fanout = rng.choice((1, 2, 4, 8))
    return {"kind": kind, "rows": _log(rng, 1, 32768 // fanout), "fanout": fanout, "groups": _log(rng, 8, 64),
            "k": _width(rng, 64, 2048), "m": _width(rng, 64, 2560), "type": t,
            "act": rng.choice(("silu", "gelu", "gelu_tanh")), "skew": round(rng.uniform(0, 1), 2)}


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _randn(g, *shape, dtype=torch.float32, std=1.0):
    return torch.randn(*shape, device="cuda", dtype=dtype, generator=g).mul_(std)


def _choices(g, case):
    """[rows, fanout] groups per row: a router's best, with a bias per group where the load is uneven."""
    rows, fanout, groups = case["rows"], case["fanout"], case["groups"]
    if fanout == 1:
        u = torch.rand(rows, 1, device="cuda", generator=g) ** (1.0 + case["skew"])
        return (u * groups).long().clamp_(max=groups - 1)
    score = _randn(g, rows, groups) + case["skew"] * _randn(g, groups)
    return score.topk(fanout, dim=1).indices


def prepare(case, seed):
    g = _gen(seed)
    kind, t = case["kind"], _TYPES[case["type"]]
    s = {"case": case}
    k = case["k"]
    if kind in ("norm", "norm_train"):
        w = _TYPES[case["weight"]]
        # rows of a residual stream: an offset and a size of their own
        n = case["rows"]
        size = torch.rand(n, 1, device="cuda", generator=g) * 2 + 0.5
        s["values"] = ((_randn(g, n, k) + 0.3 * _randn(g, n, 1)) * size).to(t)
        s["weight"] = (_randn(g, k, std=0.2) + 1).to(w)
        s["bias"] = _randn(g, k, std=0.2).to(w) if case["bias"] else None
        if kind == "norm_train":
            s["grad"] = _randn(g, n, k, dtype=t)
        return s
    if kind in ("loss", "loss_train"):
        n, v, picks = case["rows"], case["vocab"], case["picks"]
        s["weights"] = _randn(g, v, k, dtype=t, std=2 * k ** -0.5)
        hot = torch.randint(0, v, (n, picks), device="cuda", generator=g)
        # rows that lean towards what they should answer
        s["values"] = (_randn(g, n, k) + s["weights"][hot[:, 0]].float()).to(t)
        none = torch.rand(n, device="cuda", generator=g) < 0.05  # padding
        s["target"] = torch.where(none[:, None], -100, hot)
        s["probs"] = None
        if picks == 1:
            s["target"] = s["target"].view(-1).contiguous()
        else:
            s["probs"] = _randn(g, n, picks, std=2.0).softmax(1)
        if kind == "loss_train":
            s["grad"] = torch.rand(n, device="cuda", generator=g) + 0.5
        return s
    m, groups = case["m"], case["groups"]
    flat = _choices(g, case).view(-1)
    _, at = flat.sort(stable=True)
    counts = torch.bincount(flat, minlength=groups)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)])
    s["order"] = at // case["fanout"]
    s["longest"] = max(1, int(counts.max()))
    s["values"] = _randn(g, case["rows"], k, dtype=t)
    s["weights"] = _randn(g, groups, 2 * m, k, dtype=t, std=k ** -0.5)  # the gate's rows, then the other's
    if kind == "gated_train":
        s["grad"] = _randn(g, flat.numel(), m, dtype=t)
    return s


# -------------------------------------------------------------- plain forms

def _act(x, name):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return x * 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
    return x * 0.5 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _act_slope(x, name):
    if name == "silu":
        y = 1 / (1 + torch.exp(-x))
        return y * (1 + x * (1 - y))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1 / math.sqrt(2 * math.pi))
    c = math.sqrt(2 / math.pi)
    y = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1 + y) + 0.5 * x * (1 - y * y) * c * (1 + 3 * 0.044715 * x * x)


def _pad(x, offsets, longest):
    at = offsets[:-1, None] + torch.arange(longest, device=offsets.device)
    there = at < offsets[1:, None]
    return torch.where(there[..., None], x[torch.where(there, at, 0)].float(), 0.0)


def _unpad(y, offsets, n):
    row = torch.arange(n, device=offsets.device)
    group = torch.searchsorted(offsets[1:].contiguous(), row, right=True)
    return y[group, row - offsets[group]]


def _plain_gated(s):
    case, off, longest = s["case"], s["offsets"], s["longest"]
    m, t, n = case["m"], s["values"].dtype, s["order"].numel()
    x = _pad(s["values"][s["order"]], off, longest)
    w = s["weights"].float()
    pre = _unpad(torch.bmm(x, w.transpose(1, 2).contiguous()), off, n)
    gate, up = pre[:, :m], pre[:, m:]
    out = (_act(gate, case["act"]) * up).to(t)
    if case["kind"] == "gated":
        return out
    g = s["grad"].float()
    grad = torch.cat([g * up * _act_slope(gate, case["act"]), g * _act(gate, case["act"])], 1)
    full = _pad(grad, off, longest)
    grad_rows = _unpad(torch.bmm(full, w), off, n)
    grad_weights = torch.bmm(full.transpose(1, 2).contiguous(), x)
    return out, grad.to(t), grad_rows.to(t), grad_weights.to(t)


def _plain_norm(s):
    case, t = s["case"], s["values"].dtype
    x, w = s["values"].float(), s["weight"].float()
    if case["center"]:
        x = x - x.mean(1, keepdim=True)
    r = 1 / torch.sqrt((x * x).mean(1, keepdim=True) + 1e-5)
    unit = x * r
    out = unit * w
    if s["bias"] is not None:
        out = out + s["bias"].float()
    if case["kind"] == "norm":
        return out.to(t)
    g = s["grad"].float()
    gw = g * w
    back = gw - unit * (gw * unit).mean(1, keepdim=True)
    if case["center"]:
        back = back - gw.mean(1, keepdim=True)
    grads = [(back * r).to(t), (g * unit).sum(0).to(s["weight"].dtype)]
    if s["bias"] is not None:
        grads.append(g.sum(0).to(s["weight"].dtype))
    return [out.to(t)] + grads


def _plain_loss(s):
    x, w = s["values"].float(), s["weights"].float()
    target = s["target"].view(x.shape[0], -1)
    there = (target >= 0) & (target < w.shape[0])
    at = torch.where(there, target, 0)
    p = torch.where(there, s["probs"] if s["probs"] is not None else 1.0, 0.0)
    z = x @ w.t()
    top = z.max(1, keepdim=True).values
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    lse = (top + torch.log(total)).squeeze(1)
    share = p.sum(1)
    loss = share * lse - (p * z.gather(1, at)).sum(1)
    if s["case"]["kind"] == "loss":
        return loss, lse
    e *= share[:, None] / total
    e.scatter_add_(1, at, -p)
    e *= s["grad"][:, None]
    t = s["values"].dtype
    return loss, lse, (e @ w).to(t), (e.t() @ x).to(t)


def _plain(s):
    kind = s["case"]["kind"]
    if kind in ("norm", "norm_train"):
        return _plain_norm(s)
    if kind in ("loss", "loss_train"):
        return _plain_loss(s)
    return _plain_gated(s)


# ---------------------------------------------------------- the library's calls

def _calls(s):
    import segmented_reduction_amd as sr
    case, kind = s["case"], s["case"]["kind"]
    if kind in ("norm", "norm_train"):
        out = sr.norm(s["values"], s["weight"], s["bias"], eps=1e-5, center=case["center"])
        if kind == "norm":
            return out
        grad, grad_weight, grad_bias = sr.norm_grad(s["grad"], s["values"], s["weight"], eps=1e-5,
                                                    center=case["center"], want_bias=case["bias"])
        return [out, grad, grad_weight] + ([grad_bias] if case["bias"] else [])
    if kind in ("loss", "loss_train"):
        loss, lse, picked = sr.cross_entropy(s["values"], s["weights"], s["target"], probs=s["probs"])
        if kind == "loss":
            return loss, lse
        grad, grad_weights = sr.cross_entropy_grad(s["grad"], s["values"], s["weights"], s["target"], lse, picked,
                                                   probs=s["probs"])
        return loss, lse, grad, grad_weights
    out = sr.gated(s["values"], s["weights"], s["offsets"], activation=case["act"], rows=s["order"])
    if kind == "gated":
        return out
    grad = sr.gated_grad(s["grad"], s["values"], s["weights"], s["offsets"], activation=case["act"], rows=s["order"])
    grad_rows = sr.matmul(grad, s["weights"], s["offsets"])
    grad_weights = sr.outer(grad, s["values"], s["offsets"], right_rows=s["order"])
    return out, grad, grad_rows, grad_weights


def run(state):
    return _calls(state) if own else _plain(state)


# --------------------------------------------------------------------- work

def work(case):
    kind, k = case["kind"], case["k"]
    e = 4 if case["type"] == "f32" else 2
    if kind in ("norm", "norm_train"):
        n, params = case["rows"], (2 if case["bias"] else 1) * k * (4 if case["weight"] == "f32" else 2)
        if kind == "norm":
            return {"bytes": 2 * e * n * k + params, "flops": 8 * n * k}
        # values and gradient read once, both results and the parameters' gradients written
        return {"bytes": 4 * e * n * k + 2 * params, "flops": 20 * n * k}
    if kind in ("loss", "loss_train"):
        n, v, one = case["rows"], case["vocab"], 2 * case["rows"] * case["vocab"] * k
        small = n * (12 * case["picks"] + 8)
        if kind == "loss":
            return {"bytes": e * (n + v) * k + small, "flops": one}
        return {"bytes": 2 * e * (n + v) * k + small, "flops": 3 * one}
    m, groups, n = case["m"], case["groups"], case["rows"] * case["fanout"]
    live = groups * (1 - (1 - 1 / groups) ** n)  # groups that have a row, on average
    weights = 2 * m * k
    if kind == "gated":
        return {"bytes": e * (case["rows"] * k + n * m + live * weights) + 8 * (n + groups), "flops": 2 * n * weights}
    return {"bytes": e * (case["rows"] * k + n * (4 * m + k) + (live + groups) * weights) + 8 * (n + groups),
            "flops": 6 * n * weights}


# -------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    kind, d = case["kind"], torch.float64
    x = s["values"].to(d)
    if kind in ("norm", "norm_train"):
        w = s["weight"].to(d)
        mean = x.sum(1) / x.shape[1] if case["center"] else torch.zeros_like(x[:, 0])
        spread = ((x - mean[:, None]) ** 2).sum(1) / x.shape[1]
        unit = (x - mean[:, None]) * (spread + 1e-5).rsqrt()[:, None]
        out = torch.addcmul(s["bias"].to(d), unit, w) if case["bias"] else unit * w
        if kind == "norm":
            return out
        g = s["grad"].to(d)
        # the Jacobian of one row, (I - 1/k - unit unit^T / k) / sigma, applied to g w
        gw = g * w
        along = torch.linalg.vecdot(gw, unit) / x.shape[1]
        level = gw.sum(1) / x.shape[1] if case["center"] else torch.zeros_like(along)
        back = (gw - level[:, None] - unit * along[:, None]) / (spread + 1e-5).sqrt()[:, None]
        ones = torch.ones(1, x.shape[0], dtype=d, device="cuda")
        grads = [back, (ones @ (g * unit))[0]] + ([(ones @ g)[0]] if case["bias"] else [])
        return [out] + grads
    if kind in ("loss", "loss_train"):
        w, n = s["weights"].to(d), x.shape[0]
        target = s["target"].view(n, -1)
        goal = torch.zeros(n, w.shape[0] + 1, dtype=d, device="cuda")  # the last column: no target
        at = torch.where((target < 0) | (target >= w.shape[0]), w.shape[0], target)
        for j in range(at.shape[1]):
            p = s["probs"][:, j].to(d) if s["probs"] is not None else torch.ones(n, dtype=d, device="cuda")
            goal[torch.arange(n, device="cuda"), at[:, j]] += p
        goal = goal[:, :-1]
        log_p = (x @ w.t()).log_softmax(1)
        share = goal.sum(1)
        loss = -torch.linalg.vecdot(goal, log_p)
        first = w.index_select(0, torch.zeros(1, dtype=torch.int64, device="cuda"))[0]
        lse = x @ first - log_p[:, 0]
        if kind == "loss":
            return loss, lse
        g = log_p.exp_().mul_(share[:, None]).sub_(goal).mul_(s["grad"].to(d)[:, None])
        return loss, lse, g @ w, g.t() @ x
    off, m, act = s["offsets"].tolist(), case["m"], case["act"]
    x = x.index_select(0, s["order"])
    outs, grads, rows, weights = [], [], [], []
    for i, (a, b) in enumerate(zip(off[:-1], off[1:])):
        w = s["weights"][i].to(d)
        gate, up = x[a:b] @ w[:m].t(), x[a:b] @ w[m:].t()
        if act == "silu":
            slope = torch.sigmoid(gate) + gate * torch.sigmoid(gate) * torch.sigmoid(-gate)
            y = gate * torch.sigmoid(gate)
        elif act == "gelu":
            normal = torch.distributions.Normal(torch.zeros((), dtype=d, device="cuda"), 1.0, validate_args=False)
            slope = normal.cdf(gate) + gate * normal.log_prob(gate).exp()
            y = gate * normal.cdf(gate)
        else:
            # 0.5 (1 + tanh u) = sigmoid(2 u)
            u = 2 * math.sqrt(2 / math.pi) * (gate + 0.044715 * gate ** 3)
            du = 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * gate ** 2)
            slope = torch.sigmoid(u) + gate * torch.sigmoid(u) * torch.sigmoid(-u) * du
            y = gate * torch.sigmoid(u)
        outs.append(y * up)
        if kind == "gated":
            continue
        g = s["grad"][a:b].to(d)
        grads.append(torch.cat([g * up * slope, g * y], 1))
        rows.append(grads[-1] @ w)
        weights.append(grads[-1].t() @ x[a:b])
    if kind == "gated":
        return torch.cat(outs)
    return torch.cat(outs), torch.cat(grads), torch.cat(rows), torch.stack(weights)
