"""The norms, the gated projections and the cross entropy together with the
operators over ragged groups, as a training step uses them: one block of experts
behind a norm, another norm and the loss, and the gradients of everything; on other
streams, captured and replayed, in tensors that begin anywhere and past 4 GiB (GPU
only)."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu


def _step(x, choice, prob, n1, b1, w, down, n2, vocab, target, grad):
    """loss [N], and the gradients of <grad, loss> for x, n1, b1, w, down, n2, vocab and prob."""
    h = sr.norm(x, n1, b1)
    order, position, off = sr.group(choice, w.shape[0])
    mid = sr.gated(h, w, off, activation="gelu_tanh", rows=order)
    y = sr.matmul(mid, down, off, transpose=True)
    z = sr.combine(y, position, prob) + x
    u = sr.norm(z, n2, center=False)
    loss, lse, picked = sr.cross_entropy(u, vocab, target)
    du, dvocab = sr.cross_entropy_grad(grad, u, vocab, target, lse, picked)
    dz, dn2, _ = sr.norm_grad(du, z, n2, center=False)
    dy, dprob = sr.combine_grad(dz, y, position, prob)
    dmid = sr.matmul(dy, down, off)
    ddown = sr.outer(dy, mid, off)
    pair = sr.gated_grad(dmid, h, w, off, activation="gelu_tanh", rows=order)
    dw = sr.outer(pair, h, off, right_rows=order)
    dh = sr.combine(sr.matmul(pair, w, off), position, torch.ones_like(prob))
    dx, dn1, db1 = sr.norm_grad(dh, x, n1, want_bias=True)
    return loss, dx + dz, dn1, db1, dw, ddown, dn2, dvocab, dprob


def _inputs(seed, tokens, fanout, experts, k, m, v):
    g = A.gen(seed)
    choice = torch.rand(tokens, experts, generator=g).topk(fanout, dim=1).indices
    target = torch.randint(-2, v, (tokens,), generator=g)
    return [A.randn(g, tokens, k) + 0.5, choice, torch.rand(tokens, fanout, generator=g), A.randn(g, k, std=0.2) + 1,
            A.randn(g, k, std=0.2), A.randn(g, experts, 2 * m, k, std=k ** -0.5), A.randn(g, experts, k, m, std=m ** -0.5),
            A.randn(g, k, std=0.2) + 1, A.randn(g, v, k, std=2 * k ** -0.5), target, torch.rand(tokens, generator=g) + 0.5]


def _reference(x, choice, prob, n1, b1, w, down, n2, vocab, target, grad):
    leaves = [t.double().requires_grad_() for t in (x, n1, b1, w, down, n2, vocab, prob)]
    x, n1, b1, w, down, n2, vocab, prob = leaves
    h = torch.nn.functional.layer_norm(x, x.shape[1:], n1, b1, 1e-5)
    m, z = w.shape[1] // 2, x
    for j in range(choice.shape[1]):
        pre = (w[choice[:, j]] * h[:, None]).sum(-1)
        mid = torch.nn.functional.gelu(pre[:, :m], approximate="tanh") * pre[:, m:]
        z = z + prob[:, j, None] * (down[choice[:, j]] * mid[:, None]).sum(-1)
    u = z / (z.square().mean(1, keepdim=True) + 1e-5).sqrt() * n2
    logp = (u @ vocab.t()).log_softmax(1)
    live = target >= 0
    loss = torch.where(live, -logp.gather(1, target.clamp(min=0)[:, None])[:, 0], 0.0)
    (loss * grad.double()).sum().backward()
    gx, gn1, gb1, gw, gdown, gn2, gv, gp = (t.grad for t in leaves)
    return loss.detach(), gx, gn1, gb1, gw, gdown, gn2, gv, gp


NAMES = ("loss", "dx", "dn1", "db1", "dw", "ddown", "dn2", "dvocab", "dprob")


def _near(got, want):
    """Relative to the largest value of each result: float32 sums of at most a few
    hundred terms, eight operators deep, each of which passes errors on about once,
    lose below 8 * 300 * 2^-24 < 2^-12 of it."""
    for name, a, b in zip(NAMES, got, want):
        err = float((a.cpu().double() - b).abs().max())
        assert err <= 2.0 ** -12 * float(b.abs().max()), (name, err, float(b.abs().max()))


@pytest.mark.parametrize("tokens,fanout,experts,k,m,v", [(1, 2, 4, 32, 48, 50), (60, 2, 8, 64, 40, 300), (200, 3, 5, 33, 21, 131)])
def test_step(tokens, fanout, experts, k, m, v):
    data = _inputs(tokens, tokens, fanout, experts, k, m, v)
    A.say(f"training step {tokens} {fanout} {experts} {k} {m} {v}")
    got = _step(*(t.cuda() for t in data))
    torch.cuda.synchronize()
    _near(got, _reference(*data))


def test_step_on_three_streams():
    sets = [_inputs(i, 100 + 30 * i, 2, 6, 64, 48, 200) for i in range(3)]
    dev = [[t.cuda() for t in d] for d in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    A.say("training steps on three streams")
    for _ in range(3):
        got = []
        for s, d in zip(streams, dev):
            with torch.cuda.stream(s):
                got.append(_step(*d))
    torch.cuda.synchronize()
    for g, d in zip(got, sets):
        _near(g, _reference(*d))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_step_in_two_graphs(kind):
    """Captured, replayed at once on two streams with new inputs, eager calls between: every replay as the eager call."""
    t = A.TYPES[kind]

    def load(seed):
        d = _inputs(seed, 150, 2, 6, 64, 48, 300)
        return [v.cuda().to(t) if v.dtype == torch.float32 and i not in (2, 10) else v.cuda() for i, v in enumerate(d)]

    held = [load(1), load(2)]
    _step(*held[0])  # what a first call loads is not captured
    torch.cuda.synchronize()
    side, graphs, outs = torch.cuda.Stream(), [], []
    for d in held:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            outs.append(_step(*d))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in held]
    for rep in range(4):
        A.say(f"training step graphs {kind} replay {rep}")
        for d, seed in zip(held, (10 + rep, 20 + rep)):
            for old, new in zip(d, load(seed)):
                old.copy_(new)
        want = [_step(*d) for d in held]
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            for name, a, b in zip(NAMES, got, ref):
                assert torch.equal(a, b), (rep, name)


def _odd(t):
    """The same values one element behind a 16-byte boundary."""
    return torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")[1:].view(t.shape).copy_(t)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k,v", [(7, 64, 200), (300, 128, 1000), (2100, 520, 4100)])
def test_tensors_that_begin_anywhere(kind, n, k, v):
    t, g = A.TYPES[kind], A.gen(n)
    x, w = A.randn(g, n, k, dtype=t).cuda(), A.randn(g, v, k, dtype=t, std=2 * k ** -0.5).cuda()
    target, grad = torch.randint(0, v, (n,), generator=g).cuda(), torch.randn(n, generator=g).cuda()
    A.say(f"odd places {kind} {n} {k} {v}")
    loss, lse, picked = sr.cross_entropy(_odd(x), _odd(w), target)
    dx, dw = sr.cross_entropy_grad(grad, _odd(x), _odd(w), target, lse, picked)
    torch.cuda.synchronize()
    refs, errs, _ = A.cross_entropy(x, w, target)
    A.check(loss, refs[0], errs[0], "loss")
    refs, errs = A.cross_entropy_grad(grad, x, w, target, t)
    A.check(dx, refs[0], errs[0], "dx")
    A.check(dw, refs[1], errs[1], "dw")
    m, off = 72, torch.tensor([0, n // 3, n // 3, n])
    gw, d = A.randn(g, 3, 2 * m, k, dtype=t, std=k ** -0.5).cuda(), A.randn(g, n, m, dtype=t).cuda()
    out = _odd(torch.zeros(n, m, dtype=t, device="cuda"))
    sr.gated(_odd(x), _odd(gw), off.cuda(), out=out)
    pair = sr.gated_grad(_odd(d), _odd(x), _odd(gw), off.cuda())
    A.check(out, *A.gated(x, gw, off, "silu"), "gated")
    A.check(pair, *A.gated(x, gw, off, "silu", grad=d), "gated_grad")


def test_norm_past_4_gib():
    n, k = 600_000, 4096  # 4.9 GB
    x = torch.empty(n, k, dtype=torch.bfloat16, device="cuda")
    step = 50_000
    for i in range(0, n, step):
        x[i:i + step] = torch.randn(step, k, device="cuda") + i / n
    w = torch.rand(k, device="cuda") + 0.5
    A.say("norm of 4.9 GB")
    out = sr.norm(x, w)
    dx, dw, db = sr.norm_grad(x, x, w, want_bias=True)
    torch.cuda.synchronize()
    at = torch.tensor([0, 1, 262_143, 262_144, 524_287, 524_288, 524_289, n - 1], device="cuda")
    ref, err, *_ = A.norm(x[at], w, None, 1e-5, True)
    A.check(out[at], ref, err, "out")
    refs, errs = A.norm_grad(x[at], x[at], w, 1e-5, True)
    A.check(dx[at], refs[0], errs[0], "dx")
    total = sum(x[i:i + step].double().sum(0) for i in range(0, n, step))
    size = sum(x[i:i + step].double().abs().sum(0) for i in range(0, n, step))
    # each of 512 workgroups adds its rows one by one, then they are added
    assert ((db.double() - total).abs() <= (n / 512 + 600) * A.U * size).all()


def test_vocabulary_past_4_gib():
    n, k, v = 40, 8192, 300_000  # 4.9 GB of weights
    w = torch.empty(v, k, dtype=torch.bfloat16, device="cuda")
    for i in range(0, v, 50_000):
        w[i:i + 50_000] = torch.randn(50_000, k, device="cuda") * 2 * k ** -0.5
    x = torch.randn(n, k, device="cuda").to(torch.bfloat16)
    target = torch.randint(0, v, (n,), device="cuda")
    target[:4] = torch.tensor([0, 262_143, 262_144, v - 1])
    grad = torch.rand(n, device="cuda")
    A.say("vocabulary of 4.9 GB")
    loss, lse, picked = sr.cross_entropy(x, w, target)
    dx, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked)
    torch.cuda.synchronize()
    z = torch.cat([x.double() @ w[i:i + 50_000].double().t() for i in range(0, v, 50_000)], 1)
    ref = torch.logsumexp(z, 1)
    # logits: k terms; their largest error, and 32-bit arithmetic on numbers up to 30
    ez = (k + 8) * 2 * A.U * 2 * k ** 0.5
    assert ((lse.double() - ref).abs() <= ez + 300 * A.U).all()
    assert ((loss.double() - (ref - z.gather(1, target[:, None])[:, 0])).abs() <= 2 * ez + 600 * A.U).all()
    dz = (z - ref[:, None]).exp_()
    dz[torch.arange(n, device="cuda"), target] -= 1
    dz *= grad.double()[:, None]
    at = torch.tensor([0, 1, 262_143, 262_144, 262_145, v - 1], device="cuda")
    size = (dz[:, at].abs().t() @ x.double().abs())
    # dz to bfloat16, the sum, its rounding; dz's own error is 2 ez relative to its share
    assert ((dw[at].double() - dz[:, at].t() @ x.double()).abs() <= (2.0 ** -8 * 2 + 3 * ez) * size + 1e-30).all()
    want = sum(dz[:, i:i + 50_000] @ w[i:i + 50_000].double() for i in range(0, v, 50_000))
    size = sum(dz[:, i:i + 50_000].abs() @ w[i:i + 50_000].double().abs() for i in range(0, v, 50_000))
    assert ((dx.double() - want).abs() <= (2.0 ** -8 * 2 + 3 * ez) * size).all()


def test_gated_weights_past_4_gib():
    s, m, k = 40, 4096, 8192  # 5.4 GB
    w = torch.empty(s, 2 * m, k, dtype=torch.bfloat16, device="cuda")
    for i in range(s):
        w[i] = torch.randn(2 * m, k, device="cuda") * k ** -0.5
    off = torch.arange(0, 3 * s + 1, 3, device="cuda")
    x, d = torch.randn(3 * s, k, device="cuda").to(torch.bfloat16), torch.randn(3 * s, m, device="cuda").to(torch.bfloat16)
    A.say("gated weights of 5.4 GB")
    out, pair = sr.gated(x, w, off), sr.gated_grad(d, x, w, off)
    torch.cuda.synchronize()
    for i in (0, 31, 32, s - 1):
        rows, o = slice(3 * i, 3 * i + 3), torch.tensor([0, 3])
        A.check(out[rows], *A.gated(x[rows], w[i:i + 1], o, "silu"), f"out {i}")
        A.check(pair[rows], *A.gated(x[rows], w[i:i + 1], o, "silu", grad=d[rows]), f"pair {i}")
