"""Every kernel of the cross entropy and its gradient (GPU only) on inputs whose
logits are exact and whose results single entries of the vocabulary decide: those at
the ends of tiles and pieces, at the end of the vocabulary, past 4 GiB."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A
from tests import exact_logits as X

pytestmark = pytest.mark.gpu


def _check(x, w, target, probs, grad, scale, what, weights_dtype=None):
    A.say(what)
    x, w, target, probs, grad = (a.cuda() if a is not None else None for a in (x, w, target, probs, grad))
    loss, lse, picked = sr.cross_entropy(x, w, target, probs=probs, scale=scale)
    dx, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked, probs=probs, scale=scale, weights_dtype=weights_dtype)
    torch.cuda.synchronize()
    refs, errs, _ = X.forward(x, w, target, probs, scale)
    for name, got, ref, err in zip(("loss", "lse", "picked"), (loss, lse, picked), refs, errs):
        A.check(got, ref, err, f"{what} {name}")
    refs, errs = X.backward(x, w, target, probs, grad, scale)
    A.check(dx, refs[0], errs[0], f"{what} dx")
    A.check(dw, refs[1], errs[1], f"{what} dw")


# every tile of either direction, whole units and others
KERNELS = [("bf16", 5, 256, 3001), ("f16", 8, 512, 30011), ("f32", 5, 128, 9001), ("bf16", 10, 131, 3001), ("f16", 14, 65, 500),
           ("f16", 60, 131, 3001), ("bf16", 200, 257, 3001), ("f16", 40, 520, 2001), ("bf16", 300, 257, 5003),
           ("f32", 60, 128, 3001), ("f32", 300, 128, 5003), ("f32", 100, 65, 2001), ("f32", 300, 128, 9001), ("f32", 130, 100, 257),
           ("bf16", 100, 256, 33000), ("f16", 300, 256, 16500), ("bf16", 200, 520, 20001), ("f16", 300, 1030, 20001),
           ("bf16", 256, 2048, 30011), ("f16", 2304, 1024, 4100), ("bf16", 2100, 1030, 5003), ("f16", 701, 512, 9001),
           ("bf16", 64, 1024, 13000), ("f16", 250, 512, 25001)]


@pytest.mark.parametrize("t,n,k,v", KERNELS)
def test_kernels(t, n, k, v):
    """One target a row, then several with the leading entries of other rows."""
    few = len(X.entries(v)) // n + 1 if n < 16 else 1
    for i in range(few):  # few rows take the entries in turn
        x, w, target, probs, grad, scale, _ = X.case(A.TYPES[t], n, k, v, skip=i * n)
        _check(x, w, target, probs, grad, scale, f"entries {t} {n}x{k} vocab {v} from {i * n}")
    x, w, target, probs, grad, scale, _ = X.case(A.TYPES[t], n, k, v, picks=3, seed=1, skip=3)
    _check(x, w, target, probs, grad, scale, f"entries {t} {n}x{k} vocab {v} picks 3", weights_dtype=torch.float32)


@pytest.mark.parametrize("t,n,k,v", KERNELS)
def test_logits_far_below_zero(t, n, k, v):
    """A column behind the vocabulary's end, whose logit would be 0, would have all of it."""
    _check(*X.below_zero(A.TYPES[t], n, k, v), f"below zero {t} {n}x{k} vocab {v}")


@pytest.mark.parametrize("t,n,k,v", [("bf16", 16500, 64, 9001), ("f16", 16500, 72, 8193), ("f32", 9100, 64, 9000),
                                     ("bf16", 16400, 65, 8300), ("f16", 16389, 513, 8300)])
def test_pieces(t, n, k, v):
    """More than one piece of the vocabulary: rows enough for every entry to lead one."""
    x, w, target, probs, grad, scale, _ = X.case(A.TYPES[t], n, k, v)
    lead = torch.arange(n) * 7 % v
    assert lead.unique().numel() == v
    x = (2 * w[lead].float().sign()).to(A.TYPES[t])
    _check(x, w, target, probs, grad, scale, f"entries {t} {n}x{k} vocab {v} in pieces")


def test_entries_past_4_gib():
    """4.9 GB of weights: the rows' leading entries are on both sides of 4 GiB and of every tile's end there."""
    n, k, v, far = 40, 8192, 300_000, 262_144
    g = A.gen(3)
    w = torch.empty(v, k, dtype=torch.bfloat16, device="cuda")
    for i in range(0, v, 50_000):
        w[i:i + 50_000] = (torch.randint(-8, 9, (50_000, k), device="cuda") / 8).to(torch.bfloat16)
    first = [far - 1, far, far + 1, v - 1, v - 2, far + 63, far + 64, far + 127, far + 128, far + 255, far + 256, v // 64 * 64,
             v // 256 * 256, 0, 1, 131_071, 131_072]
    lead = torch.tensor(first + torch.randint(far, v, (n - len(first),), generator=g).tolist(), device="cuda")
    x = (2 * w[lead].float().sign()).to(torch.bfloat16)
    target = torch.randint(0, v, (n,), generator=g).cuda()
    target[:4] = torch.tensor([0, far - 1, far, v - 1], device="cuda")
    grad, scale = torch.rand(n, generator=g).cuda() + 0.5, 2.0 ** -7
    A.say("entries past 4 GiB")
    loss, lse, picked = sr.cross_entropy(x, w, target, scale=scale)
    dx, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked, scale=scale)
    torch.cuda.synchronize()
    parts = [slice(i, i + 50_000) for i in range(0, v, 50_000)]
    z = scale * torch.cat([x.double() @ w[p].double().t() for p in parts], 1)
    row, ref = torch.arange(n, device="cuda"), torch.logsumexp(z, 1)
    assert ((z[row, lead] - ref).exp() > 0.99).all()
    e_lse = (8 * (z.abs().max(1).values + 30) + 64 + v / 2048 + 4 * ref.abs()) * A.U
    assert float(e_lse.max()) < 1e-3  # a leading entry that is lost moves it by more than 4, one read twice by 0.69
    A.check(lse, ref, e_lse, "lse")
    at = z[row, target]
    A.check(picked, at, torch.zeros_like(at), "picked")
    A.check(loss, ref - at, e_lse + 6 * A.U * (ref.abs() + at.abs()), "loss")
    g = (grad.double() * scale)[:, None]
    p = (z - ref[:, None]).exp()
    goal = torch.zeros_like(z)
    goal[row, target] = 1
    dz = g * (p - goal)
    e = g * (p * (e_lse[:, None] + 8 * A.U * (z.abs() + ref[:, None].abs() + 4)) + 8 * A.U * (p + goal))
    e = e + 2.0 ** -8 * (dz.abs() + e)  # half a step of bfloat16
    size = dz.abs() + e
    some = torch.cat([lead, target, torch.tensor([2, far - 2, far + 2, far + 300], device="cuda")]).unique()
    err = e[:, some].t() @ x.double().abs() + (n + 8) * 2 * A.U * (size[:, some].t() @ x.double().abs())
    A.check(dw[some], dz[:, some].t() @ x.double(), err, "dw")
    want = sum(dz[:, q] @ w[q].double() for q in parts)
    err = sum(e[:, q] @ w[q].double().abs() + (v + 8) * 2 * A.U * (size[:, q] @ w[q].double().abs()) for q in parts)
    A.check(dx, want, err, "dx")
