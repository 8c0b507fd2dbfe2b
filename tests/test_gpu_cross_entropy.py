"""segred_cross_entropy and its gradient (GPU only) against 64-bit forms: every
kernel of the dispatch, odd vocabularies and widths, rows without a target, many
targets a row, several pieces of the vocabulary."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu


def _case(t, n, k, v, picks=1, seed=0, std=2.0, none=0.1):
    g = A.gen(seed + n + 7 * k + 13 * v)
    w = A.randn(g, v, k, dtype=A.TYPES[t], std=std * k ** -0.5)
    target = torch.randint(0, v, (n, picks), generator=g)
    x = (A.randn(g, n, k) + 0.5 * w[target[:, 0]].float()).to(A.TYPES[t])
    target = torch.where(torch.rand(n, picks, generator=g) < none, torch.randint(0, 2, (n, picks), generator=g) * (v + 100) - 100, target)
    probs = torch.rand(n, picks, generator=g) if picks > 1 else None
    if picks == 1:
        target = target.view(-1)
    grad = torch.randn(n, generator=g)
    return [a.cuda() if a is not None else None for a in (x, w, target.contiguous(), probs, grad)]


def _check(x, w, target, probs, grad, what, scale=1.0, weights_dtype=None):
    A.say(what)
    loss, lse, picked = sr.cross_entropy(x, w, target, probs=probs, scale=scale)
    torch.cuda.synchronize()
    refs, errs, _ = A.cross_entropy(x, w, target, probs, scale)
    for name, got, ref, err in zip(("loss", "lse", "picked"), (loss, lse, picked), refs, errs):
        assert got.dtype == torch.float32
        A.check(got, ref, err, f"{what} {name}")
    dx, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked, probs=probs, scale=scale, weights_dtype=weights_dtype)
    torch.cuda.synchronize()
    refs, errs = A.cross_entropy_grad(grad, x, w, target, x.dtype, probs, scale)
    assert dw.dtype == (weights_dtype or w.dtype)
    A.check(dx, refs[0], errs[0], f"{what} dx")
    A.check(dw, refs[1], errs[1], f"{what} dw")
    return loss, lse, picked, dx, dw


SHAPES = [(1, 64, 100), (1, 8, 1), (3, 1, 5), (7, 72, 257), (16, 256, 64), (17, 256, 65), (20, 100, 300), (33, 33, 1000),
          (64, 128, 128), (65, 320, 511), (130, 64, 129), (200, 264, 700)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k,v", SHAPES)
def test_shapes(t, n, k, v):
    for picks in (1, 3):
        _check(*_case(t, n, k, v, picks), f"cross entropy {t} {n}x{k} vocab {v} picks {picks}")


KERNELS = [("bf16", 100, 256, 33000), ("f16", 300, 256, 16500), ("bf16", 257, 512, 20001), ("f16", 8, 512, 30011),
           ("bf16", 300, 257, 5003), ("f32", 300, 128, 5003), ("f32", 5, 128, 9001), ("f32", 100, 65, 2001),
           ("bf16", 513, 64, 9000), ("f16", 30, 1024, 3000),
           ("bf16", 2100, 1030, 5003), ("f16", 300, 1030, 70001), ("bf16", 10, 131, 3001), ("f16", 2500, 2047, 4200),
           ("bf16", 5, 256, 3001), ("f16", 40, 520, 2001), ("bf16", 128, 128, 4099), ("f16", 300, 1032, 2051),
           ("bf16", 2100, 520, 5003), ("f16", 701, 512, 9001), ("bf16", 2051, 264, 8200), ("f16", 2304, 1024, 4100)]


@pytest.mark.parametrize("t,n,k,v", KERNELS)
def test_kernels(t, n, k, v):
    _check(*_case(t, n, k, v), f"cross entropy {t} {n}x{k} vocab {v}")
    _check(*_case(t, n, k, v, 20, seed=1), f"cross entropy {t} {n}x{k} vocab {v} picks 20", scale=0.5, weights_dtype=torch.float32)


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("n,k,v", [(3, 2048, 6200), (16, 1024, 13001), (64, 1024, 13000), (250, 512, 25001)])
def test_few_rows_and_many_weights(t, n, k, v):
    """The weights' gradient from operands in the other order."""
    _check(*_case(t, n, k, v), f"cross entropy {t} {n}x{k} vocab {v}")


@pytest.mark.parametrize("t", ["bf16", "f16"])
@pytest.mark.parametrize("n,k,v", [(1, 1, 1), (1, 31, 65), (7, 33, 200), (16, 95, 64), (16, 257, 1000), (10, 1711, 7143),
                                   (3, 130, 12289), (13, 2047, 40)])
def test_few_rows_that_are_no_whole_units(t, n, k, v):
    _check(*_case(t, n, k, v, none=0.0), f"cross entropy {t} {n}x{k} vocab {v}")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,picks", [(64, 16), (64, 17), (65, 2), (1, 1024), (1, 1025), (4096, 1), (4097, 1)])
def test_rows_prepared_by_one_workgroup_or_more(t, n, picks):
    _check(*_case(t, n, 72, 300, picks), f"cross entropy {t} {n}x72 vocab 300 picks {picks}")


@pytest.mark.parametrize("t,n,k,v", [("bf16", 16500, 64, 9001), ("f16", 16500, 72, 8193), ("f32", 8200, 40, 9000),
                                     ("bf16", 16400, 65, 8300), ("bf16", 16389, 512, 8300), ("f16", 16389, 513, 8300)])
def test_pieces(t, n, k, v):
    """More than one piece of the vocabulary (256 MiB hold less)."""
    _check(*_case(t, n, k, v), f"cross entropy {t} {n}x{k} vocab {v} in pieces")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n", [12, 150])
def test_rows_without_a_target(t, n):
    """Their loss is 0 and they leave no trace, whatever stands in them."""
    x, w, target, _, grad = _case(t, n, 128, 400, none=0.0)
    none = torch.arange(n, device="cuda") % 3 == 1
    target = torch.where(none, -100, target)
    clean = torch.where(none[:, None], 0, x)
    loss, lse, picked = sr.cross_entropy(clean, w, target)
    dx, dw = sr.cross_entropy_grad(grad, clean, w, target, lse, picked)
    assert (loss[none] == 0).all() and (picked[none] == 0).all() and (dx[none] == 0).all()
    dirty = x.clone()
    dirty[none] = float("nan")
    dirty[1] = float("inf")
    loss2, lse2, picked2 = sr.cross_entropy(dirty, w, target)
    dx2, dw2 = sr.cross_entropy_grad(grad, dirty, w, target, lse2, picked2)
    if t == "f32":
        # Products in bf16 parts that meet a NaN are formed again as float products, which round
        # otherwise; either is within the bounds of the formula, to which no dead row contributes.
        refs, errs, _ = A.cross_entropy(clean, w, target)
        A.check(loss2, refs[0], errs[0], "loss beside NaN")
        refs, errs = A.cross_entropy_grad(grad, clean, w, target, x.dtype)
        A.check(dx2, refs[0], errs[0], "dx beside NaN")
        A.check(dw2, refs[1], errs[1], "dw beside NaN")
    else:
        assert torch.equal(loss, loss2) and torch.equal(dx, dx2) and torch.equal(dw, dw2)
    nothing = torch.full_like(target, -1)
    loss, lse, picked = sr.cross_entropy(dirty, w, nothing)
    dx, dw = sr.cross_entropy_grad(grad, dirty, w, nothing, lse, picked)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()


@pytest.mark.parametrize("t", ["bf16", "f16"])
def test_rows_without_a_target_among_many(t):
    x, w, target, _, grad = _case(t, 2100, 512, 4100, none=0.0)
    none = torch.arange(2100, device="cuda") % 3 == 1
    target = torch.where(none, -100, target)
    clean = _check(torch.where(none[:, None], 0, x), w, target, None, grad, f"cross entropy {t} 2100 rows, a third padding")
    x[none] = float("nan")
    loss, lse, picked = sr.cross_entropy(x, w, target)
    dx, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked)
    assert torch.equal(loss, clean[0]) and torch.equal(dx, clean[3]) and torch.equal(dw, clean[4])


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_a_bad_row_stays_alone(t):
    x, w, target, _, grad = _case(t, 100, 128, 700, none=0.0)
    loss, lse, picked = sr.cross_entropy(x, w, target)
    dx, _ = sr.cross_entropy_grad(grad, x, w, target, lse, picked)
    bad = x.clone()
    bad[40, 3] = float("nan")
    loss2, lse2, picked2 = sr.cross_entropy(bad, w, target)
    dx2, _ = sr.cross_entropy_grad(grad, bad, w, target, lse2, picked2)
    good = torch.arange(100, device="cuda") != 40
    assert loss2[40].isnan() and dx2[40].isnan().all()
    assert (loss2[good] - loss[good]).abs().max() < 1e-4 and (dx2[good] - dx[good]).abs().max() <= 2 ** -7 * dx.abs().max()


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_the_same_target_twice(t):
    x, w, target, probs, grad = _case(t, 50, 64, 300, 4, none=0.0)
    target[:, 2] = target[:, 0]
    target[:, 3] = target[:, 1]
    _check(x, w, target, probs, grad, f"cross entropy {t}, targets named twice")
    same = sr.cross_entropy(x, w, target[:, :2].contiguous(), probs=(probs[:, :2] + probs[:, 2:]).contiguous())
    assert (same[0] - sr.cross_entropy(x, w, target, probs=probs)[0]).abs().max() < 1e-4


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
def test_large_logits(t):
    """Logits in the hundreds: the sum is taken around the largest."""
    _check(*_case(t, 70, 64, 500, std=60.0), f"cross entropy {t} large logits")


@pytest.mark.parametrize("n", [40, 300])
def test_small_and_uneven_gradients_in_float16(n):
    """Gradients far below float16's smallest numbers, of rows that differ by 2^12."""
    x, w, target, _, grad = _case("f16", n, 256, 2000, none=0.0)
    grad = grad * torch.exp2(-(torch.arange(n, device="cuda") % 13).float()) * 2.0 ** -12
    _check(x, w, target, None, grad, "cross entropy f16, small gradients", weights_dtype=torch.float32)


@pytest.mark.parametrize("size", [2.0 ** -140, 2.0 ** -60, 2.0 ** 100, 2.0 ** 125])
def test_gradients_of_any_size_in_float16(size):
    """The common power of two brings them into float16's range; the weights' gradient leaves in float32."""
    x, w, target, _, grad = _case("f16", 50, 64, 300, none=0.0)
    # few and small values, so that their sums stay in float32's range
    x, w = (x.float() * 2.0 ** -6).half(), (w.float() * 2.0 ** -4).half()
    sign = grad.sign()
    grad = (sign.cpu() * size).cuda()  # made on the host, which keeps the smallest numbers
    _, lse, picked = sr.cross_entropy(x, w, target)
    _, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked, weights_dtype=torch.float32)
    one = sr.cross_entropy_grad(sign, x, w, target, lse, picked, weights_dtype=torch.float32)[1].cpu().double()
    # the same but for the power of two: exact, down to float32's own smallest step and, where the
    # power would pass 2^126, half of float16's, 2^-25 2^-126 for each slope
    more = 2.0 ** -151 * float(x.abs().float().sum(0).max()) if size < 2.0 ** -113 else 0.0
    assert ((dw.cpu().double() - one * size).abs() <= 2.0 ** -23 * one.abs() * size + 2.0 ** -149 + more).all()


@pytest.mark.parametrize("t,n,picks", [("bf16", 9, 700), ("f32", 40, 130), ("f16", 300, 4096)])
def test_many_targets(t, n, picks):
    """Up to 4,096 a row, many of them named again and again."""
    _check(*_case(t, n, 64, 900, picks), f"cross entropy {t}, {picks} targets a row")


@pytest.mark.parametrize("t", ["f32", "bf16"])
def test_one_target_of_any_probability(t):
    x, w, target, _, grad = _case(t, 60, 64, 200)
    probs = torch.linspace(-1, 3, 60, device="cuda")
    one = _check(x, w, target, probs, grad, f"cross entropy {t}, one target of any probability")
    two = _check(x, w, target[:, None].contiguous(), probs[:, None].contiguous(), grad, "the same in two dimensions")
    assert two[2].shape == (60, 1) and all(torch.equal(a, b.view(a.shape)) for a, b in zip(one, two))


def test_logits_of_minus_infinity():
    """An entry of the vocabulary that is impossible takes no part."""
    g = A.gen(2)
    x, w = torch.rand(30, 64, generator=g).cuda() + 0.5, torch.randn(200, 64, generator=g).cuda()
    target = torch.randint(0, 100, (30,), generator=g).cuda()
    w[150:, 0] = float("-inf")
    loss, lse, _ = sr.cross_entropy(x, w, target)
    ref = sr.cross_entropy(x, w[:150].contiguous(), target)
    assert (lse - ref[1]).abs().max() < 1e-5 and (loss - ref[0]).abs().max() < 1e-5


def test_parts_of_the_gradient():
    x, w, target, probs, grad = _case("bf16", 90, 128, 900)
    _, lse, picked = sr.cross_entropy(x, w, target)
    dx, dw = sr.cross_entropy_grad(grad, x, w, target, lse, picked)
    assert torch.equal(sr.cross_entropy_grad(grad, x, w, target, lse, picked, want_weights=False)[0], dx)
    only = sr.cross_entropy_grad(grad, x, w, target, lse, picked, want_values=False)
    assert only[0] is None and torch.equal(only[1], dw)


def test_no_rows():
    x, w = torch.empty(0, 16, device="cuda", dtype=torch.bfloat16), torch.ones(40, 16, device="cuda", dtype=torch.bfloat16)
    e, t = torch.empty(0, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse, picked = sr.cross_entropy(x, w, t)
    assert loss.shape == lse.shape == picked.shape == (0,)
    dx, dw = sr.cross_entropy_grad(e, x, w, t, lse, picked)
    assert dx.shape == (0, 16) and (dw == 0).all()


def test_results_repeat_bit_for_bit():
    x, w, target, probs, grad = _case("bf16", 300, 512, 20000, 3)
    def once():
        loss, lse, picked = sr.cross_entropy(x, w, target, probs=probs)
        return (loss, lse, picked, *sr.cross_entropy_grad(grad, x, w, target, lse, picked, probs=probs))
    one = once()
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(one, once()))


def test_refusals():
    x, w, target, probs, grad = _case("bf16", 6, 16, 40, 2)
    for bad in (dict(values=x.cpu()), dict(weights=w[:, :8].contiguous()), dict(weights=w[0]), dict(target=target[:5]),
                dict(target=target.int()), dict(target=target.cpu()), dict(probs=probs[:, :1]), dict(probs=probs.double()),
                dict(target=target[:, :0])):
        with pytest.raises(ValueError):
            sr.cross_entropy(**{"values": x, "weights": w, "target": target, "probs": probs, **bad})
    with pytest.raises(TypeError):
        sr.cross_entropy(x, w.float(), target)
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(sr.SegredError):
            sr.cross_entropy(x, w, target, scale=scale)
    _, lse, picked = sr.cross_entropy(x, w, target, probs=probs)
    for bad in (dict(grad=grad[:5]), dict(lse=lse.double()), dict(picked=picked.view(-1))):
        with pytest.raises(ValueError):
            sr.cross_entropy_grad(**{"grad": grad, "values": x, "weights": w, "target": target, "lse": lse, "picked": picked,
                                     "probs": probs, **bad})
    with pytest.raises(TypeError):
        sr.cross_entropy_grad(grad, x, w, target, lse, picked, probs=probs, weights_dtype=torch.float16)
