"""segred_norm and its gradient (GPU only) against 64-bit forms: widths on both
sides of every kernel's limit, odd ones, rows that no kernel holds in registers,
parameters in either type or none, rows of other strides than whole units."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu

WIDTHS = [1, 2, 7, 8, 9, 64, 127, 128, 129, 333, 512, 513, 1000, 1024, 1026, 2047, 2048, 2049, 4096, 4100, 8192, 8200,
          16384, 16389, 20001]


def _case(t, k, n, center, params, bias, seed, level=0.3):
    g = A.gen(seed)
    x = (A.randn(g, n, k) * (torch.rand(n, 1, generator=g) * 3 + 0.1) + level * torch.randn(n, 1, generator=g)).to(A.TYPES[t])
    w = (A.randn(g, k, std=0.3) + 1).to(A.TYPES[params]) if params else None
    b = A.randn(g, k, std=0.3).to(A.TYPES[params]) if params and bias else None
    return x.cuda(), w.cuda() if params else None, b.cuda() if b is not None else None, A.randn(g, n, k, dtype=A.TYPES[t]).cuda()


def _check(x, w, b, g, center, eps, what, want_bias=True):
    A.say(what)
    out = sr.norm(x, w, b, eps=eps, center=center)
    torch.cuda.synchronize()
    ref, err, *_ = A.norm(x, w, b, eps, center)
    A.check(out, ref, err, f"{what} out")
    dx, dw, db = sr.norm_grad(g, x, w, eps=eps, center=center, want_bias=want_bias)
    torch.cuda.synchronize()
    refs, errs = A.norm_grad(g, x, w, eps, center)
    A.check(dx, refs[0], errs[0], f"{what} dx")
    assert (dw is None) == (w is None)
    if dw is not None:
        assert dw.dtype == w.dtype
        A.check(dw, refs[1], errs[1], f"{what} dw")
    if want_bias:
        assert db.dtype == (w.dtype if w is not None else x.dtype)
        A.check(db, refs[2], errs[2], f"{what} db")


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("k", WIDTHS)
def test_widths(t, k):
    for i, (center, params, bias) in enumerate(((True, t, True), (False, "f32", False), (True, None, False))):
        n = (5, 67, 1)[i]
        _check(*_case(t, k, n, center, params, bias, k + i), center, 1e-5, f"norm {t} {n}x{k} center={center} params={params}")


@pytest.mark.parametrize("t,n,k", [("bf16", 9001, 96), ("f32", 3001, 130), ("f16", 2500, 1024), ("bf16", 1100, 4096),
                                   ("f32", 600, 17000), ("bf16", 4099, 2048)])
def test_many_rows(t, n, k):
    """More rows than workgroups: each walks several, and their sums are joined."""
    _check(*_case(t, k, n, True, "f32", True, n), True, 1e-5, f"norm {t} {n}x{k}")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("k,n", [(100, 16), (96, 32), (100, 33), (512, 5), (512, 8), (1000, 9), (2048, 4), (2048, 8),
                                 (2040, 9), (4096, 2), (4095, 3), (8192, 2), (16384, 2), (16384, 3), (17000, 1)])
def test_few_rows(t, k, n):
    """One workgroup leaves the parameters' gradients itself, two or more have them joined."""
    _check(*_case(t, k, n, True, t, True, n), True, 1e-5, f"norm {t} {n}x{k}")


@pytest.mark.parametrize("t", ["f32", "bf16"])
@pytest.mark.parametrize("k", [96, 1024, 4096, 17000])
def test_a_mean_far_from_zero(t, k):
    """The squares are taken around the mean, not subtracted from its square."""
    x, w, b, g = _case(t, k, 9, True, t, True, 5, level=0.0)
    x = (x.float() + 300).to(x.dtype)
    _check(x, w, b, g, True, 1e-5, f"norm {t} k={k} mean 300")


@pytest.mark.parametrize("k", [7, 100, 520, 3000, 5000])
def test_rows_that_begin_anywhere(k):
    """Tensors that begin one element behind a 16-byte boundary."""
    for t in ("bf16", "f32"):
        x, w, b, g = _case(t, k, 6, True, t, True, k)
        off = [torch.empty(v.numel() + 1, dtype=v.dtype, device="cuda")[1:].view(v.shape).copy_(v) for v in (x, w, b, g)]
        for center in (True, False):
            _check(*off, center, 1e-6, f"norm {t} k={k} from odd places")


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    assert sr.norm(x).shape == (0, 64)
    w = torch.ones(64, device="cuda")
    dx, dw, db = sr.norm_grad(x, x, w, want_bias=True)
    assert dx.shape == (0, 64) and (dw == 0).all() and (db == 0).all()


def test_in_place_and_out():
    x, w, b, g = _case("bf16", 1500, 33, True, "bf16", True, 1)
    want = sr.norm(x, w, b)
    y = x.clone()
    assert sr.norm(y, w, b, out=y) is y and torch.equal(y, want)
    x, w, b, g = _case("f32", 17000, 3, True, "f32", True, 1)
    want = sr.norm(x, w, b)
    assert torch.equal(sr.norm(x, w, b, out=x), want)


@pytest.mark.parametrize("k", [40, 700, 3000, 9000, 17000])
def test_bad_rows_stay_alone(k):
    """An infinity or a NaN of a row, or a constant row with eps = 0, reaches no other row."""
    x, w, b, g = _case("f32", k, 12, True, "f32", True, 3)
    ref, refg = sr.norm(x, w, b), sr.norm_grad(g, x, w)[0]
    bad = x.clone()
    bad[3, k // 2], bad[7, 0], bad[9] = float("nan"), float("inf"), 2.0
    good = torch.tensor([i not in (3, 7, 9) for i in range(12)], device="cuda")
    out, dx = sr.norm(bad, w, b), sr.norm_grad(g, bad, w)[0]
    assert torch.equal(out[good], ref[good]) and torch.equal(dx[good], refg[good])
    assert out[3].isnan().all() and out[7].isnan().any()
    assert torch.equal(out[9], b)  # 0 / sqrt(eps)
    assert sr.norm(bad, w, b, eps=0.0)[9].isnan().all()


def test_sums_repeat_bit_for_bit():
    x, w, b, g = _case("bf16", 2048, 3000, True, "f32", True, 8)
    one = sr.norm_grad(g, x, w, want_bias=True)
    for _ in range(3):
        two = sr.norm_grad(g, x, w, want_bias=True)
        assert all(torch.equal(p, q) for p, q in zip(one, two))


def test_parameters_that_are_not_asked_for():
    x, w, b, g = _case("f16", 300, 50, True, "f16", True, 2)
    full = sr.norm_grad(g, x, w, want_bias=True)
    dx, dw, db = sr.norm_grad(g, x, w, want_weight=False)
    assert dw is None and db is None and torch.equal(dx, full[0])
    dx, dw, db = sr.norm_grad(g, x, w, want_weight=False, want_bias=True)
    assert dw is None and torch.equal(db, full[2])
    _, dw, db = sr.norm_grad(g, x, want_weight=True, want_bias=True, dtype=torch.float32)
    refs, errs = A.norm_grad(g, x, None, 1e-5, True)
    assert dw.dtype == db.dtype == torch.float32
    A.check(dw, refs[1], errs[1], "dw without a weight")
    A.check(db, refs[2], errs[2], "db without a weight")


def test_refusals():
    x = torch.zeros(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    for bad in (dict(values=x.cpu()), dict(values=x.t()), dict(values=x[0]), dict(weight=w[:7]), dict(weight=w.cpu()),
                dict(bias=torch.ones(9, device="cuda")), dict(out=torch.empty(4, 7, device="cuda")),
                dict(out=torch.empty(4, 8, device="cuda", dtype=torch.float16))):
        with pytest.raises(ValueError):
            sr.norm(**{"values": x, "weight": w, **bad})
    for bad in (dict(values=x.double()), dict(weight=w.half()), dict(bias=w.half())):
        with pytest.raises(TypeError):
            sr.norm(**{"values": x, "weight": w, **bad})
    for eps in (-1e-5, float("nan"), float("inf")):
        with pytest.raises(sr.SegredError):
            sr.norm(x, eps=eps)
        with pytest.raises(sr.SegredError):
            sr.norm_grad(x, x, eps=eps)
    with pytest.raises(ValueError):
        sr.norm_grad(x[:3], x)
    with pytest.raises(TypeError):
        sr.norm_grad(x, x, w, dtype=torch.float16)
