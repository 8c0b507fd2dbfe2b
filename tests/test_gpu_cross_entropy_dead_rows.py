"""Rows without a target beside weights that are not finite (GPU only): they have no
gradient, whatever stands in the vocabulary."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k,v", [(1, 8, 5), (12, 128, 400), (15, 33, 300), (150, 128, 400), (300, 130, 2051), (701, 512, 9001),
                                   (2100, 1030, 4100)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_no_gradient_beside_infinite_weights(t, n, k, v, bad):
    g = A.gen(n)
    x, w = A.randn(g, n, k, dtype=A.TYPES[t]).cuda(), A.randn(g, v, k, dtype=A.TYPES[t]).cuda()
    w[v // 2, k // 3] = bad
    w[v - 1, 0] = bad
    target = torch.randint(0, v, (n, 2), generator=g).cuda()
    none = torch.arange(n, device="cuda") % 3 != 1
    target[none] = -100
    A.say(f"dead rows {t} {n}x{k} {v} {bad}")
    loss, lse, picked = sr.cross_entropy(x, w, target)
    dx, dw = sr.cross_entropy_grad(torch.ones(n, device="cuda"), x, w, target, lse, picked)
    torch.cuda.synchronize()
    assert (loss[none] == 0).all() and (picked[none] == 0).all()
    assert (dx[none] == 0).all(), f"{int((dx[none] != 0).any(1).sum())} of {int(none.sum())} rows without a target have a gradient"
    assert dx[~none].isnan().any(1).all()  # 0 times infinity, or NaN, as the formula has it
    none[:] = True
    target[:] = v
    loss, lse, picked = sr.cross_entropy(x, w, target)
    dx, dw = sr.cross_entropy_grad(torch.ones(n, device="cuda"), x, w, target, lse, picked)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
