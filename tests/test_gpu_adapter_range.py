"""Low-rank rows of bfloat16 adapters next to float's largest value (GPU only)."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows", [3, 200])
@pytest.mark.parametrize("sign", [1, -1])
def test_low_rank_rows_above_the_largest_bfloat16(rows, sign):
    """Finite in float32, and nearer to 2^128 than to the largest bfloat16: the
    row is (2 - 2^-7) 2^127 + 1.5 2^119, the result that times 2^-120, 255.75."""
    import segmented_reduction_amd as sr
    t = torch.bfloat16
    x = torch.zeros(rows, 64, dtype=t)
    x[1, 0], x[1, 9] = sign * (2 - 2.0 ** -7) * 2.0 ** 127, sign * 1.5 * 2.0 ** 119
    assert torch.isfinite(x).all()
    w = torch.zeros(96, 64, dtype=t)
    down, up = torch.ones(1, 8, 64, dtype=t), torch.zeros(1, 96, 8, dtype=t)
    up[0, :, 3] = 2.0 ** -120
    ru.say(f"adapter next to float's end rows={rows}")
    args = (w.cuda(), torch.tensor([0, rows]).cuda(), torch.tensor([0]).cuda(), down.cuda(), up.cuda())
    out, low = sr.adapter(x.cuda(), *args, want_low=torch.float32)
    out, low = out.cpu(), low.cpu()
    assert bool((low[1].double() == sign * 255.75 * 2.0 ** 120).all())
    assert bool((out[1] == sign * 256).all())  # rounded to 8 bits
    out[1] = 0
    assert not out.any()
    x[1, 9], x[2, 3] = float("inf"), float("nan")
    out = sr.adapter(x.cuda(), *args).cpu()
    assert not torch.isfinite(out[1:3]).any() and not out[0].any()
