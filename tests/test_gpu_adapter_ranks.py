"""Adapters of very high rank (GPU only): more than 2^31 elements of the second
factor in the part that one workgroup copies to whole 16-byte units."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu


def test_second_factor_of_many_ranks():
    import segmented_reduction_amd as sr
    g = ru.gen(5)
    n, k, m, r = 130, 8, 520, 2 ** 22 + 4
    used = torch.tensor([0, 5, 31, 32, 2 ** 21 + 17, 2 ** 22 - 1, 2 ** 22 + 3])
    t = torch.bfloat16
    x, w = ru.randn(g, n, k, dtype=t), ru.randn(g, m, k, dtype=t)
    d, u = ru.randn(g, 1, len(used), k, dtype=t), ru.randn(g, 1, m, len(used), dtype=t)
    ru.say(f"adapter of rank {r}")
    down = torch.zeros(1, r, k, dtype=t, device="cuda")
    down[:, used.cuda()] = d.cuda()
    up = torch.zeros(1, m, r, dtype=t, device="cuda")
    up[:, :, used.cuda()] = u.cuda()
    off, which = torch.tensor([0, 7, n]), torch.tensor([-1, 0])
    out = sr.adapter(x.cuda(), w.cuda(), off.cuda(), which.cuda(), down, up)
    torch.cuda.synchronize()
    # the other ranks add zeros
    ref, mag, part, _, _ = ru.adapter(x, w, off, which, d, u)
    ru.assert_close(out, ref, mag, 2 * k + len(used), "out", more=2.0 ** -16 * part)
