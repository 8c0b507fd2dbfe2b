"""Float products in bf16 parts keep float's bits (GPU only): rows with one
element that is not zero, so that a sum is a single product.  What is left out of
it is below 2^-22; without the third parts it would be up to 2^-17."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


def single(g, n, k):
    x = torch.zeros(n, k)
    x[torch.arange(n), torch.randint(0, k, (n,), generator=g)] = torch.randn(n, generator=g)
    return x


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k,m", [(256, 512), (131, 333)])
def test_matmul(transpose, k, m):
    g = ru.gen(k)
    off = ru.offsets([1500, 0, 700, 1200, 1300])
    assert (int(off[-1]) // 64 + 2) * ((m + 127) // 128) >= 224  # tiles of the kernel in parts
    x, w = single(g, int(off[-1]), k), ru.randn(g, 5, k, m)
    ref, mag = ru.matmul(x, w, off)
    ru.say(f"bits of matmul k={k} m={m} transpose={transpose}")
    given = w.transpose(1, 2).contiguous() if transpose else w
    got = sr().matmul(x.cuda(), given.cuda(), off.cuda(), transpose=transpose).cpu().double()
    # and one rounding to float32
    assert bool(((got - ref).abs() <= (2.0 ** -22 + 2.0 ** -24) * mag + 2.0 ** -125).all())


@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("k,m", [(640, 648), (643, 645)])
def test_adapter(transpose, k, m):
    """Rank 1: a product beside another, whose first factor is a rounded product
    (2^-24), rounded again by its scale; both off by 2^-22 and their sum rounded."""
    g = ru.gen(m)
    off, which = ru.offsets([700, 1, 1300, 0, 1500, 1600]), torch.tensor([0, 1, -1, 0, 1, 0])
    have = m if transpose else k
    x, w = single(g, 5101, have), ru.randn(g, m, k)
    down, up, scale = ru.randn(g, 2, 1, k), ru.randn(g, 2, m, 1), torch.rand(2, generator=g) + 0.5
    ref, mag, _, _, _ = ru.adapter(x, w, off, which, down, up, scale, transpose)
    ru.say(f"bits of adapter k={k} m={m} transpose={transpose}")
    got = sr().adapter(*(v.cuda() for v in (x, w, off, which, down, up)), scale=scale.cuda(), transpose=transpose)
    bound = (2.0 ** -22 + 4 * 2.0 ** -24) * mag + 2.0 ** -124
    assert bool(((got.cpu().double() - ref).abs() <= bound).all())
