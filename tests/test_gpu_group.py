"""Rows grouped by an index (GPU only): exact against a stable sort."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

# (entries, groups, fanout): one launch, one digit pass, several passes; the borders between them
CASES = [(0, 10, 1), (1, 1, 1), (7, 3, 1), (10, 0, 1), (1000, 64, 8), (1024, 64, 2), (1025, 1023, 1), (8192, 1023, 8),
         (8193, 5, 1), (50000, 255, 4), (50000, 256, 1), (70001, 1023, 1), (70001, 1024, 1), (5, 100000, 1),
         (300000, 250000, 1), (12288, 1, 3), (20000, 2 ** 21, 1),
         (4096, 2047, 8), (4097, 2047, 1), (4000, 2048, 1), (65536, 64, 8), (65537, 64, 1), (65536, 2000, 1),
         (262144, 100, 4), (270000, 100, 2), (270000, 1500, 1), (30000, 2 ** 22 + 5, 1)]


@pytest.mark.parametrize("entries,groups,fanout", CASES)
@pytest.mark.parametrize("spread", ["uniform", "outside", "few"])
def test_group(entries, groups, fanout, spread):
    import segmented_reduction_amd as sr
    g = ru.gen(entries + groups)
    if spread == "uniform":
        index = torch.randint(0, max(groups, 1), (entries,), generator=g)
    elif spread == "outside":
        index = torch.randint(-groups // 8 - 2, groups + groups // 8 + 2, (entries,), generator=g)
        index[::7] = -2 ** 40
        index[3::11] = 2 ** 32 + 1
    else:  # long runs of equal entries, most groups empty
        index = (torch.arange(entries) // 97) % max(groups // 2, 1)
    if fanout > 1:
        index = index.view(-1, fanout)
    ru.say(f"group entries={entries} groups={groups} fanout={fanout} {spread}")
    got = sr.group(index.cuda(), groups)
    torch.cuda.synchronize()
    for a, b, name in zip(got, ru.group(index, groups), ("order", "position", "offsets")):
        assert torch.equal(a.cpu(), b), name


def test_group_feeds_reduce():
    """An unsorted edge list, grouped, summed by the segmented reduction."""
    import segmented_reduction_amd as sr
    g = ru.gen(3)
    index = torch.randint(0, 500, (20000,), generator=g)
    values = ru.randn(g, 20000, 8)
    ru.say("group then reduce")
    order, _, off = sr.group(index.cuda(), 500)
    out, _ = sr.reduce(values.cuda()[order], off, "sum")
    ref = torch.zeros(500, 8, dtype=torch.float64).index_add_(0, index, values.double())
    mag = torch.zeros(500, 8, dtype=torch.float64).index_add_(0, index, values.double().abs())
    ru.assert_close(out, ref, mag, 200, "sum")


def test_refusals():
    import segmented_reduction_amd as sr
    i = torch.zeros(6, dtype=torch.int64, device="cuda")
    for bad in (lambda: sr.group(i.cpu(), 3), lambda: sr.group(i.int(), 3), lambda: sr.group(i, -1),
                lambda: sr.group(i.view(1, 2, 3), 3), lambda: sr.group(i.view(2, 3).t(), 3)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(sr.SegredError) as e:
        sr.group(i, 2 ** 31)
    assert e.value.status == 2
