"""Products of many rows per segment in 16-bit types (GPU only): sizes at which
the tiles of 128 or 256 rows by 256 columns are taken, for which segments hold
64 rows on average, K >= 256, M > 128 and there are 1,536 tiles of 64 x 128."""
import pytest
import torch

from tests import ragged_util as ru

pytestmark = pytest.mark.gpu

# Ends inside tiles of 128 and of 256, halves of them, whole ones, none and single rows.
LENGTHS = [700, 0, 128, 1, 256, 1500, 129, 2900, 64, 255, 257, 0, 90, 3000, 384, 513, 127, 1100, 640, 1000]


def sr():
    import segmented_reduction_amd
    return segmented_reduction_amd


# 5 column tiles of 256 take tiles of 128 rows in either orientation; 8 take 256 rows where the weights are transposed
@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("k", [256, 264, 328, 512])
@pytest.mark.parametrize("m", [1032, 2048, 2000])
@pytest.mark.parametrize("gathered", [False, True])
def test_large_tiles(kind, k, m, gathered):
    t, g = ru.TYPES[kind], ru.gen(k + m)
    off = ru.offsets(LENGTHS, base=3)
    n, s = int(off[-1]) + 4, len(LENGTHS)
    assert (n // 64 + s // 2) * ((m + 127) // 128) >= 1536 and n // s >= 64
    pool = 4000 if gathered else n
    x, w = ru.randn(g, pool, k, dtype=t).cuda(), ru.randn(g, s, k, m, dtype=t).cuda()
    rows = torch.randint(0, pool, (n,), generator=g)
    rows[::97], rows[5::101], rows[7::211] = -1, pool, 2 ** 40
    rows = rows.cuda() if gathered else None
    ref, mag = ru.matmul(x, w, off, rows=rows, fill=7.0)
    ref, mag = ref.cpu(), mag.cpu()
    for transpose in (False, True):
        given = w.transpose(1, 2).contiguous() if transpose else w
        ru.say(f"matmul in phases {kind} k={k} m={m} transpose={transpose} gathered={gathered}")
        out = torch.full((n, m), 7.0, dtype=t, device="cuda")
        sr().matmul(x, given, off.cuda(), transpose=transpose, rows=rows, out=out)
        again = torch.full((n, m), 7.0, dtype=t, device="cuda")
        sr().matmul(x, given, off.cuda(), transpose=transpose, rows=rows, out=again)
        torch.cuda.synchronize()
        ru.assert_close(out, ref, mag, k, "matmul")
        assert torch.equal(out, again)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("m", [1032, 2048])
def test_infinity_and_nan_of_a_row_stay_in_it(kind, m):
    """Also in rows before the first segment and behind the last, which take no part."""
    t, g, k = ru.TYPES[kind], ru.gen(m), 264
    off = ru.offsets(LENGTHS, base=2)
    n, s = int(off[-1]) + 3, len(LENGTHS)
    x, w = ru.randn(g, n, k, dtype=t), ru.randn(g, s, k, m, dtype=t)
    bad = [2, 900, 5000, int(off[-1]) - 1]
    x[:2], x[-3:] = float("nan"), float("inf")
    x[bad[0], 0], x[bad[1], 263], x[bad[2], 70], x[bad[3], 5] = float("nan"), float("inf"), float("nan"), -float("inf")
    for transpose in (False, True):
        given = w.transpose(1, 2).contiguous() if transpose else w
        ru.say(f"specials in phases {kind} m={m} transpose={transpose}")
        out = torch.full((n, m), 7.0, dtype=t, device="cuda")
        got = sr().matmul(x.cuda(), given.cuda(), off.cuda(), transpose=transpose, out=out).cpu()
        assert (got[:2] == 7).all() and (got[-3:] == 7).all()
        wrong = ~torch.isfinite(got)
        assert wrong[bad].all()
        wrong[bad] = False
        assert not wrong.any()


@pytest.mark.parametrize("m", [1032, 2048])
def test_replayed(m):
    """Captured and replayed with other rows each time, eager calls between."""
    g, k = ru.gen(m), 328
    off = ru.offsets(LENGTHS).cuda()
    n, s = int(off[-1]), len(LENGTHS)
    x, w = ru.randn(g, 3000, k, dtype=torch.bfloat16).cuda(), ru.randn(g, s, m, k, dtype=torch.bfloat16).cuda()
    rows = torch.zeros(n, dtype=torch.int64, device="cuda")
    ru.say(f"matmul in phases, replayed m={m}")
    call = lambda: sr().matmul(x, w, off, transpose=True, rows=rows)  # noqa: E731
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out = call()
    for rep in range(4):
        rows.copy_(torch.randint(-2, 3002, (n,), generator=g))
        out.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, call()), rep
        torch.cuda.synchronize()
