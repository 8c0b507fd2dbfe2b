"""Refusals of the operators over ragged groups of rows, on the host before
any device work, and the sizes of their workspaces."""
import os

import pytest

FAKE = 0x10000  # a non-null, aligned host value; never dereferenced


def _lib():
    import segmented_reduction_amd as sr
    if not os.path.exists(sr.LIB_PATH):
        from segmented_reduction_amd import build_lib
        build_lib.build()
    return sr.library()


def _args(defaults, kw):
    assert set(kw) <= set(defaults)
    return tuple({**defaults, **kw}.values())


def _mm(**kw):
    return _args(dict(values=FAKE, dtype=3, k=64, rows=None, value_rows=10, weights=FAKE, transpose=0, m=32,
                      offsets=FAKE, S=2, N=10, out=FAKE), kw)


@pytest.mark.parametrize("args,expect", [
    (_mm(dtype=5), 1), (_mm(dtype=-1), 1), (_mm(dtype=0), 2), (_mm(dtype=1), 2), (_mm(k=0), 1), (_mm(m=0), 1),
    (_mm(k=2 ** 24 + 1), 2), (_mm(m=2 ** 24 + 1), 2), (_mm(value_rows=-1), 1), (_mm(S=-1), 1), (_mm(N=-1), 1),
    (_mm(value_rows=9), 1), (_mm(values=None), 1), (_mm(weights=None), 1), (_mm(offsets=None), 1), (_mm(out=None), 1),
    (_mm(values=FAKE + 1), 1), (_mm(weights=FAKE + 1), 1), (_mm(out=FAKE + 1), 1), (_mm(dtype=2, out=FAKE + 2), 1),
    (_mm(offsets=FAKE + 4), 1), (_mm(rows=FAKE + 4), 1), (_mm(value_rows=2 ** 60), 1), (_mm(S=2 ** 60), 1),
    (_mm(rows=FAKE, N=2 ** 60), 1), (_mm(rows=FAKE, N=2 ** 44, m=2 ** 14), 2),
    (_mm(S=0, offsets=None, weights=None, out=None), 0), (_mm(N=0, values=None, value_rows=0, out=None), 0),
])
def test_matmul_argument_checks(args, expect):
    assert _lib().segred_matmul(*args, None) == expect


def _outer(**kw):
    return _args(dict(left=FAKE, left_rows=None, left_count=10, k=64, right=FAKE, right_rows=None, right_count=10, m=32,
                      dtype=4, offsets=FAKE, S=2, N=10, out=FAKE, out_dtype=4, work=None, bytes=0), kw)


@pytest.mark.parametrize("args,expect", [
    (_outer(dtype=5), 1), (_outer(dtype=0), 2), (_outer(k=0), 1), (_outer(m=0), 1), (_outer(k=2 ** 24 + 1), 2),
    (_outer(left_count=-1), 1), (_outer(left_count=9), 1), (_outer(right_count=9), 1), (_outer(S=-1), 1),
    (_outer(N=-1), 1), (_outer(left=None), 1), (_outer(right=None), 1), (_outer(offsets=None), 1),
    (_outer(out=None), 1), (_outer(out_dtype=3), 1), (_outer(out_dtype=0), 1), (_outer(left=FAKE + 1), 1),
    (_outer(out_dtype=2, out=FAKE + 2), 1), (_outer(left_rows=FAKE + 4), 1), (_outer(offsets=FAKE + 4), 1),
    (_outer(left_count=2 ** 60), 1), (_outer(S=2 ** 60), 1),
    (_outer(left_count=100000, right_count=100000, N=100000), 1),                                # no workspace
    (_outer(left_count=100000, right_count=100000, N=100000, work=FAKE, bytes=1000), 1),         # too small
    (_outer(left_count=100000, right_count=100000, N=100000, work=FAKE + 8, bytes=2 ** 40), 1),  # misaligned
    (_outer(S=0, left=None, right=None, offsets=None, out=None), 0),
])
def test_outer_argument_checks(args, expect):
    assert _lib().segred_outer(*args, None) == expect


def _group(**kw):
    return _args(dict(index=FAKE, rows=10, fanout=1, dim=5, order=FAKE, position=FAKE, offsets=FAKE, work=None,
                      bytes=0), kw)


@pytest.mark.parametrize("args,expect", [
    (_group(rows=-1), 1), (_group(fanout=0), 1), (_group(dim=-1), 1), (_group(index=None), 1), (_group(order=None), 1),
    (_group(position=None), 1), (_group(offsets=None), 1), (_group(index=FAKE + 4), 1), (_group(order=FAKE + 4), 1),
    (_group(position=FAKE + 4), 1), (_group(offsets=FAKE + 4), 1), (_group(rows=2 ** 31), 2), (_group(dim=2 ** 31 - 1), 2),
    (_group(fanout=2 ** 31), 2), (_group(rows=100000), 1), (_group(rows=100000, work=FAKE, bytes=100), 1),
    (_group(rows=100000, work=FAKE + 8, bytes=2 ** 40), 1),
])
def test_group_argument_checks(args, expect):
    assert _lib().segred_group(*args, None) == expect


def _combine(**kw):
    return _args(dict(values=FAKE, dtype=3, m=64, rows=10, position=FAKE, weights=FAKE, tokens=5, fanout=2, out=FAKE), kw)


@pytest.mark.parametrize("args,expect", [
    (_combine(dtype=5), 1), (_combine(dtype=1), 2), (_combine(m=0), 1), (_combine(rows=-1), 1), (_combine(tokens=-1), 1),
    (_combine(fanout=-1), 1), (_combine(values=None), 1), (_combine(position=None), 1), (_combine(weights=None), 1),
    (_combine(out=None), 1), (_combine(values=FAKE + 1), 1), (_combine(out=FAKE + 1), 1),
    (_combine(position=FAKE + 4), 1), (_combine(weights=FAKE + 2), 1), (_combine(rows=2 ** 60), 1),
    (_combine(tokens=2 ** 60), 1), (_combine(tokens=0, out=None), 0),
])
def test_combine_argument_checks(args, expect):
    lib = _lib()
    assert lib.segred_combine(*args, None) == expect
    if expect != 0:  # the gradient call checks the same, its own pointers too
        assert lib.segred_combine_grad(FAKE, *args, FAKE, None) == expect
    good = _combine()
    assert lib.segred_combine_grad(None, *good, FAKE, None) == 1
    assert lib.segred_combine_grad(FAKE, *good, None, None) == 1
    assert lib.segred_combine_grad(FAKE + 1, *good, FAKE, None) == 1
    assert lib.segred_combine_grad(FAKE, *good, FAKE + 2, None) == 1


def _adapter(**kw):
    return _args(dict(values=FAKE, dtype=3, k=64, weights=FAKE, m=32, offsets=FAKE, which=FAKE, S=2, N=10, down=FAKE,
                      up=FAKE, scale=FAKE, L=3, r=8, transpose=0, out=FAKE, low=FAKE, work=FAKE, bytes=2 ** 30), kw)


@pytest.mark.parametrize("args,expect", [
    (_adapter(dtype=5), 1), (_adapter(dtype=0), 2), (_adapter(k=0), 1), (_adapter(m=0), 1), (_adapter(r=0), 1),
    (_adapter(L=-1), 1), (_adapter(S=-1), 1), (_adapter(N=-1), 1), (_adapter(k=2 ** 24 + 1), 2),
    (_adapter(r=2 ** 24 + 1), 2), (_adapter(L=2 ** 31), 2), (_adapter(N=2 ** 40 + 1), 2), (_adapter(values=None), 1),
    (_adapter(weights=None), 1), (_adapter(offsets=None), 1), (_adapter(which=None), 1), (_adapter(out=None), 1),
    (_adapter(down=None), 1), (_adapter(up=None), 1), (_adapter(values=FAKE + 1), 1), (_adapter(down=FAKE + 1), 1),
    (_adapter(up=FAKE + 1), 1), (_adapter(low=FAKE + 1), 1), (_adapter(scale=FAKE + 2), 1), (_adapter(which=FAKE + 4), 1),
    (_adapter(offsets=FAKE + 4), 1), (_adapter(work=None), 1), (_adapter(work=FAKE + 8), 1), (_adapter(bytes=100), 1),
    (_adapter(S=0, values=None, weights=None, offsets=None, which=None, out=None), 0),
    (_adapter(N=0, values=None, out=None, work=None), 0),
])
def test_adapter_argument_checks(args, expect):
    assert _lib().segred_adapter(*args, None) == expect


def test_workspaces():
    lib = _lib()
    assert lib.segred_group_workspace(128, 64) == 0 and lib.segred_group_workspace(0, 64) == 0
    assert lib.segred_group_workspace(4000000, 250000) > 4 * 4 * 4000000
    assert lib.segred_group_workspace(-1, 5) == 0 and lib.segred_group_workspace(2 ** 31, 5) == 0
    assert lib.segred_outer_workspace(4096, 4096, 8, 10000) == 0  # enough tiles without pieces
    assert lib.segred_outer_workspace(64, 96, 5, 300000) > 0
    assert lib.segred_outer_workspace(0, 96, 5, 300000) == 0 and lib.segred_outer_workspace(64, 96, 0, 10) == 0
    assert 48 * (4 + 128) <= lib.segred_adapter_workspace(3, 4096, 32, 16, 48) < 48 * (4 + 128) + 512
    assert lib.segred_adapter_workspace(3, 4096, 32, 12, 48) >= 48 * (4 + 128) + 32 * 4096 * 16 * 2
    assert lib.segred_adapter_workspace(3, 64, 2, 0, 48) == 0 and lib.segred_adapter_workspace(3, 64, 2, 8, 0) == 0
    assert lib.segred_adapter_workspace(0, 64, 2, 8, 8) == 0
