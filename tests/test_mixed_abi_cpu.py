"""Refusals of the calls that take two types, on the host before any device work."""
import pytest

from tests.test_ragged_abi_cpu import FAKE, _args, _lib


def _outer(**kw):
    return _args(dict(left=FAKE, left_dtype=3, left_rows=None, left_count=10, k=64, right=FAKE, right_dtype=2,
                      right_rows=None, right_count=10, m=32, offsets=FAKE, S=2, N=10, out=FAKE, out_dtype=3, work=None,
                      bytes=0), kw)


@pytest.mark.parametrize("args,expect", [
    (_outer(left_dtype=5), 1), (_outer(right_dtype=-1), 1), (_outer(left_dtype=0), 2), (_outer(right_dtype=1), 2),
    (_outer(right_dtype=4), 2), (_outer(left_dtype=4, right_dtype=3), 2),                # two 16-bit types
    (_outer(out_dtype=4), 1), (_outer(out_dtype=1), 1), (_outer(left_dtype=2, out_dtype=3), 1),
    (_outer(left=FAKE + 1), 1), (_outer(right=FAKE + 2), 1), (_outer(left_dtype=2, right_dtype=4, out_dtype=4, left=FAKE + 2), 1),
    (_outer(out_dtype=2, out=FAKE + 2), 1), (_outer(left=None), 1), (_outer(right=None), 1), (_outer(left_count=9), 1),
    (_outer(left_count=100000, right_count=100000, N=100000), 1),
    (_outer(S=0, left=None, right=None, offsets=None, out=None), 0),
])
def test_outer_argument_checks(args, expect):
    assert _lib().segred_outer_mixed(*args, None) == expect


def _adapter(**kw):
    return _args(dict(values=FAKE, dtype=3, k=64, weights=FAKE, m=32, offsets=FAKE, which=FAKE, S=2, N=10, down=FAKE,
                      up=FAKE, scale=FAKE, L=3, r=8, transpose=0, out=FAKE, low=FAKE, low_dtype=2, work=FAKE,
                      bytes=2 ** 30), kw)


@pytest.mark.parametrize("args,expect", [
    (_adapter(dtype=5), 1), (_adapter(dtype=0, low_dtype=0), 2), (_adapter(low_dtype=4), 1), (_adapter(low_dtype=5), 1),
    (_adapter(dtype=2, low_dtype=3), 1), (_adapter(low=FAKE + 2), 1), (_adapter(low_dtype=3, low=FAKE + 1), 1),
    (_adapter(bytes=100), 1), (_adapter(S=0, values=None, weights=None, offsets=None, which=None, out=None), 0),
])
def test_adapter_argument_checks(args, expect):
    assert _lib().segred_adapter_mixed(*args, None) == expect
