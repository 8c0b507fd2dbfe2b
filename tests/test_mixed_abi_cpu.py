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


def _repeated(**kw):
    return _args(dict(grad=FAKE, values=FAKE, dtype=3, m=64, rows=10, position=FAKE, weights=FAKE, tokens=5, fanout=2,
                      grad_values=FAKE, grad_weights=FAKE, work=FAKE, bytes=2 ** 30), kw)


@pytest.mark.parametrize("args,expect", [
    (_repeated(dtype=5), 1), (_repeated(dtype=1), 2), (_repeated(m=0), 1), (_repeated(rows=-1), 1),
    (_repeated(tokens=-1), 1), (_repeated(fanout=-1), 1), (_repeated(grad=None), 1), (_repeated(values=None), 1),
    (_repeated(position=None), 1), (_repeated(weights=None), 1), (_repeated(grad_values=None), 1),
    (_repeated(grad_weights=None), 1), (_repeated(grad=FAKE + 1), 1), (_repeated(grad_weights=FAKE + 2), 1),
    (_repeated(work=None), 1), (_repeated(bytes=100), 1), (_repeated(work=FAKE + 8), 1),
    (_repeated(rows=2 ** 31 - 1), 2), (_repeated(tokens=2 ** 30, fanout=2), 2), (_repeated(rows=0, tokens=0), 0),
])
def test_repeated_rows_argument_checks(args, expect):
    assert _lib().segred_combine_grad_repeated(*args, None) == expect


def test_repeated_rows_workspace():
    lib = _lib()
    assert lib.segred_combine_grad_repeated_workspace(0, 5, 2) == 0
    assert lib.segred_combine_grad_repeated_workspace(2 ** 31, 5, 2) == 0
    assert lib.segred_combine_grad_repeated_workspace(100, 5, 2) >= 2 * 80 + 101 * 8
