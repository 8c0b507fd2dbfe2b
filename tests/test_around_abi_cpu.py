"""Refusals of the norms, the gated projections and the cross entropy, on the host
before any device work, and the sizes of their workspaces."""
import os

import pytest

FAKE = 0x10000  # a non-null, aligned host value; never dereferenced
NAN, INF = float("nan"), float("inf")


def _lib():
    import segmented_reduction_amd as sr
    if not os.path.exists(sr.LIB_PATH):
        from segmented_reduction_amd import build_lib
        build_lib.build()
    return sr.library()


def _args(defaults, kw):
    assert set(kw) <= set(defaults)
    return tuple({**defaults, **kw}.values())


def _gated(**kw):
    return _args(dict(values=FAKE, dtype=3, k=64, rows=None, value_rows=10, weights=FAKE, m=32, act=0, offsets=FAKE, S=2,
                      N=10, out=FAKE), kw)


@pytest.mark.parametrize("args,expect", [
    (_gated(dtype=5), 1), (_gated(dtype=-1), 1), (_gated(dtype=0), 2), (_gated(k=0), 1), (_gated(m=0), 1), (_gated(act=-1), 1),
    (_gated(act=4), 1), (_gated(k=2 ** 24 + 1), 2), (_gated(m=2 ** 23 + 1), 2), (_gated(value_rows=-1), 1),
    (_gated(S=-1), 1), (_gated(N=-1), 1), (_gated(value_rows=9), 1), (_gated(values=None), 1), (_gated(weights=None), 1),
    (_gated(offsets=None), 1), (_gated(out=None), 1), (_gated(values=FAKE + 1), 1), (_gated(weights=FAKE + 1), 1),
    (_gated(out=FAKE + 1), 1), (_gated(dtype=2, out=FAKE + 2), 1), (_gated(offsets=FAKE + 4), 1),
    (_gated(rows=FAKE + 4), 1), (_gated(value_rows=2 ** 60), 1), (_gated(S=2 ** 58), 1), (_gated(rows=FAKE, N=2 ** 60), 1),
    (_gated(rows=FAKE, N=2 ** 44, m=2 ** 13), 2), (_gated(S=0, offsets=None, weights=None, out=None), 0),
    (_gated(N=0, values=None, value_rows=0, out=None), 0),
])
def test_gated_argument_checks(args, expect):
    lib = _lib()
    assert lib.segred_gated(*args, None) == expect
    if expect != 0:  # the gradient call checks the same, its own pointer too
        assert lib.segred_gated_grad(FAKE, *args, None) == expect
    assert lib.segred_gated_grad(None, *_gated(), None) == 1
    assert lib.segred_gated_grad(FAKE + 1, *_gated(), None) == 1


def _norm(**kw):
    return _args(dict(values=FAKE, dtype=3, k=64, rows=10, weight=FAKE, bias=FAKE, wt=3, eps=1e-5, center=1, out=FAKE), kw)


def _norm_grad(**kw):
    return _args(dict(grad=FAKE, values=FAKE, dtype=3, k=64, rows=10, weight=FAKE, wt=3, eps=1e-5, center=1, dx=FAKE, dw=FAKE,
                      db=FAKE, work=FAKE, bytes=2 ** 30), kw)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=5), 1), (dict(dtype=0), 2), (dict(k=0), 1), (dict(rows=-1), 1), (dict(k=2 ** 24 + 1), 2), (dict(wt=4), 1),
    (dict(wt=0), 1), (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1), (dict(values=None), 1),
    (dict(values=FAKE + 1), 1), (dict(weight=FAKE + 1), 1), (dict(wt=2, weight=FAKE + 2), 1), (dict(rows=2 ** 58), 1),
])
def test_norm_argument_checks(kw, expect):
    assert _lib().segred_norm(*_norm(**kw), None) == expect
    assert _lib().segred_norm_grad(*_norm_grad(**kw), None) == expect


@pytest.mark.parametrize("kw,expect", [(dict(out=None), 1), (dict(out=FAKE + 1), 1), (dict(bias=FAKE + 1), 1),
                                       (dict(rows=0, values=None, out=None), 0)])
def test_norm_own_checks(kw, expect):
    assert _lib().segred_norm(*_norm(**kw), None) == expect


@pytest.mark.parametrize("kw,expect", [
    (dict(grad=None), 1), (dict(grad=FAKE + 1), 1), (dict(dx=None), 1), (dict(dx=FAKE + 1), 1), (dict(dw=FAKE + 1), 1),
    (dict(db=FAKE + 1), 1), (dict(rows=100, work=None), 1), (dict(work=FAKE + 8), 1), (dict(rows=100, bytes=100), 1),
    (dict(rows=0, grad=None, values=None, dx=None, dw=None, db=None, work=None, bytes=0), 0),
])
def test_norm_grad_own_checks(kw, expect):
    assert _lib().segred_norm_grad(*_norm_grad(**kw), None) == expect


def _loss(**kw):
    return _args(dict(values=FAKE, dtype=3, k=64, rows=10, weights=FAKE, vocab=100, target=FAKE, probs=FAKE, picks=2, scale=1.0,
                      loss=FAKE, lse=FAKE, picked=FAKE, work=FAKE, bytes=2 ** 40), kw)


def _loss_grad(**kw):
    return _args(dict(grad=FAKE, values=FAKE, dtype=3, k=64, rows=10, weights=FAKE, vocab=100, target=FAKE, probs=FAKE, picks=2,
                      scale=1.0, lse=FAKE, picked=FAKE, dx=FAKE, dw=FAKE, dwt=3, work=FAKE, bytes=2 ** 40), kw)


@pytest.mark.parametrize("kw,expect", [
    (dict(dtype=5), 1), (dict(dtype=1), 2), (dict(k=0), 1), (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(picks=0), 1),
    (dict(k=2 ** 24 + 1), 2), (dict(vocab=2 ** 30 + 1), 2), (dict(rows=2 ** 27 + 1), 2), (dict(picks=4097), 2),
    (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(values=None), 1),
    (dict(weights=None), 1), (dict(target=None), 1), (dict(values=FAKE + 1), 1), (dict(weights=FAKE + 1), 1),
    (dict(target=FAKE + 4), 1), (dict(probs=FAKE + 2), 1), (dict(lse=None), 1), (dict(picked=None), 1), (dict(lse=FAKE + 2), 1),
    (dict(picked=FAKE + 2), 1), (dict(work=None), 1), (dict(work=FAKE + 8), 1), (dict(bytes=100), 1),
])
def test_cross_entropy_argument_checks(kw, expect):
    assert _lib().segred_cross_entropy(*_loss(**kw), None) == expect
    assert _lib().segred_cross_entropy_grad(*_loss_grad(**kw), None) == expect


@pytest.mark.parametrize("kw,expect", [(dict(loss=None), 1), (dict(loss=FAKE + 2), 1),
                                       (dict(rows=0, values=None, target=None, loss=None, lse=None, picked=None, work=None), 0)])
def test_cross_entropy_own_checks(kw, expect):
    assert _lib().segred_cross_entropy(*_loss(**kw), None) == expect


@pytest.mark.parametrize("kw,expect", [(dict(grad=None), 1), (dict(grad=FAKE + 2), 1), (dict(dx=FAKE + 1), 1),
                                       (dict(dw=FAKE + 1), 1), (dict(dwt=4), 1), (dict(dwt=2, dw=FAKE + 2), 1)])
def test_cross_entropy_grad_own_checks(kw, expect):
    assert _lib().segred_cross_entropy_grad(*_loss_grad(**kw), None) == expect


def test_workspaces():
    lib = _lib()
    assert lib.segred_norm_grad_workspace(64, 0) == 0 and lib.segred_norm_grad_workspace(0, 5) == 0
    assert lib.segred_norm_grad_workspace(4096, 2) == 0  # one workgroup has the sums
    assert lib.segred_norm_grad_workspace(4096, 3) == 3 * 2 * 4096 * 4 and lib.segred_norm_grad_workspace(20000, 1) == 2 * 20000 * 4
    assert lib.segred_norm_grad_workspace(4096, 10 ** 9) == lib.segred_norm_grad_workspace(4096, 10 ** 6)
    assert lib.segred_cross_entropy_workspace(3, 64, 0, 10) == 0 and lib.segred_cross_entropy_workspace(0, 64, 1, 10) == 0
    assert lib.segred_cross_entropy_workspace(3, 64, 100, 6400) == 100 * 100 * 8
    for dtype, k, n, v in ((3, 2048, 4096, 65536), (2, 2048, 4096, 65536), (4, 64, 1, 2 ** 30), (3, 4096, 2 ** 20, 2 ** 17)):
        need, e = lib.segred_cross_entropy_grad_workspace(dtype, k, n, v, 3), 4 if dtype == 2 else 2
        piece = min(v, max(2 ** 28 // (n * e), 4096) + 8)
        # a piece, the rows' sums (up to 64 of them where there are few), and what the weights' sums need
        assert need <= 2 * (n + 8) * piece * e + 2 * (n + piece) * (k + 8) * e + 64 * min(n, 4096) * k * 4 + n * k * 4 + n * 64 + 2 ** 28
    assert lib.segred_cross_entropy_grad_workspace(0, 64, 10, 10, 1) == 0
