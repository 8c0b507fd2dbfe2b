"""The norms, the gated projections and the cross entropy through the C ABI (GPU
only), with every result and a workspace of exactly the size that is asked for inside
larger buffers: what lies around them stays as it was, and what a workspace held
before has no part in the results."""
import pytest
import torch

import segmented_reduction_amd as sr
from tests import around_util as A

pytestmark = pytest.mark.gpu

PAD = 8192
CODE = {"f32": 2, "bf16": 3, "f16": 4}


class Inside:
    """A buffer of `count` elements with PAD bytes before and behind it, all ones at first
    (NaN in every type); `shift` elements behind a 256-byte boundary."""

    def __init__(self, name, count, dtype, shift=0):
        size = torch.empty((), dtype=dtype).element_size()
        self.name, self.begin, self.end = name, PAD + shift * size, PAD + (shift + count) * size
        self.all = torch.full((self.end + PAD,), 255, dtype=torch.uint8, device="cuda")
        self.view = self.all[self.begin:self.end].view(dtype) if count else torch.empty(0, dtype=dtype, device="cuda")
        self.ptr = self.all.data_ptr() + self.begin

    def check(self, what):
        assert (self.all[:self.begin] == 255).all(), f"{what}: written before {self.name}"
        assert (self.all[self.end:] == 255).all(), f"{what}: written behind {self.name}"


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _same(a, b, what):
    assert torch.equal(a.view(b.shape), b), f"{what}: not what the same call gives elsewhere"


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k", [(1, 1), (3, 7), (40, 127), (70, 333), (9, 520), (33, 1001), (600, 2047), (5, 4099), (300, 5001),
                                 (7, 8192), (5, 16383), (3, 16389), (300, 17000)])
def test_norm(t, n, k):
    lib, g, T = sr.library(), A.gen(n * k), A.TYPES[t]
    x, d = A.randn(g, n, k, dtype=T).cuda(), A.randn(g, n, k, dtype=T).cuda()
    w, b = A.randn(g, k).cuda(), A.randn(g, k).cuda()
    for shift in (0, 1):
        out, dx = Inside("out", n * k, T, shift), Inside("dx", n * k, T, shift)
        dw, db = Inside("dw", k, torch.float32, shift), Inside("db", k, torch.float32, shift)
        need = lib.segred_norm_grad_workspace(k, n)
        work = Inside("workspace", need, torch.uint8)
        what = f"surroundings norm {t} {n}x{k} at {shift}"
        A.say(what)
        assert lib.segred_norm(x.data_ptr(), CODE[t], k, n, w.data_ptr(), b.data_ptr(), 2, 1e-5, 1, out.ptr, _stream()) == 0
        assert lib.segred_norm_grad(d.data_ptr(), x.data_ptr(), CODE[t], k, n, w.data_ptr(), 2, 1e-5, 1, dx.ptr, dw.ptr, db.ptr,
                                    work.ptr if need else None, need, _stream()) == 0
        torch.cuda.synchronize()
        for v in (out, dx, dw, db, work):
            v.check(what)
        _same(out.view, sr.norm(x, w, b), what)
        for v, ref in zip((dx, dw, db), sr.norm_grad(d, x, w, want_bias=True)):
            _same(v.view, ref, what)


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lengths,k,m", [([1], 1, 1), ([3, 0, 9], 64, 33), ([8] * 40, 128, 65), ([16, 15], 257, 101), ([70, 130, 1], 256, 63),
                                         ([129] * 20, 256, 499), ([300, 41], 65, 131), ([600, 1200], 192, 513),
                                         ([4500, 1361], 256, 1025)])
def test_gated(t, lengths, k, m):
    """The last segment ends at the last row, and rows are no whole units."""
    lib, g, T = sr.library(), A.gen(k * m), A.TYPES[t]
    off = A.offsets(lengths).cuda()
    n = sum(lengths)
    x, d = A.randn(g, n, k, dtype=T).cuda(), A.randn(g, n, m, dtype=T).cuda()
    w = A.randn(g, len(lengths), 2 * m, k, dtype=T, std=k ** -0.5).cuda()
    for shift in (0, 1):
        out, pair = Inside("out", n * m, T, shift), Inside("pair", n * 2 * m, T, shift)
        what = f"surroundings gated {t} {lengths[:3]} {k}x{m} at {shift}"
        A.say(what)
        args = (x.data_ptr(), CODE[t], k, None, n, w.data_ptr(), m, 1, off.data_ptr(), len(lengths), n)
        assert lib.segred_gated(*args, out.ptr, _stream()) == 0
        assert lib.segred_gated_grad(d.data_ptr(), *args, pair.ptr, _stream()) == 0
        torch.cuda.synchronize()
        for v in (out, pair):
            v.check(what)
        _same(out.view, sr.gated(x, w, off, activation="gelu"), what)
        _same(pair.view, sr.gated_grad(d, x, w, off, activation="gelu"), what)


SHAPES = [(1, 1, 1), (1, 8, 65), (5, 131, 3001), (14, 256, 3001), (16, 1024, 13001), (60, 65, 2001), (64, 520, 13003), (100, 256, 33000),
          (200, 257, 3001), (300, 1030, 5003), (300, 128, 9001), (701, 512, 9001), (256, 2048, 30011), (2100, 1030, 4099),
          (2304, 1024, 4100), (8200, 65, 8300), (16389, 72, 8193)]


@pytest.mark.parametrize("t", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("n,k,v", SHAPES)
@pytest.mark.parametrize("picks", [1, 3])
def test_cross_entropy(t, n, k, v, picks):
    lib, g, T = sr.library(), A.gen(n + k + v), A.TYPES[t]
    x, w = A.randn(g, n, k, dtype=T).cuda(), A.randn(g, v, k, dtype=T, std=2 * k ** -0.5).cuda()
    target = torch.randint(-1, v, (n, picks), generator=g).cuda()
    probs, grad = torch.rand(n, picks, generator=g).cuda(), torch.rand(n, generator=g).cuda()
    shift = (n + picks) % 2
    F = torch.float32
    loss, lse, picked = (Inside(s, c, F, shift) for s, c in (("loss", n), ("lse", n), ("picked", n * picks)))
    wide = picks == 3  # the weights' gradient in float32
    dx, dw = Inside("dx", n * k, T, shift), Inside("dw", v * k, F if wide else T, shift)
    need = lib.segred_cross_entropy_workspace(CODE[t], k, n, v)
    work = Inside("workspace", need, torch.uint8)
    back = lib.segred_cross_entropy_grad_workspace(CODE[t], k, n, v, picks)
    again = Inside("gradient's workspace", back, torch.uint8)
    what = f"surroundings cross entropy {t} {n}x{k} vocab {v} picks {picks} at {shift}"
    A.say(what)
    args = (x.data_ptr(), CODE[t], k, n, w.data_ptr(), v, target.data_ptr(), probs.data_ptr(), picks, 1.0)
    assert lib.segred_cross_entropy(*args, loss.ptr, lse.ptr, picked.ptr, work.ptr, need, _stream()) == 0
    assert lib.segred_cross_entropy_grad(grad.data_ptr(), *args, lse.ptr, picked.ptr, dx.ptr, dw.ptr, 2 if wide else CODE[t], again.ptr,
                                         back, _stream()) == 0
    torch.cuda.synchronize()
    for o in (loss, lse, picked, dx, dw, work, again):
        o.check(what)
    refs = sr.cross_entropy(x, w, target, probs=probs)
    for o, ref in zip((loss, lse, picked), refs):
        _same(o.view, ref, what)
    for o, ref in zip((dx, dw), sr.cross_entropy_grad(grad, x, w, target, *refs[1:], probs=probs, weights_dtype=F if wide else None)):
        _same(o.view, ref, what)
