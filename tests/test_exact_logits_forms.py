"""The inputs with exact logits on the CPU: what one lost, doubled or added entry of
the vocabulary does to each result is far outside the bounds."""
import pytest
import torch

from tests import exact_logits as X
from tests.around_util import TYPES, half_step

CASES = [("bf16", 5, 256, 3001, 1), ("f32", 40, 65, 2001, 3), ("f16", 48, 131, 3001, 1), ("bf16", 48, 520, 20001, 1),
         ("f16", 48, 1030, 4099, 5), ("f32", 20, 128, 9001, 1), ("bf16", 20, 2048, 30011, 1), ("bf16", 60, 64, 9001, 1)]


@pytest.mark.parametrize("t,n,k,v,picks", CASES)
def test_every_row_has_an_entry_that_decides(t, n, k, v, picks):
    x, w, target, probs, grad, scale, lead = X.case(TYPES[t], n, k, v, picks)
    # sums of multiples of 1/8 below 2^21: exact in float32 in any order
    assert torch.equal(x.float() @ w.float().t(), (x.double() @ w.double().t()).float())
    assert (x.double().abs() @ w.double().abs().t()).max() < 2 ** 21
    (loss, lse, _), (e_loss, e_lse, _), (z, goal, live, share) = X.forward(x, w, target, probs, scale)
    row = torch.arange(n)
    assert (z.argmax(1) == lead).all() and ((z[row, lead] - lse).exp() > 0.9).all()
    gone = z.clone()
    gone[row, lead] = float("-inf")
    assert ((torch.logsumexp(gone, 1) - lse).abs() > 1000 * e_lse).all()
    twice = torch.cat([z, z[row, lead, None]], 1)
    assert ((torch.logsumexp(twice, 1) - lse).abs() > 1000 * e_lse).all()
    # its share of the gradients: left out, most elements leave their bounds
    (dx, dw), (e_x, e_w) = X.backward(x, w, target, probs, grad, scale)
    part = (share * grad.double() * scale * (z[row, lead] - lse).exp())[:, None]
    seen = live & ~(goal[row, lead] > 0.5 * share)  # where the target is the entry itself little is left
    off = (part * w[lead].double()).abs() > 4 * (e_x + half_step(x.dtype, dx.abs() + e_x))
    assert (off[seen].double().mean(1) > 0.5).all()
    off = (part * x.double()).abs() > 4 * (e_w + half_step(x.dtype, dw.abs() + e_w))[lead]
    assert (off[seen].double().mean(1) > 0.5).all()


@pytest.mark.parametrize("t,n,k,v", [("bf16", 5, 256, 3001), ("f32", 40, 65, 2001), ("f16", 48, 520, 20001)])
def test_an_entry_behind_the_end_would_decide(t, n, k, v):
    x, w, target, _, grad, scale = X.below_zero(TYPES[t], n, k, v)
    (_, lse, _), (_, e_lse, _), (z, *_) = X.forward(x, w, target, None, scale)
    assert z.max() < -20
    more = torch.cat([z, torch.zeros(n, 1, dtype=z.dtype)], 1)  # what a column of zero weights gives
    assert ((torch.logsumexp(more, 1) - lse) > 1e4 * e_lse).all()
