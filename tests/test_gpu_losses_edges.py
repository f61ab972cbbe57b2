"""The sharded losses where a formula's terms vanish, overflow or pass from one
piece of the vocabulary to the next.  Bounds are loss_ref's."""
import math

import pytest
import torch

from tests import loss_ref as ref
from tests.test_gpu_losses import BF16, DT, F32, Head, device, said  # noqa: F401

pytestmark = pytest.mark.gpu


def push_down(h, by):
    """Moves every logit of a head by -by."""
    h.x[:, 0] = 8.0
    h.w[:, 0] = -by / 8.0


# --------------------------------------------------------------------------
# rows whose loss has no weight
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,vocab,topk", [(40, 64, 500, 1), (40, 65, 500, 1), (40, 64, 500, 4), (40, 65, 500, 4),
                                                 (1100, 136, 13000, 1), (1100, 136, 13000, 3)], ids=str)
@pytest.mark.parametrize("by", [0.0, 120.0, 400.0])
def test_rows_of_no_weight_have_no_gradient(dt, rows, dim, vocab, topk, by):
    """grad = 0 in a row that counts, with logits so low that exp(-lse) overflows."""
    h = Head(dt, rows, dim, vocab, topk=topk, masked=0.0)
    push_down(h, by)
    h.index[:, 0] = torch.arange(rows, device="cuda") * 7 % vocab
    h.grad[::3] = 0
    h.run()
    assert h.loss.t[::3].all() and not h.dx[0].t[::3].any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("rows,dim,topk,lead", [(40, 64, 1, 0), (40, 65, 3, 0), (60, 72, 5, 1), (1100, 136, 1, 0), (1100, 136, 4, 0)],
                         ids=str)
def test_rows_of_no_weight_may_hold_anything(dt, bad, rows, dim, topk, lead):
    """They leave dx and dw as rows without a target do, whatever their x is."""
    h = Head(dt, rows, dim, 13000 if rows > 1000 else 500, topk=topk, masked=0.0, lead=lead)
    h.index[:, 0] = 3
    h.grad[1::4] = 0
    h.x[1::4] = 0
    h.make()
    h.issue()
    torch.cuda.synchronize()
    clean = [h.dx[0].t.clone(), h.dw[0].t.clone()]
    h.x[1::4] = bad
    h.make()
    h.issue()
    torch.cuda.synchronize()
    assert torch.equal(clean[0], h.dx[0].t) and torch.equal(clean[1], h.dw[0].t)
    assert not h.dx[0].t[1::4].any() and not h.loss.t[1::4].isfinite().any()
