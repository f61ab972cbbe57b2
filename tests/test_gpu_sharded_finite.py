"""The sharded step with clipping, where the gradients' norm is not finite: no weight and no bias
moves, and the next step does."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd.sharded_step import ShardedStep
from tests.test_gpu_losses import DT, device, normal, said  # noqa: F401
from tests.test_gpu_sharded_experts import inputs

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16


def weights(s):
    return [s.router, s.head, s.experts if s.products else s.scale] + ([s.bias] if s.move_bias else [])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("products,grouped", [(True, True), (False, True), (True, False), (False, False)])
def test_not_finite(dt, bad, products, grouped):
    rows, dim, vocab = 100, 72, 150
    router = rr.GroupRouter(8, 2, 2, 1, 1, False, False) if grouped else None
    s = ShardedStep(rows, dim, vocab, shards=2, dtype=dt, router=router, bias_rate=0.25, products=products, max_norm=1.0)
    x, index = inputs(rows, dim, vocab)
    before = [w.clone() for w in weights(s)]
    spoilt = x.clone()
    spoilt[5, 3] = bad                                         # a row that has a target
    assert index[5, 0] >= 0
    s.step(spoilt, index, rate=0.5)
    torch.cuda.synchronize()
    assert not math.isfinite(s.norm.item())
    assert all(torch.equal(a, b) for a, b in zip(before, weights(s)))
    s.step(x, index, rate=0.5)
    torch.cuda.synchronize()
    assert math.isfinite(s.norm.item())
    assert not any(torch.equal(a, b) for a, b in zip(before, weights(s)))
    assert all(torch.isfinite(w.float()).all() for w in weights(s))


def test_past_the_range_of_a_float():
    """A norm that fp32 does not hold is finite: the gradients are scaled and the weights move."""
    s = ShardedStep(20, 16, 30, shards=1, dtype=F32, max_norm=1.0)
    grads = [torch.full((100,), 3e38, device="cuda"), torch.full((50,), -3e38, device="cuda")]
    norm, finite = s._clip(grads)
    torch.cuda.synchronize()
    assert norm.item() == math.inf and finite.all()
    # of 150 equal elements and a norm of 1; the factor is a subnormal number
    for g, sign in zip(grads, (1, -1)):
        assert ((g.double() - sign / math.sqrt(150)).abs() <= 3e38 * 2.0 ** -150 + 1e-7).all()
