"""The gradient of a softmax router that does not renormalize, whose logits lie anywhere: it is
computed in 64 bits and rounded once (of bf16 in 32 bits), however large the logits that all experts share."""
import pytest
import torch

import pack_rr_helper_amd as rr
from tests import expert_ref as ref
from tests.test_gpu_group_route import Route, router
from tests.test_gpu_losses import DT, device, normal, said  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16


def plain(r, logits, choice, grad_weight, dt):
    """dlogits in 64 bits, and how far a kernel's may be."""
    z, live = logits.double(), choice >= 0
    at = choice.long().clamp_min(0)
    g = torch.zeros_like(z).scatter_add_(1, at, torch.where(live, grad_weight.double(), 0.0))
    p = torch.softmax(z, dim=1)
    mean, size = (p * g).sum(dim=1, keepdim=True), (p * g.abs()).sum(dim=1, keepdim=True)
    some = live.any(dim=1, keepdim=True)
    d = torch.where(some, r.scale * p * (g - mean), 0.0)
    if dt == F32:
        # in 64 bits: each factor and the sums of them within 2^-44 of what they are at most, eight of
        # them; then rounded to 32 bits, or to half the least number
        return d, 8 * 2.0 ** -44 * abs(r.scale) * p * (g.abs() + size) + d.abs() * ref.U * 1.01 + 2.0 ** -150
    # in 32 bits: an exponential is off by two half steps and by its exponent's rounding, |log p| half steps; a
    # sum of 16 and over 64 lanes by 22, quotients and products by fewer than 16 together, the mean of up to
    # 32 terms by 34 more.  Then the type, or half its least number; a p below 2^-126 has half steps of 2^-150.
    far = -torch.log_softmax(z, dim=1).clamp_min(-200.0)
    own = (64 + far) * (g.abs() + size)
    of_mean = 64 * size + (p * g.abs() * far).sum(dim=1, keepdim=True)
    tol = ref.U * abs(r.scale) * p * (own + of_mean) + d.abs() * (ref.HALF[DT[dt]] + ref.U) * 1.01
    return d, tol + 2.0 ** -134 + 2.0 ** -148 * abs(r.scale) * (g.abs() + size)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shift", [0.0, 7.0, -90.0, 1000.0, 30000.0])
@pytest.mark.parametrize("shape", [(12, 4, 4, 2, 2), (60, 4, 5, 2, 2), (160, 6, 8, 3, 1), (256, 32, 4, 2, 2), (257, 5, 1, 1, 1),
                                   (512, 16, 64, 9, 2), (1023, 8, 33, 4, 2)], ids=str)
def test_rounded_once(dt, shift, shape):
    r = router(*shape, False, False, 2.5)
    gen = torch.Generator(device="cuda").manual_seed(shape[0])
    logits = (2 * normal(gen, 77, shape[0]) + shift + 3 * normal(gen, 77, 1)).to(DT[dt])
    x = Route(dt, 77, r, logits=logits).run()
    d, tol = plain(r, logits, x.choice.t, x.grad_weight, dt)
    off = (x.dlogits.t.double() - d).abs()
    assert (off <= tol).all(), (off / tol).max().item()
    assert all(o.untouched() for o in x.outs())


@pytest.mark.parametrize("dt", [F32, BF16])
def test_rows_of_few_live_logits(dt):
    """Logits of -inf have p = 0 and no gradient, rows of them and rows without a choice none at all."""
    r = router(32, 4, 4, 2, 2, False, False)
    gen = torch.Generator(device="cuda").manual_seed(3)
    logits = (normal(gen, 40, 32) + 500.0).to(DT[dt])
    logits[:20, 5:30] = -torch.inf
    logits[20:24] = -torch.inf
    x = Route(dt, 40, r, logits=logits).run()
    d, tol = plain(r, logits[:20], x.choice.t[:20], x.grad_weight[:20], dt)
    got = x.dlogits.t.double()
    assert ((got[:20] - d).abs() <= tol).all()
    assert not got[20:24].any() and not got[~x.keep].any() and torch.isfinite(got).all()


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_scores_are_cut(sign, sigmoid):
    """Choice scores are compared by 43 significant bits: in steps of 2^-22 from 2^20 on, of 2^-23 below, the lower index
    first in one."""
    logits = torch.full((5, 8), -20.0, device="cuda")
    # sigmoid: 1/2, 1e-7 more, 1e-6 more; softmax of these three: about a third, 1.3e-7 and 1.3e-6 apart
    logits[:, 1:4] = torch.tensor([0.0, 4e-7, 4e-6], device="cuda")
    bias = torch.full((8,), sign * 2.0 ** 20, device="cuda")
    x = Route(F32, 5, router(8, 3, 1, 1, 1, sigmoid, True), masked=0.0, bias=False, logits=logits)
    x.bias = bias
    x.run()
    z = logits[0].double()
    c = (torch.sigmoid(z) if sigmoid else torch.softmax(z, dim=0)) + bias.double()
    # the cut is towards zero: a negative bias leaves magnitudes below 2^20, whose 43 bits reach to 2^-23
    part, e = torch.frexp(c)
    cut = torch.ldexp(torch.trunc(part * 2.0 ** 43), e - 43)
    want = sorted(range(8), key=lambda i: (-cut[i].item(), i))[:3]
    assert x.choice.t.tolist() == [want] * 5
    # without a bias the same scores are apart
    x.bias = None
    x.run()
    assert x.choice.t.tolist() == [[3, 2, 1]] * 5
