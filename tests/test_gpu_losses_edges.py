"""The sharded losses where a formula's terms vanish, overflow or pass from one
piece of the vocabulary to the next.  Bounds are loss_ref's."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd.sharded_step import ShardedStep
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


# --------------------------------------------------------------------------
# scale = 0: every entry is equally likely
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,vocab", [(1, 64, 100), (40, 72, 500), (50, 65, 513), (300, 64, 256), (1100, 64, 13001)], ids=str)
@pytest.mark.parametrize("topk", [1, 4])
def test_scale_of_zero(dt, rows, dim, vocab, topk):
    h = Head(dt, rows, dim, vocab, topk=topk, scale=0.0, distill=topk > 1, masked=0.3 if rows > 1 else 0.0)
    h.index[0, 0] = vocab - 1
    h.run()
    # one part's sum and its joins: vocab equal terms, the log of their number
    assert ((h.lse.t.double() - math.log(vocab)).abs() <= (vocab + 16) * ref.U).all()
    assert not h.dx[0].t.any() and not h.dw[0].t.any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_scale_of_zero_over_shards(dt):
    h = Head(dt, 77, 96, 1000, sizes=[1, 0, 300, 699], scale=0.0).run()
    assert [s.t[0].tolist() for s in h.stats] == [[0.0, 1.0], [-math.inf, 0.0], [0.0, 300.0], [0.0, 699.0]]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("scale", [0.0, -0.0, 0.5])
def test_teacher_entries_at_minus_infinity_are_left_out(dt, scale):
    h = Head(dt, 50, 64, 500, topk=6, scale=scale, masked=0.1)
    h.index[:2] = torch.arange(6, device="cuda") * 3
    h.teacher[0, 1::2] = -math.inf
    h.teacher[1] = -math.inf                            # nothing left
    h.make()
    h.issue()
    gone = h.teacher == -math.inf
    assert not h.prob.t[gone].any() and not h.loss.t[1].any() and not h.dx[0].t[1].any()
    # the entries' logits are given all the same; the rest is as if they were not there
    picked = h.logit.t[:2].clone()
    z = scale * (h.x[:2].double() @ h.w[h.index[0]].double().t())
    size = abs(scale) * (h.x[:2].double().abs() @ h.w[h.index[0]].double().abs().t())
    assert ((picked.double() - z).abs() <= (64 + 6) * ref.U * size).all()
    h.index[gone] = -1
    h.teacher[gone] = 0
    h.logit.t[gone] = 0
    h.verify()


# --------------------------------------------------------------------------
# far logits
# --------------------------------------------------------------------------

@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size", [2.0 ** 33, 2.0 ** 66])
@pytest.mark.parametrize("rows,dim,vocab", [(3, 64, 500), (40, 65, 700), (300, 72, 513), (1100, 64, 13001)], ids=str)
def test_statistics_of_huge_logits(dt, size, rows, dim, vocab):
    """Finite logits have a finite log sum exp: the largest counts once."""
    h = Head(dt, rows, dim, vocab)
    h.x = h.x * size
    h.make()
    for v, w, s, p, (_, ws) in zip(h.v, h.vw, h.stats, h.picked, h.works):
        rr.rr_vocab_stats(v, dt, h.vx, w, h.index, s.t, p.t, workspace=ws)
    rr.rr_vocab_cross_entropy(h.v[0], h.index, [s.t for s in h.stats], [p.t for p in h.picked], h.lse.t, h.logit.t, h.loss.t)
    torch.cuda.synchronize()
    want, tol = ref.head(h.x, h.w, h.index)
    for n in ("lse", "logit", "loss"):
        ref.check(n, getattr(h, n).t, want[n], tol[n])
    sums = h.stats[0].t[:, 1]
    assert (sums >= 1).all() and (sums <= vocab).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("topk", [1, 5])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_grad_of_a_row_without_a_target(dt, topk, bad):
    h = Head(dt, 40, 64, 500, topk=topk)
    none = (h.index < 0).all(dim=1)
    assert none.any() and not none.all()
    h.grad[none] = bad
    h.run()
    assert not h.dx[0].t[none].any() and not h.loss.t[none].any()


# --------------------------------------------------------------------------
# several pieces of the vocabulary (one holds 2^28 bytes of dz, 256 entries at least)
# --------------------------------------------------------------------------

def around_pieces(h):
    """Targets of the first rows at both ends of the vocabulary and of every
    possible piece."""
    edges = torch.arange(0, h.vocab, 256, device="cuda")
    at = torch.cat([edges, edges[1:] - 1, torch.tensor([h.vocab - 1], device="cuda")])[:h.rows]
    h.index[:at.numel(), 0] = at


@pytest.mark.parametrize("dt,vocab", [(F32, 17001), (BF16, 33001)])
@pytest.mark.parametrize("dim", [40, 41])
@pytest.mark.parametrize("topk", [1, 3])
def test_wide_pieces(dt, vocab, dim, topk):
    h = Head(dt, 4200, dim, vocab, topk=topk, scale=0.5 if topk > 1 else 1.0)
    assert 4200 * vocab * (4 if dt == F32 else 2) > 1 << 28
    around_pieces(h)
    h.run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("dim,lead", [(40, 0), (41, 0), (40, 1)])
@pytest.mark.parametrize("topk", [1, 3])
def test_narrow_pieces(dt, dim, lead, topk):
    """Three pieces of 256, 256 and 188 entries for many rows, most of them
    without a target: those add nothing to a sum, so that the bounds are of the
    others alone."""
    h = Head(dt, 300000, dim, 700, topk=topk, scale=0.5 if topk > 1 else 1.0, masked=0.999, lead=lead)
    around_pieces(h)
    h.make()
    h.issue()
    torch.cuda.synchronize()
    used = (h.index >= 0).any(dim=1)
    assert 100 < used.sum() < 1000
    want, tol = ref.head(h.x[used], h.w, h.index[used], h.scale, h.teacher[used] if h.distill else None, h.grad[used])
    for n in ("lse", "logit", "loss", "dx"):
        t = (h.dx[0] if n == "dx" else getattr(h, n)).t
        ref.check(n, t[used], want[n], tol[n])
    ref.check("dw", h.dw[0].t, want["dw"], tol["dw"])
    assert not h.dx[0].t[~used].any() and not h.loss.t[~used].any()
    assert all(o.untouched() for o in h.outs())
    assert all(bool((big[ws.numel():] == 0xFF).all()) for big, ws in h.works)


# --------------------------------------------------------------------------
# the step that runs the calls together
# --------------------------------------------------------------------------

def test_step_ignores_targets_outside_the_vocabulary():
    """They are no targets: not in the mean, and not routed."""
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn(60, 24, generator=gen, device="cuda")
    index = torch.randint(0, 90, (60, 1), generator=gen, device="cuda")
    index[::3] = -1
    sides = []
    for none in (-1, 90, 1 << 40):
        s = ShardedStep(60, 24, 90, shards=2, experts=5, topk=2, dtype=F32)
        loss, balance = s.step(x, torch.where(index < 0, none, index))
        assert torch.equal(s.keep, index[:, 0] >= 0)
        sides.append([loss, balance, s.dhead, s.dlogits, *s.dx])
    assert all(torch.equal(a, b) for side in sides[1:] for a, b in zip(sides[0], side))


def test_step_distills_gradients():
    """Against autograd in 64 bits: temperature^2 times the distillation, in fp32."""
    rows, dim, vocab, experts, k, t = 40, 24, 90, 5, 4, 2.0
    s = ShardedStep(rows, dim, vocab, shards=2, experts=experts, topk=2, teacher_topk=k, temperature=t, balance=0.0, dtype=F32)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    index = torch.stack([torch.randperm(vocab, generator=gen, device="cuda")[:k] for _ in range(rows)])
    index[::6] = -1
    teacher = 2 * torch.randn(rows, k, generator=gen, device="cuda")
    loss, _ = s.step(x, index, teacher)
    keep = (index >= 0).all(dim=1)
    head, logits = s.head.double().requires_grad_(), s.logits.double().requires_grad_()
    weight, choice = torch.softmax(logits, dim=1).topk(2, dim=1)
    weight = weight / weight.sum(dim=1, keepdim=True) * keep[:, None]
    y = x.double() * (1 + (weight[:, :, None] * s.scale.double()[choice]).sum(dim=1))
    p = torch.log_softmax(teacher.double() / t, dim=1)
    q = torch.log_softmax(y @ head.t() / t, dim=1).gather(1, index.clamp_min(0))
    mean = (p.exp() * (p - q)).sum(dim=1)[keep].mean()
    (t * t * mean).backward()
    assert loss.item() == pytest.approx(mean.item(), rel=512 * ref.U)
    # a few hundred fp32 roundings along the way
    for got, want in ((s.dlogits, logits.grad), (s.dhead, head.grad)):
        assert (got.double() - want).abs().max() <= 512 * ref.U * want.abs().max()
