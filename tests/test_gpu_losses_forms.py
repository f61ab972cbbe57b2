"""The sharded losses at the sizes that choose each of their kernels' forms: wide
and narrow tiles, sums split into parts, rows that do not start at 16 bytes, one
entry per 16 lanes or per wave, lists of every length; and the step that runs
them together.  Bounds are loss_ref's."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd.sharded_step import ShardedStep
from tests import loss_ref as ref
from tests.test_gpu_losses import BF16, DT, F32, Head, Route, device, said  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,vocab", [
    (1100, 200, 13001),     # 256 x 256 tiles with ragged ends
    (1100, 201, 13001),     # the same through registers and copies
    (2300, 136, 9000),
    (520, 72, 30011),
    (90, 264, 20000),
    (3, 40, 70001),         # dx in many parts, their sums joined by eight threads each
    (40, 96, 50000),
    (6000, 64, 300),        # dw in parts
    (4100, 1, 257),
], ids=str)
def test_cross_entropy(dt, rows, dim, vocab):
    Head(dt, rows, dim, vocab).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,vocab,topk", [(300, 136, 2000, 64), (1100, 72, 9001, 40), (700, 33, 600, 100)], ids=str)
def test_distill(dt, rows, dim, vocab, topk):
    Head(dt, rows, dim, vocab, sizes=[vocab // 3, vocab - vocab // 3], topk=topk, scale=0.5, distill=True).run()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_negative_scale(dt):
    Head(dt, 150, 72, 700, scale=-0.75).run()
    Head(dt, 70, 64, 500, topk=5, scale=-2.0).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("where", ["first", "last", "edges"])
def test_targets_in_every_place_of_a_tile(dt, where):
    h = Head(dt, 600, 64, 3000, masked=0.0)
    n = torch.arange(600, device="cuda")
    h.index[:, 0] = {"first": n, "last": 2999 - n, "edges": n * 5 % 3000}[where]
    h.run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows", [70, 1100])
def test_infinite_logits_of_a_masked_row_leave_no_dz(dt, rows):
    """A masked row's own gradient is zero whatever its logits are."""
    h = Head(dt, rows, 64, 13000, masked=0.0)
    h.index[5] = -100
    h.x[5] = torch.finfo(DT[dt]).max
    h.make()
    h.issue()
    torch.cuda.synchronize()
    assert not h.dx[0].t[5].any() and h.loss.t[5] == 0


def test_many_calls_share_a_workspace():
    """A workspace carries nothing over: the same bits after another call's use."""
    a, b = Head(BF16, 300, 64, 2000), Head(BF16, 20, 136, 9000, topk=3, scale=0.5)
    a.run()
    b.run()
    first = a.bits()
    work = torch.empty(max(w[1].numel() for w in a.works + b.works), dtype=torch.uint8, device="cuda")
    a.works, b.works = [(work, work)], [(work, work)]
    b.issue()
    a.issue()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(first, a.bits()))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts", [2, 15, 16, 17, 31, 32, 33, 60, 63, 64, 65, 127, 128, 129, 255, 256, 257, 511, 513, 1000, 1023])
def test_route_every_row_form(dt, renormalize, experts):
    for topk in (1, 2, 3, 4, 5, 8, 9, 17, 32):
        if topk <= experts:
            Route(dt, 150, experts, topk, renormalize=renormalize, seed=topk).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows", [127, 128, 129, 513, 40000])
def test_route_one_and_many_workgroups(dt, rows):
    Route(dt, rows, 64, 6).run()
    Route(dt, rows, 300, 3).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("experts,topk", [(24, 4), (24, 12), (200, 8), (600, 5)])
def test_route_nan_of_either_sign(dt, experts, topk):
    """NaN ranks above every number, the lower index first; only its row knows."""
    r = Route(dt, 30, experts, topk, masked=0.0)
    clean = Route(dt, 30, experts, topk, masked=0.0)
    bits, t = (torch.int32, -0x00400000) if dt == F32 else (torch.int16, -0x0040)
    r.logits[3, experts - 1] = float("nan")
    r.logits[3].view(bits)[experts // 2] = t           # a NaN with its sign set
    assert r.logits[3].isnan().sum() == 2
    r.logits[4, 1] = math.inf
    for q in (r, clean):
        q.make()
        q.issue()
    torch.cuda.synchronize()
    assert r.choice.t[3, :2].tolist() == [experts // 2, experts - 1]
    assert r.weight.t[3].isnan().all() and r.lse.t[3].isnan()
    assert r.choice.t[4, 0] == 1
    rest = torch.arange(30, device="cuda")
    rest = rest[(rest != 3) & (rest != 4)]
    assert torch.equal(r.choice.t[rest], clean.choice.t[rest])
    assert torch.equal(r.weight.t[rest], clean.weight.t[rest]) and torch.equal(r.lse.t[rest], clean.lse.t[rest])
    left = torch.tensor([3], device="cuda")
    want = sorted(set(range(experts)) - {experts // 2, experts - 1}, key=lambda e: (-float(r.logits[3, e]), e))
    assert r.choice.t[left, 2:].flatten().tolist() == want[:topk - 2]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("experts", [24, 256, 700])
def test_route_equal_logits(dt, experts):
    r = Route(dt, 50, experts, 7, masked=0.0)
    r.logits[:] = 0.5
    r.logits[1, ::2] = -0.0
    r.logits[1, 1::2] = 0.0
    r.run()
    assert (r.choice.t == torch.arange(7, device="cuda")).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("teacher", [0, 8])
def test_sharded_step_learns(dt, teacher):
    """The calls run together: the loss falls, and a step's gradients are autograd's."""
    rows, dim, vocab = 256, 64, 500
    s = ShardedStep(rows, dim, vocab, shards=3, experts=6, topk=2, teacher_topk=teacher, temperature=2.0, dtype=dt)
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    index = torch.randint(0, vocab, (rows, max(teacher, 1)), generator=gen, device="cuda")
    index[::7] = -1
    given = torch.randn(rows, max(teacher, 1), generator=gen, device="cuda")
    first, balance = s.step(x, index, given)
    assert balance > 0.9                                # experts * sum f P: 1 where evenly used
    losses = [s.step(x, index, given, rate=10.0)[0].item() for _ in range(12)]
    assert losses[0] == pytest.approx(first.item(), rel=1e-6) and losses[-1] < 0.9 * losses[0]
    assert all(b < a + 1e-3 for a, b in zip(losses, losses[1:]))


def test_sharded_step_gradients():
    """Against autograd in 64 bits, through the router and the head, in fp32."""
    rows, dim, vocab, experts, topk, balance = 40, 24, 90, 5, 2, 0.3
    s = ShardedStep(rows, dim, vocab, shards=2, experts=experts, topk=topk, balance=balance, dtype=F32)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, dim, generator=gen, device="cuda")
    index = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
    index[::6] = -1
    s.step(x, index)
    keep, xd = (index >= 0)[:, 0], x.double()
    head, scale = s.head.double().requires_grad_(), s.scale.double()
    logits = s.logits.double().requires_grad_()
    p = torch.softmax(logits, dim=1)
    weight, choice = p.topk(topk, dim=1)
    weight = weight / weight.sum(dim=1, keepdim=True) * keep[:, None]
    y = xd * (1 + (weight[:, :, None] * scale[choice]).sum(dim=1))
    n = keep.sum()
    f = torch.bincount(choice[keep].flatten(), minlength=experts).double() / (n * topk)
    loss = torch.nn.functional.cross_entropy((y @ head.t())[keep], index[keep, 0]) + \
        balance * experts * (f * p[keep].sum(dim=0) / n).sum()
    loss.backward()
    # a few hundred fp32 roundings along the way
    for got, want in ((s.dlogits, logits.grad), (s.dhead, head.grad)):
        assert (got.double() - want).abs().max() <= 512 * ref.U * want.abs().max()
    assert rr.load() is not None


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,topk", [(2100, 520, 9), (1100, 601, 65)], ids=str)
def test_distill_rows_shared_by_a_workgroup(dt, rows, dim, topk):
    Head(dt, rows, dim, 400, sizes=[150, 250], topk=topk, scale=0.5, distill=True).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("rows,dim,topk,lead", [(40, 64, 1, 0), (40, 64, 3, 0), (40, 65, 1, 0), (60, 72, 5, 1), (1100, 136, 1, 0)],
                         ids=str)
def test_rows_without_a_target_may_hold_anything(dt, bad, rows, dim, topk, lead):
    """Their x takes no part in dw and gets no gradient, whatever it is."""
    h = Head(dt, rows, dim, 13000 if rows > 1000 else 500, topk=topk, scale=0.5 if topk > 1 else 1.0, masked=0.3, lead=lead)
    none = (h.index < 0).all(dim=1)
    assert none.any() and not none.all()
    h.x[none] = 0
    h.make()
    h.issue()
    torch.cuda.synchronize()
    clean = [h.dx[0].t.clone(), h.dw[0].t.clone(), h.loss.t.clone()]
    h.x[none] = bad
    h.make()
    h.issue()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(clean, [h.dx[0].t, h.dw[0].t, h.loss.t]))
    assert not h.dx[0].t[none].any()
