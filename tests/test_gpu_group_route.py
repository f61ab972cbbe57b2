"""Routing in groups on the GPU against its 64-bit form (expert_ref): group and row
layouts, element types, masked tokens and experts, ties, values that are not
finite, the gradient against the formula and against differences, plans, streams
and graphs.  Elements around every output must keep their values."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from tests import expert_ref as ref
from tests.test_gpu_losses import DT, Out, device, normal, said, view, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16


class Route:
    def __init__(self, dt, rows, router, masked=0.2, bias=True, lead=0, seed=0, logits=None):
        gen = torch.Generator(device="cuda").manual_seed(seed + rows + 31 * router.experts + router.topk)
        self.dt, self.rows, self.r, self.lead = dt, rows, router, lead
        e, k = router.experts, router.topk
        self.logits = (2 * normal(gen, rows, e) + normal(gen, e)).to(DT[dt]) if logits is None else logits
        self.bias = 0.3 * normal(gen, e) if bias else None
        self.keep = torch.rand(rows, generator=gen, device="cuda") >= masked if masked > 0 else None
        self.grad_weight = normal(gen, rows, k)
        self.make()

    def make(self):
        rows, e, k = self.rows, self.r.experts, self.r.topk
        self.vl = view(self.logits, self.lead)
        self.choice, self.weight, self.logit = Out(torch.int32, rows, k), Out(torch.float32, rows, k), Out(torch.float32, rows, k)
        self.lse = Out(torch.float32, rows)
        self.counts = Out(torch.int32, e + 1)
        self.dlogits = Out(DT[self.dt], rows, e, lead=self.lead)
        self.work = workspace(rr.rr_group_route_workspace(self.r, rows))

    def issue(self, stream=None):
        r = self.r
        rr.rr_group_route(r, self.dt, self.vl, self.bias, self.keep, self.choice.t, self.weight.t, self.logit.t,
                          None if r.sigmoid else self.lse.t, self.counts.t, workspace=self.work[1], stream=stream)
        rr.rr_group_route_grad(r, self.dt, self.vl if r.whole else None, self.choice.t, self.logit.t,
                               self.lse.t if r.whole else None, self.grad_weight, self.dlogits.t, stream=stream)

    def outs(self):
        return [self.choice, self.weight, self.logit, self.counts, self.dlogits] + ([] if self.r.sigmoid else [self.lse])

    def run(self):
        self.issue()
        torch.cuda.synchronize()
        return self

    def check(self, grad=True):
        want = ref.group_route(self.r, self.logits, self.bias, self.keep)
        assert torch.equal(self.choice.t, want["choice"])
        assert torch.equal(self.counts.t, want["counts"])
        assert torch.equal(self.logit.t, want["logit"])
        w = self.weight.t.double()
        assert ((w - want["weight"]).abs() <= 1.01 * ref.U * want["weight"].abs() + 1e-44).all()
        if not self.r.sigmoid:
            lse = self.lse.t.double()
            assert ((lse == want["lse"]) | ((lse - want["lse"]).abs() <= 1.01 * ref.U * want["lse"].abs() + 1e-14)).all()
        if grad:
            d, tol = ref.group_route_grad(self.r, self.logits, want["choice"], self.grad_weight, DT[self.dt])
            off = (self.dlogits.t.double() - d).abs()
            assert (off <= tol).all(), (off / tol.clamp_min(1e-300)).max().item()
        assert all(o.untouched() for o in self.outs())
        assert (self.work[0][self.work[1].numel():] == 0xFF).all()


def router(experts, topk, groups, top_groups, best, sigmoid, renormalize, scale=1.0):
    return rr.GroupRouter(experts, topk, groups, top_groups, best, sigmoid, renormalize, scale)


SHAPES = [
    (1, 1, 1, 1, 1), (2, 1, 2, 1, 1), (7, 7, 1, 1, 2), (8, 3, 8, 5, 1), (12, 4, 4, 2, 2), (60, 4, 5, 2, 2), (64, 6, 1, 1, 1),
    (64, 9, 8, 3, 2), (128, 8, 16, 4, 2), (160, 6, 8, 3, 1), (256, 8, 8, 4, 2), (256, 32, 4, 2, 2), (257, 5, 1, 1, 1),
    (260, 8, 20, 7, 2), (384, 8, 1, 1, 2), (512, 16, 64, 9, 2), (1023, 8, 33, 4, 2), (1024, 32, 32, 32, 2),
]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("sigmoid,renormalize", [(True, True), (True, False), (False, True), (False, False)])
def test_against_the_definition(dt, shape, sigmoid, renormalize):
    Route(dt, 77, router(*shape, sigmoid, renormalize, 2.5)).run().check()


@pytest.mark.parametrize("rows", [1, 15, 16, 33, 129, 4000])
@pytest.mark.parametrize("dt", [F32, BF16])
def test_rows(dt, rows):
    Route(dt, rows, router(256, 8, 8, 4, 2, True, True)).run().check()
    Route(dt, rows, router(60, 4, 5, 2, 1, False, False), masked=0.0, bias=False).run().check()
    Route(dt, rows, router(300, 10, 3, 2, 2, True, True)).run().check()


def test_no_rows():
    for r in (router(16, 2, 4, 2, 2, True, True), router(16, 2, 4, 2, 2, False, False)):
        x = Route(F32, 0, r, masked=0.0).run()
        assert not x.counts.t.any() and all(o.untouched() for o in x.outs())


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lead", [1, 3])
def test_unaligned(dt, lead):
    Route(dt, 50, router(256, 8, 8, 4, 2, True, True), lead=lead).run().check()
    Route(dt, 50, router(36, 4, 3, 2, 1, False, False), lead=lead).run().check()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_all_left_out(dt):
    x = Route(dt, 40, router(64, 4, 8, 2, 2, False, False), masked=1.5).run()
    x.check()
    assert (x.choice.t == -1).all() and not x.counts.t.any() and not x.dlogits.t.any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_equal_scores(dt, sigmoid):
    """Ties go to the lower index, of groups and of experts."""
    logits = torch.zeros(20, 64, device="cuda").to(DT[dt])
    logits[5:, 40:44] = 1.0
    logits[10:, 8] = 1.0
    x = Route(dt, 20, router(64, 6, 8, 3, 2, sigmoid, True), masked=0.0, bias=False, logits=logits).run()
    x.check()
    assert x.choice.t[0].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("sigmoid,renormalize", [(True, True), (True, False), (False, True), (False, False)])
def test_experts_taken_out(dt, sigmoid, renormalize):
    """A bias of -inf: never chosen, and places that nothing else is left for hold -1."""
    r = router(24, 6, 4, 2, 2, sigmoid, renormalize)
    x = Route(dt, 30, r, masked=0.1)
    x.bias[0:11] = -math.inf
    x.run().check()
    x.bias[:] = -math.inf
    x.bias[13] = 0.0
    x.run().check()
    kept = x.keep
    assert (x.choice.t[kept][:, 0] == 13).all() and (x.choice.t[:, 1:] == -1).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_masked_logits(dt, sigmoid):
    """Logits of -inf have s = 0; a row of them has weights of 0 and no gradient."""
    x = Route(dt, 30, router(32, 4, 4, 2, 2, sigmoid, True), masked=0.0, bias=False)
    x.logits[:, 3:20] = -math.inf
    x.logits[7] = -math.inf
    x.make()
    x.run().check(grad=False)
    assert not x.weight.t[7].any() and not x.dlogits.t[7].any()
    assert torch.isfinite(x.dlogits.t.float()).all()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_extreme_logits(dt):
    """Scores next to 0 keep their quotients, next to 1 their distance from it."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    low = (normal(gen, 20, 32) * 4 - 150).to(DT[dt])
    # scores of e^-150 are equal as choice scores once a bias is added; without one they are not
    Route(dt, 20, router(32, 4, 1, 1, 1, True, True), masked=0.0, bias=False, logits=low).run().check()
    high = (normal(gen, 20, 32) + 12).to(DT[dt])
    Route(dt, 20, router(32, 4, 1, 1, 1, True, False), masked=0.0, bias=False, logits=high).run().check()
    Route(dt, 20, router(32, 4, 1, 1, 1, False, False), masked=0.0, bias=False, logits=low).run().check()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_not_a_number(dt):
    """NaN comes before every number and reaches only its own row."""
    x = Route(dt, 12, router(32, 4, 4, 2, 2, True, False), masked=0.0)
    x.logits[3, 17] = math.nan
    x.make()
    x.run()
    assert x.choice.t[3, 0] == 17 and torch.isnan(x.weight.t[3, 0]) and not torch.isnan(x.weight.t[3, 1:]).any()
    want = ref.group_route(x.r, x.logits, x.bias, None)
    assert torch.equal(x.choice.t, want["choice"])
    rest = [i for i in range(12) if i != 3]
    assert torch.isfinite(x.dlogits.t.float()[rest]).all()


@pytest.mark.parametrize("sigmoid,renormalize", [(True, True), (True, False), (False, True), (False, False)])
def test_gradient_by_differences(sigmoid, renormalize):
    """The slope of sum grad_weight * weight along a direction, of rows whose choice stays."""
    r = router(40, 5, 4, 2, 2, sigmoid, renormalize, 1.5)
    x = Route(F32, 60, r, masked=0.1).run()
    gen = torch.Generator(device="cuda").manual_seed(9)
    d, step = normal(gen, 60, 40), 2.0 ** -8
    base, grad, choice, sides = x.logits.clone(), x.dlogits.t.double().clone(), x.choice.t.clone(), []
    same = torch.ones(60, dtype=torch.bool, device="cuda")
    for sign in (1, -1):
        x.logits = base + sign * step * d
        x.make()
        x.run()
        same &= (x.choice.t == choice).all(dim=1)
        sides.append((x.weight.t.double() * x.grad_weight.double()).sum(dim=1))
    assert same.sum() > 20
    slope, want = ((sides[0] - sides[1]) / (2 * step))[same], (grad * d.double()).sum(dim=1)[same]
    # weights' roundings over the step, and the third derivative's share: |d|^3 step^2 of a smooth
    # function of slopes below 1.5 * 5 * |g|
    mag = 1.5 * 5 * x.grad_weight.double().abs().amax(dim=1)[same] * (1 + d.double().abs().amax(dim=1)[same]) ** 3
    assert ((slope - want).abs() <= mag * (ref.U * 2 / step + step ** 2)).all()


@pytest.mark.parametrize("ranks", [1, 3, 16])
@pytest.mark.parametrize("experts", [1, 7, 256, 1024])
def test_bias(ranks, experts):
    gen = torch.Generator(device="cuda").manual_seed(ranks + experts)
    r = router(experts, 1, 1, 1, 1, True, True)
    counts = [torch.randint(0, 50, (experts + 1,), generator=gen, device="cuda").to(torch.int32) for _ in range(ranks)]
    bias, out = normal(gen, experts), Out(torch.float32, experts)
    rr.rr_route_bias(r, counts, 0.125, bias, out.t)
    n = sum(c[:experts].double() for c in counts)
    want = bias + 0.125 * torch.sign(n.sum() - n * experts).float()
    torch.cuda.synchronize()
    assert torch.equal(out.t, want) and out.untouched()
    rr.rr_route_bias(r, counts, 0.125, bias, bias)
    torch.cuda.synchronize()
    assert torch.equal(bias, want)


@pytest.mark.parametrize("rows", [3, 900])
def test_plan_graph_and_streams(rows):
    x = Route(BF16, rows, router(256, 8, 8, 4, 2, False, False)).run()
    first = [o.t.clone() for o in x.outs()]
    with rr.Plan(8) as plan:
        x.issue()

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, o.t) for a, o in zip(first, x.outs()))

    def clear():
        for o in x.outs():
            o.t.fill_(0)

    clear()
    plan()
    assert same()
    s = torch.cuda.Stream()
    clear()
    s.wait_stream(torch.cuda.current_stream())
    x.issue(stream=s)
    s.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan()
    for _ in range(3):
        clear()
        g.replay()
        assert same()
        clear()
        x.issue()
        assert same()
