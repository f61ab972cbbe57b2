"""The expert layer on the GPU against its 64-bit forms (expert_ref): slots, matrices
in 8 bits, products over segments from one choice to many, their gradients, the
sums back to rows, and a whole layer.  Elements around every output, and positions
without a choice, must keep their values."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from tests import expert_ref as ref
from tests.test_gpu_losses import DT, Out, device, normal, said, view, workspace  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16
MARK = 0x5A
Out.marker.setdefault(torch.float8_e4m3fn, 1.25)


def choices(e, total=None, masked=0.0, skew=0.0, seed=0):
    """Distinct choices of each row among `total` experts, popular ones first with `skew`."""
    gen = torch.Generator(device="cuda").manual_seed(seed + e.rows * 7 + e.experts)
    total = e.experts if total is None else total
    key = torch.rand(e.rows, total, generator=gen, device="cuda") - skew * torch.arange(total, device="cuda") / total
    c = key.topk(e.topk, dim=1)[1].to(torch.int32) if e.rows else torch.empty(0, e.topk, dtype=torch.int32, device="cuda")
    c[torch.rand(e.rows, e.topk, generator=gen, device="cuda") < masked] = -1
    return c.contiguous()


class Slots:
    """The slots of choices, checked against their definition."""

    def __init__(self, e, choice, check=True):
        self.e, self.choice, self.n = e, choice, rr.rr_expert_capacity(e)
        self.outs = [Out(torch.int32, *s) for s in ((e.rows, e.topk), (self.n,), (e.experts + 1,), (e.experts,))]
        self.place = rr.Slots(*(o.t for o in self.outs))
        self.work = workspace(rr.rr_expert_workspace(e))
        rr.rr_expert_slots(e, choice, self.place, workspace=self.work[1])
        torch.cuda.synchronize()
        assert all(o.untouched() for o in self.outs) and (self.work[0][self.work[1].numel():] == 0xFF).all()
        if check:
            slot, source, offset, count = ref.slots(e, choice, self.n)
            assert self.place.count.tolist() == count and self.place.offset.tolist() == offset
            assert self.place.slot.flatten().tolist() == slot and self.place.source.tolist() == source

    def positions(self, i):
        """Positions and choices of expert i."""
        lo, n = self.place.offset[i].item(), self.place.count[i].item()
        return slice(lo, lo + n), self.place.source[lo:lo + n].long()


@pytest.mark.parametrize("rows,topk,experts,masked,skew", [
    (0, 1, 4, 0, 0), (1, 1, 1, 0, 0), (1, 8, 64, 0, 0), (3, 2, 2, 0.5, 0), (64, 1, 3, 0, 0), (65, 4, 100, 0.1, 0), (300, 3, 7, 0, 1),
    (1000, 8, 1024, 0.3, 0), (1024, 8, 64, 0, 0), (1025, 8, 64, 0, 0), (2500, 4, 256, 0.2, 2), (20000, 2, 5, 0, 0), (513, 32, 1000, 0, 0.5)])
def test_slots(rows, topk, experts, masked, skew):
    e = rr.Experts(experts, topk, rows)
    Slots(e, choices(e, masked=masked, skew=skew))


def test_slots_of_a_rank():
    """Experts [first, first + experts) of 40; other choices are not its own, whatever they are."""
    for first, rows in ((0, 50), (8, 3000), (39, 5)):
        e = rr.Experts(min(8, 40 - first), 4, rows, first)
        c = choices(e, total=40)
        c[:, 0][:3] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 1 << 20], dtype=torch.int32, device="cuda")
        Slots(e, c)


def test_slots_same_expert_twice():
    """Nothing asks a row's choices to be distinct."""
    e = rr.Experts(4, 3, 200)
    Slots(e, torch.ones(200, 3, dtype=torch.int32, device="cuda"))


# --------------------------------------------------------------------------
# eight bits
# --------------------------------------------------------------------------

class Eight:
    """A Quantized or QuantizedWeight whose memory is marked."""

    def __init__(self, q):
        self.q = q
        self.outs = []
        for name in ("values", "powers"):
            t = getattr(q, name)
            big = torch.full((t.numel() + 128,), MARK, dtype=torch.uint8, device="cuda")
            setattr(q, name, big[64:64 + t.numel()].view(t.dtype).view(t.shape))
            self.outs.append(big)

    def untouched(self):
        return all((b[:64] == MARK).all() and (b[len(b) - 64:] == MARK).all() for b in self.outs)


def spread(gen, dt, *shape):
    """Normal values over many powers of two, with zeros, ties of the rounding, and whole blocks of zeros."""
    x = normal(gen, *shape) * torch.exp2(torch.randint(-12, 13, shape, generator=gen, device="cuda").float())
    x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.1, torch.zeros_like(x), x)
    tie = (torch.randint(8, 16, shape, generator=gen, device="cuda") + 0.5) * torch.exp2(torch.randint(-9, 5, shape, generator=gen, device="cuda").float())
    x = torch.where(torch.rand(shape, generator=gen, device="cuda") < 0.2, tie, x)
    x[..., :1, :] = 0.0
    return x.to(DT[dt])


def same(q, powers, n, want, byte):
    """The values that a Quantized stands for and its powers are the definition's, zeros past n."""
    got = ref.values(q, powers, n)
    assert torch.equal(powers[:, :byte.shape[1]], byte)
    assert torch.equal(torch.nan_to_num(got, 123456.0), torch.nan_to_num(want, 123456.0))
    tail = q.view(torch.uint8)[:, n:].reshape(q.shape[0], -1)
    # a block that is not finite is NaN to its end
    assert ((tail & 0x7F) == 0).all() or torch.isnan(want).any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim", [(1, 1), (1, 128), (3, 127), (5, 130), (17, 1000), (33, 512), (200, 2056), (2, 65536)])
@pytest.mark.parametrize("lead", [0, 1])
def test_quantize_rows(dt, rows, dim, lead):
    gen = torch.Generator(device="cuda").manual_seed(rows + dim)
    x = spread(gen, dt, rows, dim)
    q = Eight(rr.Quantized(rows, dim))
    rr.rr_quantize_rows(dt, view(x, lead), q.q)
    torch.cuda.synchronize()
    same(q.q.values, q.q.powers, dim, *ref.eight(x))
    assert q.untouched()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_quantize_borders(dt):
    """Largest magnitudes next to the borders of the powers, from the least numbers to the largest, and values
    that are not finite."""
    tops = []
    for e in (-126, -120, -119, -118, -60, -1, 0, 1, 8, 9, 60, 126, 127):
        for m in (1.0, 1.5, 1.75, 1.75 + 2.0 ** -7, 1.9921875):
            tops.append(m * 2.0 ** e if m * 2.0 ** e < 3.4e38 else 3.38e38)
    tops += [0.0, 2.0 ** -133, 2.0 ** -130, math.inf, math.nan, -math.inf]
    x = torch.zeros(len(tops), 130, device="cuda")
    x[:, 7] = torch.tensor(tops, device="cuda")
    x[:, 8] = x[:, 7] * 0.37
    x[:, 9] = -x[:, 7] * 2.0 ** -15
    x[:, 129] = 1.0                                                # the next block is finite
    x = x.to(DT[dt])
    q = Eight(rr.Quantized(len(tops), 130))
    rr.rr_quantize_rows(dt, x, q.q)
    torch.cuda.synchronize()
    same(q.q.values, q.q.powers, 130, *ref.eight(x))


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("experts,n,k", [(1, 1, 1), (2, 128, 128), (3, 130, 64), (1, 100, 300), (4, 257, 520), (2, 64, 1000)])
def test_quantize_weight(dt, experts, n, k):
    gen = torch.Generator(device="cuda").manual_seed(n + k)
    w = spread(gen, dt, experts, n, k)
    q, t = Eight(rr.QuantizedWeight(experts, n, k)), Eight(rr.QuantizedWeight(experts, k, n))
    rr.rr_quantize_weight(dt, view(w, 0), q.q, t.q)
    alone = Eight(rr.QuantizedWeight(experts, n, k))
    rr.rr_quantize_weight(dt, view(w, 1), alone.q)
    torch.cuda.synchronize()
    assert torch.equal(alone.q.values.view(torch.uint8), q.q.values.view(torch.uint8))
    for i in range(experts):
        want, byte = ref.eight(w[i], 128)
        same(q.q.values[i], q.q.powers[i].repeat_interleave(128, dim=0)[:n], k, want, byte.repeat_interleave(128, dim=0)[:n])
        same(t.q.values[i], t.q.powers[i].repeat_interleave(128, dim=0)[:k], n, want.t().contiguous(),
             byte.t().contiguous().repeat_interleave(128, dim=0)[:k])
    assert q.untouched() and t.untouched() and alone.untouched()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,topk,experts,dim", [(1, 1, 1, 1), (40, 2, 3, 64), (300, 3, 5, 130), (129, 1, 1, 520)])
@pytest.mark.parametrize("weighted", [False, True])
def test_quantize_slots(dt, rows, topk, experts, dim, weighted):
    gen = torch.Generator(device="cuda").manual_seed(rows + dim)
    e = rr.Experts(experts, topk, rows)
    s = Slots(e, choices(e, masked=0.1))
    x = spread(gen, dt, rows, dim)
    weight = normal(gen, rows, topk) if weighted else None
    src = s.place.source.long()
    live = src >= 0
    by = torch.ones(s.n, device="cuda") if weight is None else torch.where(live, weight.flatten()[src.clamp_min(0)], 0.0)
    of = torch.where(live[:, None], x.float()[src.clamp_min(0) // topk] * by[:, None], 0.0)
    end = s.place.offset[experts].item()
    want, byte = ref.eight(of.t().contiguous())
    in_order = torch.full((s.n, dim), math.nan, device="cuda").to(DT[dt])      # what no choice has may hold anything
    in_order[live] = x[src[live] // topk]
    for gather, given in ((True, x), (False, in_order)):
        q = Eight(rr.Quantized(dim, s.n))
        rr.rr_quantize_slots(e, dt, s.place, given, q.q, weight=weight, gather=gather)
        torch.cuda.synchronize()
        same(q.q.values[:, :end].contiguous(), q.q.powers, end, want[:, :end], byte[:, :end // 128])
        assert (q.q.values.view(torch.uint8)[:, end:] == MARK).all() and q.untouched()


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------

class Layer:
    """A layer's inputs in 8 bits."""

    def __init__(self, rows, topk, experts, dim, out, masked=0.1, skew=0.0, check=True, first=0, total=None, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed + rows + dim)
        self.e = e = rr.Experts(experts, topk, rows, first)
        self.s = Slots(e, choices(e, total=total, masked=masked, skew=skew), check)
        self.x, self.dy = spread(gen, BF16, rows, dim), spread(gen, BF16, rows, out)
        self.w = (normal(gen, experts, out, dim) * dim ** -0.5).bfloat16()
        self.weight = normal(gen, rows, topk)
        self.xq, self.wq, self.wt = rr.Quantized(rows, dim), rr.QuantizedWeight(experts, out, dim), rr.QuantizedWeight(experts, dim, out)
        rr.rr_quantize_rows(BF16, self.x, self.xq)
        rr.rr_quantize_weight(BF16, self.w, self.wq, self.wt)

    def x_of(self, n):
        return ref.values(self.xq.values, self.xq.powers, self.x.shape[1])[n // self.e.topk]

    def w_of(self, i):
        n, k = self.w.shape[1:]
        return ref.values(self.wq.values[i], self.wq.powers[i].repeat_interleave(128, dim=0)[:n], k)


def check_product(l, dt, gather=True, weighted=False):
    e, s, out = l.e, l.s, l.w.shape[1]
    x, rows = l.xq, e.rows
    if not gather:
        # the same rows in the order of the positions; what no choice has may hold anything
        x = rr.Quantized(s.n, l.x.shape[1])
        x.values.view(torch.uint8).fill_(0x7F)
        x.powers.fill_(255)
        src = s.place.source.long()
        x.values.view(torch.uint8)[src >= 0] = l.xq.values.view(torch.uint8)[src[src >= 0] // e.topk]
        x.powers[src >= 0] = l.xq.powers[src[src >= 0] // e.topk]
    held = Out(DT[dt], s.n, out)
    rr.rr_expert_product(e, dt, s.place, x, l.wq, held.t, weight=l.weight if weighted else None, gather=gather)
    torch.cuda.synchronize()
    for i in range(e.experts):
        at, n = s.positions(i)
        xd, wd = l.x_of(n), l.w_of(i)
        by = l.weight.flatten()[n].double()[:, None] if weighted else torch.ones(len(n), 1, dtype=torch.float64, device="cuda")
        want = by * (xd @ wd.t())
        off = (held.t[at].double() - want).abs()
        assert (off <= ref.product_bound(xd, wd, want, DT[dt], by.abs())).all(), (i, len(n))
    assert (held.t[s.place.source < 0] == -7.25).all() and held.untouched()


SIZES = [(1, 1, 1, 1, 1), (1, 8, 9, 64, 40), (2, 4, 64, 128, 33), (3, 8, 64, 200, 129), (25, 3, 3, 1024, 64), (70, 4, 8, 257, 96),
         (90, 2, 4, 384, 130), (300, 4, 8, 256, 300), (700, 2, 4, 640, 257), (999, 3, 7, 1000, 520), (600, 1, 1, 129, 700),
         (2000, 2, 3, 2048, 264)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_product(dt, size):
    l = Layer(*size)
    check_product(l, dt)
    check_product(l, dt, gather=False)
    check_product(l, dt, weighted=True)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_product_uneven(dt):
    """Every choice the same expert's, and experts without any."""
    l = Layer(300, 1, 40, 256, 136, masked=0.0, skew=100.0)
    assert (l.s.place.count > 0).sum() == 1
    check_product(l, dt)
    l = Layer(700, 1, 5, 256, 136, masked=0.5, skew=3.0)
    check_product(l, dt)
    l = Layer(40, 2, 6, 256, 136, masked=1.5)
    assert not l.s.place.count.any()
    check_product(l, dt)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_product_many_experts(dt):
    check_product(Layer(400, 6, 500, 128, 72, masked=0.0), dt)
    check_product(Layer(9, 3, 1024, 128, 72, masked=0.0), dt)
    check_product(Layer(500, 4, 10, 128, 72, first=20, total=64), dt)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_product_not_finite(dt):
    """A block that is not finite makes its row's outputs NaN and no others; so does one of the weights."""
    for rows in (6, 900):
        l = Layer(rows, 1, 2, 256, 200, masked=0.0)
        l.x[3, 5] = math.inf
        rr.rr_quantize_rows(BF16, l.x, l.xq)
        held = torch.empty(l.s.n, 200, dtype=DT[dt], device="cuda")
        rr.rr_expert_product(l.e, dt, l.s.place, l.xq, l.wq, held, gather=True)
        torch.cuda.synchronize()
        src = l.s.place.source
        assert torch.isnan(held[src == 3]).all() and torch.isfinite(held[(src >= 0) & (src != 3)]).all()
        l.x[3, 5] = 1.0
        l.w[1, 190, 3] = math.nan
        rr.rr_quantize_rows(BF16, l.x, l.xq)
        rr.rr_quantize_weight(BF16, l.w, l.wq)
        rr.rr_expert_product(l.e, dt, l.s.place, l.xq, l.wq, held, gather=True)
        torch.cuda.synchronize()
        at, _ = l.s.positions(1)
        assert torch.isnan(held[at][:, 128:]).all() and torch.isfinite(held[at][:, :128]).all()
        at, _ = l.s.positions(0)
        assert torch.isfinite(held[at]).all()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("size", [(1, 1, 1, 1, 1), (5, 2, 3, 64, 40), (130, 1, 1, 100, 300), (300, 3, 5, 256, 257), (999, 3, 7, 1000, 520),
                                  (1500, 2, 16, 512, 640), (4000, 4, 8, 2048, 1024)], ids=str)
def test_weight_grad(dt, size):
    l = Layer(*size, skew=0.5)
    e, s = l.e, l.s
    out, dim = l.w.shape[1:]
    xt, dyt = rr.Quantized(dim, s.n), rr.Quantized(out, s.n)
    # what lies behind the segments may be anything
    for q in (xt, dyt):
        q.values.view(torch.uint8).fill_(0x7F)
        q.powers.fill_(255)
    rr.rr_quantize_slots(e, BF16, s.place, l.x, xt, gather=True)
    rr.rr_quantize_slots(e, BF16, s.place, l.dy, dyt, weight=l.weight, gather=True)
    dw = Out(DT[dt], e.experts, out, dim)
    rr.rr_expert_weight_grad(e, dt, s.place, dyt, xt, dw.t)
    torch.cuda.synchronize()
    xv, dv = ref.values(xt.values, xt.powers, s.n), ref.values(dyt.values, dyt.powers, s.n)
    for i in range(e.experts):
        lo, hi = s.place.offset[i].item(), s.place.offset[i + 1].item()
        a, b = dv[:, lo:hi], xv[:, lo:hi]
        want = a @ b.t()
        off = (dw.t[i].double() - want).abs()
        assert (off <= ref.product_bound(a, b, want, DT[dt])).all(), i
    assert dw.untouched()


def test_whole_numbers():
    """Small whole numbers lose nothing in 8 bits nor in sums of 32: every result is exact, and as the layer is
    linear so are its differences."""
    rows, topk, experts, dim, out = 600, 2, 3, 200, 150
    gen = torch.Generator(device="cuda").manual_seed(4)

    def whole(*shape):
        return torch.randint(-4, 5, shape, generator=gen, device="cuda").float()

    e = rr.Experts(experts, topk, rows)
    s = Slots(e, choices(e, masked=0.1))
    x, d, w, dy, weight = whole(rows, dim), whole(rows, dim), whole(experts, out, dim), whole(rows, out), whole(rows, topk) * 0.5
    live = s.choice >= 0
    wq, wt = rr.QuantizedWeight(experts, out, dim), rr.QuantizedWeight(experts, dim, out)
    rr.rr_quantize_weight(F32, w, wq, wt)

    def forward(x, weight):
        q, held, y = rr.Quantized(rows, dim), torch.empty(s.n, out, device="cuda"), torch.empty(rows, out, device="cuda")
        rr.rr_quantize_rows(F32, x, q)
        rr.rr_expert_product(e, F32, s.place, q, wq, held, gather=True)
        rr.rr_expert_combine(e, F32, F32, s.place, held, weight, y)
        return y, held

    def plain(x, weight):
        y = torch.zeros(rows, out, device="cuda", dtype=torch.float64)
        for k in range(topk):
            of = torch.einsum("rd,rod->ro", x.double(), w.double()[s.choice[:, k].long().clamp_min(0)])
            y += torch.where(live[:, k], weight[:, k], 0.0)[:, None].double() * of
        return y

    y, held = forward(x, weight)
    assert torch.equal(y.double(), plain(x, weight))
    # the gradients
    dyq, xt, dyt = rr.Quantized(rows, out), rr.Quantized(dim, s.n), rr.Quantized(out, s.n)
    held_dx, dx, dw, dweight = (torch.empty(*n, device="cuda") for n in ((s.n, dim), (rows, dim), (experts, out, dim), (rows, topk)))
    rr.rr_expert_combine_grad(e, F32, F32, s.place, held, dy, dweight)
    rr.rr_quantize_rows(F32, dy, dyq)
    rr.rr_expert_product(e, F32, s.place, dyq, wt, held_dx, weight=weight, gather=True)
    rr.rr_expert_combine(e, F32, F32, s.place, held_dx, None, dx)
    rr.rr_quantize_slots(e, F32, s.place, x, xt, gather=True)
    rr.rr_quantize_slots(e, F32, s.place, dy, dyt, weight=weight, gather=True)
    rr.rr_expert_weight_grad(e, F32, s.place, dyt, xt, dw)
    torch.cuda.synchronize()
    # in x, in a router's weights and in the experts' weights: sums and differences are whole
    up, down = forward(d, weight)[0], forward(-d, weight)[0]
    assert ((up - down).double() * dy.double()).sum().item() == 2 * (dx.double() * d.double()).sum().item()
    turn = whole(rows, topk)
    assert (forward(x, turn)[0].double() * dy.double()).sum().item() == (torch.where(live, dweight, 0.0).double() * turn.double()).sum().item()
    assert not dweight[~live].any()
    step = whole(experts, out, dim)
    w = step
    rr.rr_quantize_weight(F32, w, wq)
    assert (forward(x, weight)[0].double() * dy.double()).sum().item() == (dw.double() * step.double()).sum().item()


# --------------------------------------------------------------------------
# rows of sums
# --------------------------------------------------------------------------

@pytest.mark.parametrize("vt,dt", [(F32, F32), (F32, BF16), (BF16, BF16), (BF16, F32)])
@pytest.mark.parametrize("rows,topk,dim,lead", [(1, 1, 1, 0), (5, 3, 100, 0), (50, 8, 520, 0), (33, 32, 1001, 0), (20, 9, 64, 1), (7, 2, 4096, 3)])
def test_combine(vt, dt, rows, topk, dim, lead):
    gen = torch.Generator(device="cuda").manual_seed(rows + dim)
    e = rr.Experts(40, topk, rows)
    s = Slots(e, choices(e, masked=0.2))
    values = torch.full((s.n, dim), math.nan, device="cuda")
    live = s.place.source >= 0
    values[live] = normal(gen, int(live.sum()), dim)
    values = values.to(DT[vt])
    weight, dy = normal(gen, rows, topk), normal(gen, rows, dim).to(DT[dt])
    v, here = view(values, lead), s.place.slot >= 0
    of = torch.where(here[:, :, None], values.double()[s.place.slot.long().clamp_min(0)], 0.0)
    for by in (weight, None):
        y = Out(DT[dt], rows, dim, lead=lead)
        rr.rr_expert_combine(e, vt, dt, s.place, v, by, y.t)
        torch.cuda.synchronize()
        terms = of * (1.0 if by is None else by.double()[:, :, None])
        want = terms.sum(dim=1)
        tol = (topk + 2) * ref.U * terms.abs().sum(dim=1) + (ref.HALF[DT[dt]] + ref.U) * want.abs()
        assert ((y.t.double() - want).abs() <= tol).all() and y.untouched()
    g = Out(torch.float32, rows, topk)
    rr.rr_expert_combine_grad(e, vt, dt, s.place, v, view(dy, lead), g.t)
    torch.cuda.synchronize()
    terms = of * dy.double()[:, None, :]
    assert ((g.t.double() - terms.sum(dim=2)).abs() <= (dim + 8) * ref.U * terms.abs().sum(dim=2)).all()
    assert not g.t[~here].any() and g.untouched()


# --------------------------------------------------------------------------
# together
# --------------------------------------------------------------------------

class Step:
    """Two layers of experts between a router in groups and a loss, forward and back, recorded."""

    def __init__(self, dt, rows, experts, topk, dim, hidden, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        t, f = DT[dt], torch.float32
        self.dt, self.rows = dt, rows
        self.r = rr.GroupRouter(experts, topk, 2, 1, 2, True, True, 1.5)
        self.e = e = rr.Experts(experts, topk, rows)
        n = rr.rr_expert_capacity(e)

        def empty(d, *shape):
            return torch.empty(*shape, dtype=d, device="cuda")

        self.x, self.dy = normal(gen, rows, dim).to(t), normal(gen, rows, dim).to(t)
        self.logits, self.bias = normal(gen, rows, experts).to(t), 0.1 * normal(gen, experts)
        self.w1 = (normal(gen, experts, hidden, dim) * dim ** -0.5).to(t)
        self.w2 = (normal(gen, experts, dim, hidden) * hidden ** -0.5).to(t)
        self.choice, self.weight, self.logit = empty(torch.int32, rows, topk), empty(f, rows, topk), empty(f, rows, topk)
        self.counts, self.place = empty(torch.int32, experts + 1), rr.Slots.empty(e)
        self.held1, self.held2, self.y = empty(t, n, hidden), empty(f, n, dim), empty(t, rows, dim)
        self.dweight, self.dlogits, self.dx = empty(f, rows, topk), empty(t, rows, experts), empty(t, rows, dim)
        self.dheld1, self.dheld0 = empty(t, n, hidden), empty(t, n, dim)
        self.dw1, self.dw2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.out1, self.out2 = torch.empty_like(self.w1), torch.empty_like(self.w2)
        self.total, self.norm = empty(torch.float64, 1), empty(f, 1)
        self.q = [rr.Quantized(rows, dim), rr.Quantized(n, hidden), rr.Quantized(rows, dim), rr.Quantized(n, hidden)]
        self.qt = [rr.Quantized(dim, n), rr.Quantized(hidden, n), rr.Quantized(dim, n), rr.Quantized(hidden, n)]
        self.wq = [rr.QuantizedWeight(experts, hidden, dim), rr.QuantizedWeight(experts, dim, hidden)]
        self.wt = [rr.QuantizedWeight(experts, dim, hidden), rr.QuantizedWeight(experts, hidden, dim)]
        self.work = workspace(max(rr.rr_group_route_workspace(self.r, rows), rr.rr_expert_workspace(e),
                                  rr.rr_grad_workspace(dt, [self.dw1, self.dw2])))[1]

    def issue(self, stream=None):
        dt, e, p, k = self.dt, self.e, self.place, {"stream": stream}
        rr.rr_group_route(self.r, dt, self.logits, self.bias, None, self.choice, self.weight, self.logit, None, self.counts,
                          workspace=self.work, **k)
        rr.rr_expert_slots(e, self.choice, p, workspace=self.work, **k)
        rr.rr_quantize_weight(dt, self.w1, self.wq[0], self.wt[0], **k)
        rr.rr_quantize_weight(dt, self.w2, self.wq[1], self.wt[1], **k)
        rr.rr_quantize_rows(dt, self.x, self.q[0], **k)
        rr.rr_expert_product(e, dt, p, self.q[0], self.wq[0], self.held1, gather=True, **k)
        rr.rr_quantize_rows(dt, self.held1, self.q[1], **k)
        rr.rr_expert_product(e, F32, p, self.q[1], self.wq[1], self.held2, **k)
        rr.rr_expert_combine(e, F32, dt, p, self.held2, self.weight, self.y, **k)
        # back
        rr.rr_expert_combine_grad(e, F32, dt, p, self.held2, self.dy, self.dweight, **k)
        rr.rr_group_route_grad(self.r, dt, None, self.choice, self.logit, None, self.dweight, self.dlogits, **k)
        rr.rr_quantize_rows(dt, self.dy, self.q[2], **k)
        rr.rr_expert_product(e, dt, p, self.q[2], self.wt[1], self.dheld1, weight=self.weight, gather=True, **k)
        rr.rr_quantize_rows(dt, self.dheld1, self.q[3], **k)
        rr.rr_expert_product(e, dt, p, self.q[3], self.wt[0], self.dheld0, **k)
        rr.rr_expert_combine(e, dt, dt, p, self.dheld0, None, self.dx, **k)
        rr.rr_quantize_slots(e, dt, p, self.x, self.qt[0], gather=True, **k)
        rr.rr_quantize_slots(e, dt, p, self.held1, self.qt[1], **k)
        rr.rr_quantize_slots(e, dt, p, self.dy, self.qt[2], weight=self.weight, gather=True, **k)
        rr.rr_quantize_slots(e, dt, p, self.dheld1, self.qt[3], **k)
        rr.rr_expert_weight_grad(e, dt, p, self.qt[3], self.qt[0], self.dw1, **k)
        rr.rr_expert_weight_grad(e, dt, p, self.qt[2], self.qt[1], self.dw2, **k)
        rr.rr_grad_square_sum(dt, [self.dw1, self.dw2], self.total, workspace=self.work, **k)
        rr.rr_grad_clip(dt, [self.total], 1.0, [self.dw1, self.dw2], [self.out1, self.out2], self.norm, **k)

    def outs(self):
        return [self.y, self.dx, self.dw1, self.dw2, self.dweight, self.dlogits, self.out1, self.out2, self.norm, self.total,
                self.counts, self.choice]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,experts,topk,dim,hidden", [(7, 6, 2, 100, 72), (500, 8, 3, 264, 520)])
def test_together(dt, rows, experts, topk, dim, hidden):
    """Every stage from the stage before it, against 64 bits."""
    st = Step(dt, rows, experts, topk, dim, hidden)
    st.issue()
    torch.cuda.synchronize()
    e, p, t = st.e, st.place, DT[dt]
    slot, source, offset, count = ref.slots(e, st.choice, rr.rr_expert_capacity(e))
    assert p.source.tolist() == source
    src = torch.tensor(source, device="cuda")
    weight = st.weight.flatten()
    x8, dy8 = ref.eight(st.x)[0], ref.eight(st.dy)[0]
    y, dx, size_y, size_dx = (torch.zeros(rows, dim, dtype=torch.float64, device="cuda") for _ in range(4))
    g = torch.zeros(rows * topk, dtype=torch.float64, device="cuda")
    for i in range(experts):
        at = slice(offset[i], offset[i] + count[i])
        n = src[at].long()
        of, by = n // topk, weight[n].double()[:, None]
        w1, w2 = ref.eight(st.w1[i], 128)[0], ref.eight(st.w2[i], 128)[0]
        h = x8[of] @ w1.t()
        assert ((st.held1[at].double() - h).abs() <= ref.product_bound(x8[of], w1, h, t)).all()
        h8 = ref.eight(st.held1[at])[0]
        o = h8 @ w2.t()
        assert ((st.held2[at].double() - o).abs() <= ref.product_bound(h8, w2, o, torch.float32)).all()
        y.index_add_(0, of, by * st.held2[at].double())
        size_y.index_add_(0, of, (by * st.held2[at].double()).abs())
        g[n] = (st.held2[at].double() * st.dy[of].double()).sum(dim=1)
        dh = by * (dy8[of] @ w2)
        assert ((st.dheld1[at].double() - dh).abs() <= ref.product_bound(dy8[of], w2.t().contiguous(), dh, t, by.abs())).all()
        dh8 = ref.eight(st.dheld1[at])[0]
        d0 = dh8 @ w1
        assert ((st.dheld0[at].double() - d0).abs() <= ref.product_bound(dh8, w1.t().contiguous(), d0, t)).all()
        dx.index_add_(0, of, st.dheld0[at].double())
        size_dx.index_add_(0, of, st.dheld0[at].double().abs())
        for dw, a, b in ((st.dw1[i], st.dheld1[at], st.x[of]), (st.dw2[i], weight[n, None] * st.dy.float()[of], st.held1[at])):
            a, b = ref.eight(a.t().contiguous())[0], ref.eight(b.t().contiguous())[0]
            want = a @ b.t()
            assert ((dw.double() - want).abs() <= ref.product_bound(a, b, want, t)).all()
    h = ref.HALF[t]
    assert ((st.y.double() - y).abs() <= (topk + 2) * ref.U * size_y + (h + ref.U) * y.abs()).all()
    assert ((st.dx.double() - dx).abs() <= (topk + 2) * ref.U * size_dx + (h + ref.U) * dx.abs()).all()
    size_g = (dim + 8) * ref.U * (st.held2.double()[p.slot.long()].abs() * st.dy.double().abs()[:, None, :]).sum(dim=2)
    assert ((st.dweight.double() - g.reshape(rows, topk)).abs() <= size_g).all()
    d, tol = ref.group_route_grad(st.r, st.logits, st.choice, st.dweight, t)
    assert ((st.dlogits.double() - d).abs() <= tol).all()
    total = (st.dw1.double() ** 2).sum() + (st.dw2.double() ** 2).sum()
    assert abs(st.total.item() - total.item()) <= 1e-12 * total.item()


@pytest.mark.parametrize("rows", [7, 1500])
def test_plan_graph_and_streams(rows):
    st = Step(BF16, rows, 8, 2, 264, 136)
    st.issue()
    torch.cuda.synchronize()
    first = [t.clone() for t in st.outs()]

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(first, st.outs()))

    def clear():
        for t in st.outs():
            t.fill_(0)

    with rr.Plan(64) as plan:
        st.issue()
    clear()
    plan()
    assert same()
    s = torch.cuda.Stream()
    clear()
    s.wait_stream(torch.cuda.current_stream())
    st.issue(stream=s)
    s.synchronize()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan()
    for _ in range(3):
        clear()
        graph.replay()
        assert same()
        clear()
        st.issue()
        assert same()


def test_weights_past_2_31_bytes():
    """Offsets that need 64 bits: the last experts' weights and gradients, the last positions."""
    experts, n, k = 132, 4096, 4096
    assert experts * n * k > 1 << 31
    w = torch.zeros(experts, n, k, dtype=torch.bfloat16, device="cuda")
    w[experts - 1, n - 1, :] = 1.0
    w[experts - 1, 5, 7] = 2.0
    e = rr.Experts(experts, 1, 300)
    s = Slots(e, torch.full((300, 1), experts - 1, dtype=torch.int32, device="cuda"))
    q = rr.QuantizedWeight(experts, n, k)
    rr.rr_quantize_weight(BF16, w, q)
    x, xq = torch.ones(300, k, dtype=torch.bfloat16, device="cuda"), rr.Quantized(300, k)
    rr.rr_quantize_rows(BF16, x, xq)
    held = torch.empty(s.n, n, device="cuda")
    for dt, out in ((F32, held), (BF16, held.bfloat16())):
        rr.rr_expert_product(e, dt, s.place, xq, q, out, gather=True)
        torch.cuda.synchronize()
        assert (out[:300, n - 1] == k).all() and (out[:300, 5] == 2).all() and not out[:300, 6:n - 1].any()
    xt, dw = rr.Quantized(k, s.n), w
    rr.rr_quantize_slots(e, BF16, s.place, x, xt, gather=True)
    rr.rr_expert_weight_grad(e, BF16, s.place, xt, xt, dw)
    torch.cuda.synchronize()
    assert not dw[0].any() and not dw[experts - 2].any() and (dw[experts - 1] == 300).all()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_many_large_tiles(dt):
    """Workgroups with several tiles in turn, of the largest kind, segments that end inside one."""
    check_product(Layer(4000, 2, 2, 136, 4096, skew=0.5, check=False), dt, weighted=True)
    check_product(Layer(4000, 2, 3, 300, 4000, skew=0.5, check=False), dt, gather=False)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows", [500, 40])
def test_weight_grad_large_tiles(dt, rows):
    """The same of the weights' gradient, with experts that have no choice among the others."""
    l = Layer(rows, 1, 17, 3900, 2048, masked=0.0, skew=0.6, check=False)
    e, s = l.e, l.s
    xt, dyt = rr.Quantized(3900, s.n), rr.Quantized(2048, s.n)
    rr.rr_quantize_slots(e, BF16, s.place, l.x, xt, gather=True)
    rr.rr_quantize_slots(e, BF16, s.place, l.dy, dyt, gather=True)
    dw = Out(DT[dt], 17, 2048, 3900)
    rr.rr_expert_weight_grad(e, dt, s.place, dyt, xt, dw.t)
    torch.cuda.synchronize()
    for i in range(17):
        lo, hi = s.place.offset[i].item(), s.place.offset[i + 1].item()
        a = ref.values(dyt.values, dyt.powers, s.n)[:, lo:hi]
        b = ref.values(xt.values, xt.powers, s.n)[:, lo:hi]
        want = a @ b.t()
        assert ((dw.t[i].double() - want).abs() <= ref.product_bound(a, b, want, DT[dt])).all(), i
    assert dw.untouched()


def test_more_tiles_than_a_table_holds():
    """Over 256 tiles for each workgroup, of products and of gradients, in whole numbers."""
    experts, n, k = 1024, 16512, 128
    gen = torch.Generator(device="cuda").manual_seed(1)
    e = rr.Experts(experts, 1, experts)
    choice = torch.randperm(experts, generator=gen, device="cuda").to(torch.int32)[:, None].contiguous()
    s = Slots(e, choice, check=False)
    w = torch.randint(-4, 5, (experts, n, k), generator=gen, device="cuda", dtype=torch.int8).to(torch.bfloat16)
    x = torch.randint(-4, 5, (experts, k), generator=gen, device="cuda").to(torch.bfloat16)
    q, xq = rr.QuantizedWeight(experts, n, k), rr.Quantized(experts, k)
    rr.rr_quantize_weight(BF16, w, q)
    rr.rr_quantize_rows(BF16, x, xq)
    held, y = torch.empty(s.n, n, dtype=torch.bfloat16, device="cuda"), torch.empty(experts, n, dtype=torch.bfloat16, device="cuda")
    rr.rr_expert_product(e, BF16, s.place, xq, q, held, gather=True)
    rr.rr_expert_combine(e, BF16, BF16, s.place, held, None, y)
    torch.cuda.synchronize()
    for r in list(range(0, experts, 97)) + [experts - 1]:
        want = (w[choice[r, 0].item()].float() @ x[r].float()).to(torch.bfloat16)
        assert torch.equal(y[r], want), r
    del w, q, held, y
    n, k = 2048, 2300
    x = torch.randint(-4, 5, (experts, k), generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randint(-4, 5, (experts, n), generator=gen, device="cuda").to(torch.bfloat16)
    xt, dyt = rr.Quantized(k, s.n), rr.Quantized(n, s.n)
    rr.rr_quantize_slots(e, BF16, s.place, x, xt, gather=True)
    rr.rr_quantize_slots(e, BF16, s.place, dy, dyt, gather=True)
    dw = torch.empty(experts, n, k, dtype=torch.bfloat16, device="cuda")
    rr.rr_expert_weight_grad(e, BF16, s.place, dyt, xt, dw)
    torch.cuda.synchronize()
    for r in list(range(0, experts, 97)) + [experts - 1]:
        assert torch.equal(dw[choice[r, 0].item()], dy[r][:, None] * x[r][None, :]), r


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("x_by,w_by", [(-121, 110), (110, -118), (-60, -70), (110, 10)])
@pytest.mark.parametrize("rows,out", [(40, 96), (900, 600)])
def test_small_and_large_elements(dt, x_by, w_by, rows, out):
    """Powers at the range's ends.  fp32 results are of operands in bf16: an element below 2^-126
    is off by half a multiple of 2^-133."""
    l = Layer(rows, 2, 3, 500, out)
    l.x, l.w = l.x * 2.0 ** x_by, l.w * 2.0 ** w_by
    rr.rr_quantize_rows(BF16, l.x, l.xq)
    rr.rr_quantize_weight(BF16, l.w, l.wq)
    held = Out(DT[dt], l.s.n, out)
    rr.rr_expert_product(l.e, dt, l.s.place, l.xq, l.wq, held.t, gather=True)
    torch.cuda.synchronize()
    for i in range(3):
        at, n = l.s.positions(i)
        x, w = l.x_of(n), l.w_of(i)
        want = x @ w.t()
        half = 2.0 ** -134
        more = half * (x.abs().sum(dim=1)[:, None] + w.abs().sum(dim=1)[None, :]) + 500 * half ** 2 if dt == F32 else 0.0
        # results, and their sums, below 2^-126 may be zero
        bound = ref.product_bound(x, w, want, DT[dt]) + more + 500 * 2.0 ** -126 * (x_by + w_by < -100)
        # a sum in 32 bits, whatever its order, holds what is below 2^128 by magnitude
        out_of_range = ~(x.abs() @ w.abs().t() < 2.0 ** 127)
        assert (((held.t[at].double() - want).abs() <= bound) | out_of_range).all(), i
        assert x_by > 0 and w_by > 0 or not out_of_range.any()
    assert held.untouched()


@pytest.mark.parametrize("rows,topk,experts", [(512, 8, 64), (1366, 3, 20), (70000, 2, 11), (9000, 20, 1024)])
def test_slots_pieces(rows, topk, experts):
    """As many choices as one workgroup places, a few more, and more than a piece each of the most workgroups."""
    e = rr.Experts(experts, topk, rows)
    Slots(e, choices(e, masked=0.2, skew=0.5))
