"""The sharded losses on the GPU against plain 64-bit forms (loss_ref), within
bounds that count roundings: sizes around the kernels' tiles, every element
type, shards, masked rows, targets in every place, unaligned views, plans,
streams and graphs.  Elements around every output must keep their values."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from tests import loss_ref as ref

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16
DT = {F32: torch.float32, BF16: torch.bfloat16}
PAD = 64


@pytest.fixture(scope="module", autouse=True)
def device():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    rr.load()
    yield
    torch.cuda.synchronize()


@pytest.fixture(autouse=True)
def said(request):
    print(request.node.name, flush=True)
    yield
    torch.cuda.synchronize()


class Out:
    """An output inside a buffer of a marker value, at an element offset."""
    marker = {torch.float32: -7.25, torch.bfloat16: -7.25, torch.int32: -77, torch.uint8: 0xA5}

    def __init__(self, dtype, *shape, lead=0):
        n = math.prod(shape)
        self.big = torch.full((n + lead + 2 * PAD,), self.marker[dtype], dtype=dtype, device="cuda")
        self.lo, self.n, self.dtype = PAD + lead, n, dtype
        self.t = self.big[self.lo:self.lo + n].view(*shape)

    def untouched(self):
        m = torch.tensor(self.marker[self.dtype], dtype=self.dtype, device="cuda")
        return bool((self.big[:self.lo] == m).all()) and bool((self.big[self.lo + self.n:] == m).all())


def view(t, lead):
    """The same values at an element offset of a larger buffer."""
    if lead == 0:
        return t.contiguous()
    big = torch.empty(t.numel() + lead, dtype=t.dtype, device=t.device)
    big[lead:] = t.flatten()
    return big[lead:].view(t.shape)


def normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def workspace(n):
    """Exactly the bytes asked for, followed by guard bytes, filled with NaN."""
    big = torch.full((n + 1024,), 0xFF, dtype=torch.uint8, device="cuda")
    return big, big[:n]


class Head:
    """One head's inputs, split into shards, and its outputs."""

    def __init__(self, dt, rows, dim, vocab, sizes=None, topk=1, scale=1.0, masked=0.2, lead=0, distill=None, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed + 1000 * rows + dim + vocab)
        self.dt, self.rows, self.dim, self.vocab, self.k, self.scale, self.lead = dt, rows, dim, vocab, topk, scale, lead
        self.distill = topk > 1 if distill is None else distill
        self.sizes = [vocab] if sizes is None else sizes
        assert sum(self.sizes) == vocab
        self.x = normal(gen, rows, dim).to(DT[dt])
        self.w = (normal(gen, vocab, dim) * (2.0 / math.sqrt(dim))).to(DT[dt])
        self.index = torch.randint(0, vocab, (rows, topk), generator=gen, device="cuda")
        drop = torch.rand(rows, generator=gen, device="cuda") < masked
        if self.distill:
            live = torch.randint(0, topk + 1, (rows, 1), generator=gen, device="cuda")
            dead = torch.arange(topk, device="cuda") >= live
            self.index[dead | drop[:, None]] = -1
        else:
            self.index[drop] = -100
        self.teacher = (normal(gen, rows, topk) * 2.0).to(DT[dt])
        self.grad = normal(gen, rows)

    def make(self):
        rows, k, lead, T = self.rows, self.k, self.lead, DT[self.dt]
        self.lse, self.logit, self.loss = Out(torch.float32, rows), Out(torch.float32, rows, k), Out(torch.float32, rows)
        self.prob = Out(torch.float32, rows, k) if self.distill else None
        self.stats = [Out(torch.float32, rows, 2) for _ in self.sizes]
        self.picked = [Out(torch.float32, rows, k) for _ in self.sizes]
        self.dx = [Out(T, rows, self.dim, lead=lead) for _ in self.sizes]
        self.dw = [Out(T, n, self.dim, lead=lead) for n in self.sizes]
        self.vx = view(self.x, lead)
        self.vw = [view(w, lead) for w in self.w.split(self.sizes)]
        firsts = [sum(self.sizes[:i]) for i in range(len(self.sizes))]
        self.v = [rr.Vocab(self.dim, n, f, self.vocab, k, self.scale) for n, f in zip(self.sizes, firsts)]
        self.works = [workspace(rr.rr_vocab_workspace(v, self.dt, rows, grad=True)) for v in self.v]

    def issue(self, stream=None):
        for v, w, s, p, (_, ws) in zip(self.v, self.vw, self.stats, self.picked, self.works):
            need = rr.rr_vocab_workspace(v, self.dt, self.rows)
            rr.rr_vocab_stats(v, self.dt, self.vx, w, self.index, s.t, p.t, workspace=ws[:need], stream=stream)
        st, pk = [s.t for s in self.stats], [p.t for p in self.picked]
        prob = None
        if self.distill:
            prob = self.prob.t
            rr.rr_vocab_distill(self.v[0], self.dt, self.index, self.teacher, st, pk, self.lse.t, self.logit.t, prob,
                                self.loss.t, stream=stream)
        else:
            rr.rr_vocab_cross_entropy(self.v[0], self.index, st, pk, self.lse.t, self.logit.t, self.loss.t, stream=stream)
        for v, w, dx, dw, (_, ws) in zip(self.v, self.vw, self.dx, self.dw, self.works):
            rr.rr_vocab_grad(v, self.dt, self.vx, w, self.index, self.lse.t, self.logit.t, prob, self.grad, dx.t, dw.t,
                             workspace=ws, stream=stream)

    def outs(self):
        return [self.lse, self.logit, self.loss, *self.stats, *self.picked, *self.dx, *self.dw] + (
            [self.prob] if self.prob else [])

    def verify(self):
        torch.cuda.synchronize()
        want, tol = ref.head(self.x, self.w, self.index, self.scale, self.teacher if self.distill else None, self.grad)
        for n in ("lse", "logit", "loss") + (("prob",) if self.distill else ()):
            ref.check(n, getattr(self, n).t, want[n], tol[n])
        h = ref.HALF[DT[self.dt]]
        # each shard's part is rounded once before the sum
        parts = torch.stack([d.t.double() for d in self.dx])
        ref.check("dx", parts.sum(dim=0), want["dx"], tol["dx"] + 2 * h * parts.abs().sum(dim=0))
        ref.check("dw", torch.cat([d.t for d in self.dw]), want["dw"], tol["dw"])
        for o in self.outs():
            assert o.untouched(), "an output's surroundings were written"
        for big, ws in self.works:
            assert bool((big[ws.numel():] == 0xFF).all()), "memory behind the workspace was written"

    def bits(self):
        return [o.t.clone() for o in self.outs()]

    def run(self):
        self.make()
        self.issue()
        self.verify()
        return self


SIZES = [  # rows, dim, vocab: single elements, tile edges either side, odd sizes
    (1, 1, 1), (1, 8, 2), (2, 7, 65), (3, 64, 63), (16, 64, 64), (17, 65, 129), (64, 128, 256), (65, 72, 257),
    (127, 200, 511), (129, 33, 1000), (255, 96, 513), (257, 264, 300), (1, 1024, 4001), (5, 520, 2003), (300, 40, 3001),
]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,vocab", SIZES)
def test_cross_entropy(dt, rows, dim, vocab):
    Head(dt, rows, dim, vocab).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim,vocab,topk,scale", [
    (1, 64, 100, 1, 0.5), (9, 40, 300, 7, 0.25), (70, 136, 1000, 64, 0.5), (33, 31, 200, 100, 1.0), (260, 64, 520, 3, 2.0)])
def test_distill(dt, rows, dim, vocab, topk, scale):
    Head(dt, rows, dim, vocab, topk=topk, scale=scale, distill=True).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("sizes", [[500, 500], [1, 998, 1], [0, 300, 700], [257, 255, 256, 232], [0, 0, 1000]], ids=str)
@pytest.mark.parametrize("topk", [1, 5])
def test_shards(dt, sizes, topk):
    Head(dt, 77, 96, sum(sizes), sizes=sizes, topk=topk, scale=0.5 if topk > 1 else 1.0).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lead", [1, 2, 3, 5])
@pytest.mark.parametrize("rows,dim", [(3, 64), (40, 72), (150, 65), (300, 128)])
def test_views_at_any_element(dt, lead, rows, dim):
    Head(dt, rows, dim, 700, lead=lead).run()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_all_rows_masked(dt):
    h = Head(dt, 37, 64, 300, masked=2.0)
    h.grad.fill_(float("nan"))
    h.make()
    h.issue()
    torch.cuda.synchronize()
    assert not h.loss.t.any() and not h.dx[0].t.any() and not h.dw[0].t.any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_non_finite_hidden_states_of_masked_rows(dt, bad):
    """A masked row may hold anything: its gradient is zero, and dw only sees
    it times zero in the formula, so its x is what the caller must keep finite."""
    h = Head(dt, 40, 64, 500)
    row = int((h.index[:, 0] < 0).nonzero()[0])
    h.grad[row] = bad
    h.teacher[:] = 0
    h.run()
    assert not h.dx[0].t[row].any() and h.loss.t[row] == 0


@pytest.mark.parametrize("dt", [F32, BF16])
def test_masked_teacher_entries_are_not_read(dt):
    h = Head(dt, 50, 64, 500, topk=6, scale=0.5)
    h.teacher[h.index < 0] = float("nan")
    live = (h.index >= 0).nonzero()
    h.teacher[live[0, 0], live[0, 1]] = -math.inf        # a live entry of no weight
    r = int((h.index >= 0).sum(dim=1).argmax())
    h.teacher[r] = torch.where(h.index[r] >= 0, torch.full_like(h.teacher[r], -math.inf), h.teacher[r])
    h.run()
    assert h.loss.t[r] == 0 and not h.prob.t[r].any() and not h.dx[0].t[r].any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_equal_entries_of_a_row(dt):
    h = Head(dt, 70, 64, 300, topk=8, scale=0.5, masked=0.0)
    h.index[:, 3] = h.index[:, 1]
    h.index[::2, 7] = h.index[::2, 1]
    h.run()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_many_entries_in_one_tile(dt):
    h = Head(dt, 200, 64, 4000, topk=100, scale=0.5, masked=0.0)
    h.index[h.index >= 0] %= 128
    h.run()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_entries_outside_the_vocabulary_do_not_count(dt):
    h = Head(dt, 30, 64, 300)
    h.index[3] = 300
    h.index[4] = 1 << 40
    h.index[5] = -(1 << 40)
    h.run()
    assert not h.loss.t[3:6].any() and not h.dx[0].t[3:6].any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_far_logits(dt):
    """Logits of thousands: the softmax is formed about its maximum."""
    h = Head(dt, 50, 64, 900)
    h.w *= 500
    h.run()
    h = Head(dt, 50, 64, 900)
    h.x *= 0
    h.run()


def test_empty_row_of_logits():
    """A whole row of -inf logits: no sum, not NaN; its lse is -inf."""
    x, w = torch.ones(3, 8, device="cuda"), torch.full((70, 8), -math.inf, device="cuda")
    ix = torch.full((3, 1), -1, device="cuda")
    v = rr.Vocab(8, 70)
    stats, picked = torch.empty(3, 2, device="cuda"), torch.empty(3, 1, device="cuda")
    lse, logit, loss = (torch.empty(3, device="cuda") for _ in range(3))
    ws = torch.empty(rr.rr_vocab_workspace(v, F32, 3), dtype=torch.uint8, device="cuda")
    rr.rr_vocab_stats(v, F32, x, w, ix, stats, picked, workspace=ws)
    rr.rr_vocab_cross_entropy(v, ix, [stats], [picked], lse, logit, loss)
    assert (stats[:, 0] == -math.inf).all() and not stats[:, 1].any()
    assert (lse == -math.inf).all() and not loss.any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_nan_spreads_to_its_row_only(dt):
    h = Head(dt, 30, 64, 300, masked=0.0)
    h.x[7, 3] = float("nan")
    h.make()
    h.issue()
    torch.cuda.synchronize()
    rest = torch.arange(30, device="cuda") != 7
    assert h.lse.t[7].isnan() and h.loss.t[7].isnan() and h.dx[0].t[7].isnan().all()
    assert not h.lse.t[rest].isnan().any() and not h.dx[0].t[rest].isnan().any()


def test_no_rows():
    h = Head(BF16, 0, 64, 300)
    h.make()
    h.issue()
    torch.cuda.synchronize()
    assert not h.dw[0].t.any()


def test_gradient_against_differences():
    """The directional derivative of the kernels' own loss."""
    h = Head(F32, 24, 48, 160, topk=4, scale=0.5, masked=0.1)
    h.run()
    gen = torch.Generator(device="cuda").manual_seed(5)
    for name, grad in (("x", h.dx[0].t), ("w", h.dw[0].t)):
        d = normal(gen, *getattr(h, name).shape)
        base, sides = getattr(h, name).clone(), []
        for step in (2.0 ** -7, -2.0 ** -7):
            setattr(h, name, base + step * d)
            h.make()
            h.issue()
            sides.append((h.grad.double() * h.loss.t.double()).sum().item())
        setattr(h, name, base)
        slope, want = (sides[0] - sides[1]) * 2.0 ** 6, (grad.double() * d.double()).sum().item()
        # fp32 losses of size 5 in 24 rows over a step of 2^-6, and the third derivative's share
        assert abs(slope - want) <= 24 * 5 * 64 * 2.0 ** -22 * 64 / 8 + 0.02 * max(abs(want), 1.0)


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows", [2, 90])
def test_plan_graph_and_streams(dt, rows):
    h = Head(dt, rows, 72, 700, topk=3, scale=0.5)
    h.run()
    first = h.bits()
    # recorded: nothing runs until the launch, every launch gives the same bits
    with rr.Plan(64) as plan:
        h.issue()
    for o in h.outs():
        o.t.fill_(0)
    torch.cuda.synchronize()
    assert not h.lse.t.any()
    for _ in range(2):
        plan()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(first, h.bits()))
    # another stream
    s = torch.cuda.Stream()
    for o in h.outs():
        o.t.fill_(0)
    s.wait_stream(torch.cuda.current_stream())
    h.issue(stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, h.bits()))
    # a graph, replayed with eager work and other inputs between
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan()
    for turn in range(3):
        h.vx.copy_(view(h.x * (1 + turn), 0))
        for o in h.outs():
            o.t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        replayed = h.bits()
        h.issue()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, h.bits()))


def test_weights_past_2_31_elements():
    """Offsets that need 64 bits, in scoring and training: rows at the far end."""
    rows, dim, vocab = 3, 32768, 66000
    need = vocab * dim
    assert need > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = normal(gen, rows, dim).to(torch.bfloat16)
    w = torch.empty(vocab, dim, dtype=torch.bfloat16, device="cuda")
    for part in w.split(8192):
        part.copy_(normal(gen, *part.shape) * (2.0 / math.sqrt(dim)))
    index = torch.tensor([[vocab - 1], [65537], [5]], device="cuda")
    v = rr.Vocab(dim, vocab)
    ws = torch.empty(rr.rr_vocab_workspace(v, BF16, rows, grad=True), dtype=torch.uint8, device="cuda")
    stats, picked = torch.empty(rows, 2, device="cuda"), torch.empty(rows, 1, device="cuda")
    lse, logit, loss = (torch.empty(rows, device="cuda") for _ in range(3))
    dx, dw, grad = torch.empty_like(x), torch.full_like(w, 9.0), torch.ones(rows, device="cuda")
    rr.rr_vocab_stats(v, BF16, x, w, index, stats, picked, workspace=ws)
    rr.rr_vocab_cross_entropy(v, index, [stats], [picked], lse, logit, loss)
    rr.rr_vocab_grad(v, BF16, x, w, index, lse, logit, None, grad, dx, dw, workspace=ws)
    xd, z = x.double(), []
    for part in w.split(8192):
        z.append(xd @ part.double().t())
    z = torch.cat(z, dim=1)
    want = torch.logsumexp(z, dim=1)
    # sums of independent roundings: eight standard deviations, sum |x w| being about 1.3 sqrt(dim)
    bound = 8 * math.sqrt(dim) * ref.U * 4 * math.sqrt(dim) + (vocab + 16) * ref.U
    assert ((lse.double() - want).abs() <= bound).all()
    assert ((loss.double() - (want - z.gather(1, index).flatten())).abs() <= 2 * bound).all()
    dz = torch.exp(z - want[:, None])
    dz.scatter_add_(1, index, -torch.ones(rows, 1, dtype=torch.float64, device="cuda"))
    for r in (0, 5, 65537, vocab - 1):
        g = dz[:, r] @ xd
        mag = dz[:, r].abs() @ xd.abs()
        assert ((dw[r].double() - g).abs() <= (2 * 2.0 ** -8 + 2 * bound) * mag + 1e-30).all(), r
    acc = torch.zeros_like(xd)
    mag = torch.zeros_like(xd)
    for i, part in enumerate(w.split(8192)):
        acc += dz[:, i * 8192:i * 8192 + part.shape[0]].contiguous() @ part.double()
        mag += dz[:, i * 8192:i * 8192 + part.shape[0]].abs().contiguous() @ part.double().abs()
    assert ((dx.double() - acc).abs() <= (2 * 2.0 ** -8 + 2 * bound) * mag + 2.0 ** -8 * acc.abs()).all()


# --------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------

class Route:
    def __init__(self, dt, rows, experts, topk, masked=0.2, renormalize=True, lead=0, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed + rows + 31 * experts + topk)
        self.dt, self.rows, self.e, self.k, self.lead = dt, rows, experts, topk, lead
        self.r = rr.Router(experts, topk, renormalize)
        self.logits = (2 * normal(gen, rows, experts) + normal(gen, experts)).to(DT[dt])
        self.keep = torch.rand(rows, generator=gen, device="cuda") >= masked if masked > 0 else None
        self.grad_loss, self.grad_weight = normal(gen, 1), normal(gen, rows, topk)

    def make(self):
        rows, e, k = self.rows, self.e, self.k
        self.vl = view(self.logits, self.lead)
        self.choice, self.weight = Out(torch.int32, rows, k), Out(torch.float32, rows, k)
        self.lse, self.counts, self.prob_sum = Out(torch.float32, rows), Out(torch.int32, e + 1), Out(torch.float32, e)
        self.loss, self.slope = Out(torch.float32, 1), Out(torch.float32, e)
        self.dlogits = Out(DT[self.dt], rows, e, lead=self.lead)
        self.work = workspace(rr.rr_route_workspace(self.r, rows))

    def issue(self, stream=None):
        rr.rr_route(self.r, self.dt, self.vl, self.keep, self.choice.t, self.weight.t, self.lse.t, self.counts.t,
                    self.prob_sum.t, workspace=self.work[1], stream=stream)
        rr.rr_balance_loss(self.r, [self.counts.t], [self.prob_sum.t], self.loss.t, self.slope.t, stream=stream)
        rr.rr_route_grad(self.r, self.dt, self.vl, self.keep, self.choice.t, self.weight.t, self.lse.t, self.slope.t,
                         self.grad_loss, self.grad_weight, self.dlogits.t, stream=stream)

    def outs(self):
        return [self.choice, self.weight, self.lse, self.counts, self.prob_sum, self.loss, self.slope, self.dlogits]

    def bits(self):
        return [o.t.clone() for o in self.outs()]

    def run(self):
        self.make()
        self.issue()
        torch.cuda.synchronize()
        want, tol = ref.route(self.logits, self.keep, self.k, self.r.renormalize, self.grad_loss, self.grad_weight)
        assert torch.equal(self.choice.t, want["choice"])
        assert torch.equal(self.counts.t, want["counts"])
        for n in ("weight", "lse", "prob_sum", "loss", "slope", "dlogits"):
            ref.check(n, getattr(self, n).t, want[n], tol[n])
        for o in self.outs():
            assert o.untouched(), "an output's surroundings were written"
        assert bool((self.work[0][self.work[1].numel():] == 0xFF).all())
        return self


ROUTES = [(1, 1, 1), (1, 64, 6), (2, 2, 2), (5, 3, 1), (17, 60, 4), (64, 8, 2), (100, 65, 8), (333, 128, 8), (1000, 256, 8),
          (50, 100, 32), (77, 1024, 9), (4099, 16, 3), (9001, 37, 5), (31, 512, 1), (129, 200, 7), (3, 32, 32)]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("rows,experts,topk", ROUTES)
def test_route(dt, renormalize, rows, experts, topk):
    Route(dt, rows, experts, topk, renormalize=renormalize).run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("masked", [0.0, 2.0])
@pytest.mark.parametrize("rows", [3, 700])
def test_route_masks(dt, masked, rows):
    r = Route(dt, rows, 64, 6, masked=masked).run()
    if masked > 1:
        assert not r.loss.t.any() and not r.dlogits.t.any() and not r.counts.t.any()


@pytest.mark.parametrize("dt", [F32, BF16])
def test_route_ties_take_the_lowest_index(dt):
    r = Route(dt, 300, 48, 5)
    r.logits = (r.logits * 1.5).round().clamp(-1, 1)
    r.logits[5] = 0
    r.logits[6, ::2] = -0.0
    r.run()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_infinite_logits(dt, renormalize):
    """Experts at -inf are never weighted; a row of nothing else has no weights."""
    r = Route(dt, 40, 24, 4, masked=0.1, renormalize=renormalize)
    r.keep[:4] = True
    r.logits[0, 3:] = -math.inf
    r.logits[1, ::2] = -math.inf
    r.logits[2] = torch.finfo(DT[dt]).min
    r.logits[3] = -math.inf
    r.run()
    assert not r.weight.t[3].any() and not r.dlogits.t[3].any() and r.lse.t[3] == -math.inf


@pytest.mark.parametrize("dt", [F32, BF16])
def test_route_nan_in_a_left_out_row(dt):
    r = Route(dt, 40, 24, 4)
    r.keep[2] = False
    r.logits[2] = float("nan")
    r.grad_weight[2] = float("nan")
    r.run()
    r = Route(dt, 40, 24, 4)
    r.keep[2] = True
    r.logits[2, 5] = float("nan")
    r.make()
    r.issue()
    torch.cuda.synchronize()
    assert r.choice.t[2, 0] == 5 and r.lse.t[2].isnan() and not r.lse.t[3:].isnan().any()


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("lead", [1, 3])
@pytest.mark.parametrize("experts", [64, 37, 256])
def test_route_views_at_any_element(dt, lead, experts):
    Route(dt, 333, experts, 4, lead=lead).run()


def test_route_no_rows():
    r = Route(F32, 0, 16, 2, masked=0.0)
    r.make()
    r.issue()
    torch.cuda.synchronize()
    assert not r.counts.t.any() and not r.prob_sum.t.any() and not r.loss.t.any() and not r.slope.t.any()


def test_balance_over_ranks():
    parts = [Route(F32, n, 20, 3, seed=n).run() for n in (50, 1, 120)]
    r = rr.Router(20, 3)
    loss, slope = torch.empty(1, device="cuda"), torch.empty(20, device="cuda")
    rr.rr_balance_loss(r, [p.counts.t for p in parts], [p.prob_sum.t for p in parts], loss, slope)
    logits = torch.cat([p.logits for p in parts])
    want, tol = ref.route(logits, torch.cat([p.keep for p in parts]), 3, True)
    ref.check("loss", loss, want["loss"], tol["loss"] + 8 * ref.U * want["loss"])
    ref.check("slope", slope, want["slope"], tol["slope"])


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows", [4, 900])
def test_route_plan_and_graph(dt, rows):
    r = Route(dt, rows, 64, 6)
    r.run()
    first = r.bits()
    with rr.Plan(8) as plan:
        r.issue()
    for o in r.outs():
        o.t.fill_(0)
    plan()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, r.bits()))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan()
    for turn in range(3):
        r.vl.copy_(r.logits * (1 - 0.5 * turn))
        for o in r.outs():
            o.t.fill_(0)
        g.replay()
        torch.cuda.synchronize()
        replayed = r.bits()
        r.issue()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(replayed, r.bits()))


def test_route_gradient_against_differences():
    for renormalize in (False, True):
        r = Route(F32, 60, 16, 3, renormalize=renormalize)
        r.run()
        gen = torch.Generator(device="cuda").manual_seed(9)
        d, base, sides = normal(gen, 60, 16), r.logits.clone(), []
        choice, slope = r.choice.t.clone(), r.slope.t.clone()
        grad = r.dlogits.t.clone()
        for step in (2.0 ** -8, -2.0 ** -8):
            r.logits = base + step * d
            r.make()
            r.issue()
            torch.cuda.synchronize()
            p = torch.softmax(r.logits.double(), dim=1)
            keep = r.keep[:, None]
            w = torch.where(keep, p.gather(1, choice.clamp_min(0).long()), 0.0)
            if renormalize:
                w = torch.where(keep, w / w.sum(dim=1, keepdim=True).clamp_min(1e-30), 0.0)
            # the choice and f are constants of the gradient
            value = r.grad_loss.double() * (torch.where(keep, p, 0.0) @ slope.double()).sum() + (r.grad_weight.double() * w).sum()
            sides.append(value.item())
        want, got = (sides[0] - sides[1]) * 2.0 ** 7, (grad.double() * d.double()).sum().item()
        assert abs(want - got) <= 1e-3 * (1 + abs(want))
