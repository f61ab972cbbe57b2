"""Refusals of the sharded losses on the CPU: every check of the C ABI returns
its status before any HIP call (the pointers are fake and never dereferenced),
and the binding rejects tensors that the C ABI cannot look at."""
import ctypes

import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd import losses

OK, EINVAL, EALIAS = 0, 1, 2
F32, BF16 = rr.F32, rr.BF16
BASE = 1 << 40


@pytest.fixture(scope="module")
def L():
    return losses._lib()


def err(L):
    return L.rr_last_error().decode()


def vocab(**kw):
    d = dict(vocab=1000, first=0, total=1000, dim=64, topk=1, scale=1.0)
    d.update(kw)
    return losses._Vocab(d["vocab"], d["first"], d["total"], d["dim"], d["topk"], d["scale"], 0)


def ptr(i):
    """Fake buffers 64 MiB apart."""
    return BASE + (i << 26)


class Call:
    """A valid call as a dict of arguments, with some replaced."""

    def __init__(self, L):
        self.L = L

    def stats(self, **kw):
        a = dict(v=vocab(), dtype=BF16, rows=8, x=ptr(0), w=ptr(1), index=ptr(2), stats=ptr(3), picked=ptr(4),
                 ws=ptr(5), n=1 << 26)
        a.update(kw)
        return self.L.rr_vocab_stats(ctypes.byref(a["v"]) if a["v"] else None, a["dtype"], a["rows"], a["x"], a["w"],
                                     a["index"], a["stats"], a["picked"], a["ws"], a["n"], None)

    def combine(self, distill=False, **kw):
        a = dict(v=vocab(), dtype=BF16, rows=8, index=ptr(0), teacher=ptr(1), stats=[ptr(2)], picked=[ptr(3)], n=1,
                 lse=ptr(4), logit=ptr(5), prob=ptr(6), loss=ptr(7))
        a.update(kw)
        s = (ctypes.c_void_p * max(len(a["stats"]), 1))(*a["stats"]) if a["stats"] is not None else None
        p = (ctypes.c_void_p * max(len(a["picked"]), 1))(*a["picked"]) if a["picked"] is not None else None
        v = ctypes.byref(a["v"])
        if distill:
            return self.L.rr_vocab_distill(v, a["dtype"], a["rows"], a["index"], a["teacher"], s, p, a["n"],
                                           a["lse"], a["logit"], a["prob"], a["loss"], None)
        return self.L.rr_vocab_cross_entropy(v, a["rows"], a["index"], s, p, a["n"], a["lse"], a["logit"],
                                             a["loss"], None)

    def grad(self, **kw):
        a = dict(v=vocab(), dtype=BF16, rows=8, x=ptr(0), w=ptr(1), index=ptr(2), lse=ptr(3), logit=ptr(4), prob=None,
                 grad=ptr(5), dx=ptr(6), dw=ptr(7), ws=ptr(8), n=1 << 26)
        a.update(kw)
        return self.L.rr_vocab_grad(ctypes.byref(a["v"]), a["dtype"], a["rows"], a["x"], a["w"], a["index"], a["lse"],
                                    a["logit"], a["prob"], a["grad"], a["dx"], a["dw"], a["ws"], a["n"], None)

    def route(self, **kw):
        a = dict(r=losses._Router(64, 4, 1, 0), dtype=BF16, rows=1000, logits=ptr(0), keep=ptr(1), choice=ptr(2),
                 weight=ptr(3), lse=ptr(4), counts=ptr(5), prob_sum=ptr(6), ws=ptr(7), n=1 << 26)
        a.update(kw)
        return self.L.rr_route(ctypes.byref(a["r"]), a["dtype"], a["rows"], a["logits"], a["keep"], a["choice"],
                               a["weight"], a["lse"], a["counts"], a["prob_sum"], a["ws"], a["n"], None)

    def balance(self, **kw):
        a = dict(r=losses._Router(64, 4, 1, 0), counts=[ptr(0)], prob_sum=[ptr(1)], n=1, loss=ptr(2), slope=ptr(3))
        a.update(kw)
        c = (ctypes.c_void_p * max(len(a["counts"]), 1))(*a["counts"]) if a["counts"] is not None else None
        p = (ctypes.c_void_p * max(len(a["prob_sum"]), 1))(*a["prob_sum"]) if a["prob_sum"] is not None else None
        return self.L.rr_balance_loss(ctypes.byref(a["r"]), c, p, a["n"], a["loss"], a["slope"], None)

    def route_grad(self, **kw):
        a = dict(r=losses._Router(64, 4, 1, 0), dtype=BF16, rows=1000, logits=ptr(0), keep=ptr(1), choice=ptr(2),
                 weight=ptr(3), lse=ptr(4), slope=ptr(5), gl=ptr(6), gw=ptr(7), d=ptr(8))
        a.update(kw)
        return self.L.rr_route_grad(ctypes.byref(a["r"]), a["dtype"], a["rows"], a["logits"], a["keep"], a["choice"],
                                    a["weight"], a["lse"], a["slope"], a["gl"], a["gw"], a["d"], None)


BAD_VOCAB = [dict(vocab=-1), dict(first=-1), dict(first=1), dict(total=0), dict(total=1 << 31), dict(vocab=1001),
             dict(dim=0), dict(dim=65537), dict(topk=0), dict(topk=1025),
             dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_VOCAB, ids=str)
def test_vocab_descriptor(L, bad):
    c = Call(L)
    v = vocab(**bad)
    assert L.rr_vocab_workspace(ctypes.byref(v), BF16, 8, 1) == -1 and err(L)
    assert c.stats(v=v) == EINVAL
    assert c.combine(v=v) == EINVAL
    assert c.combine(distill=True, v=v) == EINVAL
    assert c.grad(v=v) == EINVAL


def test_null_descriptor(L):
    assert L.rr_vocab_workspace(None, BF16, 8, 0) == -1
    assert Call(L).stats(v=None) == EINVAL
    assert L.rr_route_workspace(None, 8) == -1


@pytest.mark.parametrize("call", ["stats", "grad", "route", "route_grad"])
@pytest.mark.parametrize("bad", [dict(dtype=2), dict(dtype=-1), dict(rows=-1), dict(rows=(1 << 30) + 1)], ids=str)
def test_dtype_and_rows(L, call, bad):
    assert getattr(Call(L), call)(**bad) == EINVAL


@pytest.mark.parametrize("call,names", [
    ("stats", "x w index stats picked ws"), ("combine", "index lse logit loss"),
    ("grad", "x w index lse logit grad dx dw ws"), ("route", "logits choice weight lse counts prob_sum ws"),
    ("balance", "loss slope"), ("route_grad", "logits choice weight lse slope gl gw d")])
def test_null_and_misaligned(L, call, names):
    for n in names.split():
        assert getattr(Call(L), call)(**{n: None}) == EINVAL, n
        assert "null" in err(L)
        assert getattr(Call(L), call)(**{n: BASE + (20 << 26) + 1}) == EINVAL, n
        assert "aligned" in err(L)


def test_distill_pointers(L):
    for n in ("teacher", "prob", "logit"):
        assert Call(L).combine(distill=True, **{n: None}) == EINVAL
    assert Call(L).grad(prob=BASE + 2) == EINVAL


@pytest.mark.parametrize("call,outs,others", [
    ("stats", "stats picked ws", "x w index"), ("combine", "lse logit loss", "index"),
    ("grad", "dx dw ws", "x w index lse logit grad"), ("route", "choice weight lse counts prob_sum ws", "logits keep"),
    ("route_grad", "d", "logits keep choice weight lse slope gl gw"), ("balance", "loss slope", "")])
def test_aliases(L, call, outs, others):
    outs, others = outs.split(), others.split()
    same = ptr(20)
    for o in outs:
        for other in others + [p for p in outs if p != o]:
            assert getattr(Call(L), call)(**{o: same, other: same}) == EALIAS, (o, other)


def test_shard_counts(L):
    c = Call(L)
    for n in (0, -1, 17):
        assert c.combine(n=n) == EINVAL
        assert c.balance(n=n) == EINVAL
    assert c.combine(stats=None) == EINVAL
    assert c.combine(picked=None) == EINVAL
    assert c.combine(stats=[None]) == EINVAL
    assert c.balance(counts=None) == EINVAL
    assert c.balance(prob_sum=[None]) == EINVAL


def test_cross_entropy_has_one_target(L):
    assert Call(L).combine(v=vocab(topk=2)) == EINVAL
    assert Call(L).grad(v=vocab(topk=2)) == EINVAL
    assert "one target" in err(L)


@pytest.mark.parametrize("bad", [(0, 1), (1025, 1), (8, 0), (8, 9), (64, 33)])
def test_router_descriptor(L, bad):
    r = losses._Router(bad[0], bad[1], 1, 0)
    assert L.rr_route_workspace(ctypes.byref(r), 8) == -1
    c = Call(L)
    assert c.route(r=r) == c.balance(r=r) == c.route_grad(r=r) == EINVAL


def test_workspace_too_small(L):
    c = Call(L)
    for call, need in ((c.stats, rr.rr_vocab_workspace(rr.Vocab(64, 1000), BF16, 8)),
                       (c.grad, rr.rr_vocab_workspace(rr.Vocab(64, 1000), BF16, 8, grad=True)),
                       (c.route, rr.rr_route_workspace(rr.Router(64, 4), 1000))):
        if need:
            assert call(n=need - 1) == EINVAL and "workspace" in err(L)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_workspace_sizes(dtype):
    for rows in (0, 1, 17, 4096, 1 << 20):
        for v in (rr.Vocab(1, 1), rr.Vocab(64, 0, 10, 10), rr.Vocab(65536, 1 << 20), rr.Vocab(4096, 1 << 16), rr.Vocab(4096, 128000)):
            if rows * v.vocab > 1 << 36:
                continue
            n, g = rr.rr_vocab_workspace(v, dtype, rows), rr.rr_vocab_workspace(v, dtype, rows, grad=True)
            assert 0 <= n <= g < 1 << 62
    assert rr.rr_vocab_workspace(rr.Vocab(4096, 128000), BF16, 8192, grad=True) < 4 << 30
    for v, rows in ((rr.Vocab(0, 10), 4), (rr.Vocab(8, (1 << 24) + 1), 4), (rr.Vocab(65536, (1 << 20) + 1), 4),
                    (rr.Vocab(8, (1 << 16) + 1), 1 << 20), (rr.Vocab(8, 10), (1 << 20) + 1)):
        with pytest.raises(ValueError):
            rr.rr_vocab_workspace(v, dtype, rows)
    with pytest.raises(ValueError):
        rr.rr_route_workspace(rr.Router(8, 9), 4)


def test_no_rows_is_a_no_op(L):
    c = Call(L)
    assert c.stats(rows=0, x=None, index=None, stats=None, picked=None) == OK
    assert c.combine(rows=0) == OK
    assert c.combine(distill=True, rows=0) == OK
    assert c.route_grad(rows=0, logits=None, d=None) == OK


def test_binding_refusals():
    v, r = rr.Vocab(64, 100), rr.Router(16, 2)
    f = torch.empty(8)
    x, w, ix = torch.empty(4, 64), torch.empty(100, 64), torch.zeros(4, 1, dtype=torch.int64)
    with pytest.raises(ValueError, match="device memory"):
        rr.rr_vocab_stats(v, F32, x, w, ix, f, f)
    with pytest.raises(ValueError, match="shape"):
        rr.rr_vocab_stats(v, F32, x[:, :32], w, ix, f, f)
    with pytest.raises(ValueError, match="entries"):
        rr.rr_vocab_stats(v, F32, x, w[:99], ix, f, f)
    with pytest.raises(ValueError, match="dtype"):
        rr.rr_vocab_stats(v, 7, x, w, ix, f, f)
    with pytest.raises(ValueError, match="Tensor"):
        rr.rr_vocab_cross_entropy(v, None, [f], [f], f, f, f)
    with pytest.raises(ValueError, match="shape"):
        rr.rr_route(r, F32, x, None, ix, f, f, f, f)
    with pytest.raises(ValueError, match="dtype"):
        rr.rr_route_grad(r, 5, x, None, ix, f, f, f, f, f, f)
