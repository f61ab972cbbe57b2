"""Refusals of the expert layer and the clipping on the CPU: every check of the C ABI
returns its status before any HIP call (the pointers are fake and never
dereferenced), and the binding rejects tensors that the C ABI cannot look at."""
import ctypes

import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd import experts as ex

OK, EINVAL, EALIAS = 0, 1, 2
F32, BF16 = rr.F32, rr.BF16
BASE = 1 << 40


@pytest.fixture(scope="module")
def L():
    return ex._lib()


def err(L):
    return L.rr_last_error().decode()


def ptr(i):
    """Fake buffers 256 MiB apart."""
    return BASE + (i << 28)


def router(**kw):
    d = dict(experts=64, topk=4, groups=8, top_groups=2, group_best=2, score=1, renormalize=1, scale=1.0)
    d.update(kw)
    return ex._GroupRouter(*d.values())


def layer(**kw):
    d = dict(rows=100, experts=8, first=0, topk=2, reserved=0)
    d.update(kw)
    return ex._Experts(*d.values())


# calls: their arguments in order; pointers by name
CALLS = {
    "rr_group_route": dict(r=router(score=0), dtype=BF16, rows=1000, logits=ptr(0), bias=ptr(1), keep=ptr(2), choice=ptr(3), weight=ptr(4),
                           logit=ptr(5), lse=ptr(6), counts=ptr(7), ws=ptr(8), n=1 << 26, stream=None),
    "rr_group_route_grad": dict(r=router(score=0, renormalize=0), dtype=BF16, rows=1000, logits=ptr(0), choice=ptr(1), logit=ptr(2),
                                lse=ptr(3), grad_weight=ptr(4), dlogits=ptr(5), stream=None),
    "rr_expert_slots": dict(e=layer(rows=20000), choice=ptr(0), slot=ptr(1), source=ptr(2), offset=ptr(3), count=ptr(4), ws=ptr(5),
                            n=1 << 26, stream=None),
    "rr_quantize_rows": dict(dtype=BF16, rows=100, dim=200, x=ptr(0), values=ptr(1), powers=ptr(2), stream=None),
    "rr_quantize_slots": dict(e=layer(), dtype=BF16, dim=200, x=ptr(0), gather=1, weight=ptr(1), source=ptr(2), offset=ptr(3),
                              values=ptr(4), powers=ptr(5), stream=None),
    "rr_quantize_weight": dict(dtype=BF16, experts=8, n=64, k=200, w=ptr(0), values=ptr(1), powers=ptr(2), tvalues=ptr(3),
                               tpowers=ptr(4), stream=None),
    "rr_expert_product": dict(e=layer(), dtype=BF16, n=64, k=200, gather=1, x=ptr(0), x_powers=ptr(1), w=ptr(2), w_powers=ptr(3),
                              weight=ptr(4), source=ptr(5), offset=ptr(6), count=ptr(7), out=ptr(8), stream=None),
    "rr_expert_weight_grad": dict(e=layer(), dtype=BF16, n=64, k=200, dy=ptr(0), dy_powers=ptr(1), x=ptr(2), x_powers=ptr(3),
                                  offset=ptr(4), count=ptr(5), dw=ptr(6), stream=None),
    "rr_expert_combine": dict(e=layer(), values_dtype=F32, dtype=BF16, dim=64, values=ptr(0), slot=ptr(1), weight=ptr(2), y=ptr(3),
                              stream=None),
    "rr_expert_combine_grad": dict(e=layer(), values_dtype=F32, dtype=BF16, dim=64, values=ptr(0), slot=ptr(1), dy=ptr(2),
                                   grad_weight=ptr(3), stream=None),
}
OUTS = {
    "rr_group_route": "choice weight logit lse counts ws", "rr_group_route_grad": "dlogits", "rr_expert_slots": "slot source offset count ws",
    "rr_quantize_rows": "values powers", "rr_quantize_slots": "values powers", "rr_quantize_weight": "values powers tvalues tpowers",
    "rr_expert_product": "out", "rr_expert_weight_grad": "dw", "rr_expert_combine": "y", "rr_expert_combine_grad": "grad_weight",
}
# pointers that may be null
FREE = {"bias", "keep", "weight", "lse", "tvalues"}


def call(L, name, **kw):
    a = dict(CALLS[name])
    a.update(kw)
    args = [ctypes.byref(v) if isinstance(v, ctypes.Structure) else v for v in a.values()]
    return getattr(L, name)(*args)


def pointers(name):
    return [k for k, v in CALLS[name].items() if isinstance(v, int) and v >= BASE]


def recorded(L, fn, most=16):
    """The status of a call recorded into a plan, which enqueues nothing."""
    n = L.rr_plan_bytes(most)
    plan = (ctypes.c_uint64 * (n // 8 + 1))()
    assert L.rr_plan_begin(plan, n) == OK
    st = fn()
    launches = ctypes.c_int32()
    assert L.rr_plan_end(ctypes.byref(launches)) == OK
    return st, launches.value


@pytest.mark.parametrize("name", CALLS)
def test_valid_calls_are_recorded(L, name):
    st, launches = recorded(L, lambda: call(L, name))
    assert st == OK and launches >= 1, err(L)


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned(L, name):
    for p in pointers(name):
        if not (p in FREE and (name, p) not in {("rr_group_route_grad", "lse")}) and p != "weight":
            assert call(L, name, **{p: None}) == EINVAL, p
            assert "null" in err(L)
        if p != "keep":
            assert call(L, name, **{p: ptr(20) + 1}) == EINVAL, p
            assert "aligned" in err(L)


@pytest.mark.parametrize("name", CALLS)
def test_overlaps(L, name):
    ps = pointers(name)
    reads = [p for p in ps if p not in OUTS[name].split()]
    assert reads
    for o in OUTS[name].split():
        for p in ps:
            if p != o:
                assert call(L, name, **{o: CALLS[name][p]}) in (EALIAS, EINVAL), (o, p)
    # at the last byte of an input
    if name == "rr_quantize_rows":
        assert call(L, name, values=ptr(0) + 100 * 400 - 16 - (100 * 400 - 16) % 16) == EALIAS
        assert recorded(L, lambda: call(L, name, values=ptr(0) + 100 * 400))[0] == OK


@pytest.mark.parametrize("name", [n for n in CALLS if "dtype" in CALLS[n]])
def test_dtypes(L, name):
    for bad in (2, -1):
        assert call(L, name, dtype=bad) == EINVAL
        if "values_dtype" in CALLS[name]:
            assert call(L, name, values_dtype=bad) == EINVAL


BAD_ROUTERS = [dict(experts=0), dict(experts=1025), dict(experts=63), dict(groups=0), dict(groups=65), dict(groups=-8), dict(top_groups=0),
               dict(top_groups=9), dict(group_best=0), dict(group_best=3), dict(experts=8, group_best=2), dict(topk=0), dict(topk=17),
               dict(topk=33, top_groups=8), dict(score=2), dict(score=-1), dict(scale=float("nan")), dict(scale=float("inf"))]


@pytest.mark.parametrize("bad", BAD_ROUTERS, ids=str)
def test_router_descriptor(L, bad):
    r = router(**bad)
    assert L.rr_group_route_workspace(ctypes.byref(r), 8) == -1 and err(L)
    assert call(L, "rr_group_route", r=r) == EINVAL
    assert call(L, "rr_group_route_grad", r=r) == EINVAL
    arr = (ctypes.c_void_p * 1)(ptr(0))
    assert L.rr_route_bias(ctypes.byref(r), arr, 1, 0.1, ptr(1), ptr(2), None) == EINVAL


def test_router_rows_and_workspace(L):
    for rows in (-1, (1 << 30) + 1):
        assert call(L, "rr_group_route", rows=rows) == EINVAL
        assert call(L, "rr_group_route_grad", rows=rows) == EINVAL
    r = router()
    need = L.rr_group_route_workspace(ctypes.byref(r), 100000)
    assert need > 0 and call(L, "rr_group_route", rows=100000, n=need - 1) == EINVAL
    assert call(L, "rr_group_route", r=None) == EINVAL and L.rr_group_route_workspace(None, 1) == -1
    # what a router's gradient does not read may be missing
    for kw in (dict(score=1, renormalize=0), dict(score=1), dict(score=0, renormalize=1)):
        assert recorded(L, lambda: call(L, "rr_group_route_grad", r=router(**kw), logits=None, lse=None))[0] == OK


def test_route_bias(L):
    r = router()

    def bias(counts=(ptr(0),), n=1, rate=0.1, b=ptr(1), out=ptr(2)):
        arr = (ctypes.c_void_p * max(len(counts), 1))(*counts) if counts is not None else None
        return L.rr_route_bias(ctypes.byref(r), arr, n, rate, b, out, None)

    assert recorded(L, bias)[0] == OK and recorded(L, lambda: bias(out=ptr(1)))[0] == OK
    assert bias(n=0) == EINVAL and bias(n=17) == EINVAL and bias(counts=None) == EINVAL and bias(counts=(None,)) == EINVAL
    assert bias(rate=float("nan")) == EINVAL and bias(b=None) == EINVAL and bias(out=None) == EINVAL
    assert bias(out=ptr(1) + 4) == EALIAS and bias(out=ptr(0)) == EALIAS


BAD_LAYERS = [dict(rows=-1), dict(rows=(1 << 27) + 1), dict(experts=0), dict(experts=1025), dict(first=-1), dict(first=(1 << 30) + 1),
              dict(topk=0), dict(topk=33)]


@pytest.mark.parametrize("bad", BAD_LAYERS, ids=str)
def test_layer_descriptor(L, bad):
    e = layer(**bad)
    assert L.rr_expert_capacity(ctypes.byref(e)) == -1 and L.rr_expert_workspace(ctypes.byref(e)) == -1 and err(L)
    for name in CALLS:
        if "e" in CALLS[name]:
            assert call(L, name, e=e) == EINVAL, name
            assert call(L, name, e=None) == EINVAL, name


def test_sizes(L):
    for name, dims in (("rr_quantize_rows", ["dim"]), ("rr_quantize_slots", ["dim"]), ("rr_quantize_weight", ["n", "k"]),
                       ("rr_expert_product", ["n", "k"]), ("rr_expert_weight_grad", ["n", "k"]), ("rr_expert_combine", ["dim"]),
                       ("rr_expert_combine_grad", ["dim"])):
        for d in dims:
            for bad in (0, -1, 65537):
                assert call(L, name, **{d: bad}) == EINVAL, (name, d)
    assert call(L, "rr_quantize_rows", rows=-1) == EINVAL and call(L, "rr_quantize_rows", rows=1 << 31) == EINVAL
    assert call(L, "rr_quantize_weight", experts=0) == EINVAL and call(L, "rr_quantize_weight", experts=1025) == EINVAL
    # gathered values, and the gradient's positions, within what an offset reaches
    assert call(L, "rr_expert_product", e=layer(rows=1 << 22), k=65536) == EINVAL and "2^31" in err(L)
    assert call(L, "rr_expert_weight_grad", e=layer(rows=1 << 23), n=1, k=1) == EINVAL and "capacity" in err(L)
    e = layer(rows=20000)
    need = L.rr_expert_workspace(ctypes.byref(e))
    assert need > 0 and call(L, "rr_expert_slots", n=need - 1) == EINVAL


def test_capacity_holds_any_choices(L):
    for rows, experts, topk in ((1, 1, 1), (1, 64, 8), (5, 3, 2), (1000, 7, 3), (100, 1024, 32)):
        e = layer(rows=rows, experts=experts, topk=topk)
        n = L.rr_expert_capacity(ctypes.byref(e))
        choices, used = rows * topk, min(rows * topk, experts)
        # the worst: as many experts as can be have one choice past a multiple of 128
        worst = used * 128 + max(0, (choices - used) // 128) * 128 if choices >= used else 0
        assert n % 128 == 0 and n >= choices and n >= worst
    e = layer(rows=0)
    assert L.rr_expert_capacity(ctypes.byref(e)) == 0


# --------------------------------------------------------------------------
# clipping
# --------------------------------------------------------------------------

def arrays(ins, counts, outs=None):
    n = max(len(counts), 1)
    return ((ctypes.c_void_p * n)(*ins), (ctypes.c_int64 * n)(*counts), None if outs is None else (ctypes.c_void_p * n)(*outs))


class Clip:
    def __init__(self, L):
        self.L = L

    def sum(self, dtype=F32, ins=(ptr(0), ptr(1)), counts=(100000, 50), total=ptr(2), ws=ptr(3), n=1 << 20):
        i, c, _ = arrays(ins, counts)
        return self.L.rr_grad_square_sum(dtype, len(counts), i, c, total, ws, n, None)

    def clip(self, dtype=F32, sums=(ptr(4),), n=1, limit=1.0, ins=(ptr(0), ptr(1)), counts=(100, 50), outs=(ptr(2), ptr(3)), norm=ptr(5)):
        i, c, o = arrays(ins, counts, outs)
        s = (ctypes.c_void_p * max(len(sums), 1))(*sums) if sums is not None else None
        return self.L.rr_grad_clip(dtype, s, n, limit, len(counts), i, o, c, norm, None)


def test_square_sum(L):
    c = Clip(L)
    assert recorded(L, c.sum) == (OK, 2) and recorded(L, lambda: c.sum(ins=(), counts=()))[0] == OK
    assert recorded(L, lambda: c.sum(ins=(ptr(0), None), counts=(5, 0)))[0] == OK
    assert recorded(L, lambda: c.sum(counts=(100, 50), ws=None, n=0)) == (OK, 1)
    # read twice is no fault; overlaps with what is written are
    assert recorded(L, lambda: c.sum(ins=(ptr(0), ptr(0) + 4)))[0] == OK
    for bad in (dict(dtype=2), dict(counts=(-1, 5)), dict(counts=(1 << 40, 1)), dict(ins=(None, ptr(1))), dict(ins=(ptr(0) + 2, ptr(1))),
                dict(total=None), dict(total=ptr(2) + 4), dict(ws=None), dict(n=8)):
        assert c.sum(**bad) == EINVAL, bad
    for bad in (dict(total=ptr(0) + 392), dict(ws=ptr(1)), dict(ws=ptr(0) - 256 + 0x100), dict(total=ptr(3))):
        assert c.sum(**bad) == EALIAS, bad
    n = (ctypes.c_int64 * 1)(5)
    assert L.rr_grad_workspace(F32, 4097, n) == -1 and L.rr_grad_workspace(F32, -1, n) == -1 and L.rr_grad_workspace(3, 1, n) == -1
    assert L.rr_grad_workspace(F32, 1, None) == -1 and L.rr_grad_workspace(F32, 1, n) == 0


def test_clip(L):
    c = Clip(L)
    assert recorded(L, c.clip) == (OK, 1) and recorded(L, lambda: c.clip(outs=(ptr(0), ptr(1))))[0] == OK
    assert recorded(L, lambda: c.clip(ins=(), counts=(), outs=()))[0] == OK
    assert recorded(L, lambda: c.clip(ins=(ptr(0), ptr(0))))[0] == OK
    many = tuple(ptr(10) + 4096 * i for i in range(200))
    assert recorded(L, lambda: c.clip(ins=many, counts=(100,) * 200, outs=many)) == (OK, 3)
    for bad in (dict(dtype=-1), dict(n=0), dict(n=17), dict(sums=None), dict(sums=(None,)), dict(limit=-1.0), dict(limit=float("nan")),
                dict(limit=float("inf")), dict(norm=None), dict(norm=ptr(5) + 2), dict(outs=(ptr(2), None)), dict(outs=(ptr(2) + 1, ptr(3))),
                dict(counts=(5, -1)), dict(ins=(None, ptr(1)))):
        assert c.clip(**bad) == EINVAL, bad
    for bad in (dict(outs=(ptr(0) + 4, ptr(3))), dict(outs=(ptr(1), ptr(3))), dict(outs=(ptr(2), ptr(2) + 396)), dict(norm=ptr(2)),
                dict(norm=ptr(0)), dict(sums=(ptr(2),)), dict(norm=ptr(4)), dict(outs=(ptr(1), ptr(0))), dict(outs=(ptr(2), ptr(4) - 196))):
        assert c.clip(**bad) == EALIAS, bad


def test_largest_tensors(L):
    """More tiles than one launch has workgroups: a tensor's parts in several launches."""
    c, n = Clip(L), 1 << 40
    far = dict(total=1 << 44, ws=1 << 45, n=1 << 31)
    assert recorded(L, lambda: c.sum(ins=(BASE,), counts=(n,), **far), 100) == (OK, 16 + 1)
    far = dict(sums=(1 << 44,), norm=1 << 45)
    assert recorded(L, lambda: c.clip(ins=(BASE,), outs=(BASE,), counts=(n,), **far), 100) == (OK, 64)
    # a small one before it, so that it starts inside a launch and ends in a 65th
    assert recorded(L, lambda: c.clip(ins=(1 << 46, BASE), outs=(1 << 46, BASE), counts=(5, n - 5), **far), 100) == (OK, 65)
    # 2^23 tiles of 8 KiB fit one launch, one more element does not
    half = 1 << 35
    assert recorded(L, lambda: c.clip(dtype=BF16, ins=(BASE,), outs=(BASE,), counts=(half,), **far)) == (OK, 1)
    assert recorded(L, lambda: c.clip(dtype=BF16, ins=(BASE,), outs=(BASE,), counts=(half + 1,), **far)) == (OK, 2)


# --------------------------------------------------------------------------
# the binding
# --------------------------------------------------------------------------

def test_binding_refuses():
    x = torch.zeros(4, 128)
    e = rr.Experts(2, 1, 4)
    n = rr.rr_expert_capacity(e)
    place = rr.Slots.empty(e, device="cpu")
    q, w = rr.Quantized(4, 128, device="cpu"), rr.QuantizedWeight(2, 16, 128, device="cpu")
    r = rr.GroupRouter(8, 2)
    for fn in (lambda: rr.rr_quantize_rows(F32, x, q), lambda: rr.rr_expert_slots(e, torch.zeros(4, 1, dtype=torch.int32), place),
               lambda: rr.rr_expert_product(e, F32, place, q, w, torch.zeros(n, 16), gather=True),
               lambda: rr.rr_quantize_weight(F32, torch.zeros(2, 16, 128), w),
               lambda: rr.rr_group_route(r, F32, torch.zeros(3, 8), None, None, None, None, None, None, None),
               lambda: rr.rr_grad_clip(F32, [torch.zeros(1, dtype=torch.float64)], 1.0, [x], [x], torch.zeros(1))):
        with pytest.raises(ValueError, match="device memory|must be"):
            fn()
    with pytest.raises(ValueError, match="Quantized"):
        rr.rr_quantize_rows(F32, torch.zeros(5, 128), q)
    with pytest.raises(ValueError, match="Quantized"):
        rr.rr_quantize_weight(F32, torch.zeros(2, 16, 127), w)
    with pytest.raises(ValueError, match="shape"):
        rr.rr_expert_slots(e, torch.zeros(3, 1, dtype=torch.int32), place)
    with pytest.raises(ValueError, match="differ"):
        rr.rr_grad_clip(F32, [], 1.0, [x], [x[:2]], torch.zeros(1))
    with pytest.raises(ValueError, match="dtype"):
        rr.rr_quantize_rows(7, x, q)
    with pytest.raises(ValueError):
        rr.rr_expert_capacity(rr.Experts(0, 1, 4))
    with pytest.raises(ValueError):
        rr.rr_group_route_workspace(rr.GroupRouter(8, 2, groups=3), 4)
