"""The expert layer of librr.so and the clipping of gradients: routing in groups of
experts, the slots of an expert layer, the experts' products in 8 bits with a power
of two for each block of 128, the global gradient norm.

The functions carry the C entry points' names (documented in include/rr.h) and
marshal arguments like the sharded losses' (losses.py): caller's tensors for
outputs and workspaces, ``stream``, ``prepare=True`` and ``Plan``.

An expert layer on a rank that holds the experts [first, first + experts)::

    e = rr.Experts(experts, topk, rows, first)
    place = rr.Slots.empty(e)
    xq, wq = rr.Quantized(rows, dim), rr.QuantizedWeight(experts, out, dim)
    rr.rr_quantize_weight(rr.BF16, w, wq)                       # once, or after each update
    rr.rr_expert_slots(e, choice, place, workspace=work)
    rr.rr_quantize_rows(rr.BF16, x, xq)
    rr.rr_expert_product(e, rr.BF16, place, xq, wq, held, gather=True)
    rr.rr_expert_combine(e, rr.BF16, rr.BF16, place, held, weight, y)
"""
import ctypes
from dataclasses import dataclass

import torch

from . import RR_EINVAL, RRError, _dev, _esize, _issue, _raise, _stream, load
from .losses import _array, _f32, _keep, _rows, _tensor, _vp, _work

__all__ = [
    "GroupRouter", "Experts", "Slots", "Quantized", "QuantizedWeight", "rr_group_route_workspace", "rr_group_route",
    "rr_route_bias", "rr_group_route_grad", "rr_expert_capacity", "rr_expert_workspace", "rr_expert_slots",
    "rr_quantize_rows", "rr_quantize_slots", "rr_quantize_weight", "rr_expert_product", "rr_expert_weight_grad",
    "rr_expert_combine", "rr_expert_combine_grad", "rr_grad_workspace", "rr_grad_square_sum", "rr_grad_clip",
]

BLOCK = 128


class _GroupRouter(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("experts", "topk", "groups", "top_groups", "group_best", "score",
                                              "renormalize")] + [("scale", ctypes.c_float)]


class _Experts(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_int64), ("experts", ctypes.c_int32), ("first", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("reserved", ctypes.c_int32)]


@dataclass(frozen=True)
class GroupRouter:
    """A router in groups (see rr_group_router in rr.h)."""
    experts: int
    topk: int
    groups: int = 1
    top_groups: int = 1
    group_best: int = 1
    sigmoid: bool = True
    renormalize: bool = True
    scale: float = 1.0

    def _c(self):
        return _GroupRouter(self.experts, self.topk, self.groups, self.top_groups, self.group_best,
                            int(bool(self.sigmoid)), int(bool(self.renormalize)), self.scale)

    @property
    def whole(self):
        """Whether the gradient reaches every expert, and so needs logits and lse."""
        return not self.sigmoid and not self.renormalize


@dataclass(frozen=True)
class Experts:
    """A rank's experts and its rows' choices (see rr_experts in rr.h)."""
    experts: int
    topk: int
    rows: int
    first: int = 0

    def _c(self):
        return _Experts(self.rows, self.experts, self.first, self.topk, 0)


@dataclass(frozen=True)
class Slots:
    """What rr_expert_slots writes: int32 tensors slot [rows, topk], source
    [capacity], offset [experts + 1], count [experts]."""
    slot: torch.Tensor
    source: torch.Tensor
    offset: torch.Tensor
    count: torch.Tensor

    @staticmethod
    def empty(e, device="cuda"):
        return Slots(*(torch.empty(s, dtype=torch.int32, device=device)
                       for s in ((e.rows, e.topk), (rr_expert_capacity(e),), (e.experts + 1,), (e.experts,))))


def _ld(n):
    return -(-n // BLOCK) * BLOCK


def _lds(n):
    return -(-_ld(n) // BLOCK // 4) * 4


class Quantized:
    """A matrix [rows, n] in 8 bits, on the GPU: values [rows, ld] (float8_e4m3fn)
    and powers [rows, lds] (uint8, the power's exponent + 127)."""

    def __init__(self, rows, n, device="cuda"):
        self.rows, self.n = rows, n
        self.values = torch.empty(rows, _ld(n), dtype=torch.float8_e4m3fn, device=device)
        self.powers = torch.empty(rows, _lds(n), dtype=torch.uint8, device=device)


class QuantizedWeight:
    """Weights [experts, n, k] in 8 bits: values [experts, n, ld] and powers
    [experts, ceil(n / 128), lds]."""

    def __init__(self, experts, n, k, device="cuda"):
        self.experts, self.n, self.k = experts, n, k
        self.values = torch.empty(experts, n, _ld(k), dtype=torch.float8_e4m3fn, device=device)
        self.powers = torch.empty(experts, _ld(n) // BLOCK, _lds(k), dtype=torch.uint8, device=device)


def _bind(lib):
    vp, ci, i32, i64, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int32, ctypes.c_int64, ctypes.c_float
    pp, pn = ctypes.POINTER(ctypes.c_void_p), ctypes.POINTER(ctypes.c_int64)
    router, ex = ctypes.POINTER(_GroupRouter), ctypes.POINTER(_Experts)
    for name, res, args in [
        ("rr_group_route_workspace", i64, [router, i64]),
        ("rr_group_route", ci, [router, ci, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, i64, vp]),
        ("rr_route_bias", ci, [router, pp, ci, f, vp, vp, vp]),
        ("rr_group_route_grad", ci, [router, ci, i64, vp, vp, vp, vp, vp, vp, vp]),
        ("rr_expert_capacity", i64, [ex]),
        ("rr_expert_workspace", i64, [ex]),
        ("rr_expert_slots", ci, [ex, vp, vp, vp, vp, vp, vp, i64, vp]),
        ("rr_quantized_ld", i64, [i64]),
        ("rr_quantized_lds", i64, [i64]),
        ("rr_quantize_rows", ci, [ci, i64, i32, vp, vp, vp, vp]),
        ("rr_quantize_slots", ci, [ex, ci, i32, vp, ci, vp, vp, vp, vp, vp, vp]),
        ("rr_quantize_weight", ci, [ci, i32, i32, i32, vp, vp, vp, vp, vp, vp]),
        ("rr_expert_product", ci, [ex, ci, i32, i32, ci] + [vp] * 10),
        ("rr_expert_weight_grad", ci, [ex, ci, i32, i32] + [vp] * 8),
        ("rr_expert_combine", ci, [ex, ci, ci, i32, vp, vp, vp, vp, vp]),
        ("rr_expert_combine_grad", ci, [ex, ci, ci, i32, vp, vp, vp, vp, vp]),
        ("rr_grad_workspace", i64, [ci, ci, pn]),
        ("rr_grad_square_sum", ci, [ci, ci, pp, pn, vp, vp, i64, vp]),
        ("rr_grad_clip", ci, [ci, pp, ci, ctypes.c_double, ci, pp, pp, pn, vp, vp]),
    ]:
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def _lib():
    lib = load()
    if getattr(lib, "_experts_bound", False) is False:
        _bind(lib)._experts_bound = True
    return lib


def _i32(t, what, elems):
    return _tensor(t, what, torch.int32, elems)


def _bytes(n):
    if n < 0:
        _raise(RR_EINVAL)
    return n


# --------------------------------------------------------------------------
# routing in groups
# --------------------------------------------------------------------------

def rr_group_route_workspace(router, rows):
    """Workspace bytes of rr_group_route."""
    c = router._c()
    return _bytes(_lib().rr_group_route_workspace(ctypes.byref(c), rows))


def rr_group_route(router, dtype, logits, bias, keep, choice, weight, logit, lse, counts, workspace=None, stream=None,
                   prepare=False):
    """Choices, their weights and logits [rows, topk], this rank's counts [experts + 1],
    and of softmax the rows' lse (None: not wanted).  bias [experts] and keep [rows]
    may be None."""
    _esize(dtype)
    rows, c, e = _rows(logits, "logits", router.experts), router._c(), router.experts
    k, (ws, nbytes) = rows * router.topk, _work(workspace)
    bp = 0 if bias is None else _f32(bias, "bias", e)
    lp = 0 if lse is None else _f32(lse, "lse", rows)
    return _issue(_lib().rr_group_route,
                  (ctypes.byref(c), dtype, rows, _vp(_dev(logits, "logits", dtype, 0)), _vp(bp), _vp(_keep(keep, rows)),
                   _vp(_i32(choice, "choice", k)), _vp(_f32(weight, "weight", k)), _vp(_f32(logit, "logit", k)), _vp(lp),
                   _vp(_i32(counts, "counts", e + 1)), _vp(ws), nbytes, _stream(stream)),
                  (c, logits, bias, keep, choice, weight, logit, lse, counts, workspace), prepare)


def rr_route_bias(router, counts, rate, bias, out, stream=None, prepare=False):
    """out = bias + rate * sign(mean - count) over all ranks' counts; out may be bias."""
    c, e = router._c(), router.experts
    arr, n, keep = _array(counts, "counts", torch.int32, e + 1)
    return _issue(_lib().rr_route_bias,
                  (ctypes.byref(c), arr, n, rate, _vp(_f32(bias, "bias", e)), _vp(_f32(out, "out", e)), _stream(stream)),
                  (c, arr, keep, bias, out), prepare)


def rr_group_route_grad(router, dtype, logits, choice, logit, lse, grad_weight, dlogits, stream=None, prepare=False):
    """Gradient [rows, experts] of sum(grad_weight * weight).  logits and lse are needed
    by a softmax router that does not renormalize, else None."""
    _esize(dtype)
    rows, c, e = _rows(choice, "choice", router.topk), router._c(), router.experts
    k = rows * router.topk
    zp = lp = 0
    if logits is not None:
        if _rows(logits, "logits", e) != rows:
            raise RRError(RR_EINVAL, f"logits has {logits.shape[0]} rows, expected {rows}")
        zp = _dev(logits, "logits", dtype, 0)
    if lse is not None:
        lp = _f32(lse, "lse", rows)
    return _issue(_lib().rr_group_route_grad,
                  (ctypes.byref(c), dtype, rows, _vp(zp), _vp(_i32(choice, "choice", k)), _vp(_f32(logit, "logit", k)),
                   _vp(lp), _vp(_f32(grad_weight, "grad_weight", k)), _vp(_dev(dlogits, "dlogits", dtype, rows * e)),
                   _stream(stream)),
                  (c, logits, choice, logit, lse, grad_weight, dlogits), prepare)


# --------------------------------------------------------------------------
# slots and matrices in 8 bits
# --------------------------------------------------------------------------

def rr_expert_capacity(e):
    """Positions that hold any choices of the rows."""
    c = e._c()
    return _bytes(_lib().rr_expert_capacity(ctypes.byref(c)))


def rr_expert_workspace(e):
    """Workspace bytes of rr_expert_slots."""
    c = e._c()
    return _bytes(_lib().rr_expert_workspace(ctypes.byref(c)))


def _slots(e, place):
    """Pointers of slot, source, offset and count, and the capacity."""
    n = rr_expert_capacity(e)
    return (_i32(place.slot, "slot", e.rows * e.topk), _i32(place.source, "source", n),
            _i32(place.offset, "offset", e.experts + 1), _i32(place.count, "count", e.experts), n)


def _shape(t, what, *shape):
    if not isinstance(t, torch.Tensor) or tuple(t.shape) != shape:
        raise RRError(RR_EINVAL, f"{what} has shape {tuple(getattr(t, 'shape', ()))}, expected {shape}")
    return t


def _quantized(q, what, rows, n):
    """Pointers of a Quantized matrix of `rows` and n columns."""
    if not isinstance(q, Quantized) or (q.rows, q.n) != (rows, n):
        raise RRError(RR_EINVAL, f"{what} must be Quantized({rows}, {n})")
    return (_tensor(q.values, f"{what}.values", torch.float8_e4m3fn, rows * _ld(n)),
            _tensor(q.powers, f"{what}.powers", torch.uint8, rows * _lds(n)))


def _quantized_weight(q, what, experts, n, k):
    if not isinstance(q, QuantizedWeight) or (q.experts, q.n, q.k) != (experts, n, k):
        raise RRError(RR_EINVAL, f"{what} must be QuantizedWeight({experts}, {n}, {k})")
    return (_tensor(q.values, f"{what}.values", torch.float8_e4m3fn, experts * n * _ld(k)),
            _tensor(q.powers, f"{what}.powers", torch.uint8, experts * (_ld(n) // BLOCK) * _lds(k)))


def rr_expert_slots(e, choice, place, workspace=None, stream=None, prepare=False):
    """The slots of choice [rows, topk]."""
    _shape(choice, "choice", e.rows, e.topk)
    c, (ws, nbytes), (slot, source, offset, count, _) = e._c(), _work(workspace), _slots(e, place)
    return _issue(_lib().rr_expert_slots,
                  (ctypes.byref(c), _vp(_i32(choice, "choice", 0)), _vp(slot), _vp(source), _vp(offset), _vp(count),
                   _vp(ws), nbytes, _stream(stream)), (c, choice, place, workspace), prepare)


def rr_quantize_rows(dtype, x, q, stream=None, prepare=False):
    """x [rows, dim] to q, each row in blocks."""
    _esize(dtype)
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise RRError(RR_EINVAL, "x must be a matrix")
    rows, dim = x.shape
    values, powers = _quantized(q, "q", rows, dim)
    return _issue(_lib().rr_quantize_rows,
                  (dtype, rows, dim, _vp(_dev(x, "x", dtype, 0)), _vp(values), _vp(powers), _stream(stream)), (x, q), prepare)


def rr_quantize_slots(e, dtype, place, x, q, weight=None, gather=False, stream=None, prepare=False):
    """x [rows, dim] (gather) or [capacity, dim], times weight [rows, topk] (None: 1), to q
    [dim, capacity], in blocks of positions."""
    _esize(dtype)
    c, (_, source, offset, _, n) = e._c(), _slots(e, place)
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise RRError(RR_EINVAL, "x must be a matrix")
    dim = x.shape[1]
    _shape(x, "x", e.rows if gather else n, dim)
    values, powers = _quantized(q, "q", dim, n)
    wp = 0 if weight is None else _f32(weight, "weight", e.rows * e.topk)
    return _issue(_lib().rr_quantize_slots,
                  (ctypes.byref(c), dtype, dim, _vp(_dev(x, "x", dtype, 0)), int(bool(gather)), _vp(wp), _vp(source),
                   _vp(offset), _vp(values), _vp(powers), _stream(stream)), (c, place, x, q, weight), prepare)


def rr_quantize_weight(dtype, w, q, qt=None, stream=None, prepare=False):
    """w [experts, n, k] to q, and transposed to qt, QuantizedWeight(experts, k, n)."""
    _esize(dtype)
    if not isinstance(w, torch.Tensor) or w.dim() != 3:
        raise RRError(RR_EINVAL, "w must have three dimensions")
    experts, n, k = w.shape
    values, powers = _quantized_weight(q, "q", experts, n, k)
    tvalues, tpowers = (0, 0) if qt is None else _quantized_weight(qt, "qt", experts, k, n)
    return _issue(_lib().rr_quantize_weight,
                  (dtype, experts, n, k, _vp(_dev(w, "w", dtype, 0)), _vp(values), _vp(powers), _vp(tvalues), _vp(tpowers),
                   _stream(stream)), (w, q, qt), prepare)


# --------------------------------------------------------------------------
# products
# --------------------------------------------------------------------------

def rr_expert_product(e, dtype, place, x, w, out, weight=None, gather=False, stream=None, prepare=False):
    """out [capacity, n] of dtype: the rows of x (Quantized, of the rows if gather, else of
    the positions) times their experts' w (QuantizedWeight), times weight [rows, topk]."""
    _esize(dtype)
    c, (_, source, offset, count, m) = e._c(), _slots(e, place)
    if not isinstance(w, QuantizedWeight):
        raise RRError(RR_EINVAL, "w must be a QuantizedWeight")
    n, k = w.n, w.k
    wv, wpow = _quantized_weight(w, "w", e.experts, n, k)
    xv, xpow = _quantized(x, "x", e.rows if gather else m, k)
    wp = 0 if weight is None else _f32(weight, "weight", e.rows * e.topk)
    return _issue(_lib().rr_expert_product,
                  (ctypes.byref(c), dtype, n, k, int(bool(gather)), _vp(xv), _vp(xpow), _vp(wv), _vp(wpow), _vp(wp),
                   _vp(source), _vp(offset), _vp(count), _vp(_dev(_shape(out, "out", m, n), "out", dtype, 0)),
                   _stream(stream)), (c, place, x, w, out, weight), prepare)


def rr_expert_weight_grad(e, dtype, place, dy, x, dw, stream=None, prepare=False):
    """dw [experts, n, k] of dy, Quantized(n, capacity), and x, Quantized(k, capacity)."""
    _esize(dtype)
    c, (_, _, offset, count, m) = e._c(), _slots(e, place)
    if not isinstance(dw, torch.Tensor) or dw.dim() != 3 or dw.shape[0] != e.experts:
        raise RRError(RR_EINVAL, f"dw must have shape [{e.experts}, n, k]")
    _, n, k = dw.shape
    dv, dpow = _quantized(dy, "dy", n, m)
    xv, xpow = _quantized(x, "x", k, m)
    return _issue(_lib().rr_expert_weight_grad,
                  (ctypes.byref(c), dtype, n, k, _vp(dv), _vp(dpow), _vp(xv), _vp(xpow), _vp(offset), _vp(count),
                   _vp(_dev(dw, "dw", dtype, 0)), _stream(stream)), (c, place, dy, x, dw), prepare)


def rr_expert_combine(e, values_dtype, dtype, place, values, weight, y, stream=None, prepare=False):
    """y [rows, dim]: the sum of each row's values [capacity, dim], times weight [rows, topk]
    (None: 1)."""
    _esize(values_dtype), _esize(dtype)
    c, (slot, _, _, _, m) = e._c(), _slots(e, place)
    dim = y.shape[1] if isinstance(y, torch.Tensor) and y.dim() == 2 else 0
    _shape(y, "y", e.rows, dim), _shape(values, "values", m, dim)
    wp = 0 if weight is None else _f32(weight, "weight", e.rows * e.topk)
    return _issue(_lib().rr_expert_combine,
                  (ctypes.byref(c), values_dtype, dtype, dim, _vp(_dev(values, "values", values_dtype, 0)), _vp(slot),
                   _vp(wp), _vp(_dev(y, "y", dtype, 0)), _stream(stream)), (c, place, values, weight, y), prepare)


def rr_expert_combine_grad(e, values_dtype, dtype, place, values, dy, grad_weight, stream=None, prepare=False):
    """grad_weight [rows, topk] of dy [rows, dim]."""
    _esize(values_dtype), _esize(dtype)
    c, (slot, _, _, _, m) = e._c(), _slots(e, place)
    dim = dy.shape[1] if isinstance(dy, torch.Tensor) and dy.dim() == 2 else 0
    _shape(dy, "dy", e.rows, dim), _shape(values, "values", m, dim)
    return _issue(_lib().rr_expert_combine_grad,
                  (ctypes.byref(c), values_dtype, dtype, dim, _vp(_dev(values, "values", values_dtype, 0)), _vp(slot),
                   _vp(_dev(dy, "dy", dtype, 0)), _vp(_f32(grad_weight, "grad_weight", e.rows * e.topk)), _stream(stream)),
                  (c, place, values, dy, grad_weight), prepare)


# --------------------------------------------------------------------------
# gradient norm
# --------------------------------------------------------------------------

def _tensors(dtype, ts, what):
    """Pointers and counts of a list of tensors of one dtype, of any shape."""
    arr = (ctypes.c_void_p * max(len(ts), 1))()
    counts = (ctypes.c_int64 * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = _dev(t, f"{what}[{i}]", dtype, 0)
        counts[i] = t.numel()
    return arr, counts


def rr_grad_workspace(dtype, tensors):
    """Workspace bytes of rr_grad_square_sum."""
    _esize(dtype)
    counts = (ctypes.c_int64 * max(len(tensors), 1))(*(t.numel() for t in tensors))
    return _bytes(_lib().rr_grad_workspace(dtype, len(tensors), counts))


def rr_grad_square_sum(dtype, tensors, total, workspace=None, stream=None, prepare=False):
    """total [1] (float64): the sum of the squares of all tensors' elements."""
    _esize(dtype)
    tensors = list(tensors)
    arr, counts = _tensors(dtype, tensors, "tensors")
    ws, nbytes = _work(workspace)
    return _issue(_lib().rr_grad_square_sum,
                  (dtype, len(tensors), arr, counts, _vp(_tensor(total, "total", torch.float64, 1)), _vp(ws), nbytes,
                   _stream(stream)), (arr, counts, tensors, total, workspace), prepare)


def rr_grad_clip(dtype, totals, max_norm, tensors, outs, norm, stream=None, prepare=False):
    """norm [1], the root of the totals' sum (of ranks and dtypes), and outs: the tensors
    scaled to max_norm where norm is above it.  outs may be the tensors themselves.  Totals that are
    not finite leave the values as they are; a finite norm past fp32's range is stored as infinite
    and scales them, so ask the totals."""
    _esize(dtype)
    tensors, outs = list(tensors), list(outs)
    if [t.numel() for t in tensors] != [t.numel() for t in outs]:
        raise RRError(RR_EINVAL, "outs differ from tensors in their number or sizes")
    arr, counts = _tensors(dtype, tensors, "tensors")
    out, _ = _tensors(dtype, outs, "outs")
    sums, n, keep = _array(totals, "totals", torch.float64, 1)
    return _issue(_lib().rr_grad_clip,
                  (dtype, sums, n, float(max_norm), len(tensors), arr, out, counts, _vp(_f32(norm, "norm", 1)),
                   _stream(stream)), (arr, out, counts, tensors, outs, sums, keep, norm), prepare)
