"""The sharded losses of librr.so: cross entropy over a vocabulary split over
ranks, its distillation from a teacher's top logits, and the routing of tokens
to experts with its balance loss, each with its gradient.

The functions carry the C entry points' names (documented in include/rr.h) and
marshal arguments like the relay steps': ``stream`` defaults to torch's current
stream, ``prepare=True`` and ``Plan`` record calls, rejected arguments raise
``ValueError``.  ``rows`` is taken from the tensors.  Outputs and the workspace
are the caller's tensors; a tensor that belongs to another stream than the
call's has to be kept alive and ordered by the caller, as for any torch kernel.

A rank's step, its shard being w = head[first : first + vocab]::

    v = rr.Vocab(dim, vocab, first, total)
    work = torch.empty(rr.rr_vocab_workspace(v, rr.BF16, rows, grad=True),
                       dtype=torch.uint8, device="cuda")
    rr.rr_vocab_stats(v, rr.BF16, x, w, index, stats, picked, workspace=work)
    # exchange: every rank's stats and picked
    rr.rr_vocab_cross_entropy(v, index, all_stats, all_picked, lse, logit, loss)
    rr.rr_vocab_grad(v, rr.BF16, x, w, index, lse, logit, None, grad, dx, dw, workspace=work)
    # all-reduce: dx
"""
import ctypes
from dataclasses import dataclass

import torch

from . import RR_EINVAL, RRError, _dev, _esize, _issue, _raise, _stream, load

__all__ = [
    "Vocab", "Router", "rr_vocab_workspace", "rr_vocab_stats", "rr_vocab_cross_entropy", "rr_vocab_distill",
    "rr_vocab_grad", "rr_route_workspace", "rr_route", "rr_balance_loss", "rr_route_grad",
]


class _Vocab(ctypes.Structure):
    _fields_ = [("vocab", ctypes.c_int64), ("first", ctypes.c_int64), ("total", ctypes.c_int64),
                ("dim", ctypes.c_int32), ("topk", ctypes.c_int32), ("scale", ctypes.c_float),
                ("reserved", ctypes.c_int32)]


class _Router(ctypes.Structure):
    _fields_ = [("experts", ctypes.c_int32), ("topk", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


@dataclass(frozen=True)
class Vocab:
    """One rank's vocabulary shard (see rr_vocab in rr.h)."""
    dim: int
    vocab: int
    first: int = 0
    total: int = -1     # the shard's own size by default
    topk: int = 1
    scale: float = 1.0

    def _c(self):
        total = self.vocab if self.total < 0 else self.total
        return _Vocab(self.vocab, self.first, total, self.dim, self.topk, self.scale, 0)


@dataclass(frozen=True)
class Router:
    """A router's shape (see rr_router in rr.h)."""
    experts: int
    topk: int
    renormalize: bool = True

    def _c(self):
        return _Router(self.experts, self.topk, int(bool(self.renormalize)), 0)


def _bind(lib):
    vp, ci, i64, f = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_void_p
    pp = ctypes.POINTER(ctypes.c_void_p)
    vocab, router = ctypes.POINTER(_Vocab), ctypes.POINTER(_Router)
    for name, res, args in [
        ("rr_vocab_workspace", i64, [vocab, ci, i64, ci]),
        ("rr_vocab_stats", ci, [vocab, ci, i64, vp, vp, vp, f, f, vp, i64, vp]),
        ("rr_vocab_cross_entropy", ci, [vocab, i64, vp, pp, pp, ci, f, f, f, vp]),
        ("rr_vocab_distill", ci, [vocab, ci, i64, vp, vp, pp, pp, ci, f, f, f, f, vp]),
        ("rr_vocab_grad", ci, [vocab, ci, i64, vp, vp, vp, f, f, f, f, vp, vp, vp, i64, vp]),
        ("rr_route_workspace", i64, [router, i64]),
        ("rr_route", ci, [router, ci, i64, vp, vp, vp, f, f, vp, f, vp, i64, vp]),
        ("rr_balance_loss", ci, [router, pp, pp, ci, f, f, vp]),
        ("rr_route_grad", ci, [router, ci, i64, vp, vp, vp, f, f, f, f, f, vp, vp]),
    ]:
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


def _lib():
    lib = load()
    if getattr(lib, "_losses_bound", False) is False:
        _bind(lib)._losses_bound = True
    return lib


# --------------------------------------------------------------------------
# marshalling
# --------------------------------------------------------------------------

def _tensor(t, what, dtype, elems):
    """Device pointer of a tensor of a fixed dtype after the checks the C ABI
    cannot make."""
    if not isinstance(t, torch.Tensor):
        raise RRError(RR_EINVAL, f"{what} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise RRError(RR_EINVAL, f"{what} is on {t.device}, the kernels need device memory")
    if t.dtype != dtype:
        raise RRError(RR_EINVAL, f"{what} has dtype {t.dtype}, expected {dtype}")
    if not t.is_contiguous():
        raise RRError(RR_EINVAL, f"{what} must be contiguous")
    if t.numel() < elems:
        raise RRError(RR_EINVAL, f"{what} holds {t.numel()} elements, needs {elems}")
    return t.data_ptr()


def _f32(t, what, elems):
    return _tensor(t, what, torch.float32, elems)


def _work(t):
    """Pointer and bytes of a workspace (None: none)."""
    if t is None:
        return 0, 0
    return _tensor(t, "workspace", torch.uint8, 0), t.numel()


def _rows(t, what, width):
    """Rows of a matrix whose rows hold `width` elements."""
    if not isinstance(t, torch.Tensor):
        raise RRError(RR_EINVAL, f"{what} must be a torch.Tensor")
    if t.dim() != 2 or t.shape[1] != width:
        raise RRError(RR_EINVAL, f"{what} has shape {tuple(t.shape)}, expected [rows, {width}]")
    return t.shape[0]


def _index(v, index, rows):
    if _rows(index, "index", v.topk) != rows:
        raise RRError(RR_EINVAL, f"index has {index.shape[0]} rows, expected {rows}")
    return _tensor(index, "index", torch.int64, 0)


def _array(ts, what, dtype, elems):
    ts = [ts] if isinstance(ts, torch.Tensor) else list(ts)
    arr = (ctypes.c_void_p * max(len(ts), 1))()
    for i, t in enumerate(ts):
        arr[i] = _tensor(t, f"{what}[{i}]", dtype, elems)
    return arr, len(ts), ts


def _head(v, dtype, x, w):
    _esize(dtype)
    rows = _rows(x, "x", v.dim)
    if _rows(w, "w", v.dim) != v.vocab:
        raise RRError(RR_EINVAL, f"w has {w.shape[0]} rows, the shard {v.vocab} entries")
    return rows, _dev(x, "x", dtype, 0), _dev(w, "w", dtype, 0)


def _vp(p):
    return ctypes.c_void_p(p)


# --------------------------------------------------------------------------
# vocabulary head
# --------------------------------------------------------------------------

def rr_vocab_workspace(v, dtype, rows, grad=False):
    """Workspace bytes of rr_vocab_stats, or (grad) of rr_vocab_grad and both."""
    c = v._c()
    n = _lib().rr_vocab_workspace(ctypes.byref(c), dtype, rows, int(bool(grad)))
    if n < 0:
        _raise(RR_EINVAL)
    return n


def rr_vocab_stats(v, dtype, x, w, index, stats, picked, workspace=None, stream=None, prepare=False):
    """This shard's softmax statistics [rows, 2] and the logits of the entries
    that it holds [rows, topk], from x [rows, dim] and w [vocab, dim]."""
    rows, xp, wp = _head(v, dtype, x, w)
    ip, (ws, nbytes), c = _index(v, index, rows), _work(workspace), v._c()
    return _issue(_lib().rr_vocab_stats,
                  (ctypes.byref(c), dtype, rows, _vp(xp), _vp(wp), _vp(ip), _vp(_f32(stats, "stats", 2 * rows)),
                   _vp(_f32(picked, "picked", rows * v.topk)), _vp(ws), nbytes, _stream(stream)),
                  (c, x, w, index, stats, picked, workspace), prepare)


def _shards(v, rows, stats, picked):
    s, n, ls = _array(stats, "stats", torch.float32, 2 * rows)
    p, m, lp = _array(picked, "picked", torch.float32, rows * v.topk)
    if n != m:
        raise RRError(RR_EINVAL, f"{n} shards' stats and {m} shards' picked logits")
    return s, p, n, (ls, lp)


def rr_vocab_cross_entropy(v, index, stats, picked, lse, logit, loss, stream=None, prepare=False):
    """Cross entropy [rows] of all shards' statistics (lists in the same order)."""
    rows = _rows(index, "index", v.topk)
    s, p, n, keep = _shards(v, rows, stats, picked)
    c = v._c()
    return _issue(_lib().rr_vocab_cross_entropy,
                  (ctypes.byref(c), rows, _vp(_index(v, index, rows)), s, p, n, _vp(_f32(lse, "lse", rows)),
                   _vp(_f32(logit, "logit", rows * v.topk)), _vp(_f32(loss, "loss", rows)), _stream(stream)),
                  (c, s, p, keep, index, lse, logit, loss), prepare)


def rr_vocab_distill(v, dtype, index, teacher, stats, picked, lse, logit, prob, loss, stream=None, prepare=False):
    """Divergence [rows] from the teacher's top logits [rows, topk], and its
    probabilities [rows, topk]."""
    _esize(dtype)
    rows = _rows(index, "index", v.topk)
    s, p, n, keep = _shards(v, rows, stats, picked)
    c, k = v._c(), rows * v.topk
    return _issue(_lib().rr_vocab_distill,
                  (ctypes.byref(c), dtype, rows, _vp(_index(v, index, rows)), _vp(_dev(teacher, "teacher", dtype, k)),
                   s, p, n, _vp(_f32(lse, "lse", rows)), _vp(_f32(logit, "logit", k)), _vp(_f32(prob, "prob", k)),
                   _vp(_f32(loss, "loss", rows)), _stream(stream)),
                  (c, s, p, keep, index, teacher, lse, logit, prob, loss), prepare)


def rr_vocab_grad(v, dtype, x, w, index, lse, logit, prob, grad, dx, dw, workspace=None, stream=None, prepare=False):
    """Gradients of sum(grad * loss): this shard's part of dx [rows, dim], and
    dw [vocab, dim].  prob is None for cross entropy."""
    rows, xp, wp = _head(v, dtype, x, w)
    ip, (ws, nbytes), c, k = _index(v, index, rows), _work(workspace), v._c(), rows * v.topk
    pp = 0 if prob is None else _f32(prob, "prob", k)
    return _issue(_lib().rr_vocab_grad,
                  (ctypes.byref(c), dtype, rows, _vp(xp), _vp(wp), _vp(ip), _vp(_f32(lse, "lse", rows)),
                   _vp(_f32(logit, "logit", k)), _vp(pp), _vp(_f32(grad, "grad", rows)),
                   _vp(_dev(dx, "dx", dtype, rows * v.dim)), _vp(_dev(dw, "dw", dtype, v.vocab * v.dim)),
                   _vp(ws), nbytes, _stream(stream)),
                  (c, x, w, index, lse, logit, prob, grad, dx, dw, workspace), prepare)


# --------------------------------------------------------------------------
# router
# --------------------------------------------------------------------------

def rr_route_workspace(router, rows):
    """Workspace bytes of rr_route."""
    c = router._c()
    n = _lib().rr_route_workspace(ctypes.byref(c), rows)
    if n < 0:
        _raise(RR_EINVAL)
    return n


def _keep(keep, rows):
    if keep is None:
        return 0
    if not isinstance(keep, torch.Tensor) or keep.dtype not in (torch.bool, torch.uint8):
        raise RRError(RR_EINVAL, "keep must be a bool or uint8 tensor")
    return _tensor(keep, "keep", keep.dtype, rows)


def rr_route(router, dtype, logits, keep, choice, weight, lse, counts, prob_sum, workspace=None, stream=None,
             prepare=False):
    """Choices, weights [rows, topk] and this rank's counts [experts + 1] and
    probability sums [experts].  keep [rows] leaves tokens out (None: none)."""
    _esize(dtype)
    rows, c, e = _rows(logits, "logits", router.experts), router._c(), router.experts
    k, (ws, nbytes) = rows * router.topk, _work(workspace)
    return _issue(_lib().rr_route,
                  (ctypes.byref(c), dtype, rows, _vp(_dev(logits, "logits", dtype, 0)), _vp(_keep(keep, rows)),
                   _vp(_tensor(choice, "choice", torch.int32, k)), _vp(_f32(weight, "weight", k)),
                   _vp(_f32(lse, "lse", rows)), _vp(_tensor(counts, "counts", torch.int32, e + 1)),
                   _vp(_f32(prob_sum, "prob_sum", e)), _vp(ws), nbytes, _stream(stream)),
                  (c, logits, keep, choice, weight, lse, counts, prob_sum, workspace), prepare)


def rr_balance_loss(router, counts, prob_sum, loss, slope, stream=None, prepare=False):
    """Balance loss [1] of all ranks' counts and probability sums, and its slope
    [experts] in a token's probabilities."""
    c, e = router._c(), router.experts
    n_arr, n, keep_n = _array(counts, "counts", torch.int32, e + 1)
    p_arr, m, keep_p = _array(prob_sum, "prob_sum", torch.float32, e)
    if n != m:
        raise RRError(RR_EINVAL, f"{n} ranks' counts and {m} ranks' probability sums")
    return _issue(_lib().rr_balance_loss,
                  (ctypes.byref(c), n_arr, p_arr, n, _vp(_f32(loss, "loss", 1)), _vp(_f32(slope, "slope", e)),
                   _stream(stream)),
                  (c, n_arr, p_arr, keep_n, keep_p, loss, slope), prepare)


def rr_route_grad(router, dtype, logits, keep, choice, weight, lse, slope, grad_loss, grad_weight, dlogits,
                  stream=None, prepare=False):
    """Gradient [rows, experts] of grad_loss * loss + sum(grad_weight * weight)."""
    _esize(dtype)
    rows, c, e = _rows(logits, "logits", router.experts), router._c(), router.experts
    k = rows * router.topk
    return _issue(_lib().rr_route_grad,
                  (ctypes.byref(c), dtype, rows, _vp(_dev(logits, "logits", dtype, 0)), _vp(_keep(keep, rows)),
                   _vp(_tensor(choice, "choice", torch.int32, k)), _vp(_f32(weight, "weight", k)),
                   _vp(_f32(lse, "lse", rows)), _vp(_f32(slope, "slope", e)), _vp(_f32(grad_loss, "grad_loss", 1)),
                   _vp(_f32(grad_weight, "grad_weight", k)), _vp(_dev(dlogits, "dlogits", dtype, rows * e)),
                   _stream(stream)),
                  (c, logits, keep, choice, weight, lse, slope, grad_loss, grad_weight, dlogits), prepare)
