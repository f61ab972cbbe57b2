"""Plain 64-bit forms of the expert layer and the clipping, and bounds on how far a
kernel may be from them.

The bounds count roundings: u = 2^-24 is fp32's half step, h the element type's
(2^-8 for bf16).  A sum of n products is off by at most (n + 8) u of the sum of their
magnitudes.  Products of e4m3 by the 8-bit matrix instruction lose, each, up to 2^-17 of
the largest product that it is summed with (results in bf16 only)."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
BLOCK = 128


# --------------------------------------------------------------------------
# routing in groups
# --------------------------------------------------------------------------

def order(v):
    """Indices of each row's values, falling, the lower index first among equals, NaN first."""
    return torch.where(torch.isnan(v), math.inf, v).sort(dim=1, descending=True, stable=True)[1]


def group_route(r, logits, bias, keep):
    """The choices, weights, logits of the choices, lse and counts."""
    rows, e = logits.shape
    size, z = e // r.groups, logits.double()
    if r.sigmoid:
        s = torch.sigmoid(z)
        lse = torch.zeros(rows, dtype=torch.float64, device=z.device)
    else:
        s = torch.softmax(z, dim=1)
        s = torch.where((z == -math.inf).all(dim=1, keepdim=True), 0.0, s)
        lse = torch.logsumexp(z, dim=1)
    c = s if bias is None else s + bias.double()
    # a -inf counts as a finite number below all others, so that groups with fewer of them come first
    low = torch.where(c == -math.inf, -1e270, c)
    of = low.reshape(rows, r.groups, size)
    of = torch.where(torch.isnan(of), 1e300, of).sort(dim=2, descending=True)[0][:, :, :r.group_best].sum(dim=2)
    best = order(of)[:, :r.top_groups]
    live = torch.zeros_like(of).scatter_(1, best, 1.0).repeat_interleave(size, dim=1) > 0
    pick = order(torch.where(live, c, -math.inf))[:, :r.topk]
    p = s.gather(1, pick)
    ok = torch.ones(rows, dtype=torch.bool, device=z.device) if keep is None else keep.bool()
    ok = ok[:, None] & (c.gather(1, pick) != -math.inf)
    p = torch.where(ok, p, 0.0)
    total = p.sum(dim=1, keepdim=True) if r.renormalize else torch.ones_like(p[:, :1])
    weight = torch.where(ok & (total != 0), r.scale * p / total, 0.0)
    kept = rows if keep is None else int(keep.bool().sum())
    counts = torch.zeros(e + 1, dtype=torch.int64, device=z.device)
    counts[:e] = torch.bincount(pick[ok], minlength=e)
    counts[e] = kept
    if keep is not None:
        lse = torch.where(keep.bool(), lse, 0.0)
    return {"choice": torch.where(ok, pick, -1).to(torch.int32), "weight": weight,
            "logit": torch.where(ok, logits.float().gather(1, pick), -math.inf), "lse": lse, "counts": counts.to(torch.int32)}


def group_route_grad(r, logits, choice, grad_weight, dtype):
    """dlogits and its bound, of finite logits."""
    z, live = logits.double(), choice >= 0
    at, g = choice.long().clamp_min(0), torch.where(live, grad_weight.double(), 0.0)
    chosen = z.gather(1, at)
    s = torch.sigmoid(z) if r.sigmoid else torch.softmax(z, dim=1)
    p = torch.where(live, s.gather(1, at), 0.0)
    if r.renormalize:
        total = p.sum(dim=1, keepdim=True)
        w = torch.where(total > 0, p / total, 0.0)
        term = r.scale * w * (g - (w * g).sum(dim=1, keepdim=True))
    else:
        term = r.scale * p * g
    if r.sigmoid:
        term = term * torch.sigmoid(-chosen)
    term = torch.where(live, term, 0.0)
    d = torch.zeros_like(z).scatter_add_(1, at, term)
    # computed in 64 bits: quotients, products and a mean of up to topk terms, each within 2^-53 of the
    # largest |grad_weight| (s, its quotients and 1 - s are at most 1), then rounded to 32 bits and to the type
    wide = (4 * r.topk + 32) * 2.0 ** -53 * abs(r.scale) * g.abs().amax(dim=1, keepdim=True)
    tol = d.abs() * (1.01 * U + HALF[dtype]) + wide + 1e-44
    if not r.sigmoid and not r.renormalize:
        some = live.any(dim=1, keepdim=True)
        dot, mag = term.sum(dim=1, keepdim=True), term.abs().sum(dim=1, keepdim=True)
        d = torch.where(some, d - s * dot, 0.0)
        # in 32 bits: the exponents' roundings, the difference of the chosen's own terms
        lse = torch.logsumexp(z, dim=1, keepdim=True)
        spread = (4 * (z.abs() + lse.abs()).amax(dim=1, keepdim=True) + 2 * r.topk + 32) * U
        own = torch.zeros_like(z).scatter_add_(1, at, torch.where(live, abs(r.scale) * g.abs(), 0.0))
        tol = spread * s * (own + mag) + HALF[dtype] * 1.01 * d.abs() + 1e-44
    return d, tol


# --------------------------------------------------------------------------
# slots
# --------------------------------------------------------------------------

def slots(e, choice, capacity):
    """slot, source, offset, count as lists of whole numbers, by definition."""
    flat = choice.flatten().tolist()
    of = [[] for _ in range(e.experts)]
    for n, c in enumerate(flat):
        if e.first <= c < e.first + e.experts:
            of[c - e.first].append(n)
    slot, source, offset = [-1] * len(flat), [-1] * capacity, [0]
    for ns in of:
        for i, n in enumerate(ns):
            slot[n] = offset[-1] + i
            source[offset[-1] + i] = n
        offset.append(offset[-1] + -(-len(ns) // BLOCK) * BLOCK)
    return slot, source, offset, [len(ns) for ns in of]


# --------------------------------------------------------------------------
# eight bits
# --------------------------------------------------------------------------

def power(e):
    """2^e, of whole numbers in the range of doubles."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def eight(x, high=1):
    """x [rows, n] by blocks of `high` x 128: values (64 bits, NaN blocks) and the powers' bytes."""
    rows, n = x.shape
    full = torch.zeros(-(-rows // high) * high, -(-n // BLOCK) * BLOCK, dtype=torch.float64, device=x.device)
    full[:rows, :n] = x.double()
    v = full.reshape(full.shape[0] // high, high, full.shape[1] // BLOCK, BLOCK)
    fine = torch.isfinite(v).all(dim=3, keepdim=True).all(dim=1, keepdim=True)
    v = torch.where(fine, v, 0.0)
    top = v.abs().amax(dim=(1, 3), keepdim=True)
    part, e = torch.frexp(torch.where(top > 0, top, torch.full_like(top, 448 * 2.0 ** -127)) / 448)
    e = (e - (part == 0.5).to(e.dtype)).clamp_min(-127)
    v = v * power(-e)
    step = power(torch.frexp(v.abs().clamp_min(2.0 ** -6))[1] - 4)
    q = torch.where(fine, torch.round(v / step) * step * power(e), math.nan)
    byte = torch.where(fine, e + 127, 255).reshape(v.shape[0], v.shape[2])
    return q.reshape(full.shape)[:rows, :n], byte.to(torch.uint8)


def values(q, powers, n):
    """What a Quantized matrix stands for, [rows, n] in 64 bits."""
    v = q.float().double()[:, :n]
    p = torch.where(powers == 255, math.nan, power(powers.int() - 127))
    return v * p.repeat_interleave(BLOCK, dim=1)[:, :n]


def product_bound(x, w, out, dtype, by=1.0):
    """Of out = by * (x @ w.t()), x [m, k] and w [n, k] in 64 bits."""
    k = x.shape[1]
    mag = x.abs() @ w.abs().t()
    tol = (k + 16) * U * mag * by + (HALF[dtype] + 2 * U) * out.abs() + 1e-44
    if dtype == torch.bfloat16:
        for b in range(0, k, BLOCK):
            top = x[:, b:b + BLOCK].abs().amax(dim=1)[:, None] * w[:, b:b + BLOCK].abs().amax(dim=1)[None, :]
            tol = tol + BLOCK * 2.0 ** -17 * top * by
    return tol
