"""Plain 64-bit forms of the sharded losses, and bounds on how far a kernel that
accumulates in fp32 may be from them.

The bounds count roundings.  u = 2^-24 is fp32's half step, h the element
type's (2^-8 for bf16).  With d the dimension, a logit sum of d products is off
by at most (d + 4) u sum |x w|; a sum of n terms by (n + 4) u of the sum of
their magnitudes; exp and log by a few u, and u of their argument's size."""
import math

import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def head(x, w, index, scale=1.0, teacher=None, grad=None):
    """(values, bounds) of one unsharded head: dicts with lse, logit, prob,
    loss, and with grad dx, dw.  x, w in their element type."""
    h = HALF[x.dtype]
    xd, wd = x.double(), w.double()
    rows, vocab = x.shape[0], w.shape[0]
    z = scale * (xd @ wd.t())
    size = abs(scale) * (xd.abs() @ wd.abs().t())
    ez = (x.shape[1] + 4) * U * size.amax(dim=1)                    # logit bound per row
    lse = torch.logsumexp(z, dim=1)
    top = z.amax(dim=1)
    elogsum = (vocab + 16) * U
    spread = (top[:, None] - z).clamp_max(100.0).amax(dim=1)
    elogsum = elogsum + 4 * U * spread
    elz = ez + elogsum + 4 * U * (lse.abs() + top.abs())
    live = (index >= 0) & (index < vocab)
    at = index.clamp(0, vocab - 1)
    logit = torch.where(live, z.gather(1, at), 0.0)
    if teacher is None:
        p = live.double()
        ep = torch.zeros_like(p)
        logp = torch.zeros_like(p)
    else:
        t = torch.where(live, scale * teacher.double(), -math.inf)
        best = t.amax(dim=1, keepdim=True)
        some = best > -math.inf
        e = torch.where(live & some, torch.exp(t - best), 0.0)
        s = e.sum(dim=1, keepdim=True)
        p = torch.where(some, e / s.clamp_min(1e-300), 0.0)
        logp = torch.where(p > 0, t - best - torch.log(s.clamp_min(1e-300)), 0.0)
        depth = torch.where(p > 0, best - t, 0.0)
        size_t = torch.where(live & some, t.abs() + best.abs(), 0.0).nan_to_num(0.0, 0.0, 0.0)
        ep = p * U * (index.shape[1] + 16 + 4 * depth + 4 * size_t)
    used = p.sum(dim=1) > 0
    terms = torch.where(p > 0, p * (logp - logit + lse[:, None]), 0.0)
    loss = terms.sum(dim=1)
    eterm = p * (ez + elz)[:, None] + (ep + 8 * U * p) * (logp.abs() + logit.abs() + lse.abs()[:, None] + 1.0)
    out = {"lse": lse, "logit": logit, "prob": p, "loss": loss}
    tol = {"lse": elz, "logit": ez[:, None] + 2 * U * logit.abs(), "prob": ep,
           "loss": torch.where(p > 0, eterm, 0.0).sum(dim=1) + (index.shape[1] + 4) * U * terms.abs().sum(dim=1)}
    if grad is None:
        return out, tol
    g = torch.where(used, grad.double() * scale, 0.0)[:, None]
    soft = torch.where(used[:, None], torch.exp(z - lse[:, None]), 0.0)
    target = torch.zeros_like(soft)
    etarget = torch.zeros_like(soft)
    for k in range(index.shape[1]):
        r = live[:, k].nonzero().flatten()
        target[r, index[r, k]] += p[r, k]
        etarget[r, index[r, k]] += ep[r, k] + 4 * U * p[r, k]
    dz = g * (soft - target)
    edz = g.abs() * (soft * (ez + elz + 16 * U + 4 * U * (lse.abs() + spread))[:, None] + etarget) + (h + 4 * U) * dz.abs()
    out["dx"], out["dw"] = dz @ wd, dz.t() @ xd
    mag = dz.abs() + edz
    tol["dx"] = edz @ wd.abs() + (vocab + 8) * U * (mag @ wd.abs()) + h * out["dx"].abs() + 1e-37
    tol["dw"] = edz.t() @ xd.abs() + (rows + 8) * U * (mag.t() @ xd.abs()) + h * out["dw"].abs() + 1e-37
    return out, tol


def route(logits, keep, topk, renormalize, grad_loss=None, grad_weight=None):
    """(values, bounds) of one rank's router.  choice, counts are exact."""
    h = HALF[logits.dtype]
    z = logits.double()
    rows, e = z.shape
    keep = torch.ones(rows, dtype=torch.bool, device=z.device) if keep is None else keep.bool()
    # largest first, NaN above all, the lower index first among equals
    key = torch.where(z.isnan(), math.inf, z)
    order = key.sort(dim=1, descending=True, stable=True)[1]
    if z.isnan().any():
        order = torch.stack([torch.tensor(sorted(range(e), key=lambda i: (not math.isnan(r[i]), -r[i] if not math.isnan(r[i]) else 0, i)),
                                          device=z.device) for r in z.tolist()])
    pick = order[:, :topk]
    top = z.amax(dim=1, keepdim=True)
    ez = torch.where(z == -math.inf, 0.0, torch.exp(z - top))
    total = ez.sum(dim=1, keepdim=True)
    p = torch.where(total == 0, 0.0, ez / total)
    lse = (top + torch.log(total)).squeeze(1)
    depth = torch.where(p > 0, top - z, 0.0).nan_to_num(0.0, 0.0, 0.0)
    size = torch.where(p > 0, z.abs() + top.abs(), 0.0).nan_to_num(0.0, 0.0, 0.0)
    ep = p * U * (e + 16 + 4 * depth + 4 * size)
    w = p.gather(1, pick)
    ew = ep.gather(1, pick) + 2 * U * w
    if renormalize:
        s = w.sum(dim=1, keepdim=True)
        ew = torch.where(s == 0, 0.0, ew / s + w / s * (ew.sum(dim=1, keepdim=True) / s + (topk + 4) * U))
        w = torch.where(s == 0, 0.0, w / s)
    k1 = keep[:, None]
    p0, ep0 = torch.where(k1, p, 0.0), torch.where(k1, ep, 0.0)
    choice = torch.where(k1, pick, -1).to(torch.int32)
    counts = torch.zeros(e + 1, dtype=torch.int64, device=z.device)
    counts[:e] = torch.bincount(pick[keep].flatten(), minlength=e)
    counts[e] = keep.sum()
    out = {"choice": choice, "weight": torch.where(k1, w, 0.0), "lse": torch.where(keep, lse, 0.0),
           "counts": counts.to(torch.int32), "prob_sum": p0.sum(dim=0)}
    tol = {"weight": torch.where(k1, ew, 0.0),
           "lse": (e + 16) * U + 4 * U * (lse.abs() + top.squeeze(1).abs()).nan_to_num(0.0, 0.0, 0.0),
           "prob_sum": ep0.sum(dim=0) + (rows + 8) * U * p0.sum(dim=0)}
    n = float(keep.sum())
    f = counts[:e].double() / max(n * topk, 1.0)
    out["loss"] = e * (f * out["prob_sum"]).sum().reshape(1) / max(n, 1.0)
    out["slope"] = e * f / max(n, 1.0)
    tol["loss"] = e * (f * (tol["prob_sum"] + (e + 12) * U * out["prob_sum"])).sum().reshape(1) / max(n, 1.0)
    tol["slope"] = 8 * U * out["slope"]
    if grad_loss is None:
        return out, tol
    gl, gw = grad_loss.double(), torch.where(k1, grad_weight.double(), 0.0)
    a = (gl * out["slope"]).expand_as(p).clone()
    w0, ew0 = out["weight"], tol["weight"]
    if not renormalize:
        a.scatter_add_(1, pick, gw)
    dot, edot = (p0 * a).sum(dim=1, keepdim=True), ((ep0 + (e + 12) * U * p0) * a.abs()).sum(dim=1, keepdim=True)
    dz = p0 * (a - dot)
    edz = ep0 * (a - dot).abs() + p0 * (edot + 12 * U * (a.abs() + dot.abs()))
    if renormalize:
        mean, emean = (w0 * gw).sum(dim=1, keepdim=True), ((ew0 + (topk + 4) * U * w0) * gw.abs()).sum(dim=1, keepdim=True)
        dz = dz.scatter_add(1, pick, w0 * (gw - mean))
        edz = edz.scatter_add(1, pick, ew0 * (gw - mean).abs() + w0 * (emean + 6 * U * (gw.abs() + mean.abs())))
    # the kernel forms p from the rounded lse
    edz = edz + p0 * (2 * tol["lse"][:, None]) * ((a - dot).abs() + (p0 * (a - dot).abs()).sum(dim=1, keepdim=True))
    out["dlogits"] = dz
    tol["dlogits"] = edz + (h + 4 * U) * (dz.abs() + edz) + 1e-37
    return out, tol


def check(name, got, want, bound):
    """Every element within its bound; NaN and infinities in the same places."""
    got, bound = got.double(), bound + 1e-30
    assert got.shape == want.shape, f"{name}: {tuple(got.shape)} against {tuple(want.shape)}"
    same = (got == want) | (got.isnan() & want.isnan())
    off = torch.where(same, torch.zeros_like(got), (got - want).abs() / bound)
    off = torch.where(off.isnan(), torch.full_like(off, math.inf), off)
    worst = off.max().item() if off.numel() else 0.0
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound, at {off.argmax().item()} of {tuple(off.shape)}"
