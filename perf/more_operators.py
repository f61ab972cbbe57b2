"""The experts of a sharded training step and the clipping of its gradients, as cases to be timed.

A case is one pass through an operator: the routing of tokens in groups of experts, the experts' products in
8 bits with a scale for each block of 128, or the global gradient norm with the clipping; forward alone
(serving, scoring) or forward and gradient (training).  ``own`` chooses between the plain torch form and this
repository's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_BLOCK = 128


def listed():
    """The cases that are timed by name."""
    return [
        # the router of one decoded token: latency
        _route("route_one_token", "f32", False, 1, 8, 32, 4, 2, 8, "sigmoid", True, 2.5),
        # a batch of prompts, fine experts in groups of 20 of which the best expert speaks for its group
        _route("route_prompts", "bf16", False, 4096, 8, 20, 3, 1, 6, "softmax", False, 16.0),
        # the router of a training step: many experts balanced by a bias
        _route("route_train", "bf16", True, 65536, 8, 32, 4, 2, 8, "sigmoid", True, 2.5),
        # few experts, padding tokens left out, odd sizes, the softmax's whole gradient
        _route("route_train_f32_odd", "f32", True, 30011, 5, 12, 2, 2, 4, "softmax", False, 1.0, masked=0.15),
        # one decoded token through the experts that it chose: bound by their weights
        _experts("experts_one_token", "bf16", False, 1, 64, 8, 2048, 1024),
        # a batch of decoding sequences: every expert's weights for a few tokens each
        _experts("experts_decode", "bf16", False, 96, 64, 6, 2048, 1408),
        # prompts
        _experts("experts_prompts", "bf16", False, 4096, 16, 4, 2048, 1408),
        # the largest: a training step, weights quantised anew in each
        _experts("experts_train", "bf16", True, 8192, 32, 8, 4096, 2048),
        # a small one in full precision at odd sizes, some tokens left out
        _experts("experts_train_f32_odd", "f32", True, 999, 7, 3, 1000, 520, masked=0.1),
        # a small model's gradients: latency
        _clip("clip_small", "f32", 14, 40000, 1.0),
        # a large model's, 300 matrices and vectors
        _clip("clip_train", "bf16", 300, 600_000_000, 1.0),
        # odd sizes within the limit: nothing to scale
        _clip("clip_f32_odd_within", "f32", 37, 50_000_003, 1e6),
    ]


def _route(name, dtype, train, rows, groups, size, top_groups, best, topk, score, renormalize, scale, masked=0.0):
    return {"name": name, "op": "route", "dtype": dtype, "train": train, "rows": rows, "groups": groups, "size": size,
            "top_groups": top_groups, "best": best, "topk": topk, "score": score, "renormalize": renormalize,
            "scale": scale, "masked": masked}


def _experts(name, dtype, train, rows, experts, topk, dim, out, masked=0.0):
    return {"name": name, "op": "experts", "dtype": dtype, "train": train, "rows": rows, "experts": experts,
            "topk": topk, "dim": dim, "out": out, "masked": masked}


def _clip(name, dtype, tensors, total, limit):
    return {"name": name, "op": "clip", "dtype": dtype, "tensors": tensors, "total": total, "limit": limit}


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["route", "experts", "experts", "clip"])
    dtype, train = rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.5
    masked = rng.choice([0.0, 0.05, 0.3])
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 5, 8, 8, 16])
        size = _log_int(rng, max(2, 8 // groups), 384 // groups)
        top_groups = rng.randint(1, groups)
        case = _route("", dtype, train, _log_int(rng, 1, 65536), groups, size, top_groups, rng.choice([1, 2]),
                      rng.randint(1, min(10, top_groups * size)), rng.choice(["sigmoid", "sigmoid", "softmax"]),
                      rng.random() < 0.5, rng.choice([1.0, 2.5]), masked)
    elif op == "experts":
        experts = _log_int(rng, 1, 64)
        rows, dim, out = _log_int(rng, 1, 8192), _log_int(rng, 64, 4096), _log_int(rng, 64, 4096)
        if rng.random() < 0.6:
            dim, out = max(64, dim // 64 * 64), max(64, out // 64 * 64)
        topk = rng.randint(1, min(8, experts))
        while rows * topk * dim * out > 1 << 38:
            rows //= 2
        while experts * dim * out > 1 << 27:
            out = max(64, out // 2)
        case = _experts("", dtype, train, rows, experts, topk, dim, out, masked)
    else:
        tensors = _log_int(rng, 1, 300)
        case = _clip("", dtype, tensors, _log_int(rng, tensors * 100, 300_000_000), rng.choice([0.5, 1.0, 1e6]))
    del case["name"]
    return case


def _sizes(case):
    """The tensors' elements: a few large matrices, many smaller ones, vectors, one that is empty."""
    n, total = case["tensors"], case["total"]
    share = [1.0 if i % 7 == 0 else 0.25 if i % 3 else 0.002 for i in range(n)]
    sizes = [max(1, int(total * s / sum(share))) + i % 5 for i, s in enumerate(share)]
    if n > 4:
        sizes[3] = 0
    return sizes


def _inputs(case, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = _DT[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    if case["op"] == "clip":
        # layers differ in the size of their gradients
        return {"grads": [(normal(n) * 10.0 ** (i % 4 - 4)).to(dt) for i, n in enumerate(_sizes(case))]}
    rows, k = case["rows"], case["topk"]
    keep = torch.rand(rows, generator=gen, device="cuda") >= case["masked"]
    if case["op"] == "route":
        e = case["groups"] * case["size"]
        # a trained router: a preference shared by all tokens beside each token's own, and a bias against it
        shared = normal(e)
        st = {"logits": (normal(rows, e) + 0.5 * shared).to(dt), "bias": -0.1 * shared, "keep": keep}
        if case["train"]:
            st["grad_weight"] = normal(rows, k) / rows
        return st
    experts, dim, out = case["experts"], case["dim"], case["out"]
    # distinct experts for each token, some of them more popular
    key = torch.rand(rows, experts, generator=gen, device="cuda") * (0.5 + torch.rand(experts, generator=gen, device="cuda"))
    choice = key.topk(k, dim=1)[1].to(torch.int32)
    choice[~keep] = -1
    weight = torch.rand(rows, k, generator=gen, device="cuda") + 0.1
    weight = torch.where(keep[:, None], weight / weight.sum(dim=1, keepdim=True), torch.zeros_like(weight))
    st = {"x": normal(rows, dim).to(dt), "w": torch.empty(experts, out, dim, dtype=dt, device="cuda"),
          "choice": choice, "weight": weight}
    for e in range(experts):
        st["w"][e] = normal(out, dim) * dim ** -0.5
    if case["train"]:
        st["dy"] = (normal(rows, out) / rows).to(dt)
    return st


def prepare(case, seed):
    """Inputs, with serving the quantised weights, and with the kernels the buffers and the recorded plan that a
    loop keeps."""
    st = _inputs(case, seed)
    st["case"] = case
    if own:
        {"route": _record_route, "experts": _record_experts, "clip": _record_clip}[case["op"]](case, st)
    elif case["op"] == "experts" and not case["train"]:
        st["wq"] = _rounded(st["w"], _BLOCK)
    return st


def run(st):
    """One pass."""
    if own:
        st["plan"]()
        return st["result"]
    return {"route": _plain_route, "experts": _plain_experts, "clip": _plain_clip}[st["case"]["op"]](st)


# ---- the kernels' calls ---------------------------------------------------------------

def _empty(dtype, *shape):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def _record_route(case, st):
    import pack_rr_helper_amd as rr
    dt = rr.BF16 if case["dtype"] == "bf16" else rr.F32
    rows, e, k = case["rows"], case["groups"] * case["size"], case["topk"]
    router = rr.GroupRouter(experts=e, topk=k, groups=case["groups"], top_groups=case["top_groups"],
                            group_best=case["best"], sigmoid=case["score"] == "sigmoid",
                            renormalize=case["renormalize"], scale=case["scale"])
    whole = case["train"] and case["score"] == "softmax" and not case["renormalize"]
    choice, weight, logit = _empty(torch.int32, rows, k), _empty(torch.float32, rows, k), _empty(torch.float32, rows, k)
    lse = _empty(torch.float32, rows) if whole else None
    counts = _empty(torch.int32, e + 1)
    work = _empty(torch.uint8, max(rr.rr_group_route_workspace(router, rows), 1))
    out = {"choice": choice, "weight": weight, "counts": counts}
    with rr.Plan(16) as plan:
        rr.rr_group_route(router, dt, st["logits"], st["bias"], st["keep"], choice, weight, logit, lse, counts,
                          workspace=work)
        if case["train"]:
            # the next step's bias: from this one's, which stays as it is here
            out["bias"] = _empty(torch.float32, e)
            rr.rr_route_bias(router, [counts], 0.001, st["bias"], out["bias"])
            out["dlogits"] = torch.empty_like(st["logits"])
            rr.rr_group_route_grad(router, dt, st["logits"] if whole else None, choice, logit, lse,
                                   st["grad_weight"], out["dlogits"])
    st["plan"], st["result"] = plan, out


def _record_experts(case, st):
    import pack_rr_helper_amd as rr
    dt = rr.BF16 if case["dtype"] == "bf16" else rr.F32
    t, rows, k, dim, out = _DT[case["dtype"]], case["rows"], case["topk"], case["dim"], case["out"]
    ex = rr.Experts(experts=case["experts"], topk=k, rows=rows)
    n = rr.rr_expert_capacity(ex)
    slot, source = _empty(torch.int32, rows, k), _empty(torch.int32, n)
    offset, count = _empty(torch.int32, ex.experts + 1), _empty(torch.int32, ex.experts)
    work = _empty(torch.uint8, max(rr.rr_expert_workspace(ex), 1))
    place = rr.Slots(slot, source, offset, count)
    xq = rr.Quantized(rows, dim)
    wq = rr.QuantizedWeight(ex.experts, out, dim)
    # the router's gradient is a sum over what the experts gave: training keeps that in 32 bits
    hd = rr.F32 if case["train"] else dt
    held, y = _empty(torch.float32 if case["train"] else t, n, out), _empty(t, rows, out)
    res = {"y": y}

    def forward():
        rr.rr_expert_slots(ex, st["choice"], place, workspace=work)
        rr.rr_quantize_rows(dt, st["x"], xq)
        rr.rr_expert_product(ex, hd, place, xq, wq, held, gather=True)
        rr.rr_expert_combine(ex, hd, dt, place, held, st["weight"], y)

    if not case["train"]:
        rr.rr_quantize_weight(dt, st["w"], wq)
        with rr.Plan(32) as plan:
            forward()
        st["plan"], st["result"] = plan, res
        return
    wt = rr.QuantizedWeight(ex.experts, dim, out)              # the transposed weights
    dyq, xt, dyt = rr.Quantized(rows, out), rr.Quantized(dim, n), rr.Quantized(out, n)
    held_dx = _empty(t, n, dim)
    res["dx"], res["dw"], res["dweight"] = torch.empty_like(st["x"]), torch.empty_like(st["w"]), _empty(torch.float32, rows, k)
    with rr.Plan(64) as plan:
        rr.rr_quantize_weight(dt, st["w"], wq, wt)
        forward()
        rr.rr_expert_combine_grad(ex, hd, dt, place, held, st["dy"], res["dweight"])
        rr.rr_quantize_rows(dt, st["dy"], dyq)
        rr.rr_expert_product(ex, dt, place, dyq, wt, held_dx, weight=st["weight"], gather=True)
        rr.rr_expert_combine(ex, dt, dt, place, held_dx, None, res["dx"])
        rr.rr_quantize_slots(ex, dt, place, st["x"], xt, gather=True)
        rr.rr_quantize_slots(ex, dt, place, st["dy"], dyt, weight=st["weight"], gather=True)
        rr.rr_expert_weight_grad(ex, dt, place, dyt, xt, res["dw"])
    st["plan"], st["result"] = plan, res


def _record_clip(case, st):
    import pack_rr_helper_amd as rr
    dt = rr.BF16 if case["dtype"] == "bf16" else rr.F32
    grads = st["grads"]
    total, norm = _empty(torch.float64, 1), _empty(torch.float32, 1)
    flat = _empty(_DT[case["dtype"]], sum(_sizes(case)))        # the optimiser's flat buffer
    outs = list(flat.split(_sizes(case)))
    work = _empty(torch.uint8, max(rr.rr_grad_workspace(dt, grads), 1))
    with rr.Plan(256) as plan:
        rr.rr_grad_square_sum(dt, grads, total, workspace=work)
        rr.rr_grad_clip(dt, [total], case["limit"], grads, outs, norm)
    st["plan"], st["result"] = plan, {"norm": norm, "grads": flat}


# ---- the plain forms ------------------------------------------------------------------

def _plain_route(st):
    case, keep = st["case"], st["keep"]
    k, g, size = case["topk"], case["groups"], case["size"]
    # the choice in 64 bits: values next to each other decide it
    z = st["logits"].double()
    if case["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-z))
    else:
        s = torch.exp(z - z.amax(dim=1, keepdim=True))
        s = s / s.sum(dim=1, keepdim=True)
    c = s + st["bias"].double()
    groups = c.reshape(-1, g, size).sort(dim=2, descending=True)[0][:, :, :min(case["best"], size)].sum(dim=2)
    best = groups.sort(dim=1, descending=True, stable=True)[1][:, :case["top_groups"]]
    live = torch.zeros_like(groups, dtype=torch.bool).scatter_(1, best, True)
    c = torch.where(live[:, :, None].expand(-1, -1, size).reshape(c.shape), c, -math.inf)
    pick = c.sort(dim=1, descending=True, stable=True)[1][:, :k]
    z, s = z.float(), s.float()
    chosen = s.gather(1, pick)
    total = chosen.sum(dim=1, keepdim=True) if case["renormalize"] else torch.ones_like(chosen[:, :1])
    weight = case["scale"] * chosen / total
    counts = torch.zeros(g * size + 1, dtype=torch.int32, device=z.device)
    counts[:-1].scatter_add_(0, pick.reshape(-1), keep[:, None].to(torch.int32).expand(-1, k).reshape(-1))
    counts[-1] = keep.sum()
    out = {"choice": torch.where(keep[:, None], pick, -1).to(torch.int32),
           "weight": torch.where(keep[:, None], weight, torch.zeros_like(weight)), "counts": counts}
    if not case["train"]:
        return out
    out["bias"] = st["bias"] + 0.001 * torch.sign(counts[:-1].sum() - counts[:-1].long() * (g * size)).float()
    gw = torch.where(keep[:, None], st["grad_weight"], torch.zeros_like(weight))
    ds = case["scale"] / total * gw
    if case["renormalize"]:
        ds = ds - case["scale"] / total * (gw * chosen).sum(dim=1, keepdim=True) / total
    if case["score"] == "sigmoid":
        dz = torch.zeros_like(z).scatter_(1, pick, ds * chosen / (1 + torch.exp(z.gather(1, pick))))
    else:
        dz = torch.zeros_like(z).scatter_(1, pick, ds * chosen)
        if not case["renormalize"]:                             # renormalised, the sum is zero
            dz = dz - s * (ds * chosen).sum(dim=1, keepdim=True)
    out["dlogits"] = dz.to(_DT[case["dtype"]])
    return out


def _power(e):
    """2 to the whole number e in [-127, 127], exactly."""
    return torch.where(e >= -126, (e + 127) << 23, 1 << 22).to(torch.int32).view(torch.float32)


def _rounded(x, high=1):
    """x [..., rows, n] in e4m3 with one power of two for each block of `high` x 128, as the values that it stands for."""
    rows, n = x.shape[-2:]
    v = torch.nn.functional.pad(x.float(), (0, -n % _BLOCK, 0, -rows % high))
    v = v.reshape(*x.shape[:-2], v.shape[-2] // high, high, v.shape[-1] // _BLOCK, _BLOCK)
    m, e = torch.frexp(v.abs().amax(dim=(-1, -3), keepdim=True))   # m 2^e, m in [1/2, 1); 448 = 7/8 * 2^9
    e = (e - 9 + (m > 0.875).to(e.dtype)).clamp_min(-127)
    q = (v * _power(-e)).to(torch.float8_e4m3fn).float() * _power(e)
    return q.reshape(*x.shape[:-2], q.shape[-4] * high, -1)[..., :rows, :n].contiguous()


def _segments(case, st):
    """Choices of each expert, in order, on the host."""
    order = st["choice"].reshape(-1).long().sort(stable=True)[1]
    counts = torch.bincount(st["choice"].reshape(-1).long() + 1, minlength=case["experts"] + 1).tolist()
    return order.split(counts)[1:]


def _plain_experts(st):
    case, x, w = st["case"], st["x"], st["w"]
    k, dt = case["topk"], _DT[case["dtype"]]
    segments = _segments(case, st)
    xq = _rounded(x)
    wq = _rounded(w, _BLOCK) if case["train"] else st["wq"]
    weight = st["weight"].reshape(-1)
    held = torch.zeros(case["rows"] * k, case["out"], device=x.device)
    for e, s in enumerate(segments):
        held[s] = xq[s // k] @ wq[e].t()
    out = {"y": (held * weight[:, None]).reshape(-1, k, case["out"]).sum(dim=1).to(dt)}
    if not case["train"]:
        return out
    dy = st["dy"].float()
    out["dweight"] = (held.reshape(-1, k, case["out"]) * dy[:, None, :]).sum(dim=2)
    del held
    dyq = _rounded(st["dy"])
    held = torch.zeros(case["rows"] * k, case["dim"], device=x.device)
    out["dw"] = torch.zeros_like(w)
    for e, s in enumerate(segments):
        held[s] = weight[s, None] * (dyq[s // k] @ wq[e])
        # along the expert's tokens, 128 of them to a block
        a, b = _rounded((weight[s, None] * dy[s // k]).t()), _rounded(x[s // k].t())
        out["dw"][e] = (a @ b.t()).to(dt)
    out["dx"] = held.reshape(-1, k, case["dim"]).sum(dim=1).to(dt)
    return {n: out[n] for n in ("y", "dx", "dw", "dweight")}


def _plain_clip(st):
    # the sum in 64 bits: it is a long one
    norm = torch.sqrt(torch.stack([g.double().square().sum() for g in st["grads"]]).sum())
    factor = torch.where(norm > st["case"]["limit"], st["case"]["limit"] / norm, torch.ones_like(norm)).float()
    return {"norm": norm.float().reshape(1), "grads": torch.cat([(g.float() * factor).to(g.dtype) for g in st["grads"]])}


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    """What run returns, from the definitions in 64 bits."""
    st = _inputs(case, seed)
    return {"route": _exact_route, "experts": _exact_experts, "clip": _exact_clip}[case["op"]](case, st)


def _largest(v, n):
    """Indices of the n largest of each row, falling, the lower index first among equals."""
    work, picks = v.clone(), []
    at = torch.arange(v.shape[1], device=v.device)
    for _ in range(n):
        best = work.max(dim=1, keepdim=True)[0]
        pick = torch.where(work == best, at, v.shape[1]).amin(dim=1, keepdim=True)
        picks.append(pick)
        work.scatter_(1, pick, -math.inf)
    return torch.cat(picks, dim=1)


def _exact_route(case, st):
    rows, e, k = case["rows"], case["groups"] * case["size"], case["topk"]
    kept = st["keep"].nonzero().flatten()
    choice = torch.full((rows, k), -1, dtype=torch.int32, device="cuda")
    weight = torch.zeros(rows, k, dtype=torch.float64, device="cuda")
    full = torch.zeros(rows, e, dtype=torch.float64, device="cuda")
    counts = torch.zeros(e + 1, dtype=torch.int32, device="cuda")
    if kept.numel():
        z = st["logits"][kept].double()
        s = torch.sigmoid(z) if case["score"] == "sigmoid" else torch.softmax(z, dim=1)
        c = s + st["bias"].double()
        of = c.reshape(-1, case["size"]).topk(min(case["best"], case["size"]), dim=1)[0].sum(dim=1).reshape(-1, case["groups"])
        allowed = torch.zeros_like(of).scatter_(1, _largest(of, case["top_groups"]), 1.0)
        c = c.masked_fill(allowed.repeat_interleave(case["size"], dim=1) == 0, -math.inf)
        pick = _largest(c, k)
        p = s.gather(1, pick)
        w = case["scale"] * (p / p.sum(dim=1, keepdim=True) if case["renormalize"] else p)
        choice[kept], weight[kept] = pick.to(torch.int32), w
        counts[:e] = torch.bincount(pick.flatten(), minlength=e).to(torch.int32)
        counts[e] = kept.numel()
        if case["train"]:
            g = st["grad_weight"][kept].double()
            if case["renormalize"]:
                g = w * (g - (g * w).sum(dim=1, keepdim=True) / case["scale"])
            else:
                g = w * g                                       # s d/ds
            if case["score"] == "sigmoid":
                dz = torch.zeros_like(z).scatter_(1, pick, g * torch.sigmoid(-z.gather(1, pick)))
            else:
                dz = torch.zeros_like(z).scatter_(1, pick, g) - s * g.sum(dim=1, keepdim=True)
            full[kept] = dz
    out = {"choice": choice, "weight": weight, "counts": counts}
    if case["train"]:
        n = counts[:e].double()
        out["bias"] = st["bias"].double() + 0.001 * torch.sign(n.sum() / e - n)
        out["dlogits"] = full
    return out


def _blocks(x, high=1):
    """x [rows, n] rounded to e4m3 by blocks of `high` x 128, in 64 bits: steps of an eighth of the value's power of
    two, of 2^-9 at the least, below the largest that 448 holds."""
    rows, n = x.shape
    full = torch.zeros(-(-rows // high) * high, -(-n // _BLOCK) * _BLOCK, dtype=torch.float64, device=x.device)
    full[:rows, :n] = x.double()
    v = full.reshape(full.shape[0] // high, high, full.shape[1] // _BLOCK, _BLOCK)
    top = v.abs().amax(dim=(1, 3), keepdim=True)
    def power(e):
        return ((e.long() + 1023) << 52).view(torch.float64)

    part, e = torch.frexp(torch.where(top > 0, top, torch.ones_like(top)) / 448)
    e = (e - (part == 0.5).to(e.dtype)).clamp_min(-127)
    v = v * power(-e)
    step = power(torch.frexp(v.abs().clamp_min(2.0 ** -6))[1] - 4)
    return (torch.round(v / step) * step * power(e)).reshape(full.shape)[:rows, :n]


def _exact_experts(case, st):
    rows, k, dim, n = case["rows"], case["topk"], case["dim"], case["out"]
    x, w, weight = st["x"], st["w"], st["weight"].double().flatten()
    choice = st["choice"].flatten()
    xq = _blocks(x)
    y = torch.zeros(rows, n, dtype=torch.float64, device="cuda")
    dx, dw = torch.zeros(rows, dim, dtype=torch.float64, device="cuda"), []
    dweight = torch.zeros(rows * k, dtype=torch.float64, device="cuda")
    if case["train"]:
        dy, dyq = st["dy"].double(), _blocks(st["dy"])
    for e in range(case["experts"]):
        at = (choice == e).nonzero().flatten()
        of = at // k
        wq = _blocks(w[e], _BLOCK)
        o = xq[of] @ wq.t()
        y.index_add_(0, of, o * weight[at, None])
        if case["train"]:
            dweight[at] = (o * dy[of]).sum(dim=1)
            dx.index_add_(0, of, (dyq[of] @ wq) * weight[at, None])
            # the product of a weight and an element of dy is a 32-bit number
            g = (st["weight"].flatten()[at, None] * st["dy"].float()[of]).t()
            dw.append(_blocks(g) @ _blocks(x[of].t()).t())
    if not case["train"]:
        return {"y": y}
    return {"y": y, "dx": dx, "dw": torch.stack(dw), "dweight": dweight.reshape(rows, k)}


def _exact_clip(case, st):
    norm = math.sqrt(math.fsum(float((g.double() ** 2).sum()) for g in st["grads"]))
    by = case["limit"] / norm if norm > case["limit"] else 1.0
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"), "grads": torch.cat([g.double() * by for g in st["grads"]])}


def work(case):
    """Bytes and operations of one pass that no form can leave out."""
    es = _DT[case["dtype"]].itemsize
    if case["op"] == "clip":
        n = sum(_sizes(case))
        return {"bytes": 2 * n * es + 4, "flops": 3 * n}
    rows, k = case["rows"], case["topk"]
    if case["op"] == "route":
        e = case["groups"] * case["size"]
        b, f = rows * e * es + rows + e * 4 + rows * k * 8 + (e + 1) * 4, rows * e * 4
        if case["train"]:
            b, f = b + rows * e * es + rows * k * 4 + e * 4, f + rows * k * 8
        return {"bytes": b, "flops": f}
    dim, out = case["dim"], case["out"]
    choices = round(rows * (1 - case["masked"])) * k
    used = min(case["experts"], choices)
    product = 2 * choices * dim * out
    b = rows * (dim + out) * es + rows * k * 8
    if not case["train"]:
        return {"bytes": b + used * dim * out, "flops": product}
    b += case["experts"] * dim * out * es * 2 + rows * (dim + out) * es + rows * k * 4
    return {"bytes": b, "flops": 3 * product}
