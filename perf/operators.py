"""The loss operators of a sharded training step, as cases to be timed.

A case is one pass through an operator: the vocabulary head's cross entropy, its
distillation from a teacher's top logits, or the experts' router with its balance
loss; forward alone (scoring) or forward and gradient (training).  ``own`` chooses
between the plain torch form, computed in 32 bits, and this repository's kernels.
"""
import math

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def listed():
    """The cases that are timed by name."""
    return [
        # scoring one next token: latency, bound by one read of the weights
        _head("ce_score_one_token", "ce", "bf16", False, 1, 1024, 32000),
        # scoring a handful of continuations
        _head("ce_score_rows_48", "ce", "bf16", False, 48, 2048, 50001, masked=0.1),
        # evaluating a batch of documents, a third of the positions being prompt
        _head("ce_score_batch", "ce", "bf16", False, 4096, 2048, 50001, masked=0.3),
        # a small model's training step
        _head("ce_train_small", "ce", "bf16", True, 1023, 1024, 32000, masked=0.05),
        # a large head's training step over four vocabulary shards, as a group of four
        # ranks holds it
        _head("ce_train_shards_4", "ce", "bf16", True, 2048, 2048, 64000, shards=4, masked=0.05),
        # the largest: a long batch, a wide model and a large vocabulary
        _head("ce_train_large", "ce", "bf16", True, 8192, 4096, 128000, masked=0.02),
        # full precision at odd sizes, over two shards
        _head("ce_train_f32_odd", "ce", "f32", True, 777, 1000, 10007, shards=2, masked=0.2),
        # distillation of a student from a teacher's 64 top logits
        _head("kd_train", "kd", "bf16", True, 4096, 2048, 64000, topk=64, scale=0.5, masked=0.1),
        # the same in full precision, short teacher rows, odd sizes
        _head("kd_train_f32_odd", "kd", "f32", True, 129, 520, 5003, topk=7, scale=0.25, masked=0.25),
        # the router of one decoded token: latency
        _route("route_one_token", "f32", False, 1, 64, 6),
        # the router of a training step, many fine experts
        _route("route_train", "bf16", True, 65536, 256, 8),
        # few experts, padding tokens left out, odd sizes
        _route("route_train_f32_odd", "f32", True, 100003, 60, 4, masked=0.15, renormalize=False),
    ]


def _head(name, op, dtype, train, rows, dim, vocab, shards=1, topk=1, scale=1.0, masked=0.0):
    return {"name": name, "op": op, "dtype": dtype, "train": train, "rows": rows, "dim": dim, "vocab": vocab,
            "shards": shards, "topk": topk, "scale": scale, "masked": masked}


def _route(name, dtype, train, rows, experts, topk, masked=0.0, renormalize=True):
    return {"name": name, "op": "route", "dtype": dtype, "train": train, "rows": rows, "experts": experts,
            "topk": topk, "masked": masked, "renormalize": renormalize}


def _log_int(rng, lo, hi):
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return min(max(v, lo), hi)


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["ce", "ce", "kd", "kd", "route"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    train = rng.random() < 0.65
    masked = rng.choice([0.0, 0.05, 0.3])
    if op == "route":
        experts = _log_int(rng, 8, 256)
        case = _route("", dtype, train, _log_int(rng, 1, 131072), experts, rng.randint(1, min(8, experts)),
                      masked, rng.random() < 0.5)
    else:
        rows, vocab = _log_int(rng, 1, 8192), _log_int(rng, 1000, 128000)
        dim = _log_int(rng, 64, 4096)
        if rng.random() < 0.7:
            dim = max(64, dim // 64 * 64)
        limit = 8192 * 4096 * 128000 // (1 if dtype == "bf16" else 40)
        while rows * dim * vocab > limit:
            rows = max(1, rows // 2)
        case = _head("", op, dtype, train, rows, dim, vocab, rng.choice([1, 1, 2, 4]),
                     rng.choice([1, 5, 16, 64, 100]) if op == "kd" else 1,
                     rng.choice([1.0, 0.5]) if op == "kd" else 1.0, masked)
    del case["name"]
    return case


def _shard_sizes(case):
    """Vocabulary rows of each shard: as even as whole rows allow."""
    q, r = divmod(case["vocab"], case["shards"])
    return [q + (i < r) for i in range(case["shards"])]


def _inputs(case, seed):
    """The inputs of a case, on the GPU, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt, rows = _DT[case["dtype"]], case["rows"]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    keep = torch.rand(rows, generator=gen, device="cuda") >= case["masked"]
    grad = 1.0 / rows
    if case["op"] == "route":
        # trained routers prefer some experts: a shared bias beside the token's own preference
        e = case["experts"]
        logits = (normal(rows, e) + 0.5 * normal(e)).to(dt)
        return {"logits": logits, "keep": keep, "grad_loss": normal(1).abs() * 0.01,
                "grad_weight": normal(rows, case["topk"]) * grad}
    dim, vocab, k = case["dim"], case["vocab"], case["topk"]
    x = normal(rows, dim).to(dt)                       # a normed hidden state
    w = (normal(vocab, dim) * (2.0 / math.sqrt(dim))).to(dt)
    st = {"x": x, "w": w, "grad": torch.full((rows,), grad, device="cuda")}
    if case["op"] == "ce":
        index = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
        index[~keep] = -100                            # prompt and padding positions
    else:
        # k distinct indices a row, spread over the vocabulary, falling teacher logits; some
        # rows hold fewer entries, masked ones none
        start = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
        step = max(vocab // k, 1)
        index = (start + torch.arange(k, device="cuda") * step) % vocab
        live = torch.randint(max(k // 2, 1), k + 1, (rows, 1), generator=gen, device="cuda")
        index[(torch.arange(k, device="cuda") >= live) | ~keep[:, None]] = -1
        st["teacher"] = (normal(rows, k) * 2.0).sort(dim=1, descending=True)[0].to(dt)
        st["grad"] /= case["scale"] ** 2               # the usual square of the temperature
    st["index"] = index
    return st


def prepare(case, seed):
    """Inputs, and with the kernels the buffers and the recorded plan that a loop keeps."""
    st = _inputs(case, seed)
    st["case"] = case
    if case["op"] != "route":
        sizes = _shard_sizes(case)
        st["ws"] = list(st["w"].split(sizes))
        st["firsts"] = [sum(sizes[:i]) for i in range(len(sizes))]
    if own:
        (_record_route if case["op"] == "route" else _record_head)(case, st)
    return st


def run(st):
    """One pass."""
    if own:
        st["plan"]()
        return st["out"]
    return (_plain_route if st["case"]["op"] == "route" else _plain_head)(st)


# ---- the kernels' calls ---------------------------------------------------------------

def _record_head(case, st):
    import pack_rr_helper_amd as rr
    dt = rr.BF16 if case["dtype"] == "bf16" else rr.F32
    x, index, rows, k = st["x"], st["index"], case["rows"], case["topk"]

    def f32(*shape):
        return torch.empty(*shape, dtype=torch.float32, device="cuda")

    vocabs = [rr.Vocab(dim=case["dim"], vocab=w.shape[0], first=f, total=case["vocab"], topk=k, scale=case["scale"])
              for w, f in zip(st["ws"], st["firsts"])]
    need = max(rr.rr_vocab_workspace(v, dt, rows, grad=case["train"]) for v in vocabs)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    stats = [f32(rows, 2) for _ in vocabs]
    picked = [f32(rows, k) for _ in vocabs]
    lse, logit, loss = f32(rows), f32(rows, k), f32(rows)
    prob = f32(rows, k) if case["op"] == "kd" else None
    out = {"loss": loss, "lse": lse}
    with rr.Plan(512) as plan:
        for v, w, s, p in zip(vocabs, st["ws"], stats, picked):
            rr.rr_vocab_stats(v, dt, x, w, index, s, p, workspace=work)
        if case["op"] == "kd":
            rr.rr_vocab_distill(vocabs[0], dt, index, st["teacher"], stats, picked, lse, logit, prob, loss)
        else:
            rr.rr_vocab_cross_entropy(vocabs[0], index, stats, picked, lse, logit, loss)
        if case["train"]:
            out["dx"] = [torch.empty_like(x) for _ in vocabs]
            dw = torch.empty_like(st["w"])
            out["dw"] = dw
            for v, w, dxp, dwp in zip(vocabs, st["ws"], out["dx"], dw.split([w.shape[0] for w in st["ws"]])):
                rr.rr_vocab_grad(v, dt, x, w, index, lse, logit, prob, st["grad"], dxp, dwp, workspace=work)
    st["plan"], st["out"] = plan, out


def _record_route(case, st):
    import pack_rr_helper_amd as rr
    dt = rr.BF16 if case["dtype"] == "bf16" else rr.F32
    rows, e, k = case["rows"], case["experts"], case["topk"]
    router = rr.Router(experts=e, topk=k, renormalize=case["renormalize"])

    def empty(dtype, *shape):
        return torch.empty(*shape, dtype=dtype, device="cuda")

    work = empty(torch.uint8, max(rr.rr_route_workspace(router, rows), 1))
    choice, weight = empty(torch.int32, rows, k), empty(torch.float32, rows, k)
    lse, counts, prob_sum = empty(torch.float32, rows), empty(torch.int32, e + 1), empty(torch.float32, e)
    loss, slope = empty(torch.float32, 1), empty(torch.float32, e)
    out = {"choice": choice, "weight": weight, "counts": counts, "loss": loss}
    with rr.Plan(16) as plan:
        rr.rr_route(router, dt, st["logits"], st["keep"], choice, weight, lse, counts, prob_sum, workspace=work)
        rr.rr_balance_loss(router, [counts], [prob_sum], loss, slope)
        if case["train"]:
            out["dlogits"] = torch.empty_like(st["logits"])
            rr.rr_route_grad(router, dt, st["logits"], st["keep"], choice, weight, lse, slope, st["grad_loss"],
                             st["grad_weight"], out["dlogits"])
    st["plan"], st["out"] = plan, out


# ---- the plain forms ------------------------------------------------------------------

def _soft_targets(case, st, index, real):
    """Target probabilities [rows, topk] of the entries that count, zero elsewhere."""
    live = index >= 0
    if case["op"] == "ce":
        return live.to(real)
    t = (st["teacher"].to(real) * case["scale"]).masked_fill(~live, -math.inf)
    top = t.amax(dim=1, keepdim=True)
    e = torch.where(live, torch.exp(t - top), torch.zeros((), dtype=real, device=t.device))
    return e / e.sum(dim=1, keepdim=True).clamp_min(torch.finfo(real).tiny)


def _plain_head(st):
    case, index = st["case"], st["index"]
    real, dt, scale = torch.float32, _DT[case["dtype"]], case["scale"]
    x = st["x"].to(real)
    ws = [w.to(real) for w in st["ws"]]
    z = [scale * (x @ w.t()) for w in ws]
    top = torch.stack([s.amax(dim=1) for s in z]).amax(dim=0)
    lse = top + torch.log(sum(torch.exp(s - top[:, None]).sum(dim=1) for s in z))
    p = _soft_targets(case, st, index, real)
    logit = torch.zeros_like(p)
    for s, first in zip(z, st["firsts"]):
        here = (index >= first) & (index < first + s.shape[1])
        logit = torch.where(here, s.gather(1, (index - first).clamp(0, s.shape[1] - 1)), logit)
    used = p.sum(dim=1) > 0
    entropy = torch.where(p > 0, p * torch.log(torch.where(p > 0, p, torch.ones_like(p))), torch.zeros_like(p))
    loss = torch.where(used, (entropy + p * (lse[:, None] - logit)).sum(dim=1), torch.zeros_like(lse))
    out = {"loss": loss, "lse": lse}
    if not case["train"]:
        return out
    g = torch.where(used, st["grad"] * scale, torch.zeros_like(lse))[:, None]
    out["dx"], dws = [], []
    for s, w, first in zip(z, ws, st["firsts"]):
        dz = g * torch.exp(s - lse[:, None])
        here = (index >= first) & (index < first + s.shape[1])
        dz.scatter_add_(1, (index - first).clamp(0, s.shape[1] - 1),
                        torch.where(here, -g * p, torch.zeros_like(p)))
        out["dx"].append((dz @ w).to(dt))
        dws.append((dz.t() @ x).to(dt))
    out["dw"] = torch.cat(dws)
    return out


def _plain_route(st):
    case = st["case"]
    real, k, e = torch.float32, case["topk"], case["experts"]
    z, keep = st["logits"].to(real), st["keep"]
    top = z.amax(dim=1, keepdim=True)
    ez = torch.exp(z - top)
    p = ez / ez.sum(dim=1, keepdim=True)
    choice = z.sort(dim=1, descending=True, stable=True)[1][:, :k]
    weight = p.gather(1, choice)
    if case["renormalize"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    weight = torch.where(keep[:, None], weight, torch.zeros_like(weight))
    p = torch.where(keep[:, None], p, torch.zeros_like(p))
    counts = torch.zeros(e + 1, dtype=torch.int32, device=z.device)
    ones = keep[:, None].to(torch.int32).expand(-1, k)
    counts[:e].scatter_add_(0, choice.reshape(-1), ones.reshape(-1))
    rows = keep.sum()
    counts[e] = rows
    n = rows.to(real).clamp_min(1)
    frac = counts[:e].to(real) / (n * k)
    loss = (e * (frac * (p.sum(dim=0) / n)).sum()).reshape(1)
    out = {"choice": torch.where(keep[:, None], choice, torch.full_like(choice, -1)).to(torch.int32),
           "weight": weight, "counts": counts, "loss": loss}
    if not case["train"]:
        return out
    a = (st["grad_loss"] * e * frac / n).expand_as(p)
    gw = st["grad_weight"]
    if case["renormalize"]:
        dz = p * (a - (p * a).sum(dim=1, keepdim=True))
        dz = dz.scatter_add(1, choice, weight * (gw - (weight * gw).sum(dim=1, keepdim=True)))
    else:
        a = a.scatter_add(1, choice, torch.where(keep[:, None], gw, torch.zeros_like(gw)))
        dz = p * (a - (p * a).sum(dim=1, keepdim=True))
    out["dlogits"] = dz.to(_DT[case["dtype"]])
    return out


# ---- the definitions in 64 bits -------------------------------------------------------

def exact(case, seed):
    """What run returns, from the definitions in 64 bits."""
    st = _inputs(case, seed)
    return (_exact_route if case["op"] == "route" else _exact_head)(case, st)


def _exact_head(case, st):
    rows, vocab, scale = case["rows"], case["vocab"], case["scale"]
    if rows * vocab * case["dim"] > 3 << 41:
        return None
    x, index = st["x"].double(), st["index"]
    live = index >= 0
    used = live.any(dim=1)
    if case["op"] == "ce":
        logp = torch.zeros(index.shape, dtype=torch.float64, device=x.device)
    else:
        t = torch.where(live, st["teacher"].double() * scale, -math.inf)
        logp = t - torch.logsumexp(torch.where(used[:, None], t, 0.0), dim=1, keepdim=True)
    logp = torch.where(live, logp, 0.0)
    p = torch.where(live, logp.exp(), 0.0)
    # blocks of the vocabulary small enough for 64-bit logits
    block = max(1, min(vocab, (1 << 28) // rows))
    at = [(v, min(v + block, vocab)) for v in range(0, vocab, block)]

    def logits(v0, v1):
        return torch.matmul(x, st["w"][v0:v1].double().t().contiguous()) * scale

    parts, logit = [], torch.zeros_like(p)
    for v0, v1 in at:
        z = logits(v0, v1)
        parts.append(torch.logsumexp(z, dim=1))
        inside = live & (index >= v0) & (index < v1)
        r, c = inside.nonzero(as_tuple=True)
        logit[r, c] = z[r, index[r, c] - v0]
    lse = torch.logsumexp(torch.stack(parts), dim=0)
    loss = (p * (logp - logit + lse[:, None])).sum(dim=1)
    out = {"loss": loss, "lse": lse}
    if not case["train"]:
        return out
    sizes = _shard_sizes(case)
    ends = [sum(sizes[:i + 1]) for i in range(len(sizes))]
    g = st["grad"].double() * scale * used
    dx = [torch.zeros_like(x) for _ in sizes]
    dw = torch.empty(vocab, case["dim"], dtype=torch.float64, device=x.device)
    for v0, v1 in at:
        dz = torch.exp(logits(v0, v1) - lse[:, None])
        inside = live & (index >= v0) & (index < v1)
        r, c = inside.nonzero(as_tuple=True)
        dz.index_put_((r, index[r, c] - v0), -p[r, c], accumulate=True)
        dz *= g[:, None]
        dw[v0:v1] = dz.t().contiguous() @ x
        for i, end in enumerate(ends):
            lo, hi = max(v0, end - sizes[i]), min(v1, end)
            if lo < hi:
                dx[i] += dz[:, lo - v0:hi - v0].contiguous() @ st["w"][lo:hi].double()
    out["dx"], out["dw"] = dx, dw
    return out


def _exact_route(case, st):
    e, k = case["experts"], case["topk"]
    z, keep = st["logits"].double(), st["keep"].nonzero().flatten()
    z = z[keep]
    n, total = keep.numel(), case["rows"]
    # the k largest, the lower index first among equals
    work, picks = z.clone(), []
    for _ in range(k):
        best = work.max(dim=1, keepdim=True)[0] if n else work[:, :1]
        at = torch.where(work == best, torch.arange(e, device=z.device), e).amin(dim=1, keepdim=True)
        picks.append(at)
        work.scatter_(1, at, -math.inf)
    pick = torch.cat(picks, dim=1)
    logp = torch.log_softmax(z, dim=1)
    chosen = logp.gather(1, pick)
    w = torch.softmax(chosen, dim=1) if case["renormalize"] else chosen.exp()
    choice = torch.full((total, k), -1, dtype=torch.int32, device=z.device)
    weight = torch.zeros(total, k, dtype=torch.float64, device=z.device)
    choice[keep], weight[keep] = pick.to(torch.int32), w
    counts = torch.cat([torch.bincount(pick.flatten(), minlength=e),
                        torch.tensor([n], device=z.device)]).to(torch.int32)
    if n:
        f = counts[:e].double() / (n * k)
        loss = e * (f @ logp.exp().mean(dim=0)).reshape(1)
    else:
        f, loss = torch.zeros(e, dtype=torch.float64, device=z.device), torch.zeros(1, dtype=torch.float64, device=z.device)
    out = {"choice": choice, "weight": weight, "counts": counts, "loss": loss}
    if not case["train"]:
        return out
    p = logp.exp()
    slope = st["grad_loss"].double() * e * f / max(n, 1)
    dz = p * (slope - (p @ slope)[:, None])
    gw = st["grad_weight"][keep].double()
    if case["renormalize"]:
        dz.scatter_add_(1, pick, w * (gw - (w * gw).sum(dim=1, keepdim=True)))
    else:
        dz.scatter_add_(1, pick, w * gw)
        dz -= p * (w * gw).sum(dim=1, keepdim=True)
    full = torch.zeros(total, e, dtype=torch.float64, device=z.device)
    full[keep] = dz
    out["dlogits"] = full
    return out


def work(case):
    """Bytes and operations of one pass that no form can leave out."""
    es, rows, k = _DT[case["dtype"]].itemsize, case["rows"], case["topk"]
    if case["op"] == "route":
        e = case["experts"]
        b = rows * e * es + rows + rows * k * 8 + (e + 1) * 4 + 4
        f = rows * e * 4
        if case["train"]:
            b += rows * e * es + rows * k * 4 + 4      # the logits' gradient, the weights' gradient
            f += rows * e * 4
        return {"bytes": b, "flops": f}
    n = rows * case["dim"] + case["vocab"] * case["dim"]
    b = n * es + rows * k * 8 + rows * 8
    if case["op"] == "kd":
        b += rows * k * es
    product = 2 * rows * case["dim"] * case["vocab"]
    if not case["train"]:
        return {"bytes": b, "flops": product}
    b += (rows * case["dim"] * case["shards"] + case["vocab"] * case["dim"]) * es + rows * 4
    # the logits, and the two products of their gradient
    return {"bytes": b, "flops": 3 * product}
