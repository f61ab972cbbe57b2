"""A training step with the sharded losses, all ranks on one GPU.

A batch of tokens goes through a layer of experts and a vocabulary head that is
split over ``shards`` ranks.  Every rank's calls are issued one after the other
here, and what ranks would exchange (statistics, picked logits, partial input
gradients) simply lies side by side.  The calls are recorded once into plans;
torch supplies the memory, the router's and the experts' own small products and
the weight updates::

    y       = x * (1 + sum_k weight_k * scale[choice_k])      the experts
    loss    = sum over targets of cross entropy(y, head) / n + balance * balance loss

With a teacher's top logits the head's loss is the distillation instead, times
the square of the temperature as usual.

With a router in groups (``router``) the choice is balanced by a bias, which each
step moves by ``bias_rate``, and there is no balance loss.  With ``products`` the
experts are matrices, multiplied in 8 bits::

    y       = x + sum_k weight_k * (experts[choice_k] x)

With ``max_norm`` the gradients are clipped to that norm over all weights before an
update; a step whose gradients have no finite sum of squares changes no weight and no bias.

    python -m pack_rr_helper_amd.sharded_step --steps 20
    python -m pack_rr_helper_amd.sharded_step --groups 4 --products --max-norm 1
"""
import argparse

import torch

from . import (BF16, F32, Experts, GroupRouter, Plan, Quantized, QuantizedWeight, Router, Slots, Vocab, rr_balance_loss,
               rr_expert_capacity, rr_expert_combine, rr_expert_combine_grad, rr_expert_product, rr_expert_slots,
               rr_expert_weight_grad, rr_expert_workspace, rr_grad_clip, rr_grad_square_sum, rr_grad_workspace,
               rr_group_route, rr_group_route_grad, rr_group_route_workspace, rr_quantize_rows, rr_quantize_slots,
               rr_quantize_weight, rr_route, rr_route_bias, rr_route_grad, rr_route_workspace, rr_vocab_cross_entropy,
               rr_vocab_distill, rr_vocab_grad, rr_vocab_stats, rr_vocab_workspace)

TORCH = {F32: torch.float32, BF16: torch.bfloat16}


class ShardedStep:
    """Weights, buffers and recorded calls of one step; ``step`` runs it."""

    def __init__(self, rows, dim, vocab, shards=2, experts=8, topk=2, teacher_topk=0, temperature=1.0, balance=0.01,
                 dtype=BF16, device="cuda", seed=0, router=None, bias_rate=0.001, products=False, max_norm=None):
        if router is not None:
            experts, topk = router.experts, router.topk
        gen = torch.Generator(device=device).manual_seed(seed)
        t, k = TORCH[dtype], max(teacher_topk, 1)
        self.rows, self.entries, self.balance, self.distills = rows, vocab, balance, teacher_topk > 0
        self.temperature = temperature if self.distills else 1.0

        def normal(*shape):
            return torch.randn(*shape, generator=gen, device=device)

        def empty(dt, *shape):
            return torch.empty(*shape, dtype=dt, device=device)

        f32 = torch.float32
        self.head = (normal(vocab, dim) * dim ** -0.5).to(t)
        self.router = normal(experts, dim) * dim ** -0.5
        self.scale = normal(experts, dim) * 0.1
        sizes = [vocab // shards + (i < vocab % shards) for i in range(shards)]
        firsts = [sum(sizes[:i]) for i in range(shards)]
        self.shards = [Vocab(dim, n, first, vocab, k, 1.0 / self.temperature) for n, first in zip(sizes, firsts)]
        # what a caller fills before a step
        self.y, self.logits = empty(t, rows, dim), empty(t, rows, experts)
        self.keep = torch.ones(rows, dtype=torch.bool, device=device)
        self.index = torch.full((rows, k), -1, dtype=torch.int64, device=device)
        self.teacher = torch.zeros(rows, k, dtype=t, device=device)
        self.grad, self.grad_weight = empty(f32, rows), empty(f32, rows, topk)
        self.grad_balance = torch.full((1,), balance, device=device)
        # what the calls fill
        self.choice, self.weight = empty(torch.int32, rows, topk), empty(f32, rows, topk)
        self.loss, self.balance_loss = empty(f32, rows), empty(f32, 1)
        self.dx = [empty(t, rows, dim) for _ in range(shards)]
        self.dhead, self.dlogits = torch.empty_like(self.head), empty(t, rows, experts)

        self.move_bias = None
        if router is None:
            r = Router(experts, topk)
            counts, prob_sum, slope, lse = (empty(torch.int32, experts + 1), empty(f32, experts), empty(f32, experts),
                                            empty(f32, rows))
            work = empty(torch.uint8, max(rr_route_workspace(r, rows), 1))
            with Plan(8) as self.route:
                rr_route(r, dtype, self.logits, self.keep, self.choice, self.weight, lse, counts, prob_sum, workspace=work)
                rr_balance_loss(r, [counts], [prob_sum], self.balance_loss, slope)
            with Plan(8) as self.route_grad:
                rr_route_grad(r, dtype, self.logits, self.keep, self.choice, self.weight, lse, slope, self.grad_balance,
                              self.grad_weight, self.dlogits)
        else:
            self._group_router(router, dtype, bias_rate, empty)
        self.products, self.max_norm = products, max_norm
        if products:
            self.experts = (normal(experts, dim, dim) * 0.1 * dim ** -0.5).to(t)
            self._products(experts, topk, dtype, empty)
        stats, picked = [empty(f32, rows, 2) for _ in sizes], [empty(f32, rows, k) for _ in sizes]
        lse, logit = empty(f32, rows), empty(f32, rows, k)
        prob = empty(f32, rows, k) if self.distills else None
        work = empty(torch.uint8, max(rr_vocab_workspace(v, dtype, rows, grad=True) for v in self.shards))
        parts = list(zip(self.shards, self.head.split(sizes), stats, picked, self.dx, self.dhead.split(sizes)))
        with Plan(1024) as self.vocab:
            for v, w, s, p, _, _ in parts:
                rr_vocab_stats(v, dtype, self.y, w, self.index, s, p, workspace=work)
            if self.distills:
                rr_vocab_distill(self.shards[0], dtype, self.index, self.teacher, stats, picked, lse, logit, prob, self.loss)
            else:
                rr_vocab_cross_entropy(self.shards[0], self.index, stats, picked, lse, logit, self.loss)
            for v, w, _, _, dx, dw in parts:
                rr_vocab_grad(v, dtype, self.y, w, self.index, lse, logit, prob, self.grad, dx, dw, workspace=work)

    def _group_router(self, r, dtype, bias_rate, empty):
        """Records a router in groups and what moves its bias."""
        self.bias, logit = torch.zeros_like(self.router[:, 0]), torch.empty_like(self.weight)
        self.counts = empty(torch.int32, r.experts + 1)
        self.balance_loss.zero_()
        lse = empty(torch.float32, self.rows) if r.whole else None
        work = empty(torch.uint8, max(rr_group_route_workspace(r, self.rows), 1))
        with Plan(8) as self.route:
            rr_group_route(r, dtype, self.logits, self.bias, self.keep, self.choice, self.weight, logit, lse, self.counts,
                           workspace=work)
        with Plan(8) as self.route_grad:
            rr_group_route_grad(r, dtype, self.logits if r.whole else None, self.choice, logit, lse, self.grad_weight,
                                self.dlogits)
        with Plan(8) as self.move_bias:                                # of all ranks' counts
            rr_route_bias(r, [self.counts], bias_rate, self.bias, self.bias)

    def _products(self, experts, topk, dtype, empty):
        """Records the experts' products: forward, and the gradients of the experts and the router's weights."""
        e, dim = Experts(experts, topk, self.rows), self.experts.shape[2]
        n, t = rr_expert_capacity(e), TORCH[dtype]
        self.x, self.dy, self.mix = (empty(t, self.rows, dim) for _ in range(3))
        self.dexperts = torch.empty_like(self.experts)
        place, held = Slots.empty(e, self.x.device), empty(torch.float32, n, dim)
        xq, wq = Quantized(self.rows, dim, self.x.device), QuantizedWeight(experts, dim, dim, self.x.device)
        xt, dyt = (Quantized(dim, n, self.x.device) for _ in range(2))
        work = empty(torch.uint8, max(rr_expert_workspace(e), 1))
        with Plan(16) as self.mixing:
            rr_expert_slots(e, self.choice, place, workspace=work)
            rr_quantize_weight(dtype, self.experts, wq)
            rr_quantize_rows(dtype, self.x, xq)
            rr_expert_product(e, F32, place, xq, wq, held, gather=True)
            rr_expert_combine(e, F32, dtype, place, held, self.weight, self.mix)
        with Plan(16) as self.mixing_grad:
            rr_expert_combine_grad(e, F32, dtype, place, held, self.dy, self.grad_weight)
            rr_quantize_slots(e, dtype, place, self.x, xt, gather=True)
            rr_quantize_slots(e, dtype, place, self.dy, dyt, weight=self.weight, gather=True)
            rr_expert_weight_grad(e, dtype, place, dyt, xt, self.dexperts)

    def _clip(self, grads):
        """Scales the gradients in place to the norm that they may have over all weights, and returns theirs and
        whether it is finite; if not, the gradients become zeros.  The sums of squares tell, as the norm is a
        float: infinite too where a finite norm is past fp32's range."""
        totals, kinds = [], []
        for dtype, t in TORCH.items():
            these = [g for g in grads if g.dtype == t]
            if these:
                totals.append(torch.empty(1, dtype=torch.float64, device=these[0].device))
                kinds.append((dtype, these))
                work = torch.empty(max(rr_grad_workspace(dtype, these), 1), dtype=torch.uint8, device=these[0].device)
                rr_grad_square_sum(dtype, these, totals[-1], workspace=work)
        norm = torch.empty(1, device=grads[0].device)
        for dtype, these in kinds:
            rr_grad_clip(dtype, totals, self.max_norm, these, these, norm)
        finite = torch.isfinite(sum(totals))
        for g in grads:
            g.masked_fill_(~finite, 0)
        return norm, finite

    def step(self, x, index, teacher=None, rate=0.0):
        """One step on x [rows, dim]; index [rows, k] holds the targets (below 0,
        or not below the vocabulary's size: none), teacher [rows, k] the teacher's
        logits for them.  Returns the mean cross entropy or divergence of the rows
        that have a target, without the temperature's square and the balance, and
        the balance loss."""
        self.index.copy_(index)
        if self.distills:
            self.teacher.copy_(teacher)
        torch.any((self.index >= 0) & (self.index < self.entries), dim=1, out=self.keep)
        n = self.keep.sum().clamp_min(1)
        self.grad.copy_(self.temperature ** 2 / n)
        x = x.float()
        self.logits.copy_(x @ self.router.t())
        self.route()
        if self.products:
            self.x.copy_(x)
            self.mixing()
            self.y.copy_(x + self.mix.float())
            self.vocab()
            self.dy.copy_(sum(d.float() for d in self.dx))             # an all-reduce over the shards' ranks
            self.mixing_grad()
        else:
            keep = self.keep[:, None]
            choice = self.choice.long().clamp_min(0)
            mixed = self.scale[choice]                                 # [rows, topk, dim]
            gain = 1 + (self.weight[:, :, None] * mixed).sum(dim=1)
            self.y.copy_(x * gain)
            self.vocab()
            dgain = sum(d.float() for d in self.dx) * x                # an all-reduce over the shards' ranks
            self.grad_weight.copy_((dgain[:, None, :] * mixed).sum(dim=2))
        self.route_grad()
        if rate:
            drouter = self.dlogits.float().t() @ x
            if self.products:
                dexperts = self.dexperts
            else:
                dexperts = torch.zeros_like(self.scale).index_add_(
                    0, choice.flatten(), ((self.weight * keep)[:, :, None] * dgain[:, None, :]).flatten(0, 1))
            finite = None
            if self.max_norm is not None:
                self.norm, finite = self._clip([drouter, dexperts, self.dhead])
            self.router -= rate * drouter
            if self.move_bias is not None:
                before = None if finite is None else self.bias.clone()
                self.move_bias()
                if finite is not None:
                    self.bias.copy_(torch.where(finite, self.bias, before))
            if self.products:
                self.experts -= (rate * dexperts.float()).to(self.experts.dtype)
            else:
                self.scale -= rate * dexperts
            self.head -= (rate * self.dhead.float()).to(self.head.dtype)
        return self.loss.sum() / n, self.balance_loss[0]


def main(argv=None):
    ap = argparse.ArgumentParser(description="train a small sharded head with experts on random text")
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rows", type=int, default=1024)
    ap.add_argument("--dim", type=int, default=256)
    ap.add_argument("--vocab", type=int, default=4000)
    ap.add_argument("--shards", type=int, default=4)
    ap.add_argument("--teacher-topk", type=int, default=0)
    ap.add_argument("--groups", type=int, default=0, help="route in this many groups of four experts, balanced by a bias")
    ap.add_argument("--products", action="store_true", help="experts that are matrices, multiplied in 8 bits")
    ap.add_argument("--max-norm", type=float, default=None, help="clip the gradients to this norm")
    a = ap.parse_args(argv)
    router = GroupRouter(4 * a.groups, 2, a.groups, max(a.groups // 2, 1), 2) if a.groups else None
    s = ShardedStep(a.rows, a.dim, a.vocab, a.shards, teacher_topk=a.teacher_topk, temperature=2.0, router=router,
                    products=a.products, max_norm=a.max_norm)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.rows, a.dim, generator=gen, device="cuda")
    k = max(a.teacher_topk, 1)
    index = torch.randint(0, a.vocab, (a.rows, k), generator=gen, device="cuda")
    index[::10] = -1                                                   # prompt positions
    teacher = torch.randn(a.rows, k, generator=gen, device="cuda")
    for i in range(a.steps):
        loss, balance = s.step(x, index, teacher, rate=20.0)
        print(f"step {i}: loss {loss.item():.4f}, balance {balance.item():.4f}", flush=True)


if __name__ == "__main__":
    main()
