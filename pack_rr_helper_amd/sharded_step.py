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

    python -m pack_rr_helper_amd.sharded_step --steps 20
"""
import argparse

import torch

from . import (BF16, F32, Plan, Router, Vocab, rr_balance_loss, rr_route, rr_route_grad, rr_route_workspace,
               rr_vocab_cross_entropy, rr_vocab_distill, rr_vocab_grad, rr_vocab_stats, rr_vocab_workspace)

TORCH = {F32: torch.float32, BF16: torch.bfloat16}


class ShardedStep:
    """Weights, buffers and recorded calls of one step; ``step`` runs it."""

    def __init__(self, rows, dim, vocab, shards=2, experts=8, topk=2, teacher_topk=0, temperature=1.0, balance=0.01,
                 dtype=BF16, device="cuda", seed=0):
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
        keep = self.keep[:, None]
        choice = self.choice.long().clamp_min(0)
        mixed = self.scale[choice]                                     # [rows, topk, dim]
        gain = 1 + (self.weight[:, :, None] * mixed).sum(dim=1)
        self.y.copy_(x * gain)
        self.vocab()
        dgain = sum(d.float() for d in self.dx) * x                    # an all-reduce over the shards' ranks
        self.grad_weight.copy_((dgain[:, None, :] * mixed).sum(dim=2))
        self.route_grad()
        if rate:
            drouter = self.dlogits.float().t() @ x
            dscale = torch.zeros_like(self.scale).index_add_(
                0, choice.flatten(), ((self.weight * keep)[:, :, None] * dgain[:, None, :]).flatten(0, 1))
            self.router -= rate * drouter
            self.scale -= rate * dscale
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
    a = ap.parse_args(argv)
    s = ShardedStep(a.rows, a.dim, a.vocab, a.shards, teacher_topk=a.teacher_topk, temperature=2.0)
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
