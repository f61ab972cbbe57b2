"""The sharded step with a router in groups, experts as 8-bit products and clipping:
each of its gradients against 64 bits from the stages before it, and its updates."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd import sharded_step
from pack_rr_helper_amd.sharded_step import ShardedStep
from tests import expert_ref as ref
from tests.test_gpu_losses import DT, device, normal, said  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16


def inputs(rows, dim, vocab):
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x = normal(gen, rows, dim)
    index = torch.randint(0, vocab, (rows, 1), generator=gen, device="cuda")
    index[::7] = -1
    return x, index


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,dim", [(60, 136), (700, 64)])
def test_gradients(dt, rows, dim):
    vocab, r = 300, rr.GroupRouter(8, 2, 4, 2, 2, True, True, 1.5)
    s = ShardedStep(rows, dim, vocab, shards=2, dtype=dt, router=r, products=True)
    x, index = inputs(rows, dim, vocab)
    loss, balance = s.step(x, index)
    torch.cuda.synchronize()
    assert math.isfinite(loss.item()) and balance.item() == 0.0
    t, keep = DT[dt], (index >= 0).flatten()
    want = ref.group_route(r, s.logits, s.bias, keep)
    assert torch.equal(s.choice, want["choice"]) and torch.equal(s.counts, want["counts"])
    x8 = ref.eight(x.to(t))[0]
    mix, size = (torch.zeros(rows, dim, dtype=torch.float64, device="cuda") for _ in range(2))
    g, size_g = (torch.zeros(rows * 2, dtype=torch.float64, device="cuda") for _ in range(2))
    weight, choice = s.weight.flatten(), s.choice.flatten()
    for i in range(8):
        n = (choice == i).nonzero().flatten()
        of, w8 = n // 2, ref.eight(s.experts[i], 128)[0]
        o = x8[of] @ w8.t()
        tol = ref.product_bound(x8[of], w8, o, torch.float32)
        by = weight[n].double()[:, None]
        mix.index_add_(0, of, by * o)
        size.index_add_(0, of, by.abs() * (tol + 8 * ref.U * o.abs()))
        dy = s.dy[of].double()
        g[n] = (o * dy).sum(dim=1)
        size_g[n] = ((tol + (dim + 8) * ref.U * o.abs()) * dy.abs()).sum(dim=1)
        # the contraction over an expert's rows in blocks of 128
        a, b = ref.eight((weight[n, None] * s.dy.float()[of]).t().contiguous())[0], ref.eight(x.to(t)[of].t().contiguous())[0]
        dw = a @ b.t()
        assert ((s.dexperts[i].double() - dw).abs() <= ref.product_bound(a, b, dw, t)).all()
    assert ((s.mix.double() - mix).abs() <= size + (ref.HALF[t] + ref.U) * mix.abs()).all()
    assert ((s.grad_weight.double() - g.reshape(rows, 2)).abs() <= size_g.reshape(rows, 2)).all()
    d, tol = ref.group_route_grad(r, s.logits, s.choice, s.grad_weight, t)
    assert ((s.dlogits.double() - d).abs() <= tol).all()
    assert not s.bias.any()                                            # moves with an update only


@pytest.mark.parametrize("products", [False, True])
@pytest.mark.parametrize("limit", [1e-3, 1e6])
def test_update_and_clip(products, limit):
    rows, dim, vocab, rate = 200, 72, 150, 0.5
    r = rr.GroupRouter(8, 2, 2, 1, 1, False, False)
    s = ShardedStep(rows, dim, vocab, shards=3, dtype=F32, router=r, bias_rate=0.25, products=products, max_norm=limit)
    x, index = inputs(rows, dim, vocab)
    s.step(x, index)
    router, head, experts = s.router.clone(), s.head.clone(), (s.experts if products else s.scale).clone()
    dhead, dlogits = s.dhead.double().clone(), s.dlogits.double().clone()
    counts = s.counts.clone()
    s.step(x, index, rate=rate)
    torch.cuda.synchronize()
    norm, by = s.norm.item(), min(1.0, limit / s.norm.item())
    drouter = dlogits.t() @ x.double()
    # the experts' gradient from what the update took away
    dexperts = (experts - (s.experts if products else s.scale)).double() / (rate * by)
    want = math.sqrt(drouter.square().sum().item() + dhead.square().sum().item() + dexperts.square().sum().item())
    # differences of weights about 1 and below, over the rate and the factor
    lost = 2.0 ** -23 / (rate * by) * math.sqrt(experts.numel() + head.numel()) + 1e-4 * want
    assert abs(norm - want) <= lost
    assert ((s.head.double() - (head.double() - rate * by * dhead)).abs() <= 4 * ref.U * (head.abs() + rate * by * dhead.abs()) + 1e-30).all()
    moved = rate * by * drouter
    mag = rate * by * (dlogits.abs().t() @ x.double().abs())
    assert ((s.router.double() - (router.double() - moved)).abs() <= 4 * ref.U * router.abs() + (rows + 16) * ref.U * mag + 1e-30).all()
    n = counts[:8].double()
    assert torch.equal(s.bias, (0.25 * torch.sign(n.sum() - n * 8)).float())


def test_command():
    """The command runs with each of its options."""
    sharded_step.main("--steps 2 --rows 64 --dim 32 --vocab 100 --shards 2 --groups 4 --products --max-norm 1".split())
    sharded_step.main("--steps 2 --rows 64 --dim 32 --vocab 100 --shards 2 --groups 2 --teacher-topk 4".split())
    sharded_step.main("--steps 2 --rows 64 --dim 32 --vocab 100 --shards 2 --products --max-norm 0.1".split())
