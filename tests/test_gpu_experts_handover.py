"""What tiles of one step of k hand over: choices, rows and weights of a tile are fetched by all
waves of a workgroup while the tiles before it are computed, and every position's result must be
of its own row, its row's power and its own weight."""
import pytest
import torch

import pack_rr_helper_amd as rr
from tests.test_gpu_experts import Layer, check_product
from tests.test_gpu_losses import DT, device, normal, said  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16


def layer(rows, topk, experts, dim, out):
    """Rows of magnitudes 2^-20 .. 2^20, so that a row, its power or its weight taken from another position shows."""
    l = Layer(rows, topk, experts, dim, out, check=False)
    gen = torch.Generator(device="cuda").manual_seed(rows + out)
    l.x = l.x * torch.exp2(torch.randint(-20, 21, (rows, 1), generator=gen, device="cuda").float()).bfloat16()
    l.weight = normal(gen, rows, topk) + 3.0
    rr.rr_quantize_rows(BF16, l.x, l.xq)
    return l


# three tiles of a workgroup and more: of 256 x 256 with results in bf16 (the first two), of 128 x 128
# (the last two), of 128 x 128 with results in fp32 (all)
@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("rows,topk,experts,dim,out", [(8192, 4, 4, 128, 4096), (8192, 4, 6, 64, 4096), (32768, 4, 6, 128, 260),
                                                       (32768, 4, 4, 64, 260)])
def test_tiles_of_one_step(dt, rows, topk, experts, dim, out):
    l = layer(rows, topk, experts, dim, out)
    check_product(l, dt)
    check_product(l, dt, weighted=True)
    check_product(l, dt, gather=False, weighted=True)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_input_gradient_of_few_outputs(dt):
    """The product by the transposed weights, out <= 128 being its k."""
    l = layer(8192, 2, 3, 96, 2048)
    e, s = l.e, l.s
    wq, wt = rr.QuantizedWeight(3, 96, 2048), rr.QuantizedWeight(3, 2048, 96)
    w = l.w.transpose(1, 2).contiguous()                       # 96 results of 2048 inputs
    rr.rr_quantize_weight(BF16, w, wq, wt)
    l.wq, l.w = wt, l.w
    check_product(l, dt, weighted=True)


def test_weight_gradient_of_short_segments():
    """An expert's positions are one step of the weights' gradient, and none of some experts."""
    experts, n, k, rows = 60, 1024, 1024, 3000
    gen = torch.Generator(device="cuda").manual_seed(2)
    e = rr.Experts(experts, 1, rows)
    choice = (torch.randint(0, 40, (rows, 1), generator=gen, device="cuda") * 3 // 2).to(torch.int32)
    place = rr.Slots.empty(e)
    work = torch.empty(max(rr.rr_expert_workspace(e), 1), dtype=torch.uint8, device="cuda")
    rr.rr_expert_slots(e, choice, place, workspace=work)
    x = torch.randint(-4, 5, (rows, k), generator=gen, device="cuda").bfloat16()
    dy = torch.randint(-4, 5, (rows, n), generator=gen, device="cuda").bfloat16()
    m = rr.rr_expert_capacity(e)
    xt, dyt = rr.Quantized(k, m), rr.Quantized(n, m)
    rr.rr_quantize_slots(e, BF16, place, x, xt, gather=True)
    rr.rr_quantize_slots(e, BF16, place, dy, dyt, gather=True)
    for dt in (F32, BF16):
        dw = torch.empty(experts, n, k, dtype=DT[dt], device="cuda")
        rr.rr_expert_weight_grad(e, dt, place, dyt, xt, dw)
        torch.cuda.synchronize()
        for i in range(experts):
            of = (choice.flatten() == i).nonzero().flatten()
            want = dy[of].double().t() @ x[of].double()        # whole numbers, exact in 32 bits
            assert torch.equal(dw[i], want.to(DT[dt])), i
