"""Slots of many positions to 8 bits: more blocks than a launch may have go in several launches,
none of which the runtime refuses for its threads."""
import pytest
import torch

import pack_rr_helper_amd as rr
from pack_rr_helper_amd import experts as ex
from tests.test_experts_host import BF16, OK, call, layer, recorded


def test_recorded_launches():
    L = ex._lib()
    # fake buffers a pebibyte apart, which no call reads here
    far = {n: (i + 1) << 50 for i, n in enumerate(("x", "weight", "source", "offset", "values", "powers"))}

    def launches(rows, topk, dim):
        return recorded(L, lambda: call(L, "rr_quantize_slots", e=layer(rows=rows, topk=topk, experts=1), dim=dim, **far), 2000)

    # a launch has less than 2^32 threads, 256 to a block of 128 x 128
    for rows, topk, dim in ((1 << 23, 32, 65536), (1 << 28, 1, 897), (1 << 20, 16, 65536), (1 << 27, 1, 1), (1 << 28, 1, 1)):
        blocks = -(-dim // 128) * -(-(rows * topk + 127) // 128)
        st, n = launches(rows, topk, dim)
        assert st == OK and n >= -(-blocks * 256 // ((1 << 32) - 1)), (rows, topk, dim)
    assert launches(1 << 22, 4, 2048) == (OK, 2 + 1)
    assert launches(65536, 8, 4096) == (OK, 1) and launches(1, 1, 1) == (OK, 1)


@pytest.mark.gpu
def test_positions_in_two_launches():
    """Positions of two launches, a block on both sides of the border and the last one looked at."""
    rows, topk = (1 << 27) // 32 + 100, 32
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("not the memory for it")
    e = rr.Experts(2, topk, rows)
    gen = torch.Generator(device="cuda").manual_seed(1)
    choice = torch.zeros(rows, topk, dtype=torch.int32, device="cuda")
    choice[rows // 2:] = 1
    place, n = rr.Slots.empty(e), rr.rr_expert_capacity(e)
    assert n // 128 > 1 << 20
    work = torch.empty(max(rr.rr_expert_workspace(e), 1), dtype=torch.uint8, device="cuda")
    rr.rr_expert_slots(e, choice, place, workspace=work)
    x = torch.randint(-8, 9, (rows, 1), generator=gen, device="cuda").bfloat16()
    q = rr.Quantized(1, n)
    q.values.view(torch.uint8).fill_(0x5A)
    q.powers.fill_(0x5A)
    rr.rr_quantize_slots(e, BF16, place, x, q, gather=True)
    torch.cuda.synchronize()
    end = place.offset[2].item()
    src = place.source[:end].long()
    want = torch.where(src >= 0, x[src.clamp_min(0) // topk, 0].float(), 0.0)
    power = torch.exp2(q.powers[0, :end // 128].float() - 127)
    got = q.values[0, :end].float() * power.repeat_interleave(128)
    assert torch.equal(got, want)                              # whole numbers up to 8 have four bits
    assert (q.values[0, end:].view(torch.uint8) == 0x5A).all()
    del x, q, choice, place, src, want, got, power
    torch.cuda.empty_cache()
