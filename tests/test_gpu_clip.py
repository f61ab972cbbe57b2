"""The global gradient norm and the clipping on the GPU against 64 bits: sizes from
none to more than a launch's tensors, alignments, several dtypes and ranks, values
that are not finite, in place, plans and graphs."""
import math

import pytest
import torch

import pack_rr_helper_amd as rr
from tests.test_gpu_losses import DT, device, normal, said  # noqa: F401

pytestmark = pytest.mark.gpu

F32, BF16 = rr.F32, rr.BF16
U = 2.0 ** -24
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


def tensors(dt, sizes, seed=0, scale=1.0, lead=0):
    """Tensors with marked elements around them, at element offset 8 + lead."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    big = [torch.full((n + 16 + lead,), -7.25, device="cuda").to(DT[dt]) for n in sizes]
    ts = [b[8 + lead:8 + lead + n] for b, n in zip(big, sizes)]
    for t in ts:
        t.copy_(normal(gen, t.numel()) * scale)
    return big, ts


def around(big, lead=0):
    return all((b[:8 + lead] == -7.25).all() and (b[len(b) - 8:] == -7.25).all() for b in big)


def square_sum(dt, ts, stream=None):
    n = rr.rr_grad_workspace(dt, ts)
    total = torch.full((1,), -1.0, dtype=torch.float64, device="cuda")
    work = torch.full((n + 256,), 0xFF, dtype=torch.uint8, device="cuda")
    rr.rr_grad_square_sum(dt, ts, total, workspace=work[:n], stream=stream)
    torch.cuda.synchronize()
    assert (work[n:] == 0xFF).all()
    return total


def exact(ts):
    return sum((t.double() ** 2).sum().item() for t in ts)


def check(dt, ts, outs, norm, sums, limit):
    n = math.sqrt(sums)
    assert abs(norm.item() - n) <= 1.01 * U * n + 1e-44
    by = limit / n if n > limit else 1.0
    for t, o in zip(ts, outs):
        want = t.double() * by
        assert ((o.double() - want).abs() <= (HALF[dt] + 2.01 * U) * want.abs() + 1e-44).all()
        if by == 1.0:
            assert torch.equal(t, o)


SIZES = [[], [0], [1], [5], [8], [2047], [2048 * 8], [16384], [16385, 3], [1, 0, 7, 100003, 0, 64], [65536] * 91, list(range(200)),
         [3_000_001]]


@pytest.mark.parametrize("dt", [F32, BF16])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s, default=0)}")
@pytest.mark.parametrize("lead", [0, 1])
def test_against_64_bits(dt, sizes, lead):
    big, ts = tensors(dt, sizes, lead=lead)
    total = square_sum(dt, ts)
    want = exact(ts)
    # at most as many roundings in 64 bits as there are elements
    assert abs(total.item() - want) <= (sum(sizes) + 8) * 2.0 ** -52 * want
    for limit in (0.5, 1e9):
        big_out, outs = tensors(dt, sizes, seed=1, lead=3 - lead)
        norm = torch.full((1,), -1.0, device="cuda")
        rr.rr_grad_clip(dt, [total], limit, ts, outs, norm)
        torch.cuda.synchronize()
        check(dt, ts, outs, norm, want, limit)
        assert around(big, lead) and around(big_out, 3 - lead)
    # in place
    copies = [t.clone() for t in ts]
    norm = torch.empty(1, device="cuda")
    for limit in (1e9, 0.5):
        rr.rr_grad_clip(dt, [total], limit, ts, ts, norm)
        torch.cuda.synchronize()
        check(dt, copies, ts, norm, want, limit)
    assert around(big, lead)


@pytest.mark.parametrize("limit", [0.0, 0.25, 1e3])
def test_dtypes_and_ranks(limit):
    """The sums of a rank's bf16 and fp32 tensors, and of other ranks, in one norm."""
    _, a = tensors(F32, [1000, 17], seed=1)
    _, b = tensors(BF16, [333, 4096], seed=2)
    sums = [square_sum(F32, a), square_sum(BF16, b), torch.full((1,), 7.5, dtype=torch.float64, device="cuda")]
    want = exact(a) + exact(b) + 7.5
    for dt, ts in ((F32, a), (BF16, b)):
        outs = [torch.empty_like(t) for t in ts]
        norm = torch.empty(1, device="cuda")
        rr.rr_grad_clip(dt, sums, limit, ts, outs, norm)
        torch.cuda.synchronize()
        check(dt, ts, outs, norm, want, limit)


def test_shapes_are_free():
    x = torch.randn(7, 5, 3, device="cuda")
    y = torch.empty_like(x)
    total, norm = square_sum(F32, [x]), torch.empty(1, device="cuda")
    rr.rr_grad_clip(F32, [total], 1.0, [x], [y], norm)
    torch.cuda.synchronize()
    check(F32, [x.flatten()], [y.flatten()], norm, exact([x]), 1.0)


@pytest.mark.parametrize("dt", [F32, BF16])
def test_large_and_small_values(dt):
    """Squares that 32 bits do not hold: finite tensors have a finite sum."""
    for v in (3e38, 1e-38, 1e-41):
        x = torch.full((1000,), v, device="cuda").to(DT[dt])
        total, norm, y = square_sum(dt, [x]), torch.empty(1, device="cuda"), torch.empty_like(x)
        assert abs(total.item() - exact([x])) <= 1e-12 * exact([x])
        rr.rr_grad_clip(dt, [total], 1.0, [x], [y], norm)
        torch.cuda.synchronize()
        # a norm past fp32's range is told as infinite, the tensors are scaled all the same
        n = math.sqrt(exact([x]))
        if n > 1:
            # the factor may be a subnormal number, rounded to steps of 2^-149
            assert abs(y.double().norm().item() - 1.0) <= HALF[dt] * 2 + 1e-6 + n * 2.0 ** -150
            assert norm.item() == math.inf or abs(norm.item() - n) <= 1.01 * U * n
        else:
            assert torch.equal(x, y)


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_not_finite(bad):
    """The norm tells, the values stay."""
    x = torch.randn(5000, device="cuda")
    x[1234] = bad
    total, norm, y = square_sum(F32, [x]), torch.empty(1, device="cuda"), torch.zeros_like(x)
    rr.rr_grad_clip(F32, [total], 1.0, [x], [y], norm)
    torch.cuda.synchronize()
    assert not math.isfinite(norm.item()) and math.isnan(norm.item()) == math.isnan(bad)
    assert torch.equal(x.view(torch.int32), y.view(torch.int32))


def test_past_2_31_elements():
    n = (1 << 31) + 12345
    x = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    x[0], x[1 << 31], x[n - 1] = 1.0, 2.0, -4.0
    total, norm = square_sum(BF16, [x]), torch.empty(1, device="cuda")
    assert total.item() == 21.0
    rr.rr_grad_clip(BF16, [total], 0.5, [x], [x], norm)
    torch.cuda.synchronize()
    by = 0.5 / math.sqrt(21.0)
    for i, v in ((0, 1.0), (1 << 31, 2.0), (n - 1, -4.0)):
        assert abs(x[i].item() - v * by) <= 2.0 ** -7 * abs(v * by)


def test_plan_graph_and_streams():
    _, ts = tensors(BF16, [100000, 33, 0, 4097] * 30)
    outs, norm = [torch.empty_like(t) for t in ts], torch.empty(1, device="cuda")
    total = torch.empty(1, dtype=torch.float64, device="cuda")
    work = torch.empty(rr.rr_grad_workspace(BF16, ts), dtype=torch.uint8, device="cuda")

    def issue(stream=None):
        rr.rr_grad_square_sum(BF16, ts, total, workspace=work, stream=stream)
        rr.rr_grad_clip(BF16, [total], 1.0, ts, outs, norm, stream=stream)

    issue()
    torch.cuda.synchronize()
    first = [t.clone() for t in (*outs, norm, total)]

    def same():
        torch.cuda.synchronize()
        return all(torch.equal(a, b) for a, b in zip(first, (*outs, norm, total)))

    def clear():
        for t in (*outs, norm, total):
            t.fill_(0)

    with rr.Plan(16) as plan:
        issue()
    clear()
    plan()
    assert same()
    s = torch.cuda.Stream()
    clear()
    s.wait_stream(torch.cuda.current_stream())
    issue(stream=s)
    s.synchronize()
    assert same()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        plan()
    for _ in range(3):
        clear()
        g.replay()
        assert same()
        clear()
        issue()
        assert same()


def test_more_tiles_than_a_launch():
    """A tensor that takes two launches to scale, its last elements in the second."""
    n = (1 << 35) + 5
    if torch.cuda.mem_get_info()[0] < 2 * n + (8 << 30):
        pytest.skip("not the memory for it")
    t = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    t[0], t[n - 6], t[n - 5], t[n - 1] = 2, 1, 2, 4
    total = square_sum(BF16, [t])
    norm = torch.full((1,), -1.0, device="cuda")
    rr.rr_grad_clip(BF16, [total], 2.5, [t], [t], norm)
    torch.cuda.synchronize()
    assert total.item() == 25.0 and norm.item() == 5.0
    assert [t[i].item() for i in (0, 1, n - 6, n - 5, n - 4, n - 1)] == [1.0, 0.0, 0.5, 1.0, 0.0, 2.0]
    del t
    torch.cuda.empty_cache()
