"""Rows at the ends of bf16's range through the quantiser, the products and the
weights' gradient; at the lower one: what the quantiser makes of them decodes exactly, in
bf16 too, and nothing is lost on the way to an fp32 result that has room."""
import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from test_gpu_fp8_rows import BF16, BYTE, gen, say

pytestmark = pytest.mark.gpu

N, K = 136, 272


def test_what_the_quantiser_makes_is_bf16():
    """Every magnitude up to the least scale's largest value, each alone with every block maximum of a power of two: the
    value that the codes stand for is a bf16 (the CPU's form of the quantiser, which the kernel's is compared with)."""
    say("what the quantiser makes is bf16")
    bits = torch.arange(0, 0x0880, dtype=torch.int32).to(torch.int16)  # up to 2^-110
    v = bits.view(BF16)
    for top in range(-133, -109):
        small = v[v <= 2.0 ** top]
        x = torch.zeros(len(small), 128, dtype=BF16)
        x[:, 0], x[:, 1] = 2.0 ** top, small
        q, sf = (torch.empty(len(x), c, dtype=BYTE, device="cuda") for c in (128, 1))
        moe.moe_quantize_fp8(x.cuda(), q, sf)
        rq, rs = ref.quantize(x)
        assert torch.equal(q.cpu(), rq) and torch.equal(sf.cpu(), rs)
        kept = ref.rows(rq, rs)
        assert torch.equal(kept.to(BF16).double(), kept)


@pytest.mark.parametrize("low", [-133, -131, -127, -126, -124, -110])
@pytest.mark.parametrize("M", [7, 40, 600])
def test_products(low, M):
    """Whole numbers times 2^low with weights, or a gradient, times 2^100: sums of whole numbers, exact."""
    say(f"products of small values 2^{low}, {M} rows")
    x = (torch.randint(-3, 4, (M, K), generator=gen(M)).double() * 2.0 ** low).to(BF16)
    q, sf = (torch.empty(M, c, dtype=BYTE, device="cuda") for c in (K, 3))
    moe.moe_quantize_fp8(x.cuda(), q, sf)
    w = ref.encode(torch.randint(-2, 3, (N, K), generator=gen(2)).double()).cuda()
    w_sf = torch.full((2, 3), 2.0 ** 100, device="cuda")
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_fp8(q, sf, w, w_sf, y)
    xv = x.double().cuda()
    assert torch.equal(y, torch.mm(xv, ref.weights(w, w_sf).t().contiguous()).float())
    dy = (torch.randint(-3, 4, (M, N), generator=gen(3)).double() * 2.0 ** 100).to(BF16).cuda()
    dw = torch.empty(N, K, device="cuda")
    moe.moe_linear_fp8_wgrad(dy, q, sf, dw)
    assert torch.equal(dw, torch.mm(dy.double().t().contiguous(), xv).float())


@pytest.mark.parametrize("M", [4, 40])
def test_the_largest_values(M):
    """What is kept as 2^128 multiplies as that; the weights' gradient has an infinity of it."""
    say(f"the largest values, {M} rows")
    x = torch.zeros(M, K, dtype=BF16)
    x[1, 3], x[2, 5], x[3, 7] = 3.38e38, -3.3e38, 3.2e38
    q, sf = (torch.empty(M, c, dtype=BYTE, device="cuda") for c in (K, 3))
    moe.moe_quantize_fp8(x.cuda(), q, sf)
    kept = ref.rows(*ref.quantize(x))
    assert kept[1, 3] == 2.0 ** 128 and kept[2, 5] == -2.0 ** 128 and kept[3, 7] < 2.0 ** 128
    w = ref.encode(torch.full((N, K), 0.5).double()).cuda()
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_fp8(q, sf, w, torch.ones(2, 3, device="cuda"), y)
    assert torch.equal(y.cpu(), (kept.sum(1, keepdim=True) * 0.5).float().expand(-1, N))
    dw = torch.empty(N, K, device="cuda")
    moe.moe_linear_fp8_wgrad(torch.full((M, N), 2.0 ** -9, dtype=BF16, device="cuda"), q, sf, dw)
    want = (kept * 2.0 ** -9).sum(0)
    want[3], want[5] = float("inf"), -float("inf")
    assert torch.equal(dw.cpu(), want.float().expand(N, -1))
