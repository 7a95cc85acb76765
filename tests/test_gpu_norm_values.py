"""moe_rmsnorm at the ends of the number range."""
import pytest
import torch

import mixture_experts_forward_moe_amd as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.mark.parametrize("H", [64, 512, 6144, 16384])
@pytest.mark.parametrize("wdtype", [torch.float32, BF16])
def test_rows_whose_squares_overflow(H, wdtype):
    """r is 0 and y is 0, whatever h * weight would be; an infinity among them
    is NaN, in its place alone; the gradients are those of a constant."""
    print(f"norm overflow H={H} {wdtype}", flush=True)
    x = torch.ones(5, H)
    x[0] = 3.0e38
    x[1] = -3.3e38
    x[2, 1] = 2.0e19
    x[3] = 1.0e20
    x[3, 3] = float("inf")
    x = x.to(BF16)
    w = torch.linspace(-40, 40, H).to(wdtype)
    y, r = torch.full((5, H), 7, dtype=BF16, device="cuda"), torch.full((5,), 7.0, device="cuda")
    q, sf = torch.full((5, H), 7, dtype=torch.uint8, device="cuda"), torch.full((5, H // 32), 7, dtype=torch.uint8, device="cuda")
    moe.moe_rmsnorm(x.cuda(), w.cuda(), y=y, q=q, q_sf=sf, rstd=r)
    y, r = y.cpu(), r.cpu()
    assert bool((r[:4] == 0).all()) and abs(r[4].item() - 1) < 1e-6
    assert bool((y[:3] == 0).all())
    assert bool(torch.isnan(y[3, 3])) and bool((y[3, torch.arange(H) != 3] == 0).all())
    assert bool(((y[4].double() - w.double()).abs() <= w.double().abs() * (2.0 ** -8 + 2.0 ** -19)).all())
    assert bool(((q[:3].cpu() & 127) == 0).all()) and bool((sf[:3].cpu() == 0).all())
    dy, dh = torch.ones(3, H, dtype=BF16, device="cuda"), torch.full((3, H), 0.5, dtype=BF16, device="cuda")
    dx, dw = torch.empty_like(dy), torch.empty(H, device="cuda")
    moe.moe_rmsnorm_backward(dy, x[:3].cuda(), w.cuda(), r[:3].cuda(), dx, dw, dh=dh)
    assert torch.equal(dx, dh) and bool((dw == 0).all())
