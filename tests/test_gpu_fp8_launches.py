"""Launches of the calls on rows in 8 bits at the ends of their documented
ranges: recorded with the largest sizes (placeholder addresses; nothing runs),
and run past 2^32 threads in all, where memory allows it."""
import ctypes

import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from hip_kernels import launches_of
from test_gpu_fp8_rows import BF16, BYTE, I32, gen, say

pytestmark = pytest.mark.gpu

F = 0x10000
H = 16384


def plan_args(M, k=1, tile=16, El=1):
    p = moe.Plan()
    n = moe.lib().moe_plan_workspace_size(M, k, El, tile)
    assert moe.lib().moe_plan_init(ctypes.byref(p), ctypes.c_void_p(F), n, M, k, El, tile) == 0
    return p


M22 = 1 << 22
ENDS = {
    "dispatch, rows": ("moe_dispatch", lambda s: (F, 0, ctypes.byref(plan_args(M22)), H, F, None, None, s), M22 * 32),
    "dispatch, codes": ("moe_dispatch", lambda s: (F, 0, ctypes.byref(plan_args(M22)), H, None, F, F, s), M22 * 16),
    "dispatch, both": ("moe_dispatch", lambda s: (F, 0, ctypes.byref(plan_args(M22)), H, F, F, F, s), M22 * 16),
    "dispatch backward": ("moe_dispatch_backward", lambda s: (F, ctypes.byref(plan_args(M22)), H, 0, F, s), M22 * 32),
    "finalize backward": ("moe_finalize_backward",
                          lambda s: (F, F, ctypes.byref(plan_args(M22)), F, H, 1.0, F, F, F, F, s), M22 * 4),
    "quantize": ("moe_quantize_fp8", lambda s: (F, 0, 1 << 25, 2048, F, F, s), 1 << 25),
    "quantize, a long row": ("moe_quantize_fp8", lambda s: (F, 0, 64, 1 << 30, F, F, s), 1 << 25),
    "quantize weights": ("moe_quantize_fp8_weight", lambda s: (F, 1 << 23, 128, 128, F, F, F, F, s), 1 << 25),
    "act": ("moe_gated_act_fp8", lambda s: (F, None, 1 << 25, 1024, 0, 1.0, 0.0, moe.FLT_MAX, F, F, F, F, s), 1 << 25),
    "act backward": ("moe_gated_act_fp8_backward",
                     lambda s: (F, F, F, None, 1 << 25, 1024, 0, 1.0, 0.0, moe.FLT_MAX, F, F, F, s), 1 << 25),
    # the products: a workgroup a tile while few are at work, else as many as the GPU holds
    "linear, columns": ("moe_linear_fp8", lambda s: (F, F, F, F, F, 16, 1 << 26, 16, 0, F, 0, s), 1 << 24),
    "linear, rows": ("moe_linear_fp8", lambda s: (F, F, F, F, F, 1 << 26, 1 << 10, 1 << 20, 0, F, 1, s), 1),
    "grouped, tiles of 16": ("moe_grouped_linear_fp8",
                             lambda s: (F, F, ctypes.byref(plan_args((1 << 23) - 64)), F, F, 256, 64, F, s), 1 << 24),
    "grouped, tiles of 256": ("moe_grouped_linear_fp8",
                              lambda s: (F, F, ctypes.byref(plan_args((1 << 20) - 256, tile=256)), F, F, 1 << 16, 64, F, s), 1),
    "wgrad": ("moe_linear_fp8_wgrad", lambda s: (F, F, F, 1 << 26, 1 << 16, 1 << 16, 0, F, s), 1 << 19),
    "grouped wgrad": ("moe_grouped_linear_fp8_wgrad",
                      lambda s: (F, F, F, ctypes.byref(plan_args(1 << 20, El=32)), 1 << 16, 1 << 16, 0, F, s), 1 << 24),
    "grouped wgrad, small": ("moe_grouped_linear_fp8_wgrad",
                             lambda s: (F, F, F, ctypes.byref(plan_args(1 << 20, El=512)), 8, 16, 0, F, s), 1 << 12),
}


@pytest.mark.parametrize("name", ENDS)
def test_launch_at_the_end_of_the_range(name):
    say(f"launch {name}")
    call, args, waves = ENDS[name]

    def record(stream):
        status = getattr(moe.lib(), call)(*args(ctypes.c_void_p(stream.cuda_stream)))
        assert status == 0, moe.status_string(status)
    launched = launches_of(record)
    assert len(launched) == 1
    _, grid, block = launched[0]
    assert all(g * b < 1 << 32 for g, b in zip(grid, block)), (grid, block)
    assert grid[1] < 1 << 16 and grid[2] == 1
    assert grid[0] * grid[1] * block[0] // 64 >= waves, (grid, block)


@pytest.fixture
def room():
    torch.cuda.empty_cache()
    yield torch.cuda.mem_get_info()[0]
    torch.cuda.empty_cache()


def few_routes(M, at):
    """The plan of M tokens of which `at` have a route."""
    ids = torch.full((M, 1), -1, dtype=I32, device="cuda")
    ids[at] = 0
    plan = moe.moe_sort(ids, 1, 1, 0, 16)
    assert torch.equal(plan.expanded_to_permuted[at].cpu(), torch.arange(len(at), dtype=I32))
    return plan


# tokens whose wavefronts lie past 2^32 threads: from 2^21 on in pieces of 512, from 2^22 in two pieces
MARKS = [0, 1, (1 << 20) + 7, (1 << 21) - 1, 1 << 21, (1 << 21) + 4]


def test_dispatch_rows_and_back(room):
    M = (1 << 21) + 5
    say(f"dispatch {M} x {H} and back")
    if room < 150 << 30:
        pytest.skip("needs 150 GB of free GPU memory")
    plan = few_routes(M, MARKS)
    n = len(MARKS)
    v = torch.randint(-3, 4, (n, H), generator=gen(1)).to(BF16).cuda()
    x, rows = (torch.empty(r, H, dtype=BF16, device="cuda") for r in (M, plan.route_slots))
    x[MARKS] = v
    rows[:n + 2] = 7
    moe.moe_dispatch(x, plan, rows=rows)
    assert torch.equal(rows[:n], v) and bool((rows[n:n + 2] == 7).all())
    x.fill_(5)
    moe.moe_dispatch_backward(rows, plan, x)
    assert torch.equal(x[MARKS], v)
    x[MARKS] = 0
    for i in range(0, M, 1 << 17):
        assert not bool(x[i:i + (1 << 17)].any()), "a token without a route gets 0"
    x[MARKS] = 2
    moe.moe_dispatch_backward(rows, plan, x, accumulate=True)
    assert torch.equal(x[MARKS], v + 2)


def test_dispatch_codes(room):
    M = 1 << 22
    say(f"dispatch {M} x {H}, codes")
    if room < 210 << 30:
        pytest.skip("needs 210 GB of free GPU memory")
    at = [*MARKS, (1 << 22) - 1]
    plan = few_routes(M, at)
    v = torch.randn(len(at), H, generator=gen(2)).to(BF16)
    x = torch.empty(M, H, dtype=BF16, device="cuda")
    x[at] = v.cuda()
    q, sf = (torch.empty(plan.route_slots, c, dtype=BYTE, device="cuda") for c in (H, H // 128))
    moe.moe_dispatch(x, plan, q=q, q_sf=sf)
    want, want_sf = ref.quantize(v)
    assert torch.equal(q[:len(at)].cpu(), want) and torch.equal(sf[:len(at)].cpu(), want_sf)
