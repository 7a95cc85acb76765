"""Products of rows in 8 bits and the gradients of their weights on the GPU.
Small whole numbers under powers of two make every sum exact, so that most
tests compare bits; the others have tolerances that count what is lost."""
import math

import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from fp8_ref import U8, U24
from test_gpu_fp8_rows import BF16, BYTE, F32, F64, I32, Guarded, gen, near, plan_of, say, untouched

pytestmark = pytest.mark.gpu

NAN_CODE = ref.NAN_CODE


def nb(n):
    return -(-n // 128)


def whole_rows(M, K, seed):
    """(codes, E8M0): whole numbers -2 .. 2 and scales 1/4 .. 4."""
    g = gen(seed)
    q = ref.encode(torch.randint(-2, 3, (M, K), generator=g).double())
    return q.cuda(), torch.randint(125, 130, (M, nb(K)), generator=g).to(BYTE).cuda()


def whole_weights(B, N, K, seed):
    g = gen(seed)
    q = ref.encode(torch.randint(-2, 3, (B, N, K), generator=g).double())
    sf = torch.exp2(torch.randint(-2, 3, (B, nb(N), nb(K)), generator=g).float())
    return q.cuda(), sf.cuda()


def product(x, w):
    """fp64 x w^T on the GPU."""
    return torch.mm(x, w.t().contiguous())


# Sums of multiples of 2^-4 that stay below 4 K 16: exact in fp32 while K <= 2^13.
SHAPES = [(1, 1, 16), (1, 17, 128), (3, 64, 144), (8, 300, 1040), (16, 16, 8192), (8, 4096, 6144), (17, 128, 256),
          (31, 33, 400), (33, 136, 2064), (64, 200, 512), (65, 1000, 1552), (100, 129, 4096), (128, 128, 128),
          (129, 257, 272), (200, 520, 96), (256, 256, 1024), (300, 1024, 2048), (511, 2056, 1568), (513, 768, 640),
          (1000, 3000, 528), (1237, 2056, 1568), (2048, 2048, 512), (2500, 1111, 1024), (4096, 4096, 1168),
          (5000, 520, 160), (7001, 264, 4112), (1, 8200, 160), (5, 8193, 400), (16, 9011, 1168), (12, 16384, 144)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear_exact(M, N, K):
    say(f"linear {M} x {N} x {K}")
    x, x_sf = whole_rows(M, K, M + K)
    w, w_sf = whole_weights(1, N, K, N + K)
    g = gen(N)
    bias = torch.randint(-8, 9, (N,), generator=g).float().cuda()
    want = product(ref.rows(x, x_sf), ref.weights(w[0], w_sf[0]))
    old = torch.randint(-64, 65, (M, N), generator=g).float().cuda()
    for dtype in (F32, BF16):
        for b in (None, bias):
            for acc in (False, True):
                out = Guarded()
                y = out(M, N, dtype=dtype)
                if acc:
                    y.copy_(old)
                moe.moe_linear_fp8(x, x_sf, w[0], w_sf[0], y, bias=b, accumulate=acc)
                out.check()
                full = want + (0 if b is None else b.double()) + (old.double() if acc else 0)
                assert torch.equal(y, full.to(dtype)), (dtype, b is not None, acc)


@pytest.mark.parametrize("M,N,K", [(5, 72, 144), (40, 264, 1040), (300, 520, 2064), (1025, 1032, 528)])
def test_linear_alignment(M, N, K):
    """y at every alignment of its elements: the same sums."""
    say(f"linear alignment {M} x {N} x {K}")
    x, x_sf = whole_rows(M, K, 1)
    w, w_sf = whole_weights(1, N, K, 2)
    want = product(ref.rows(x, x_sf), ref.weights(w[0], w_sf[0]))
    for dtype, offsets in ((BF16, (1, 2, 4)), (F32, (1, 2))):
        for o in offsets:
            room = torch.zeros(M * N + 16, dtype=dtype, device="cuda")
            y = room[o:o + M * N].view(M, N)
            moe.moe_linear_fp8(x, x_sf, w[0], w_sf[0], y)
            assert torch.equal(y, want.to(dtype))
            assert bool((room[:o] == 0).all()) and bool((room[o + M * N:] == 0).all())


@pytest.mark.parametrize("M,N,K", [(7, 136, 6144), (40, 200, 4096), (130, 384, 1040), (600, 520, 2064),
                                   (2048, 1536, 1024)])
def test_linear_random(M, N, K):
    """Ordinary values and scales of any size against fp64, with what the instruction and fp32 may lose."""
    say(f"linear random {M} x {N} x {K}")
    g = gen(K)
    xb = (torch.randn(M, K, generator=g) * torch.exp2(torch.randint(-3, 4, (M, 1), generator=g).float())).to(BF16)
    wb = torch.randn(N, K, generator=g).to(BF16)
    x, x_sf = torch.empty(M, K, dtype=BYTE, device="cuda"), torch.empty(M, nb(K), dtype=BYTE, device="cuda")
    w, w_sf = torch.empty(N, K, dtype=BYTE, device="cuda"), torch.empty(nb(N), nb(K), device="cuda")
    moe.moe_quantize_fp8(xb.cuda(), x, x_sf)
    moe.moe_quantize_fp8_weight(wb.cuda(), w, w_sf)
    w_sf *= torch.rand(w_sf.shape, generator=g).cuda() + 0.5  # any scales
    some = torch.linspace(0, M - 1, min(M, 9)).long().unique().cuda()
    xv, wv = ref.rows(x, x_sf)[some], ref.weights(w, w_sf)
    want, size = product(xv, wv), product(xv.abs(), wv.abs())
    # 16 groups of a block and the blocks, one after another (what is cut off counts twice), and up to 8 parts
    tol = ref.product_bound(xv, wv) + 2 * (16 + nb(K) + 8) * U24 * size
    for dtype in (F32, BF16):
        y = torch.empty(M, N, dtype=dtype, device="cuda")
        moe.moe_linear_fp8(x, x_sf, w, w_sf, y)
        near(y[some], want, tol + (want.abs() * U8 if dtype == BF16 else 0))
        again = torch.empty_like(y)
        moe.moe_linear_fp8(x, x_sf, w, w_sf, again)
        assert torch.equal(y, again)


@pytest.mark.parametrize("M,N,K", [(6, 144, 272), (130, 264, 400), (1030, 1040, 1168)])
def test_linear_nan_stays_in_its_row(M, N, K):
    """NaN codes, the last chunk of an odd K and the first among them, reach their row or column alone."""
    say(f"linear nan {M} x {N} x {K}")
    x, x_sf = whole_rows(M, K, 3)
    w, w_sf = whole_weights(1, N, K, 4)
    x[1, 0] = x[M - 1, K - 1] = x[M // 2, K // 2] = NAN_CODE
    w[0, N - 1, 0] = w[0, N // 2, K - 1] = NAN_CODE
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_fp8(x, x_sf, w[0], w_sf[0], y)
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[[1, M - 1, M // 2]] = True
    bad[:, [N - 1, N // 2]] = True
    assert torch.equal(torch.isnan(y), bad)


def test_linear_extreme_scales():
    """Products below and above fp32's range, scales of 0, negative and subnormal ones."""
    say("linear extreme scales")
    M, N, K = 20, 136, 256
    x, x_sf = whole_rows(M, K, 5)
    w, w_sf = whole_weights(1, N, K, 6)
    x_sf[:5] = 1
    x_sf[5:9] = 247
    w_sf[0, 0, 0], w_sf[0, 0, 1], w_sf[0, 1, 0], w_sf[0, 1, 1] = 0.0, -3.0, 2.0 ** -140, 1.0
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_fp8(x, x_sf, w[0], w_sf[0], y)
    want = product(ref.rows(x, x_sf), ref.weights(w[0], w_sf[0]))
    big = want.abs() >= 2.0 ** -118
    assert torch.equal(y[big], want[big].float())
    assert float(y[~big].abs().max()) < 2.0 ** -110


# ------------------------------------------------------------------ experts

GROUPS = [(1, 1, 1, 1, 0, 16, "random"), (5, 2, 4, 4, 0, 16, "same"), (64, 8, 32, 4, 8, 16, "random"),
          (67, 4, 9, 9, 0, 32, "padded"), (130, 6, 60, 15, 30, 64, "random"), (133, 8, 16, 16, 0, 128, "padded"),
          (1301, 3, 8, 8, 0, 256, "random"), (12, 4, 8, 4, 2, 16, "nowhere"), (700, 2, 3, 3, 0, 256, "same"),
          (900, 2, 5, 5, 0, 128, "random"), (301, 4, 6, 3, 3, 64, "padded"), (2100, 1, 2, 2, 0, 16, "random")]
NK = [(8, 16), (136, 144), (256, 1024), (520, 2064), (768, 4096)]


def group_inputs(p, K, seed):
    M, k, E, El, off, tile, kind = p
    plan, slot = plan_of(M, k, E, El, off, tile, seed, kind)
    n = plan.route_slots
    x, x_sf = whole_rows(n, K, seed)
    s = slot[slot >= 0]
    rest = torch.ones(n, dtype=torch.bool)
    rest[s] = False
    x[rest.cuda()], x_sf[rest.cuda()] = NAN_CODE, 255  # what padding slots hold is not read
    return plan, x, x_sf, rest


def ranges(plan):
    first, counts = plan.expert_offsets.tolist(), plan.expert_counts.tolist()
    return [(e, slice(first[e], first[e] + counts[e])) for e in range(plan.num_local_experts)]


@pytest.mark.parametrize("p", range(len(GROUPS)))
@pytest.mark.parametrize("N,K", NK)
def test_grouped_linear(p, N, K):
    say(f"grouped linear {GROUPS[p]} {N} x {K}")
    plan, x, x_sf, rest = group_inputs(GROUPS[p], K, p)
    w, w_sf = whole_weights(plan.num_local_experts, N, K, p + 1)
    out = Guarded()
    y = out(plan.route_slots, N, dtype=BF16)
    moe.moe_grouped_linear_fp8(x, x_sf, plan, w, w_sf, y)
    out.check()
    for e, at in ranges(plan):
        want = product(ref.rows(x[at], x_sf[at]), ref.weights(w[e], w_sf[e]))
        assert torch.equal(y[at], want.to(BF16)), e
    assert untouched(y.cpu()[rest]), "a padding slot was written"


# ------------------------------------------------------------------ weight gradients

def whole_dy(M, N, seed):
    return torch.randint(-3, 4, (M, N), generator=gen(seed)).to(BF16).cuda()


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (2, 64, 128), (31, 136, 144), (33, 128, 128), (64, 200, 272),
                                   (100, 520, 1040), (129, 256, 512), (300, 2056, 1568), (1237, 2056, 1568),
                                   (2000, 264, 400), (4096, 1024, 512), (8191, 136, 272), (777, 4096, 2048),
                                   (65, 8, 8192), (500, 6144, 16)])
def test_wgrad_exact(M, N, K):
    """Sums of multiples of 1/4 below 2^20: exact in fp32."""
    say(f"wgrad {M} x {N} x {K}")
    x, x_sf = whole_rows(M, K, M + K)
    dy = whole_dy(M, N, M + N)
    want = torch.mm(dy.double().t().contiguous(), ref.rows(x, x_sf))
    old = torch.randint(-64, 65, (N, K), generator=gen(1)).float().cuda()
    for acc in (False, True):
        out = Guarded()
        dw = out(N, K, dtype=F32)
        if acc:
            dw.copy_(old)
        moe.moe_linear_fp8_wgrad(dy, x, x_sf, dw, accumulate=acc)
        out.check()
        assert torch.equal(dw, (want + (old.double() if acc else 0)).float()), acc


@pytest.mark.parametrize("M,N,K", [(50, 136, 400), (1000, 264, 528), (3000, 512, 1024)])
def test_wgrad_random(M, N, K):
    say(f"wgrad random {M} x {N} x {K}")
    g = gen(M)
    x, x_sf = torch.empty(M, K, dtype=BYTE, device="cuda"), torch.empty(M, nb(K), dtype=BYTE, device="cuda")
    moe.moe_quantize_fp8((torch.randn(M, K, generator=g) * 3).to(BF16).cuda(), x, x_sf)
    dy = (torch.randn(M, N, generator=g) * 0.01).to(BF16).cuda()
    dw, again = torch.empty(N, K, device="cuda"), torch.empty(N, K, device="cuda")
    moe.moe_linear_fp8_wgrad(dy, x, x_sf, dw)
    moe.moe_linear_fp8_wgrad(dy, x, x_sf, again)
    assert torch.equal(dw, again)
    a, b = dy.double().t().contiguous(), ref.rows(x, x_sf)
    # products are exact; M of them are added, in fp32 steps that may cut off
    near(dw, torch.mm(a, b), 2 * M * U24 * torch.mm(a.abs(), b.abs()))


def test_wgrad_by_differences():
    """The loss sum(y c) changes by dW at a weight: whole numbers make both sides exact."""
    say("wgrad by differences")
    M, N, K = 37, 24, 48
    x, x_sf = whole_rows(M, K, 8)
    w, w_sf = whole_weights(1, N, K, 9)
    w_sf.fill_(1.0)
    c = whole_dy(M, N, 10)
    dw = torch.empty(N, K, device="cuda")
    moe.moe_linear_fp8_wgrad(c, x, x_sf, dw)
    y = torch.empty(M, N, device="cuda")

    def loss():
        moe.moe_linear_fp8(x, x_sf, w[0], w_sf[0], y)
        return float((y.double() * c.double()).sum())
    for n, k in [(0, 0), (23, 47), (7, 16), (12, 31)]:
        w[0, n, k] = ref.encode(torch.tensor([1.0], dtype=F64))[0]
        a = loss()
        w[0, n, k] = 0
        assert a - loss() == float(dw[n, k])


def test_wgrad_nan_and_no_rows():
    say("wgrad nan, no rows")
    N, K = 136, 272
    x, x_sf = whole_rows(70, K, 3)
    dy = whole_dy(70, N, 4)
    x[69, K - 1] = NAN_CODE
    dy[3, 5] = math.nan
    dw = torch.empty(N, K, device="cuda")
    moe.moe_linear_fp8_wgrad(dy, x, x_sf, dw)
    bad = torch.zeros(N, K, dtype=torch.bool, device="cuda")
    bad[5] = True
    bad[:, K - 1] = True
    assert torch.equal(torch.isnan(dw), bad)
    moe.moe_linear_fp8_wgrad(dy[:0], x[:0], x_sf[:0], dw)
    assert bool((dw == 0).all())
    dw.fill_(3)
    moe.moe_linear_fp8_wgrad(dy[:0], x[:0], x_sf[:0], dw, accumulate=True)
    assert bool((dw == 3).all())


@pytest.mark.parametrize("p", range(len(GROUPS)))
@pytest.mark.parametrize("N,K", NK)
def test_grouped_wgrad(p, N, K):
    say(f"grouped wgrad {GROUPS[p]} {N} x {K}")
    plan, x, x_sf, rest = group_inputs(GROUPS[p], K, p)
    El = plan.num_local_experts
    dy = whole_dy(plan.route_slots, N, p)
    dy[rest.cuda()] = math.nan
    old = torch.randint(-64, 65, (El, N, K), generator=gen(1)).float().cuda()
    for acc in (False, True):
        out = Guarded()
        dw = out(El, N, K, dtype=F32)
        if acc:
            dw.copy_(old)
        moe.moe_grouped_linear_fp8_wgrad(dy, x, x_sf, plan, dw, accumulate=acc)
        out.check()
        for e, at in ranges(plan):
            want = torch.mm(dy[at].double().t().contiguous(), ref.rows(x[at], x_sf[at]))
            assert torch.equal(dw[e], (want + (old[e].double() if acc else 0)).float()), (e, acc)


def test_empty():
    say("empty")
    e = lambda *s, dtype=BYTE: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    plan = moe.moe_sort(e(0, 2, dtype=I32), 4, 4, 0, 16)
    w, w_sf = whole_weights(4, 16, 64, 1)
    moe.moe_linear_fp8(e(0, 64), e(0, 1), w[0], w_sf[0], e(0, 16, dtype=BF16))
    moe.moe_linear_fp8(e(3, 64), e(3, 1), e(0, 64), e(0, 1, dtype=F32), e(3, 0, dtype=BF16))
    moe.moe_grouped_linear_fp8(e(0, 64), e(0, 1), plan, w, w_sf, e(0, 16, dtype=BF16))
    dw = torch.full((4, 16, 64), 2.0, device="cuda")
    moe.moe_grouped_linear_fp8_wgrad(e(0, 16, dtype=BF16), e(0, 64), e(0, 1), plan, dw, accumulate=True)
    assert bool((dw == 2).all())
    moe.moe_grouped_linear_fp8_wgrad(e(0, 16, dtype=BF16), e(0, 64), e(0, 1), plan, dw)
    assert bool((dw == 0).all())
