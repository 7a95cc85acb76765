"""Rows in 8 bits on the GPU: quantisers, dispatch, the gradients of the way
back, activations; codes bit for bit, sums with tolerances that count roundings."""
import math

import numpy as np
import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from fp8_ref import U4, U8, U24

pytestmark = pytest.mark.gpu

BF16, F32, F64, BYTE, I32 = torch.bfloat16, torch.float32, torch.float64, torch.uint8, torch.int32
GUARD = 173


def say(*a):
    print(*a, flush=True)


def gen(seed):
    return torch.Generator().manual_seed(seed)


class Guarded:
    """Outputs whose bytes all start as GUARD, with room behind them."""

    def __init__(self):
        self.all = []

    def __call__(self, *shape, dtype=BYTE):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        room = torch.full((n + 512,), GUARD, dtype=BYTE, device="cuda")
        self.all.append((room, n))
        return room[:n].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for room, n in self.all:
            assert bool((room[n:] == GUARD).all()), "written past the end"


def untouched(t):
    return bool((t.contiguous().view(BYTE) == GUARD).all())


def near(got, want, tol, what=""):
    got, want = got.cpu().double(), want.cpu().double()
    tol = torch.as_tensor(tol, dtype=F64).cpu().expand(want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what
    over = ((got - want).abs() - tol)[fin]
    if over.numel() and over.max() > 0:
        i = int(over.argmax())
        raise AssertionError(f"{what}: {got[fin][i]} against {want[fin][i]}, tolerance {tol[fin][i]}")


def values(M, n, seed, special=False):
    """bf16 rows of many sizes; `special`: zeros, blocks of zeros, infinities, NaN, the borders of a scale."""
    g = gen(seed)
    x = torch.randn(M, n, generator=g) * torch.exp2(torch.randint(-20, 20, (M, 1), generator=g).float())
    x = x.to(BF16)
    if special:
        x[0] = 0
        x[M // 2, : n // 2] = 0
        x[-1, n // 3] = math.inf
        x[-1, 0] = -math.inf
        x[M // 3, n - 1] = math.nan
        x[M // 3, 1] = 2.0 ** -133
        for i, v in enumerate((448, 450, 1.75, 1.7578125, 3.38e38, 2.0 ** -126, 2.0 ** -118)):
            x[(3 * i + 1) % M, (128 * i + 5) % n] = v
    return x


# ------------------------------------------------------------------ quantisers

@pytest.mark.parametrize("M,n", [(1, 16), (1, 128), (3, 144), (2, 400), (17, 528), (5, 2064), (64, 6144), (4097, 1040),
                                 (1500, 4128), (2, 16384)])
def test_quantize(M, n):
    say(f"quantize {M} x {n}")
    x = values(M, n, M + n, special=True)
    out = Guarded()
    q, sf = out(M, n), out(M, -(-n // 128))
    moe.moe_quantize_fp8(x.cuda(), q, sf)
    out.check()
    rq, rs = ref.quantize(x)
    assert torch.equal(sf.cpu(), rs)
    assert ref.same_codes(q.cpu(), rq)


def test_quantize_strided_and_every_value():
    """Every finite bf16 next to a block's largest one, from rows that are apart."""
    say("quantize strided, every value")
    bits = torch.arange(0, 65536, dtype=I32).to(torch.int16).view(BF16)
    finite = bits[torch.isfinite(bits)]
    for top in (448.0, 1.0, 3.0e38, 2.0 ** -100):
        v = finite[finite.abs() <= top]
        v = torch.cat((v, v.new_zeros(-v.numel() % 127))).view(-1, 127)
        x = torch.cat((torch.full((v.shape[0], 1), top, dtype=BF16), v), 1)
        wide = torch.full((x.shape[0], 192), 9.0, dtype=BF16)
        wide[:, 8:136] = x
        q = torch.empty(x.shape, dtype=BYTE, device="cuda")
        sf = torch.empty(x.shape[0], 1, dtype=BYTE, device="cuda")
        moe.moe_quantize_fp8(wide.cuda()[:, 8:136], q, sf)
        rq, rs = ref.quantize(x)
        assert torch.equal(sf.cpu(), rs) and ref.same_codes(q.cpu(), rq), top


@pytest.mark.parametrize("B,N,K,special", [(1, 8, 16, False), (1, 128, 128, False), (3, 136, 264, False),
                                           (2, 304, 392, True), (1, 1, 24, False), (5, 256, 1024, True)])
def test_quantize_weight(B, N, K, special):
    say(f"quantize weight {B} x {N} x {K}")
    w = torch.stack([values(max(N, 1), K, 7 * i + N, special=special) for i in range(B)])
    out = Guarded()
    nn, nk = -(-N // 128), -(-K // 128)
    q, sf = out(B, N, K), out(B, nn, nk, dtype=F32)
    if N % 8 == 0:
        qt, sft = out(B, K, N), out(B, nk, nn, dtype=F32)
        moe.moe_quantize_fp8_weight(w.cuda(), q, sf, qt, sft)
    else:
        moe.moe_quantize_fp8_weight(w.cuda(), q, sf)
    out.check()
    for b in range(B):
        rq, rs = ref.quantize_weight(w[b])
        assert torch.equal(sf[b].cpu(), rs)
        assert ref.same_codes(q[b].cpu(), rq)
    if N % 8 == 0:
        assert torch.equal(qt, q.transpose(1, 2)) and torch.equal(sft, sf.transpose(1, 2))
        q2, sf2 = torch.empty_like(q), torch.empty_like(sf)
        moe.moe_quantize_fp8_weight(w.cuda(), q2, sf2)
        assert torch.equal(q, q2) and torch.equal(sf, sf2)
        moe.moe_quantize_fp8_weight(w[0].cuda(), q2[0], sf2[0])
        assert torch.equal(q[0], q2[0])


# ------------------------------------------------------------------ plans

def plan_of(M, k, E, El, off, tile, seed, kind="random"):
    """(plan, slot of every route on the CPU) of ids that are distinct, equal, padded or nowhere local."""
    g = gen(seed)
    ids = torch.stack([torch.randperm(E, generator=g)[:k] for _ in range(M)]) if M else torch.zeros(0, k)
    if kind == "same":       # the same expert at every place of a token
        ids[:] = off
    if kind == "nowhere":
        ids[:] = -1
    if kind == "padded":
        ids[torch.rand(M, generator=g) < 0.4] = -1
        ids[torch.rand(M, k, generator=g) < 0.1] = E + 3
    plan = moe.moe_sort(ids.to(I32).cuda(), E, El, off, tile)
    torch.cuda.synchronize()
    return plan, plan.expanded_to_permuted.cpu().long().view(M, k)


PLANS = [(1, 1, 1, 1, 0, 16, "random"), (5, 2, 4, 4, 0, 16, "same"), (8, 8, 32, 4, 8, 16, "random"),
         (67, 4, 9, 9, 0, 32, "padded"), (130, 6, 60, 15, 30, 64, "random"), (33, 8, 16, 16, 0, 128, "padded"),
         (301, 3, 8, 8, 0, 256, "random"), (12, 4, 8, 4, 2, 16, "nowhere"), (9, 64, 64, 64, 0, 16, "random")]
WIDTHS = [16, 128, 400, 2064, 6144]


@pytest.mark.parametrize("p", range(len(PLANS)))
@pytest.mark.parametrize("H", WIDTHS)
def test_dispatch(p, H):
    M, k, E, El, off, tile, kind = PLANS[p]
    say(f"dispatch {PLANS[p]} H={H}")
    plan, slot = plan_of(M, k, E, El, off, tile, p, kind)
    n = plan.route_slots
    x = values(M, H, p + H, special=M > 4)
    out = Guarded()
    rows, q, sf = out(n, H, dtype=BF16), out(n, H), out(n, -(-H // 128))
    moe.moe_dispatch(x.cuda(), plan, rows=rows, q=q, q_sf=sf)
    out.check()
    t = (torch.arange(M * k) // k)[slot.flatten() >= 0]
    s = slot.flatten()[slot.flatten() >= 0]
    rq, rs = ref.quantize(x)
    assert torch.equal(rows.cpu().view(torch.int16)[s], x.view(torch.int16)[t])
    assert ref.same_codes(q.cpu()[s], rq[t]) and torch.equal(sf.cpu()[s], rs[t])
    rest = torch.ones(n, dtype=torch.bool)
    rest[s] = False
    for v in (rows, q, sf):
        assert untouched(v.cpu()[rest]), "a padding slot was written"
    # one output without the other, from rows that are apart
    wide = torch.zeros(M, H + 24, dtype=BF16)
    wide[:, 8:8 + H] = x
    q2, sf2 = torch.full_like(q, GUARD), torch.full_like(sf, GUARD)
    rows2 = torch.full_like(q, GUARD).repeat(1, 2).view(BF16)
    if n:
        moe.moe_dispatch(wide.cuda()[:, 8:8 + H], plan, q=q2, q_sf=sf2)
        moe.moe_dispatch(wide.cuda()[:, 8:8 + H], plan, rows=rows2)
        assert torch.equal(q, q2) and torch.equal(sf, sf2)
        assert torch.equal(rows.view(BYTE), rows2.view(BYTE))


@pytest.mark.parametrize("p", range(len(PLANS)))
@pytest.mark.parametrize("H", [16, 400, 2064, 6144])
def test_dispatch_backward(p, H):
    M, k, E, El, off, tile, kind = PLANS[p]
    say(f"dispatch backward {PLANS[p]} H={H}")
    plan, slot = plan_of(M, k, E, El, off, tile, p, kind)
    n = plan.route_slots
    g = gen(p + H)
    d = torch.randn(n, H, generator=g).to(BF16)
    local = slot >= 0
    room = torch.zeros(n, dtype=torch.bool)
    room[slot[local]] = True
    d[~room] = math.nan  # padding
    terms = torch.where(local.unsqueeze(-1), d[slot.clamp(min=0)].double(), 0.0)
    old = torch.randn(M, H, generator=g).to(BF16)
    for acc in (False, True):
        out = Guarded()
        dx = out(M, H, dtype=BF16)
        if acc:
            dx.copy_(old)
        moe.moe_dispatch_backward(d.cuda(), plan, dx, accumulate=acc)
        out.check()
        want = terms.sum(1) + (old.double() if acc else 0)
        size = terms.abs().sum(1) + (old.double().abs() if acc else 0)
        near(dx, want, want.abs() * U8 + (k + 1) * U24 * size * (1 + U8), f"accumulate={acc}")
        none = ~local.any(1)
        assert torch.equal(dx.cpu()[none], old[none] if acc else torch.zeros_like(old)[none])


@pytest.mark.parametrize("p", range(len(PLANS)))
@pytest.mark.parametrize("H", [16, 400, 2064, 4128, 6144, 8208])
def test_finalize_backward(p, H):
    M, k, E, El, off, tile, kind = PLANS[p]
    say(f"finalize backward {PLANS[p]} H={H}")
    plan, slot = plan_of(M, k, E, El, off, tile, p, kind)
    n, rsf = plan.route_slots, 1.75
    g = gen(3 * p + H)
    dout, y2 = torch.randn(M, H, generator=g).to(BF16), torch.randn(n, H, generator=g).to(BF16)
    w = torch.rand(M, k, generator=g)
    local = slot >= 0
    w[~local] = math.nan  # a route that is not local has no weight
    r = local.flatten().nonzero().flatten()
    s, t = slot.flatten()[r], r // k
    room = torch.zeros(n, dtype=torch.bool)
    room[s] = True
    y2[~room] = math.nan
    out = Guarded()
    dy2, q, sf = out(n, H, dtype=BF16), out(n, H), out(n, -(-H // 128))
    dw = out(M, k, dtype=F32)
    moe.moe_finalize_backward(dout.cuda(), y2.cuda(), plan, w.cuda(), dy2=dy2, q=q, q_sf=sf, d_topk_weights=dw,
                              routed_scaling_factor=rsf)
    out.check()
    want = ((w * torch.tensor(rsf)).flatten()[r, None] * dout.float()[t]).to(BF16)  # fp32 products, one rounding
    assert torch.equal(dy2.cpu()[s], want)
    rq, rs = ref.quantize(want)
    assert ref.same_codes(q.cpu()[s], rq) and torch.equal(sf.cpu()[s], rs)
    for v in (dy2, q, sf):
        assert untouched(v.cpu()[~room]), "a padding slot was written"
    prod = dout.double()[t] * y2.double()[s]
    got, exact = dw.cpu().flatten(), torch.zeros(M * k, dtype=F64)
    exact[r] = rsf * prod.sum(1)
    tol = torch.zeros(M * k, dtype=F64)
    # a lane's fused sums (64 at most), the 6 + 3 that join lanes and wavefronts, the factor
    tol[r] = rsf * (64 + 9 + 1) * U24 * prod.abs().sum(1)
    near(got, exact, tol, "d_topk_weights")
    assert bool((got[~local.flatten()] == 0).all())
    if not n:
        return
    # outputs by themselves, in place, and the same bits
    dw2, q2, sf2 = torch.empty_like(dw), torch.full_like(q, GUARD), torch.full_like(sf, GUARD)
    moe.moe_finalize_backward(dout.cuda(), y2.cuda(), plan, w.cuda(), d_topk_weights=dw2, routed_scaling_factor=rsf)
    moe.moe_finalize_backward(dout.cuda(), None, plan, w.cuda(), q=q2, q_sf=sf2, routed_scaling_factor=rsf)
    both = y2.cuda()
    dw3 = torch.empty_like(dw)
    moe.moe_finalize_backward(dout.cuda(), both, plan, w.cuda(), dy2=both, d_topk_weights=dw3,
                              routed_scaling_factor=rsf)
    assert torch.equal(dw, dw2) and torch.equal(dw, dw3) and torch.equal(q, q2) and torch.equal(sf, sf2)
    assert torch.equal(both.cpu()[s], want)


# ------------------------------------------------------------------ activations

KINDS = [("geglu", {}), ("swiglu", {}), ("swiglu", dict(alpha=1.702, beta=1.0, limit=7.0))]


def kwargs(kind, kw):
    return {"activation": moe.ACT_GEGLU_TANH if kind == "geglu" else moe.ACT_SWIGLU,
            **{"swiglu_" + n: v for n, v in kw.items()}}


def act_rows(M, I, seed):
    """Gates and ups of ordinary sizes, some at and past the limits, some far out."""
    g = gen(seed)
    h = (torch.randn(M, 2 * I, generator=g) * 3).to(BF16)
    h[0, ::3] = 7.0
    h[0, 1::7] = -7.0
    h[-1, ::5] *= 64
    h[M // 2, :] = 0
    return h


def loose(got, want, what):
    """E4M3 values whose bf16 source may have been rounded the other way: half a step of the code, one and a half of
    bf16 (its own rounding, and the neighbour that a last bit of fp32 makes of it), half the smallest code."""
    codes, sf = got
    v = ref.rows(codes.cpu(), sf.cpu())
    step = ref.spread(torch.exp2(sf.cpu().double() - 127), v.shape[-1]) * 2.0 ** -10
    near(v, want, want.abs() * (U4 * (1 + U8) + 3 * U8) + step, what)


@pytest.mark.parametrize("kind,kw", KINDS)
@pytest.mark.parametrize("M,I", [(1, 16), (3, 128), (7, 400), (33, 1536), (2, 8208), (1100, 2048)])
def test_act(M, I, kind, kw):
    say(f"act {kind} {kw} {M} x {I}")
    h = act_rows(M, I, M + I)
    nb = -(-I // 128)
    out = Guarded()
    y, y_sf, hq, hq_sf = out(M, I), out(M, nb), out(M, 2 * I), out(M, 2 * nb)
    moe.moe_gated_act_fp8(h.cuda(), y, y_sf, hq=hq, hq_sf=hq_sf, **kwargs(kind, kw))
    dh, dq, dq_sf = out(M, 2 * I, dtype=BF16), out(M, 2 * I), out(M, 2 * nb)
    dy = torch.randn(M, I, generator=gen(I)).to(BF16)
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy.cuda(), dh=dh, dq=dq, dq_sf=dq_sf, **kwargs(kind, kw))
    out.check()
    rq, rs = ref.halves(h)
    assert torch.equal(hq.cpu(), rq) and torch.equal(hq_sf.cpu(), rs)
    f, _, up, _ = ref.act(kind, h[:, :I].double(), h[:, I:].double(), **kw)
    loose((y, y_sf), f * up, "y")
    # the gradient at the rows that were kept
    kept = ref.halves_rows(rq, rs)
    f, df, up, dup = ref.act(kind, kept[:, :I], kept[:, I:], **kw)
    d = dy.double()
    want = torch.cat((d * df * up, d * f * dup), 1)
    # fp32: about a dozen roundings of values that make f' (each below 1 + |alpha g|), then bf16
    g = kept[:, :I].abs()
    size = torch.cat((d.abs() * up.abs() * (1.2 + 2 * g), d.abs() * g * dup), 1)
    near(dh, want, want.abs() * U8 + 24 * U24 * size * (1 + U8) + 2.0 ** -133, "dh")
    rq, rs = ref.halves(dh.cpu())
    assert ref.same_codes(dq.cpu(), rq) and torch.equal(dq_sf.cpu(), rs)
    # outputs by themselves: the same bits
    y2, s2, dh2, dq2, ds2 = (torch.empty_like(t) for t in (y, y_sf, dh, dq, dq_sf))
    moe.moe_gated_act_fp8(h.cuda(), y2, s2, **kwargs(kind, kw))
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy.cuda(), dh=dh2, **kwargs(kind, kw))
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy.cuda(), dq=dq2, dq_sf=ds2, **kwargs(kind, kw))
    assert torch.equal(y, y2) and torch.equal(y_sf, s2) and torch.equal(dh, dh2)
    assert torch.equal(dq, dq2) and torch.equal(dq_sf, ds2)


@pytest.mark.parametrize("kind,kw", KINDS)
def test_act_far_out(kind, kw):
    """Gates so large that intermediate values overflow, NaN and infinities: gradients are 0, the up part, or NaN,
    never a NaN from finite values."""
    say(f"act far out {kind} {kw}")
    I = 128
    vals = [1e4, -1e4, 1e19, -1e19, 3e25, -3e25, 1e30, -1e30, 0.0, -0.0, 1e-30, 60.0, -60.0, -104.0, 88.0]
    g = torch.tensor(vals, dtype=BF16)
    h = torch.zeros(len(vals) + 1, 2 * I, dtype=BF16)
    h[:-1, :I] = g[:, None]
    h[:, I:] = 0.5
    h[-1, 3], h[-1, I + 9] = math.nan, math.nan
    M = h.shape[0]
    y, y_sf, hq, hq_sf = (torch.empty(M, n, dtype=BYTE, device="cuda") for n in (I, 1, 2 * I, 2))
    dh = torch.empty(M, 2 * I, dtype=BF16, device="cuda")
    dy = torch.full((M, I), 0.25, dtype=BF16, device="cuda")
    moe.moe_gated_act_fp8(h.cuda(), y, y_sf, hq=hq, hq_sf=hq_sf, **kwargs(kind, kw))
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy, dh=dh, **kwargs(kind, kw))
    d = dh.cpu().double()
    assert bool(torch.isfinite(d[:-1]).all())
    kept = ref.halves_rows(hq.cpu(), hq_sf.cpu())[:-1]
    f, df, up, dup = ref.act(kind, kept[:, :I], kept[:, I:], **kw)
    near(dh[:-1], 0.25 * torch.cat((df * up, f * dup), 1),
         0.25 * torch.cat((df * up, f * dup), 1).abs() * 2 * U8 + 64 * U24, "dh")
    # of a gate: both halves; of an up value: the gate's (the up half's gradient has no u)
    assert set(torch.isnan(d[-1]).nonzero().flatten().tolist()) == {3, 9, I + 3}
    codes = y.cpu()[-1] & 127
    assert int(codes[3]) == 127 and int(codes[9]) == 127


@pytest.mark.parametrize("p", range(len(PLANS)))
def test_act_of_a_plan(p):
    M, k, E, El, off, tile, kind = PLANS[p]
    say(f"act of a plan {PLANS[p]}")
    plan, slot = plan_of(M, k, E, El, off, tile, p, kind)
    n, I = plan.route_slots, 272
    nb = 3
    s = slot[slot >= 0]
    rest = torch.ones(n, dtype=torch.bool)
    rest[s] = False
    h = act_rows(max(n, 2), I, p)[:n]
    h[rest] = math.nan
    out = Guarded()
    y, y_sf, hq, hq_sf = out(n, I), out(n, nb), out(n, 2 * I), out(n, 2 * nb)
    dh, dq, dq_sf = out(n, 2 * I, dtype=BF16), out(n, 2 * I), out(n, 2 * nb)
    dy = torch.randn(n, I, generator=gen(p)).to(BF16).cuda()
    moe.moe_gated_act_fp8(h.cuda(), y, y_sf, hq=hq, hq_sf=hq_sf, plan=plan)
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy, dh=dh, dq=dq, dq_sf=dq_sf, plan=plan)
    out.check()
    if not n:
        return
    got = [y, y_sf, hq, hq_sf, dh, dq, dq_sf]
    for v in got:
        assert untouched(v.cpu()[rest]), "a padding slot was written"
    want = [torch.empty_like(v) for v in got]
    moe.moe_gated_act_fp8(h.cuda(), want[0], want[1], hq=want[2], hq_sf=want[3])
    moe.moe_gated_act_fp8_backward(want[2], want[3], dy, dh=want[4], dq=want[5], dq_sf=want[6])
    for a, b in zip(got, want):
        assert torch.equal(a.cpu()[s].view(BYTE), b.cpu()[s].view(BYTE))


def test_empty():
    say("empty")
    e = lambda *s, dtype=BYTE: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
    plan = moe.moe_sort(e(0, 2, dtype=I32), 4, 4, 0, 16)
    moe.moe_quantize_fp8(e(0, 64, dtype=BF16), e(0, 64), e(0, 1))
    moe.moe_dispatch(e(0, 64, dtype=BF16), plan, q=e(0, 64), q_sf=e(0, 1))
    moe.moe_dispatch_backward(e(0, 64, dtype=BF16), plan, e(0, 64, dtype=BF16))
    moe.moe_finalize_backward(e(0, 64, dtype=BF16), e(0, 64, dtype=BF16), plan, e(0, 2, dtype=F32),
                              dy2=e(0, 64, dtype=BF16), d_topk_weights=e(0, 2, dtype=F32))
    moe.moe_gated_act_fp8(e(0, 64, dtype=BF16), e(0, 32), e(0, 1))
    moe.moe_gated_act_fp8(e(0, 64, dtype=BF16), e(0, 32), e(0, 1), plan=plan)
    torch.cuda.synchronize()
