"""The gated activations on rows in 8 bits at single gates: every E4M3 value
under several scales, against fp64 within what fp32 and one rounding lose of
each value, however small it is."""
import math

import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from fp8_ref import U4, U8, U24
from test_gpu_fp8_rows import BF16, BYTE, F64, kwargs, near, say

pytestmark = pytest.mark.gpu

KINDS = [("geglu", {}), ("swiglu", {}), ("swiglu", dict(alpha=1.702, beta=1.0, limit=7.0)),
         ("swiglu", dict(alpha=1.702))]
SCALES = range(119, 132)   # E8M0 codes: gates from 2^-17 to 7168
UPS = (1.0, -0.875, 7.0, -7.5, 0.0, 48.0)


def exact(kind, g, u, kw):
    """f, f' and up, up' in fp64, and by how many half steps of fp32 of which sizes f and f' may be off.

    GeGLU, z = c (g + 0.044715 g^3), s = sigmoid(2z): z has two rounded constants and five operations on terms of one
    sign, so 2z is off by 7 half steps, s by 14 |z| of them, and the exponential, the sum and the quotient by 6 more;
    f has one product more, f' the terms s and 2 g s (1 - s) z', the second with two such factors and ten operations.
    SwiGLU, s = sigmoid(a g): one operation in a g, then as before; 1 - s is a difference from 1."""
    f, df, up, dup = ref.act(kind, g, u, **kw)
    if kind == "geglu":
        z = math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)
        s = torch.sigmoid(2 * z)
        f = g * s  # (fp64's 1 + tanh cancels too)
        slope = 2 * g * s * torch.sigmoid(-2 * z) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * g * g)
        df = s + slope
        off = 14 * z.abs() + 6
        return f, df, up, dup, f.abs() * (off + 1), s * off + slope.abs() * (2 * off + 10) + df.abs()
    ag = kw.get("alpha", 1.0) * g.clamp(max=kw.get("limit", math.inf))
    s, off = torch.sigmoid(ag), 2 * ag.abs() + 6
    return f, df, up, dup, f.abs() * (off + 1), s * (1 + ag.abs()) * (2 * off + 6) * (df != 0)


@pytest.mark.parametrize("kind,kw", KINDS)
def test_gradient_at_every_gate(kind, kw):
    say(f"gradient at every gate {kind} {kw}")
    I = 256
    codes = torch.arange(256, dtype=torch.int64).to(BYTE)
    codes[(codes & 127) == 127] = 0
    n = len(SCALES) * len(UPS)
    hq, hq_sf = torch.empty(n, 2 * I, dtype=BYTE), torch.empty(n, 4, dtype=BYTE)
    for i, sc in enumerate(SCALES):
        for j, up in enumerate(UPS):
            r = len(UPS) * i + j
            hq[r, :I], hq[r, I:] = codes, ref.encode(torch.full((I,), up, dtype=F64))
            hq_sf[r] = torch.tensor([sc, sc, 127, 127], dtype=BYTE)
    dy = torch.randn(n, I, generator=torch.Generator().manual_seed(1)).to(BF16)
    dh = torch.empty(n, 2 * I, dtype=BF16, device="cuda")
    moe.moe_gated_act_fp8_backward(hq.cuda(), hq_sf.cuda(), dy.cuda(), dh=dh, **kwargs(kind, kw))
    kept, d = ref.halves_rows(hq, hq_sf), dy.double()
    f, df, up, dup, f_off, df_off = exact(kind, kept[:, :I], kept[:, I:], kw)
    # up + beta, two products, the rounding to bf16; what lies below fp32's normal range (a gate's factor, or a product)
    tiny = 2.0 ** -126
    for name, got, want, size in (
            ("gate", dh[:, :I], d * df * up, d.abs() * up.abs() * (df_off + 3 * df.abs())),
            ("up", dh[:, I:], d * f * dup, d.abs() * dup * (f_off + 2 * f.abs()))):
        small = tiny * (1 + d.abs() * (1 + kept[:, :I].abs()) * (1 + up.abs())) + 2.0 ** -134
        near(got, want, want.abs() * U8 + size * U24 * (1 + U8) + small, name)


@pytest.mark.parametrize("kind,kw", KINDS)
def test_value_at_every_gate(kind, kw):
    """A gate a row, so that its block's scale is its own."""
    say(f"value at every gate {kind} {kw}")
    I = 128
    g = torch.cat((torch.linspace(-12, 12, 769), torch.tensor([-60.0, -30.0, -20.0, 20.0, 60.0]))).to(BF16)
    u = torch.tensor([1.0, -0.75] * (I // 2)).to(BF16)
    h = torch.cat((g[:, None].expand(-1, I), u.expand(len(g), -1)), 1).contiguous()
    y, y_sf = torch.empty(len(g), I, dtype=BYTE, device="cuda"), torch.empty(len(g), 1, dtype=BYTE, device="cuda")
    moe.moe_gated_act_fp8(h.cuda(), y, y_sf, **kwargs(kind, kw))
    f, _, up, _, f_off, _ = exact(kind, h[:, :I].double(), h[:, I:].double(), kw)
    want = f * up
    # fp32, bf16 and E4M3, each of the one before; below the least scale half a step of the smallest code
    tol = want.abs() * ((1 + U4) * (1 + U8) - 1) + f_off * up.abs() * 2 * U24 * (1 + U4) + f.abs() * U24
    low = 2.0 ** -126 * 2.0 ** -10 + 2.0 ** -126 * (h[:, :I].double().abs() + 1)
    near(ref.rows(y.cpu(), y_sf.cpu()), want, tol + low, "y")


FAR = [2.0e38, 2.5e38, 3.2e38]
PAST = [3.29e38, 3.32e38, 3.38e38]  # kept as codes that stand for 2^128


@pytest.mark.parametrize("values", [FAR, PAST])
@pytest.mark.parametrize("kind,kw", [("geglu", {}), ("swiglu", {}), ("swiglu", dict(alpha=1.702)),
                                     ("swiglu", dict(alpha=-3.0)), ("swiglu", dict(alpha=1.702, beta=1.0, limit=7.0))])
def test_gradient_of_the_largest_values(kind, kw, values):
    """Gates and ups at the end of bf16's range, one at a time: gradients of finite values are finite numbers."""
    say(f"gradient of the largest values {kind} {kw} {values}")
    I = 128
    large = torch.tensor(values + [-v for v in values]).to(BF16)
    n = len(large)
    h = torch.full((2 * n + 1, 2 * I), 0.5).to(BF16)
    h[:n, :I] = large[:, None]
    h[n:2 * n, I:] = large[:, None]
    h[2 * n, 0], h[2 * n, I + 1], h[2 * n, 2] = math.nan, math.nan, -math.inf
    M = len(h)
    y, y_sf, hq, hq_sf = (torch.empty(M, c, dtype=BYTE, device="cuda") for c in (I, 1, 2 * I, 2))
    dh = torch.empty(M, 2 * I, dtype=BF16, device="cuda")
    dy = torch.full((M, I), 2.0 ** -9).to(BF16)
    dy[:, 1::2] = 0
    moe.moe_gated_act_fp8(h.cuda(), y, y_sf, hq=hq, hq_sf=hq_sf, **kwargs(kind, kw))
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy.cuda(), dh=dh, **kwargs(kind, kw))
    got = dh.cpu().double()
    assert bool(torch.isfinite(got[:-1]).all())
    top = torch.finfo(torch.float32).max
    kept = ref.halves_rows(hq.cpu(), hq_sf.cpu())[:-1].clamp(-top, top)
    f, df, up, dup = ref.act(kind, kept[:, :I], kept[:, I:], **kw)
    f = torch.where(torch.isnan(f), 0.0, f)
    d = dy.double()[:-1]
    want = torch.cat((d * df * up, d * f * dup), 1)
    # ordinary values at 0.5, all else the value itself or 0: fp32's dozen roundings, and bf16's
    near(got[:-1], want, want.abs() * (U8 + 32 * U24) + 2.0 ** -134, "dh")
    # a gate's NaN reaches both halves, an up value's the gate's
    assert set(torch.isnan(got[-1]).nonzero().flatten().tolist()) == {0, 1, 2, I, I + 2}
