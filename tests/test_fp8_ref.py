"""The fp64 forms of tests/fp8_ref.py against other definitions of the same:
torch's own E4M3, scales by hand, derivatives by differences."""
import math

import pytest
import torch

import fp8_ref as ref


def test_table_is_torch_s():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(want), torch.isnan(ref.TABLE))
    fin = ~torch.isnan(want)
    assert torch.equal(want[fin], ref.TABLE[fin])


def test_encode_is_torch_s():
    g = torch.Generator().manual_seed(1)
    v = torch.cat((torch.randn(20000, generator=g) * torch.exp2(torch.randint(-12, 9, (20000,), generator=g).float()),
                   torch.linspace(-448, 448, 4097), torch.arange(-40, 41) * 2.0 ** -11)).clamp(-448, 448)
    assert torch.equal(ref.encode(v.double()), v.to(torch.float8_e4m3fn).view(torch.uint8))


@pytest.mark.parametrize("amax,exponent", [(448, 0), (450, 1), (449.99, 1), (1.0, -8), (1.75, -8), (1.7578125, -7), (0, -126),
                                           (2.0 ** -118, -126), (3e38, 120)])
def test_scale(amax, exponent):
    x = torch.tensor([[amax, -amax / 2, 0.0, math.inf]]).to(torch.bfloat16)
    if amax == 449.99:
        exponent = 1 if x[0, 0] > 448 else 0
    q, sf = ref.quantize(x)
    assert int(sf[0, 0]) == exponent + 127
    assert (int(q[0, 3]) & 127) == 127
    if amax:
        assert abs(ref.rows(q, sf)[0, 0] / x[0, 0].double() - 1) <= ref.U4


@pytest.mark.parametrize("kind,kw", [("geglu", {}), ("swiglu", {}), ("swiglu", dict(alpha=1.702, beta=1.0, limit=7.0))])
def test_derivatives_by_differences(kind, kw):
    g = torch.linspace(-9, 9, 271, dtype=ref.F64)[:, None]
    u = torch.linspace(-8.3, 8.4, 19, dtype=ref.F64)[None, :]
    g, u = (v.contiguous() for v in torch.broadcast_tensors(g, u))
    e = 1e-6
    f, df, up, dup = ref.act(kind, g, u, **kw)

    def value(g, u):
        f, _, up, _ = ref.act(kind, g, u, **kw)
        return f * up
    limit = kw.get("limit", math.inf)
    inside = ((g - limit).abs() > 2 * e) & ((u.abs() - limit).abs() > 2 * e)
    # central differences: third derivatives stay below 100; a value is below 85 and has four roundings of
    # 2^-53 of it, twice in a difference of 2 e
    tol = 100 * e * e + 8 * 2.0 ** -53 * 85 / (2 * e)
    assert ((df * up - (value(g + e, u) - value(g - e, u)) / (2 * e))[inside]).abs().max() < tol
    assert ((f * dup - (value(g, u + e) - value(g, u - e)) / (2 * e))[inside]).abs().max() < tol


def test_weight_codes_by_hand():
    w = torch.zeros(130, 256, dtype=torch.bfloat16)
    w[0, 0], w[127, 127], w[5, 200], w[129, 130] = 448, -224, 1.0, 0.5
    q, sf = ref.quantize_weight(w)
    assert sf.shape == (2, 2)
    assert float(sf[0, 0]) == 1.0 and float(sf[1, 0]) == 2.0 ** -126
    assert ref.TABLE[int(q[0, 0])] == 448 and ref.TABLE[int(q[127, 127])] == -224
    assert ref.TABLE[int(q[5, 200])] == 448 and ref.TABLE[int(q[129, 130])] == 448
