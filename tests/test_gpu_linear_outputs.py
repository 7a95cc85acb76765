"""The ways out of moe_linear_mx: every width of the stored pieces, at every
alignment of y, in every kernel."""
import pytest
import torch

import mixture_experts_forward_moe_amd as moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
GUARD = 173


def say(*a):
    print(*a, flush=True)


def whole_operands(M, N, K, elem, seed=1):
    """x, w and their scales whose products are multiples of 1/4 up to 36 and
    whose sums stay below 2^22: every order of the sums gives the same fp32."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda *s: torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    t = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device="cuda")
    t = torch.cat((t, -t))
    val = lambda q: t[torch.stack((q & 15, q >> 4), -1).flatten(-2).long()]  # noqa: E731
    xq, wq = byte(M, K // 2), byte(N, K // 2)
    prod = val(xq) @ val(wq).t()
    if elem == 0:
        xq = val(xq).to(torch.float8_e4m3fn).view(torch.uint8)
    one = lambda n: torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    return (xq, one(M), wq, one(N)), prod


def placed(M, N, dtype, offset):
    """y at `offset` elements behind an aligned address, and a check of what
    lies around it."""
    size = torch.empty(0, dtype=dtype).element_size()
    room = torch.full(((M * N + offset) * size + 512,), GUARD, dtype=torch.uint8, device="cuda")
    at, end = offset * size, (offset + M * N) * size

    def check():
        assert bool((room[:at] == GUARD).all()) and bool((room[end:] == GUARD).all()), "written outside of y"
    return room[at:end].view(dtype).view(M, N), check


@pytest.mark.parametrize("M,N,K", [
    (7, 515, 1536), (70, 200, 160),                                     # 16 x 16 tiles
    (300, 512, 1536), (300, 515, 1536), (300, 516, 2048), (300, 514, 1024),
    (1100, 1252, 160), (1237, 2056, 1568), (1237, 2055, 1568), (2111, 1110, 736), (600, 4100, 2080),
    (2500, 2576, 544), (4096, 4096, 1024), (3900, 4090, 1120),
])
@pytest.mark.parametrize("elem", [0, 1])
def test_ways_out(M, N, K, elem):
    say(f"ways out M={M} N={N} K={K} elem={elem}")
    args, prod = whole_operands(M, N, K, elem)
    for offset in (0, 1, 2, 4):
        y, check = placed(M, N, BF16, offset)
        moe.moe_linear_mx(*args, y, x_elem=elem)
        torch.cuda.synchronize()
        check()
        assert torch.equal(y, prod.to(BF16)), offset
        y32, check = placed(M, N, F32, offset)
        moe.moe_linear_mx(*args, y32, x_elem=elem)
        torch.cuda.synchronize()
        check()
        assert torch.equal(y32, prod), offset
        # (fp32: a sum of two multiples of 1/4 below 2^22; bf16: rounded once)
        moe.moe_linear_mx(*args, y32, x_elem=elem, accumulate=True)
        assert torch.equal(y32, 2 * prod), offset
        y.fill_(3)
        moe.moe_linear_mx(*args, y, x_elem=elem, accumulate=True)
        torch.cuda.synchronize()
        check()
        assert torch.equal(y, (prod + 3).to(BF16)), offset


def mixed_operands(M, N, K, elem, seed=2):
    """Random codes and scales of 2^-10 .. 2^10: sums that round at every step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    byte = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
    xq = byte(0, 256, M, K // 2)
    if elem == 0:  # E4M3 codes of both signs, without NaN
        xq = byte(0, 126, M, K) | (byte(0, 2, M, K) << 7)
    return xq, byte(117, 138, M, K // 32), byte(0, 256, N, K // 2), byte(117, 138, N, K // 32)


@pytest.mark.parametrize("M,N,K", [
    (8, 520, 1536), (70, 200, 1120),                                    # 16 x 16 tiles
    (300, 512, 1536), (300, 512, 2048), (300, 520, 4096),               # 64 x 64, K split in two from 2048 on
    (512, 4096, 4096), (1024, 1032, 2080), (520, 4104, 2048),           # E4M3: K split in two
    (1237, 2056, 1568), (1100, 4096, 2048), (2500, 2576, 544), (4096, 4096, 1024), (3900, 4096, 1120),
])
@pytest.mark.parametrize("elem", [0, 1])
def test_one_sum_whatever_becomes_of_it(M, N, K, elem):
    """y's type, alignment and the accumulation change no bit of the sums."""
    say(f"one sum M={M} N={N} K={K} elem={elem}")
    args = mixed_operands(M, N, K, elem)
    g = torch.Generator(device="cuda").manual_seed(3)
    alpha, bias = torch.tensor([0.7], device="cuda"), torch.randn(N, generator=g, device="cuda") * 1e4
    for kw in (dict(), dict(alpha=alpha), dict(bias=bias), dict(alpha=alpha, bias=bias)):
        y32, _ = placed(M, N, F32, 0)
        moe.moe_linear_mx(*args, y32, x_elem=elem, **kw)
        assert bool(torch.isfinite(y32).all())
        for dtype, offset, acc in ((F32, 1, False), (F32, 0, True), (F32, 3, True), (BF16, 0, False), (BF16, 1, False),
                                   (BF16, 2, False), (BF16, 4, False), (BF16, 0, True), (BF16, 1, True)):
            y, check = placed(M, N, dtype, offset)
            if acc:
                y.zero_()
            moe.moe_linear_mx(*args, y, x_elem=elem, accumulate=acc, **kw)
            torch.cuda.synchronize()
            check()
            assert torch.equal(y, y32.to(dtype)), (list(kw), dtype, offset, acc)


@pytest.mark.parametrize("M", [16, 300, 3000])
@pytest.mark.parametrize("elem", [0, 1])
def test_bits_of_a_product_that_count(M, elem):
    """What the header says of the products beside a large one: E4M3 ones count
    down to 2^-13 of it in its group of 8 consecutive k, and to fp32's last bit
    in others; E2M1 ones all."""
    say(f"product bits M={M} elem={elem}")
    N, K = 1024, 1056
    code = {0: {256.0: 0x78, 2.0 ** -5: 0x10, 2.0 ** -9: 0x01}, 1: {4.0: 6, 0.5: 1}}[elem]
    big, small, least = (256.0, 2.0 ** -5, 2.0 ** -9) if elem == 0 else (4.0, 0.5, 0.5)
    x = torch.zeros(M, K, dtype=torch.uint8)
    want = torch.zeros(M)
    for m in range(M):
        i = (37 * m) % K                       # the large one
        j = i - i % 8 + (i + 1 + m % 7) % 8    # in its group
        far = (i + 8 * (1 + m // 8 % 100)) % K # in another
        x[m, i], x[m, j], x[m, far] = code[big], code[small], code[least]
        want[m] = big + small + least
    if elem == 1:
        x = x[:, 0::2] | (x[:, 1::2] << 4)
    w = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # 1 everywhere
    one = lambda n: torch.full((n, K // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    y = torch.empty(M, N, device="cuda")
    moe.moe_linear_mx(x.cuda(), one(M), w, one(N), y, x_elem=elem)
    assert torch.equal(y, want.cuda()[:, None].expand(M, N))
