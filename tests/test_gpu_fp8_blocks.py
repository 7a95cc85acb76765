"""The products of rows in 8 bits by kernel and by blocks of K: each kernel,
with each way out, at K of few blocks, whole and ragged, where every block of a
row has a scale of its own.  Each case is seen to launch the kernel it is for."""
import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from hip_kernels import kernels_of
from test_gpu_fp8_products import nb, product, ranges, whole_weights
from test_gpu_fp8_rows import BF16, BYTE, F32, Guarded, gen, plan_of, say, untouched

pytestmark = pytest.mark.gpu


def tile(*p):
    """The part of a kernel's name that says which Tile it has."""
    return "4TileI" + "".join(f"Li{v}E" for v in p) + "E"


STREAM1, STREAM2 = "fp8_stream_kernelILi1EE", "fp8_stream_kernelILi2EE"
BIG, MIDDLE, SMALL, LOW = tile(4, 2, 4, 8, 2, 1), tile(2, 2, 4, 4, 2, 1), tile(2, 2, 2, 4, 3, 1), tile(1, 4, 2, 4, 2, 1)
SPLIT2, SPLIT4, SPLIT4_LOW = tile(2, 2, 2, 4, 3, 2), tile(2, 1, 2, 4, 2, 4), tile(1, 1, 2, 4, 2, 4)
FEW = (1, 2, 3, 4, 5, 7)

# Kernel, M and N (whole tiles, and K of whole blocks; ragged ones in turn), blocks of K.  K is split in four only
# where rows and columns have work enough: from two and from three blocks on; the
# largest tiles take one matrix from 1024 on.
ONE = [
    (STREAM1, [(16, 64), (13, 131)], FEW),
    (STREAM2, [(16, 8192), (5, 8193)], FEW),
    (SPLIT4_LOW, [(512, 1024), (387, 1027), (64, 8192), (256, 2048)], (3, 4, 5, 7, 9)),
    (SPLIT4, [(1024, 1024), (1000, 1001), (512, 2048)], (2, 3, 4, 5, 7, 9)),
    (SPLIT2, [(1024, 2048), (1001, 2041)], FEW),
    (SMALL, [(2048, 2048), (1999, 2001)], FEW),
    (MIDDLE, [(2176, 2048), (2100, 2049)], FEW),
    (BIG, [(4096, 4096), (4001, 4003)], (9, 10, 11)),
]
CASES = [(name, M, N, 128 * b - (112 if i % 2 else 0)) for name, sizes, blocks in ONE
         for i, (M, N) in enumerate(sizes) for b in blocks]


def rows_of(M, K, seed):
    """(codes, E8M0): whole numbers -2 .. 2 under scales 1/4 .. 4, none of them twice in five blocks of a row."""
    g = gen(seed)
    q = ref.encode(torch.randint(-2, 3, (M, K), generator=g).double())
    first = torch.randint(0, 5, (M, 1), generator=g)
    step = torch.randint(1, 5, (M, 1), generator=g)
    return q.cuda(), (125 + (first + step * torch.arange(nb(K))) % 5).to(BYTE).cuda()


@pytest.mark.parametrize("name,M,N,K", CASES)
def test_linear(name, M, N, K):
    """Sums of multiples of 2^-4 below 2^17: exact in fp32, on every way out."""
    say(f"linear {name} {M} x {N} x {K}")
    x, x_sf = rows_of(M, K, M + K)
    w, w_sf = whole_weights(1, N, K, N + K)
    g = gen(N)
    bias = torch.randint(-8, 9, (N,), generator=g).float().cuda()
    old = torch.randint(-64, 65, (M, N), generator=g).float().cuda()
    want = product(ref.rows(x, x_sf), ref.weights(w[0], w_sf[0]))
    for dtype in (BF16, F32):
        for b, acc in ((None, False), (bias, True)):
            out = Guarded()
            y = out(M, N, dtype=dtype)
            if acc:
                y.copy_(old)

            def call(stream=None):
                moe.moe_linear_fp8(x, x_sf, w[0], w_sf[0], y, bias=b, accumulate=acc, stream=stream)
            launched = kernels_of(call)
            assert len(launched) == 1 and name in launched[0], launched
            call()
            out.check()
            full = want + (b.double() + old.double() if acc else 0)
            assert torch.equal(y, full.to(dtype)), (dtype, acc)


@pytest.mark.parametrize("name,rows", [(STREAM1, 16), (STREAM2, 16), (LOW, 32), (SMALL, 64), (MIDDLE, 128), (BIG, 256)])
@pytest.mark.parametrize("blocks", [1, 2, 3, 4, 5, 7, 9])
def test_grouped_linear(name, rows, blocks):
    M, k, E = 701, 2, 5
    N = 520 if name == STREAM2 else 16 if name == STREAM1 else 776
    for K in (128 * blocks, 128 * blocks - 112):
        say(f"grouped linear {name} tile {rows} {N} x {K}")
        plan, slot = plan_of(M, k, E, E, 0, rows, blocks, "random")
        x, x_sf = rows_of(plan.route_slots, K, blocks)
        w, w_sf = whole_weights(E, N, K, blocks + 1)
        out = Guarded()
        y = out(plan.route_slots, N, dtype=BF16)

        def call(stream=None):
            moe.moe_grouped_linear_fp8(x, x_sf, plan, w, w_sf, y, stream=stream)
        launched = kernels_of(call)
        assert len(launched) == 1 and name in launched[0], launched
        call()
        out.check()
        for e, at in ranges(plan):
            assert torch.equal(y[at], product(ref.rows(x[at], x_sf[at]), ref.weights(w[e], w_sf[e])).to(BF16)), e
        rest = torch.ones(plan.route_slots, dtype=torch.bool)
        rest[slot[slot >= 0]] = False
        assert untouched(y.cpu()[rest]), "a padding slot was written"
