"""Rows in 8 bits whose elements pass 2^31 and 2^32: rows at the start, on both
sides of those marks and at the end hold small whole numbers (every sum is
exact), the others zeros, so that an offset cut off to 32 bits shows."""
import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from test_gpu_fp8_rows import BF16, BYTE, F32, F64, I32, gen, say

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def room():
    """Some tens of GB, given back after each test."""
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of free GPU memory")
    yield
    torch.cuda.empty_cache()


def nb(n):
    return -(-n // 128)


def marks(rows, cols):
    """Rows at the ends and around the elements 2^31 and 2^32."""
    assert rows * cols > (1 << 32) + cols
    at = {0, 1, rows - 1}
    for m in (1 << 31, 1 << 32):
        at |= {m // cols - 1, m // cols, m // cols + 1}
    return sorted(at)


def sparse(rows, cols, dtype, seed):
    """(tensor on the GPU, marked rows, their fp64 values): whole numbers -2 .. 2."""
    at = marks(rows, cols)
    v = torch.randint(-2, 3, (len(at), cols), generator=gen(seed)).double()
    t = torch.zeros(rows, cols, dtype=dtype, device="cuda")
    t[at] = (ref.encode(v) if dtype == BYTE else v.to(dtype)).cuda()
    return t, at, v


def ones(rows, cols):
    """Scales of 1."""
    return torch.full((rows, nb(cols)), 127, dtype=BYTE, device="cuda")


def whole(rows, cols, seed):
    v = torch.randint(-2, 3, (rows, cols), generator=gen(seed)).double()
    return ref.encode(v).cuda(), v


def same(got, want, what):
    got = got.cpu().double()
    assert torch.equal(got, want.to(F64)), f"{what}: {int((got != want).sum())} differ"


def test_quantize():
    rows, cols = 66000, 65552
    say(f"quantize {rows} x {cols}")
    x, at, v = sparse(rows, cols, BF16, 1)
    q, sf = torch.full((rows, cols), 9, dtype=BYTE, device="cuda"), torch.zeros(rows, nb(cols), dtype=BYTE, device="cuda")
    moe.moe_quantize_fp8(x, q, sf)
    torch.cuda.synchronize()
    want, want_sf = ref.quantize(v.to(BF16))
    assert torch.equal(q[at].cpu(), want) and torch.equal(sf[at].cpu(), want_sf)
    q[at] = 0
    for i in range(0, rows, 4096):
        assert not bool(q[i:i + 4096].any())


def test_quantize_weight():
    N, K = 66048, 65536
    say(f"weights {N} x {K}")
    w, at, v = sparse(N, K, BF16, 2)
    q, qt = (torch.full(s, 9, dtype=BYTE, device="cuda") for s in ((N, K), (K, N)))
    sf, sft = (torch.zeros(s, device="cuda") for s in ((nb(N), nb(K)), (nb(K), nb(N))))
    moe.moe_quantize_fp8_weight(w, q, sf, qt, sft)
    torch.cuda.synchronize()
    assert torch.equal(sf.t().contiguous(), sft)
    for n in at:
        rows = w[n // 128 * 128:n // 128 * 128 + 128].cpu()
        want, want_sf = ref.quantize_weight(rows)
        assert torch.equal(q[n].cpu(), want[n % 128]) and torch.equal(sf[n // 128].cpu(), want_sf[0])
    for i in range(0, K, 4096):
        assert torch.equal(qt[i:i + 4096], q[:, i:i + 4096].t().contiguous())


def test_dispatch_and_its_gradients():
    """Each token at two experts; their rows pass 2^32 elements, x's 2^31."""
    M, k, E, H = 140000, 2, 4, 16384
    say(f"dispatch {M} x {H}")
    x = torch.empty(M, H, dtype=BF16, device="cuda").normal_()
    ids = torch.rand(M, E, generator=gen(3)).topk(k, 1).indices.to(I32).cuda()
    p = moe.moe_sort(ids, E, E, 0, 256)
    S = p.route_slots
    assert S * H > 1 << 32
    slots = p.expanded_to_permuted.view(M, k).long()
    rows, q = torch.empty(S, H, dtype=BF16, device="cuda"), torch.empty(S, H, dtype=BYTE, device="cuda")
    sf = torch.empty(S, nb(H), dtype=BYTE, device="cuda")
    moe.moe_dispatch(x, p, rows, q, sf)
    dx = torch.empty(M, H, dtype=BF16, device="cuda")
    moe.moe_dispatch_backward(rows, p, dx)
    torch.cuda.synchronize()
    tokens = torch.cat((torch.arange(3), torch.randint(0, M, (40,), generator=gen(4)), torch.tensor([M - 1]))).cuda()
    last = p.permuted_to_expanded[p.permuted_to_expanded >= 0][-3:].long() // k  # of the last slots
    tokens = torch.cat((tokens, last))
    want, want_sf = ref.quantize(x[tokens].cpu())
    for j in range(k):
        s = slots[tokens, j]
        assert torch.equal(rows[s], x[tokens])
        assert torch.equal(q[s].cpu(), want) and torch.equal(sf[s].cpu(), want_sf)
    for i in range(0, M, 4096):
        assert torch.equal(dx[i:i + 4096], x[i:i + 4096] * 2)
    # the gradients of the way back: weights that are powers of two, y2 over dy2
    weights = torch.exp2(torch.randint(-2, 3, (M, k), generator=gen(5)).float()).cuda()
    y2, dw = rows, torch.empty(M, k, device="cuda")
    y = y2[slots[tokens]].double()
    moe.moe_finalize_backward(x, y2, p, weights, dy2=y2, q=q, q_sf=sf, d_topk_weights=dw)
    torch.cuda.synchronize()
    for j in range(k):
        s = slots[tokens, j]
        w = (x[tokens].float() * weights[tokens, j, None]).to(BF16)
        assert torch.equal(y2[s], w)
        want, want_sf = ref.quantize(w.cpu())
        assert torch.equal(q[s].cpu(), want) and torch.equal(sf[s].cpu(), want_sf)
        terms = x[tokens].double() * y[:, j]
        assert bool(((dw[tokens, j].double() - terms.sum(1)).abs() <= H * ref.U24 * terms.abs().sum(1)).all())


def test_act():
    rows, I = 140000, 16384
    say(f"act {rows} x {I}")
    h, at, v = sparse(rows, 2 * I, BF16, 6)
    y, hq, dq = (torch.full((rows, n), 9, dtype=BYTE, device="cuda") for n in (I, 2 * I, 2 * I))
    y_sf, hq_sf, dq_sf = (torch.zeros(rows, n, dtype=BYTE, device="cuda") for n in (nb(I), 2 * nb(I), 2 * nb(I)))
    moe.moe_gated_act_fp8(h, y, y_sf, hq, hq_sf)
    torch.cuda.synchronize()
    want, want_sf = ref.halves(v.to(BF16))
    assert torch.equal(hq[at].cpu(), want) and torch.equal(hq_sf[at].cpu(), want_sf)
    few = [torch.zeros(len(at), *t.shape[1:], dtype=t.dtype, device="cuda") for t in (y, y_sf, hq, hq_sf)]
    moe.moe_gated_act_fp8(h[at], *few)
    for got, one in zip((y, y_sf, hq, hq_sf), few):
        assert torch.equal(got[at], one)
    dy = torch.zeros(rows, I, dtype=BF16, device="cuda")
    dy[at] = torch.randn(len(at), I, generator=gen(7)).to(BF16).cuda()
    dh = h
    moe.moe_gated_act_fp8_backward(hq, hq_sf, dy, dh, dq, dq_sf)
    one = [torch.zeros(len(at), *t.shape[1:], dtype=t.dtype, device="cuda") for t in (dh, dq, dq_sf)]
    moe.moe_gated_act_fp8_backward(hq[at], hq_sf[at], dy[at], *one)
    for got, o in zip((dh, dq, dq_sf), one):
        assert torch.equal(got[at], o)
    dq[at] = 0
    for i in range(0, rows, 8192):
        assert not bool(dq[i:i + 8192].any())


def test_linear_rows():
    """x and y past the marks."""
    M = 70000
    for N, K in ((64, 65536), (65536, 128)):
        say(f"linear {M} x {N} x {K}")
        if K > N:
            x, at, v = sparse(M, K, BYTE, 8)
        else:
            at = marks(M, N)
            v = torch.randint(-2, 3, (len(at), K), generator=gen(9)).double()
            x = torch.zeros(M, K, dtype=BYTE, device="cuda")
            x[at] = ref.encode(v).cuda()
        w, wv = whole(N, K, 10)
        y = torch.full((M, N), 7, dtype=BF16, device="cuda")
        moe.moe_linear_fp8(x, ones(M, K), w, torch.ones(nb(N), nb(K), device="cuda"), y)
        torch.cuda.synchronize()
        same(y[at], (v @ wv.t()).to(BF16), "y")
        y[at] = 0
        for i in range(0, M, 8192):
            assert not bool(y[i:i + 8192].any())


@pytest.mark.parametrize("M", [5, 100])
def test_linear_weights(M):
    N, K = 70000, 65536
    say(f"linear {M} x {N} x {K}")
    w, at, wv = sparse(N, K, BYTE, 11)
    x, v = whole(M, K, 12)
    y = torch.full((M, N), 7, dtype=F32, device="cuda")
    moe.moe_linear_fp8(x, ones(M, K), w, torch.ones(nb(N), nb(K), device="cuda"), y)
    torch.cuda.synchronize()
    same(y[:, at], v @ wv.t(), "y")
    y[:, at] = 0
    assert not bool(y.any())


@pytest.mark.parametrize("tile", [16, 32, 256])
def test_experts(tile):
    """Weights and their gradient past the marks; rows at the first and the last experts."""
    E, N, K, M = 17, 16384, 16400, 40
    say(f"experts {E} x {N} x {K}, tile {tile}")
    ids = torch.tensor([0, 1, 7, 8, 15, 16])[torch.randint(0, 6, (M, 2), generator=gen(13))].to(I32).cuda()
    p = moe.moe_sort(ids, E, E, 0, tile)
    S = p.route_slots
    w = torch.empty(E, N, K, dtype=BYTE, device="cuda")
    codes = whole(N, K, 100)[0]
    for e in range(E):  # (each expert's a little further on)
        w[e] = torch.roll(codes, e, 1)
    w_sf = torch.ones(E, nb(N), nb(K), device="cuda")
    x, v = whole(S, K, 14)
    y = torch.zeros(S, N, dtype=BF16, device="cuda")
    moe.moe_grouped_linear_fp8(x, ones(S, K), p, w, w_sf, y)
    dy = torch.randint(-2, 3, (S, N), generator=gen(15)).to(BF16)
    dw = torch.full((E, N, K), 7.0, device="cuda")
    moe.moe_grouped_linear_fp8_wgrad(dy.cuda(), x, ones(S, K), p, dw)
    torch.cuda.synchronize()
    offsets, counts = p.expert_offsets.cpu().tolist(), p.expert_counts.cpu().tolist()
    cols = [0, 1, 777, N - 2, N - 1]
    for e in range(E):
        r = slice(offsets[e], offsets[e] + counts[e])
        wv = ref.TABLE[w[e][cols].cpu().long()]
        same(y[r][:, cols], (v[r] @ wv.t()).to(BF16), f"y of expert {e}")
        same(dw[e][cols], dy[r][:, cols].double().t() @ v[r], f"dw of expert {e}")
        if counts[e] == 0:
            assert not bool(dw[e].any())


def test_wgrad_rows():
    """dy and x past the marks."""
    M = 70000
    for N, K in ((65536, 16), (8, 65536)):
        say(f"wgrad {M} x {N} x {K}")
        if N > K:
            dy, at, d = sparse(M, N, BF16, 16)
            v = torch.randint(-2, 3, (len(at), K), generator=gen(17)).double()
            x = torch.zeros(M, K, dtype=BYTE, device="cuda")
            x[at] = ref.encode(v).cuda()
        else:
            x, at, v = sparse(M, K, BYTE, 18)
            d = torch.randint(-2, 3, (len(at), N), generator=gen(19)).double()
            dy = torch.zeros(M, N, dtype=BF16, device="cuda")
            dy[at] = d.to(BF16).cuda()
        dw = torch.full((N, K), 7.0, device="cuda")
        moe.moe_linear_fp8_wgrad(dy, x, ones(M, K), dw)
        torch.cuda.synchronize()
        same(dw, d.t() @ v, "dw")
