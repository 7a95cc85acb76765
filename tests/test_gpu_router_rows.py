"""A token's experts, weights and gradients hang on its own logits alone,
and tokens that are hard to choose for cost the others nothing."""
import pytest
import torch

import layer_ref as ref
import mixture_experts_forward_moe_amd as moe

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def say(*a):
    print(*a, flush=True)


def topk(l, k, **kw):
    ids = torch.empty(l.shape[0], k, dtype=torch.int32, device="cuda")
    w = torch.empty(l.shape[0], k, device="cuda")
    moe.moe_router_topk(l, ids, w, **kw)
    return ids, w


def gradient(l, ids, dw, grad, **kw):
    d = torch.empty_like(l)
    moe.moe_router_backward(l, ids, d, d_topk_weights=dw, prob_grad=grad, **kw)
    return d


def median_us(f, n=20):
    """Median time of a call in a replayed graph of n."""
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(n):
            f()
    times = []
    for _ in range(9):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        g.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 1e3 / n)
    return sorted(times)[4]


# what stands beside the tokens looked at: rows that choose by another way
BESIDE = {
    "equal": lambda l: torch.zeros_like(l),
    "negative": lambda l: -5 - l.abs(),
    "nothing": lambda l: torch.full_like(l, -INF),
    "nan": lambda l: torch.full_like(l, NAN),
    "two slots": lambda l: torch.where(torch.arange(l.shape[1], device="cuda") % (l.shape[1] // 20 + 1) == 0, 9.0, l),
}


@pytest.mark.parametrize("E,k", [(40, 4), (100, 7), (159, 6), (256, 8), (500, 16), (128, 20), (1000, 8)])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_do_not_hang_on_their_neighbours(E, k, dtype):
    g = torch.Generator(device="cuda").manual_seed(E + k)
    M = 203
    l = torch.randn(M, E, generator=g, device="cuda").to(dtype)
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    dw, grad = torch.randn(M, k, generator=g, device="cuda"), torch.randn(E, generator=g, device="cuda")
    out = [torch.empty(E, dtype=torch.int32, device="cuda"), torch.empty(E, device="cuda"),
           torch.empty(E, device="cuda"), torch.empty(1, device="cuda")]
    names = ("expert_counts", "mean_probs", "prob_grad", "loss")
    for score in (0, 1):
        for renorm in (True, False):
            for b in (None, bias):
                kw = dict(score=score, renormalize=renorm, select_bias=b)
                ids, w = topk(l, k, **kw)
                d = gradient(l, ids, dw, grad, score=score, renormalize=renorm)
                fused = topk(l, k, coef=0.1, **dict(zip(names, out)), **kw)
                assert torch.equal(fused[0], ids) and torch.equal(fused[1], w)
                for what, change in BESIDE.items():
                    say(f"rows E={E} k={k} {dtype} score={score} renorm={renorm} bias={b is not None} {what}")
                    for first in (0, 2):
                        at = torch.arange(M, device="cuda") % 4 != first
                        other = torch.where(at[:, None], l, change(l).to(dtype))
                        ids2, w2 = topk(other, k, **kw)
                        assert torch.equal(ids2[at], ids[at]) and torch.equal(w2[at], w[at])
                        d2 = gradient(other, ids2, dw, grad, score=score, renormalize=renorm)
                        assert torch.equal(d2[at], d[at])
                        ids64, w64 = ref.router_topk(other.cpu(), k, score, renorm, None if b is None else b.cpu())
                        assert torch.equal(ids2.cpu(), ids64)
                        on = at.to(torch.uint8)
                        ids2, w2 = topk(other, k, token_mask=on, **kw)
                        assert torch.equal(ids2[at], ids[at]) and torch.equal(w2[at], w[at])
                        assert bool((ids2[~at] == -1).all()) and bool((w2[~at] == 0).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_padding_rows_cost_no_more_than_others(dtype):
    """A masked row's choice is thrown away, whatever it holds: a batch whose
    padding has equal logits (every key a candidate) takes the time of one
    whose padding is random.  (Chosen by rounds, those rows made it 4.7 times.)"""
    say(f"padding {dtype}")
    M, E, k = 65536, 256, 8
    l = torch.randn(M, E, device="cuda").to(dtype)
    mask = (torch.arange(M, device="cuda") % 5 != 4).to(torch.uint8)
    same = torch.where(mask.bool()[:, None], l, torch.zeros_like(l))
    t = [median_us(lambda: topk(x, k, token_mask=mask)) for x in (l, same)]
    say(t)
    assert t[1] <= 2 * t[0]


@pytest.mark.parametrize("E,k", [(16, 4), (40, 4), (64, 8), (128, 6), (159, 6), (256, 8), (256, 3), (500, 10), (1000, 8)])
@pytest.mark.parametrize("score", [0, 1])
def test_one_pair_closer_than_fp32_resolves(E, k, score):
    """Two experts whose scores plus bias agree to fp32's last bits, among
    others that are far apart: the fp64 order, wherever the pair lies."""
    say(f"one close pair E={E} k={k} score={score}")
    for seed in range(12):
        g = torch.Generator().manual_seed(seed)
        M = 64
        b = torch.randn(E, generator=g) * 0.1
        i, j = torch.randperm(E, generator=g)[:2].tolist()
        if score:  # the others differ from token to token
            l = torch.randn(M, E, generator=g)
            l[:, i], l[:, j] = 2.5, 1.0
        else:      # the same logits in another order, so that the pair's softmax stays
            others = torch.tensor([e for e in range(E) if e not in (i, j)])
            row = torch.randn(E, generator=g)
            row[i], row[j] = 1.5, 0.75
            l = row.repeat(M, 1)
            for m in range(M):
                l[m, others] = row[others[torch.randperm(E - 2, generator=g)]]
        s = ref.scores(l[:1], score)[0][0]
        b[i] = 0.5
        b[j] = (s[i] + 0.5 - s[j]).float()
        ids, _ = topk(l.cuda(), k, score=score, select_bias=b.cuda())
        assert torch.equal(ids.cpu(), ref.router_topk(l, k, score, True, b)[0]), seed


@pytest.mark.parametrize("E,k", [(40, 4), (128, 7), (300, 16), (1000, 9)])
def test_infinite_keys_beside_other_tokens(E, k):
    """A bias of +inf, in tokens with few candidates and with many (which go by
    rounds and must leave the candidates of the others alone)."""
    g = torch.Generator().manual_seed(E)
    M = 70
    l = torch.randn(M, E, generator=g)
    l[1::4] = 0.5
    mask = torch.ones(M, dtype=torch.uint8)
    mask[2::4] = 0
    for count in (1, 2, k, k + 2, E):
        bias = torch.randn(E, generator=g) * 0.1
        bias[torch.randperm(E, generator=g)[:count]] = INF
        for score in (0, 1):
            for m in (None, mask):
                say(f"infinite E={E} k={k} count={count} score={score} mask={m is not None}")
                ids, w = topk(l.cuda(), k, score=score, select_bias=bias.cuda(),
                              token_mask=None if m is None else m.cuda())
                ids64, w64 = ref.router_topk(l, k, score, True, bias, m)
                assert torch.equal(ids.cpu(), ids64)
                assert bool(((w.cpu().double() - w64).abs() <= w64 * (k + 40) * ref.U24).all())


@pytest.mark.parametrize("E,k", [(40, 4), (60, 6), (256, 8), (300, 16), (1000, 9)])
def test_bias_that_takes_experts_out_or_puts_them_first(E, k):
    """Biases far from the scores: their own rounding errors are larger than
    any difference of scores, which the other experts must not feel."""
    g = torch.Generator().manual_seed(E)
    M = 61
    l = torch.randn(M, E, generator=g)
    l[7] = 0.25
    base = torch.randn(E, generator=g) * 0.1
    at = torch.randperm(E, generator=g)
    big = torch.finfo(F32).max
    cases = {"one out": {-1e9: 1}, "lowest": {-big: 2}, "three out": {-1e9: 1, -999999936.0: 1, -3e4: 1},
             "all but three out": {-1e9: E - 3}, "one first": {1e9: 1}, "many first": {1e9: k + 3},
             "first and out": {1e9: 2, -1e9: 2, -big: 1}, "infinite": {INF: 1, -INF: 1}, "infinite first": {INF: k + 2},
             "largest": {big: 3}}
    for what, values in cases.items():
        bias, n = base.clone(), 0
        for v, count in values.items():
            bias[at[n:n + count]] = v
            n += count
        for score in (0, 1):
            for b in (bias, torch.where(bias == base, 0.0, bias)):
                say(f"bias E={E} k={k} {what} score={score}")
                for dtype in (F32, BF16):
                    x = l.to(dtype)
                    ids, w = topk(x.cuda(), k, score=score, select_bias=b.cuda())
                    ids64, w64 = ref.router_topk(x, k, score, True, b)
                    assert torch.equal(ids.cpu(), ids64)
                    # half a dozen steps of |l| <= 6 and of the sum of k scores
                    assert bool(((w.cpu().double() - w64).abs() <= w64 * (k + 40) * ref.U24).all())


@pytest.mark.parametrize("score", [0, 1])
def test_expert_taken_out_costs_the_others_nothing(score):
    """One expert at -1e9: the others keep the time of an ordinary bias (8 times
    that, when the errors of its key counted for all)."""
    say(f"expert out score={score}")
    M, E, k = 65536, 256, 8
    l = torch.randn(M, E, device="cuda")
    bias = torch.randn(E, device="cuda") * 0.1
    out = bias.clone()
    out[3] = -1e9
    t = [median_us(lambda: topk(l, k, score=score, select_bias=b)) for b in (bias, out)]
    say(t)
    assert t[1] <= 2 * t[0]


def test_scores_below_the_normal_range():
    """Scores that fp32 does not hold, beside biases of their size."""
    say("tiny scores")
    for l, bias in [([-87.5, -200.0], [0.0, 7e-39]), ([-88.0, -200.0], [1.2e-38, 1.5e-38]),
                    ([-90.0, -89.0], [1.2e-38, 1.2e-38]), ([-200.0, -87.5, -100.0], [8e-39, 0.0, 3e-39])]:
        l, bias = torch.tensor([l] * 5), torch.tensor(bias)
        for k in (1, 2):
            ids, _ = topk(l.cuda(), k, score=1, select_bias=bias.cuda())
            assert torch.equal(ids.cpu(), ref.router_topk(l, k, 1, True, bias)[0])


@pytest.mark.parametrize("E,k", [(5, 5), (60, 16), (300, 40), (1000, 64)])
def test_equal_ids_add_up_in_one_order(E, k):
    """Many places of a token with the same expert: the same bits wherever the
    token stands and on every run."""
    say(f"equal ids E={E} k={k}")
    g = torch.Generator(device="cuda").manual_seed(E)
    M = 1003
    l = torch.randn(1, E, generator=g, device="cuda").expand(M, E).contiguous()
    ids = torch.randint(0, 3, (1, k), generator=g, device="cuda", dtype=torch.int32).expand(M, k).contiguous()
    dw = torch.randn(1, k, generator=g, device="cuda") * 10 ** torch.randn(1, k, generator=g, device="cuda")
    dw = dw.expand(M, k).contiguous()
    for score in (0, 1):
        for renorm in (True, False):
            kw = dict(score=score, renormalize=renorm)
            d = gradient(l, ids, dw, None, **kw)
            assert torch.equal(d, d[:1].expand(M, E))
            for _ in range(5):
                assert torch.equal(gradient(l, ids, dw, None, **kw), d)
            want, size = ref.router_backward(l[:1].cpu(), ids[:1].cpu(), score, renorm, dw[:1].cpu())
            # (a place more is a rounding more: k of them on top of the weights')
            assert bool(((d[:1].cpu().double() - want).abs() <= size * (k + 100) * ref.U24 + 1e-37).all())
