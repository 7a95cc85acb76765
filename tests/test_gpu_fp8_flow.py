"""The operators on rows in 8 bits as they are used together: a training step of
an MoE layer's experts -- tokens dispatched and quantised, both products, the
activation that keeps its input, the way back, and every gradient -- on streams,
captured into graphs, and several at once."""
import pytest
import torch

import fp8_ref as ref
import mixture_experts_forward_moe_amd as moe
from fp8_ref import F64, U4, U8, U24
from test_gpu_fp8_rows import BF16, BYTE, F32, GUARD, I32, gen, near, say

pytestmark = pytest.mark.gpu


def nb(n):
    return -(-n // 128)


class Step:
    """One training step of the local experts E0 .. E0 + El - 1 of E; tokens of a
    padded batch (the last ones) have no expert, one token has the same one k times."""

    def __init__(self, M, H, I, E, El, E0, k, tile, seed, padded=3, act=moe.ACT_SWIGLU):
        g = gen(seed)
        self.M, self.H, self.I, self.E, self.El, self.E0, self.k, self.tile, self.act = M, H, I, E, El, E0, k, tile, act
        self.x = torch.randn(M, H, generator=g).to(BF16).cuda()
        ids = torch.rand(M, E, generator=g).topk(k, 1).indices
        ids[ids == E0 + 1] = E0              # (an expert without a row)
        ids[M // 2] = E0                     # (the same index k times)
        if padded:
            ids[-padded:] = -1
        self.ids = ids.to(I32).cuda()
        self.weights = torch.rand(M, k, generator=g).cuda()
        self.dout = torch.randn(M, H, generator=g).to(BF16).cuda()
        self.w1, self.w2 = (torch.randn(El, n, m, generator=g).mul(m ** -0.5).to(BF16).cuda()
                            for n, m in ((2 * I, H), (H, I)))
        self.plan = moe.MoePlan(M, k, El, tile)
        self.slots = S = self.plan.route_slots

        def guarded(*shape, dtype=BYTE):
            n = torch.empty(shape, dtype=dtype).numel() * torch.empty(0, dtype=dtype).element_size()
            return torch.full((n,), GUARD, dtype=BYTE, device="cuda").view(dtype).view(shape)
        self.b = b = {}
        for name, rows, cols in (("w1", 2 * I, H), ("w2", H, I)):
            b[name + "q"], b[name + "sf"] = guarded(El, rows, cols), guarded(El, nb(rows), nb(cols), dtype=F32)
            b[name + "t"], b[name + "tsf"] = guarded(El, cols, rows), guarded(El, nb(cols), nb(rows), dtype=F32)
        for name, n in (("x", H), ("a", I), ("dy2", H)):
            b[name + "q"], b[name + "sf"] = guarded(S, n), guarded(S, nb(n))
        for name, blocks in (("h", 2 * nb(I)), ("dh", nb(2 * I))):
            b[name + "q"], b[name + "sf"] = guarded(S, 2 * I), guarded(S, blocks)
            b[name] = guarded(S, 2 * I, dtype=BF16)
        for name, n in (("y2", H), ("dy2", H), ("da", I), ("dxp", H)):
            b[name] = guarded(S, n, dtype=BF16)
        b["out"], b["dx"] = guarded(M, H, dtype=BF16), guarded(M, H, dtype=BF16)
        b["dweights"] = guarded(M, k, dtype=F32)
        b["dw1"], b["dw2"] = guarded(El, 2 * I, H, dtype=F32), guarded(El, H, I, dtype=F32)

    def run(self, stream=None):
        b, p, s = self.b, self.plan, stream
        moe.moe_sort(self.ids, self.E, self.El, self.E0, self.tile, plan=p, stream=s)
        moe.moe_quantize_fp8_weight(self.w1, b["w1q"], b["w1sf"], b["w1t"], b["w1tsf"], stream=s)
        moe.moe_quantize_fp8_weight(self.w2, b["w2q"], b["w2sf"], b["w2t"], b["w2tsf"], stream=s)
        moe.moe_dispatch(self.x, p, q=b["xq"], q_sf=b["xsf"], stream=s)
        moe.moe_grouped_linear_fp8(b["xq"], b["xsf"], p, b["w1q"], b["w1sf"], b["h"], stream=s)
        moe.moe_gated_act_fp8(b["h"], b["aq"], b["asf"], b["hq"], b["hsf"], p, self.act, stream=s)
        moe.moe_grouped_linear_fp8(b["aq"], b["asf"], p, b["w2q"], b["w2sf"], b["y2"], stream=s)
        moe.moe_finalize(b["y2"], p, self.weights, self.H, b["out"], stream=s)
        moe.moe_finalize_backward(self.dout, b["y2"], p, self.weights, b["dy2"], b["dy2q"], b["dy2sf"], b["dweights"],
                                  stream=s)
        moe.moe_grouped_linear_fp8_wgrad(b["dy2"], b["aq"], b["asf"], p, b["dw2"], stream=s)
        moe.moe_grouped_linear_fp8(b["dy2q"], b["dy2sf"], p, b["w2t"], b["w2tsf"], b["da"], stream=s)
        if self.I % 128 == 0:
            moe.moe_gated_act_fp8_backward(b["hq"], b["hsf"], b["da"], b["dh"], b["dhq"], b["dhsf"], p, self.act, stream=s)
        else:  # (the blocks of the halves are not those of a row of 2I)
            moe.moe_gated_act_fp8_backward(b["hq"], b["hsf"], b["da"], b["dh"], plan=p, activation=self.act, stream=s)
            moe.moe_quantize_fp8(b["dh"], b["dhq"], b["dhsf"], stream=s)
        moe.moe_grouped_linear_fp8_wgrad(b["dh"], b["xq"], b["xsf"], p, b["dw1"], stream=s)
        moe.moe_grouped_linear_fp8(b["dhq"], b["dhsf"], p, b["w1t"], b["w1tsf"], b["dxp"], stream=s)
        moe.moe_dispatch_backward(b["dxp"], p, b["dx"], stream=s)

    def clear(self):
        for v in self.b.values():
            v.view(BYTE).fill_(GUARD)

    def bits(self):
        return {n: v.clone() for n, v in self.b.items()}

    def same(self, want, what):
        for n, v in self.b.items():
            assert torch.equal(v.view(BYTE), want[n].view(BYTE)), f"{what}: {n}"


class Bounded:
    """An fp64 value and how far the kernels' one may be from it."""

    def __init__(self, v, e):
        self.v, self.e = v, e


def kept_bf16(b):
    """Rounded to bf16."""
    return Bounded(b.v, b.e + U8 * (b.v.abs() + b.e) + 2.0 ** -134)


def quantised(b):
    """Rows rounded to E4M3 under the power of two of a block, less than twice the largest value / 448: half a step
    of the value, or of the smallest step, 2^-9."""
    top = ref.blocks(b.v.abs() + b.e).amax(-1) * 2 / 448
    return Bounded(b.v, b.e + U4 * (b.v.abs() + b.e) + ref.spread(top, b.v.shape[-1]) * 2.0 ** -10)


def product(b, w, lossy):
    """b w^T in fp32, lossy: by the matrix instruction for 8 bits, which loses less than 8 * 2^-13 of the largest of 8
    products twice over (a power of two and the value below it); fp32 sums of K terms."""
    mag = (b.v.abs() + b.e) @ w.abs().t().contiguous()
    loss = (2.0 ** -10 if lossy else 0.0) + b.v.shape[1] * U24
    return Bounded(b.v @ w.t().contiguous(), b.e @ w.abs().t().contiguous() + loss * mag)


SHAPES = [(37, 256, 256, 8, 6, 1, 3, 16, moe.ACT_SWIGLU), (150, 272, 144, 6, 6, 0, 2, 32, moe.ACT_GEGLU_TANH),
          (301, 512, 384, 5, 4, 0, 2, 64, moe.ACT_SWIGLU), (700, 384, 272, 4, 3, 1, 2, 128, moe.ACT_SWIGLU),
          (1300, 272, 128, 3, 3, 0, 2, 256, moe.ACT_GEGLU_TANH)]


@pytest.mark.parametrize("M,H,I,E,El,E0,k,tile,act", SHAPES)
def test_step(M, H, I, E, El, E0, k, tile, act):
    """Every result against fp64: the forward pass at each call's own inputs, the gradients from the loss's on, with
    bounds that follow each rounding on its way; what a step keeps (rows and h in 8 bits) is where they are taken."""
    say(f"step {M} x {H} x {I}, {El} of {E} experts, tile {tile}")
    s = Step(M, H, I, E, El, E0, k, tile, M, act=act)
    s.run()
    torch.cuda.synchronize()
    b = {n: v.cpu() for n, v in s.b.items()}
    slots = s.plan.expanded_to_permuted.cpu().view(M, k)
    offsets, counts = s.plan.expert_offsets.cpu().tolist(), s.plan.expert_counts.cpu().tolist()
    ids, weights, dout, x = s.ids.cpu(), s.weights.cpu().double(), s.dout.cpu().double(), s.x.cpu()
    local = (ids >= E0) & (ids < E0 + El)
    assert torch.equal(slots >= 0, local) and int(local.sum()) == sum(counts)
    routes = local.nonzero()                                    # (token, which of its routes)
    at = slots[local].long()
    pad = torch.ones(s.slots, dtype=torch.bool)
    pad[at] = False
    kind = "geglu" if act == moe.ACT_GEGLU_TANH else "swiglu"
    dx = Bounded(torch.zeros(M, H, dtype=F64), torch.zeros(M, H, dtype=F64))
    for e in range(El):
        rows = slice(offsets[e], offsets[e] + counts[e])
        mine = (at >= offsets[e]) & (at < offsets[e] + counts[e])
        tok = torch.empty(counts[e], dtype=torch.long)
        wt = torch.empty(counts[e], 1, dtype=F64)
        tok[at[mine] - offsets[e]] = routes[mine][:, 0]
        wt[at[mine] - offsets[e], 0] = weights[local][mine]
        w1, w2 = (ref.weights(b[n + "q"][e], b[n + "sf"][e]) for n in ("w1", "w2"))
        exact = lambda v: Bounded(v, torch.zeros_like(v))  # noqa: E731
        # forward, at what each call was given
        q, sf = ref.quantize(x[tok])
        assert torch.equal(b["xq"][rows], q) and torch.equal(b["xsf"][rows], sf)
        xv, hv = ref.rows(q, sf), b["h"][rows].double()
        want = kept_bf16(product(exact(xv), w1, True))
        near(b["h"][rows], want.v, want.e, f"h of expert {e}")
        qh, sfh = ref.halves(b["h"][rows])
        assert torch.equal(b["hq"][rows], qh) and torch.equal(b["hsf"][rows], sfh)
        f, _, up, _ = ref.act(kind, hv[:, :I], hv[:, I:])
        fp32 = 16 * U24 * (f * up).abs() + 2.0 ** -20 * up.abs()  # (the exponential's and the product's few steps)
        want = quantised(kept_bf16(Bounded(f * up, fp32)))
        av = ref.rows(b["aq"][rows], b["asf"][rows])
        near(av, want.v, want.e, f"a of expert {e}")
        want = kept_bf16(product(exact(av), w2, True))
        near(b["y2"][rows], want.v, want.e, f"y2 of expert {e}")
        # backward, from dout on
        dy2 = kept_bf16(Bounded(wt * dout[tok], U24 * (wt * dout[tok]).abs()))
        near(b["dy2"][rows], dy2.v, dy2.e, f"dy2 of expert {e}")
        da = kept_bf16(product(quantised(dy2), w2.t().contiguous(), True))
        near(b["da"][rows], da.v, da.e, f"da of expert {e}")
        kept = ref.halves_rows(qh, sfh)
        f, df, up, dup = ref.act(kind, kept[:, :I], kept[:, I:])
        factor = torch.cat((df * up, f * dup), 1)
        off = 2.0 ** -18 * torch.cat((up.abs(), torch.ones_like(up)), 1)  # of f and f' in fp32
        dh = kept_bf16(Bounded(torch.cat((da.v, da.v), 1) * factor,
                               torch.cat((da.e, da.e), 1) * (factor.abs() + off) + torch.cat((da.v, da.v), 1).abs() * off))
        near(b["dh"][rows], dh.v, dh.e, f"dh of expert {e}")
        for name, d, v in (("dw2", dy2, av), ("dw1", dh, xv)):
            t = product(Bounded(d.v.t().contiguous(), d.e.t().contiguous()), v.t().contiguous(), False)
            near(b[name][e], t.v, t.e, f"{name} of expert {e}")
        dxp = kept_bf16(product(quantised(dh), w1.t().contiguous(), True))
        near(b["dxp"][rows], dxp.v, dxp.e, f"dxp of expert {e}")
        dx.v.index_add_(0, tok, dxp.v)
        dx.e.index_add_(0, tok, dxp.e)
    dx.e += k * U24 * (dx.v.abs() + dx.e)
    want = kept_bf16(dx)
    near(b["dx"], want.v, want.e, "dx")
    want = torch.zeros(M, k, dtype=F64)
    mag = torch.zeros(M, k, dtype=F64)
    terms = dout[routes[:, 0]] * b["y2"][at].double()
    want[local], mag[local] = terms.sum(1), terms.abs().sum(1)
    near(b["dweights"], want, H * U24 * mag, "dweights")
    assert bool((b["dx"][~local.any(1)] == 0).all()) and bool((b["out"][~local.any(1)] == 0).all())
    for e in range(El):
        if counts[e] == 0:
            assert bool((b["dw1"][e] == 0).all()) and bool((b["dw2"][e] == 0).all())
    assert min(counts) == 0
    for n in ("xq", "xsf", "aq", "asf", "h", "hq", "hsf", "y2", "dy2", "dy2q", "dy2sf", "da", "dh", "dhq", "dhsf", "dxp"):
        if n in ("dhq", "dhsf") and I % 128:
            continue
        assert bool((b[n][pad].contiguous().view(BYTE) == GUARD).all()), f"{n}: a padding slot was written"


def eager(s):
    s.clear()
    s.run()
    torch.cuda.synchronize()
    return s.bits()


def captured(s):
    """The step as a graph, and the results of an eager run."""
    want = eager(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run()
    return graph, want


def test_the_same_bits_again_on_other_streams():
    s = Step(301, 512, 384, 5, 4, 0, 2, 64, 7)
    want = eager(s)
    for _ in range(3):
        eager(s)
        s.same(want, "again")
    other = torch.cuda.Stream()
    s.clear()
    other.wait_stream(torch.cuda.current_stream())
    s.run(stream=other)                      # named
    other.synchronize()
    s.same(want, "a named stream")
    s.clear()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):           # current
        s.run()
    other.synchronize()
    s.same(want, "the current stream")


@pytest.mark.parametrize("tile", [16, 32, 64, 128, 256])
def test_graph(tile):
    """Captured once, replayed with other work and other inputs between."""
    s = Step(200, 384, 256, 6, 5, 0, 2, tile, 11)
    graph, want = captured(s)
    for i in range(4):
        s.clear()
        graph.replay()
        torch.cuda.synchronize()
        s.same(want, f"replay {i}")
        eager(s)
        torch.randn(64, 64, device="cuda").sum()
    # the same graph at other values, routes included
    g = gen(99)
    s.x.copy_(torch.randn(s.M, s.H, generator=g).to(BF16))
    s.ids.copy_(torch.randint(-1, s.E, (s.M, s.k), generator=g).to(I32))
    s.w1.copy_(torch.randn(s.w1.shape, generator=g).mul(0.1).to(BF16))
    want = eager(s)
    s.clear()
    graph.replay()
    torch.cuda.synchronize()
    s.same(want, "other values")


def test_two_graphs_and_an_eager_step_at_once():
    """None of them has anything that another one uses."""
    steps = [Step(130 + 100 * i, 272 + 128 * i, 128, 5, 4, 0, 2, 32, 20 + i) for i in range(3)]
    (g0, want0), (g1, want1), want2 = captured(steps[0]), captured(steps[1]), eager(steps[2])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(4):
        for s in steps:
            s.clear()
        torch.cuda.synchronize()
        for _ in range(2):
            with torch.cuda.stream(streams[0]):
                g0.replay()
            with torch.cuda.stream(streams[1]):
                g1.replay()
            with torch.cuda.stream(streams[2]):
                steps[2].run()
        torch.cuda.synchronize()
        for s, want in zip(steps, (want0, want1, want2)):
            s.same(want, f"round {i}")


def test_single_products_in_a_graph():
    """The products of one matrix, each way of splitting one among wavefronts."""
    g = gen(5)
    shapes = [(1, 512, 1024), (40, 1024, 512), (70, 512, 1040), (200, 1024, 512), (600, 520, 1568), (1100, 2056, 1040),
              (3100, 4104, 1024)]
    calls, outs = [], []
    for M, N, K in shapes:
        x = torch.randint(0, 120, (M, K), generator=g).to(BYTE).cuda()
        x_sf = torch.randint(120, 130, (M, nb(K)), generator=g).to(BYTE).cuda()
        w = torch.randint(0, 120, (N, K), generator=g).to(BYTE).cuda()
        w_sf = torch.rand(nb(N), nb(K), generator=g).cuda()
        y, dw = torch.zeros(M, N, dtype=BF16, device="cuda"), torch.zeros(N, K, device="cuda")
        dy = torch.randn(M, N, generator=g).to(BF16).cuda()
        calls.append((x, x_sf, w, w_sf, y, dy, dw))
        outs += [y, dw]

    def run():
        for x, x_sf, w, w_sf, y, dy, dw in calls:
            moe.moe_linear_fp8(x, x_sf, w, w_sf, y)
            moe.moe_linear_fp8_wgrad(dy, x, x_sf, dw)
    run()
    torch.cuda.synchronize()
    want = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(3):
        for o in outs:
            o.fill_(7)
        graph.replay()
        torch.cuda.synchronize()
        for j, (a, b) in enumerate(zip(outs, want)):
            assert torch.equal(a, b), f"replay {i}, output {j}"
        run()
        torch.cuda.synchronize()
