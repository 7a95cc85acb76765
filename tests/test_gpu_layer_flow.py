"""The operators around the routed experts as they are used together: the
input of an MoE layer, its router, the routed experts and a shared expert;
on other streams, captured into a graph, and several at once."""
import numpy as np
import pytest
import torch

import layer_ref as ref
import mixture_experts_forward_moe_amd as moe
import oracle
import synth

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def say(*a):
    print(*a, flush=True)


class Layer:
    """An MXFP8 x MXFP4 MoE layer with a shared linear part, one step:
    norm -> router -> shared product into out -> routed experts on top."""

    def __init__(self, M, H=512, I=256, E=8, k=2, seed=1):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std)  # noqa: E731
        self.M, self.H, self.I, self.E, self.k = M, H, I, E, k

        def mx(rows, cols, std):
            v = rnd(rows, cols, std=std).to(BF16).view(torch.int16).numpy().view(np.uint16)
            q, s = oracle.mx_quantize_bf16(v, 1)
            return torch.from_numpy(np.asarray(q)).cuda(), torch.from_numpy(np.asarray(s)).cuda()

        self.x, self.res = rnd(M, H).to(BF16).cuda(), rnd(M, H).to(BF16).cuda()
        self.weight = (1 + 0.1 * rnd(H)).cuda()
        self.wg = rnd(E, H, std=H ** -0.5).cuda()
        w1, s1 = mx(E * 2 * I, H, 0.05)
        w2, s2 = mx(E * H, I, 0.05)
        self.w1, self.w1_sf = w1.view(E, 2 * I, H // 2), s1.view(E, 2 * I, H // 32)
        self.w2, self.w2_sf = w2.view(E, H, I // 2), s2.view(E, H, I // 32)
        self.one = torch.ones(E, device="cuda")
        self.ws, self.ws_sf = mx(H, H, 0.05)
        e = lambda *s, dtype=F32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.h, self.y = e(M, H, dtype=BF16), e(M, H, dtype=BF16)
        self.q, self.sf = e(M, H, dtype=torch.uint8), e(M, H // 32, dtype=torch.uint8)
        self.rstd, self.logits = e(M), e(M, E)
        self.ids, self.w = e(M, k, dtype=torch.int32), e(M, k)
        self.counts, self.mean, self.grad, self.loss = e(E, dtype=torch.int32), e(E), e(E), e(1)
        self.d_logits, self.dw = e(M, E), rnd(M, k).cuda()
        self.dx, self.dweight = e(M, H, dtype=BF16), e(H)
        self.dy = rnd(M, H).to(BF16).cuda()
        self.out = e(M, H, dtype=BF16)
        self.tile = 32
        n = moe.workspace_size(M, H, I, k, E, self.tile, moe.MXFP8_MXFP4)
        self.space = torch.empty(n, dtype=torch.uint8, device="cuda")
        self.bspace = torch.empty(moe.balance_workspace_size(M, E), dtype=torch.uint8, device="cuda")
        self.nspace = torch.empty(moe.rmsnorm_backward_workspace_size(M, H), dtype=torch.uint8, device="cuda")

    def forward(self, stream=None):
        moe.moe_rmsnorm(self.x, self.weight, y=self.y, residual=self.res, residual_out=self.h, q=self.q, q_sf=self.sf,
                        rstd=self.rstd, stream=stream)
        torch.sum(self.y.float()[:, None, :] * self.wg, -1, out=self.logits)
        moe.moe_router_topk(self.logits, self.ids, self.w, coef=0.1, expert_counts=self.counts, mean_probs=self.mean,
                            prob_grad=self.grad, loss=self.loss, workspace=self.bspace, stream=stream)
        moe.moe_linear_mx(self.q, self.sf, self.ws, self.ws_sf, self.out, stream=stream)
        moe.moe_forward(self.q, self.sf, self.ids, self.w, self.w1, self.w1_sf, self.one, self.w2, self.w2_sf,
                        self.one, self.E, self.k, self.E, 0, moe.MXFP8_MXFP4, self.out, self.H, self.I,
                        workspace=self.space, tile=self.tile, accumulate=True, stream=stream)

    def backward(self, stream=None):
        moe.moe_router_backward(self.logits, self.ids, self.d_logits, d_topk_weights=self.dw, prob_grad=self.grad,
                                stream=stream)
        moe.moe_rmsnorm_backward(self.dy, self.h, self.weight, self.rstd, self.dx, self.dweight,
                                 workspace=self.nspace, stream=stream)

    def results(self):
        return [t.clone() for t in (self.h, self.y, self.q, self.sf, self.ids, self.w, self.counts, self.mean,
                                    self.grad, self.loss, self.out, self.d_logits, self.dx, self.dweight)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8) if x.dtype != torch.int32 else x,
                           y.view(torch.uint8) if y.dtype != torch.int32 else y) for x, y in zip(a, b))


@pytest.mark.parametrize("M", [1, 24, 300])
def test_layer_against_the_oracle(M):
    """The whole run: routed experts by the CPU oracle from the GPU's own
    input codes and routing, the shared product in fp64."""
    say(f"layer M={M}")
    L = Layer(M)
    L.forward()
    torch.cuda.synchronize()
    hx, r64, y64 = ref.rmsnorm(L.x.cpu(), L.res.cpu(), L.weight.cpu(), 1e-6)
    assert torch.equal(L.h.cpu(), hx)
    ids64, w64 = ref.router_topk(L.logits.cpu(), L.k, 0, True)
    assert torch.equal(L.ids.cpu(), ids64)
    assert int(L.counts.sum()) == M * L.k
    n = lambda t: np.ascontiguousarray(t.cpu().numpy())  # noqa: E731
    p = oracle.Problem(mode=oracle.MXFP8_MXFP4, M=M, H=L.H, I=L.I, num_experts=L.E, num_local_experts=L.E,
                       local_expert_offset=0, top_k=L.k, x=n(L.q), x_sf=n(L.sf), topk_ids=n(L.ids),
                       topk_weights=n(L.w), w1=n(L.w1), w1_sf=n(L.w1_sf), w1_alpha=np.ones(L.E, np.float32),
                       w2=n(L.w2), w2_sf=n(L.w2_sf), w2_alpha=np.ones(L.E, np.float32))
    routed = synth.bf16_to_f32(oracle.forward_tokens(p, np.arange(M))).astype(np.float64)
    shared = ref.mx_values(L.q.cpu(), L.sf.cpu(), 0) @ ref.mx_values(L.ws.cpu(), L.ws_sf.cpu(), 1).t()
    want = routed + shared.numpy()
    got = L.out.cpu().double().numpy()
    assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(want)


def test_layer_replayed_from_a_graph():
    """Forward and backward captured once, replayed with the eager run of
    another layer in between; every replay equals the eager result."""
    say("layer graph")
    L, other = Layer(70), Layer(90, seed=2)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        L.forward()
        L.backward()
    torch.cuda.synchronize()
    want = L.results()
    logits = L.logits.clone()
    g = torch.cuda.CUDAGraph()

    def step():
        moe.moe_rmsnorm(L.x, L.weight, y=L.y, residual=L.res, residual_out=L.h, q=L.q, q_sf=L.sf, rstd=L.rstd)
        moe.moe_router_topk(L.logits, L.ids, L.w, coef=0.1, expert_counts=L.counts, mean_probs=L.mean,
                            prob_grad=L.grad, loss=L.loss, workspace=L.bspace)
        moe.moe_linear_mx(L.q, L.sf, L.ws, L.ws_sf, L.out)
        moe.moe_forward(L.q, L.sf, L.ids, L.w, L.w1, L.w1_sf, L.one, L.w2, L.w2_sf, L.one, L.E, L.k, L.E, 0,
                        moe.MXFP8_MXFP4, L.out, L.H, L.I, workspace=L.space, tile=L.tile, accumulate=True)
        L.backward()

    with torch.cuda.graph(g):
        step()
    for i in range(4):
        for t in (L.h, L.y, L.q, L.sf, L.ids, L.w, L.counts, L.mean, L.grad, L.loss, L.out, L.d_logits, L.dx,
                  L.dweight):
            t.fill_(3)
        L.bspace.fill_(255)
        L.nspace.fill_(255)
        assert torch.equal(L.logits, logits)
        g.replay()
        other.forward()
        other.backward()
        torch.cuda.synchronize()
        assert same(L.results(), want), i


def test_layers_on_two_streams():
    """Two layers in flight at once, each on a stream of its own."""
    say("layers on two streams")
    layers = [Layer(130, seed=3), Layer(41, seed=4)]
    want = []
    for L in layers:
        L.forward()
        L.backward()
        torch.cuda.synchronize()
        want.append(L.results())
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(3):
        for L, s in zip(layers, streams):
            with torch.cuda.stream(s):
                L.forward()
                L.backward()
        torch.cuda.synchronize()
        for L, w in zip(layers, want):
            assert same(L.results(), w), i


def test_stream_argument():
    """A stream passed to a call is the one it runs on, its workspace too."""
    say("stream argument")
    L = Layer(64, seed=5)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    want = L.results()
    s = torch.cuda.Stream()
    for t in (L.d_logits, L.dx, L.dweight, L.counts, L.mean, L.grad, L.loss):
        t.fill_(1)
    torch.cuda.synchronize()
    moe.moe_balance_loss(L.logits, L.ids, 0.1, L.counts, L.mean, L.grad, L.loss, stream=s)
    moe.moe_router_backward(L.logits, L.ids, L.d_logits, d_topk_weights=L.dw, prob_grad=L.grad, stream=s)
    moe.moe_rmsnorm_backward(L.dy, L.h, L.weight, L.rstd, L.dx, L.dweight, stream=s)
    s.synchronize()
    assert same(L.results(), want)


def test_own_workspace_is_of_the_calls_stream(monkeypatch):
    """A workspace that a call allocates comes from the memory of the stream it
    runs on: a block of another stream's may still be in use there."""
    say("own workspace")
    L = Layer(64, seed=5)
    L.forward()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    seen = []
    alloc = moe._alloc
    monkeypatch.setattr(moe, "_alloc", lambda *a: seen.append(torch.cuda.current_stream()) or alloc(*a))
    moe.moe_balance_loss(L.logits, L.ids, 0.1, L.counts, L.mean, L.grad, L.loss, stream=s)
    moe.moe_rmsnorm_backward(L.dy, L.h, L.weight, L.rstd, L.dx, L.dweight, stream=s)
    moe.moe_rmsnorm_backward(L.dy, L.h, L.weight, L.rstd, L.dx, L.dweight)
    s.synchronize()
    torch.cuda.synchronize()
    assert seen == [s, s, torch.cuda.current_stream()]


def test_padded_tokens_do_not_reach_the_experts():
    """Masked tokens get no route: the forward leaves their rows zero."""
    say("padded tokens")
    L = Layer(50, seed=6)
    L.forward()
    mask = torch.ones(50, dtype=torch.uint8, device="cuda")
    mask[20:] = 0
    moe.moe_router_topk(L.logits, L.ids, L.w, token_mask=mask)
    out = torch.full_like(L.out, 9)
    moe.moe_forward(L.q, L.sf, L.ids, L.w, L.w1, L.w1_sf, L.one, L.w2, L.w2_sf, L.one, L.E, L.k, L.E, 0,
                    moe.MXFP8_MXFP4, out, L.H, L.I)
    torch.cuda.synchronize()
    assert bool((out[20:] == 0).all()) and bool((out[:20] != 0).any(-1).all())
