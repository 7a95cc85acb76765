"""Calls of several host threads at once, each on a stream of its own."""
import threading

import pytest
import torch

import mixture_experts_forward_moe_amd as moe

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def say(*a):
    print(*a, flush=True)


class Work:
    """Calls of every operator around the routed experts, of other sizes for
    each seed."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        e = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        M, H, E, k = 200 + 64 * seed, 512, 40 + 50 * seed, 6
        self.x, self.w = rnd(M, H).to(BF16), rnd(H)
        self.y, self.q, self.sf = e(M, H, dtype=BF16), e(M, H, dtype=torch.uint8), e(M, H // 32, dtype=torch.uint8)
        self.rstd, self.dx, self.dw = e(M), e(M, H, dtype=BF16), e(H)
        self.logits, self.ids, self.wt = rnd(M, E), e(M, k, dtype=torch.int32), e(M, k)
        self.stats = dict(expert_counts=e(E, dtype=torch.int32), mean_probs=e(E), prob_grad=e(E), loss=e(1))
        self.d = e(M, E)
        self.linears = []
        for m, n, kk, elem in ((M, 264, H, 0), (1200, 2048, 1024, seed % 2), (4096, 4096, 1024, seed % 2)):
            byte = lambda *s, hi=126: torch.randint(0, hi, s, generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
            one = lambda r: torch.full((r, kk // 32), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
            self.linears.append((byte(m, kk if elem == 0 else kk // 2), one(m), byte(n, kk // 2, hi=256), one(n),
                                 e(m, n, dtype=BF16), elem))
        self.stream = torch.cuda.Stream()

    def run(self, stream=None):
        moe.moe_rmsnorm(self.x, self.w, y=self.y, q=self.q, q_sf=self.sf, rstd=self.rstd, stream=stream)
        moe.moe_rmsnorm_backward(self.y, self.x, self.w, self.rstd, self.dx, self.dw, stream=stream)
        moe.moe_router_topk(self.logits, self.ids, self.wt, coef=0.1, stream=stream, **self.stats)
        moe.moe_router_backward(self.logits, self.ids, self.d, d_topk_weights=self.wt,
                                prob_grad=self.stats["prob_grad"], stream=stream)
        for *args, elem in self.linears:
            moe.moe_linear_mx(*args, x_elem=elem, stream=stream)

    def outputs(self):
        return [self.y, self.q, self.sf, self.rstd, self.dx, self.dw, self.ids, self.wt, self.d, *self.stats.values(),
                *(v[4] for v in self.linears)]


def test_threads_at_once():
    say("threads")
    works = [Work(s) for s in range(6)]
    torch.cuda.synchronize()
    gate, errors = threading.Barrier(len(works)), []

    def body(w):
        try:
            gate.wait()
            for _ in range(5):
                w.run(w.stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=body, args=(w,)) for w in works]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors
    for i, w in enumerate(works):
        got = [t.clone() for t in w.outputs()]
        w.run()
        torch.cuda.synchronize()
        for n, (a, b) in enumerate(zip(got, w.outputs())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), (i, n)
