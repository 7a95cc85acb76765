"""Every value between the steps of a layer's run, forward and backward,
against fp64 from the step's own inputs."""
import pytest
import torch

import layer_ref as ref
from layer_ref import U8, U24
from test_gpu_layer import R_TOL, near, weight_tol
from test_gpu_layer_flow import Layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M", [1, 24, 300])
def test_values_between_the_steps(M):
    print(f"layer steps M={M}", flush=True)
    L = Layer(M)
    L.forward()
    L.backward()
    torch.cuda.synchronize()
    h, r64, y64 = ref.rmsnorm(L.x.cpu(), L.res.cpu(), L.weight.cpu(), 1e-6)
    assert torch.equal(L.h.cpu(), h)
    near(L.rstd, r64, r64 * R_TOL, "rstd")
    near(L.y, y64, y64.abs() * (U8 + R_TOL + 2 * U24) + 2.0 ** -133, "y")
    logits, ids = L.logits.cpu(), L.ids.cpu()
    ids64, w64 = ref.router_topk(logits, L.k, 0, True)
    assert torch.equal(ids, ids64)
    tol = weight_tol(logits, L.E)
    near(L.w, w64, w64 * tol + 1e-37, "weights")
    n64, m64, g64, l64 = ref.balance(logits, ids, L.k, 0, 0.1)
    assert torch.equal(L.counts.cpu().long(), n64)
    near(L.mean, m64, m64 * (tol.max().item() + 9 * U24) + 1e-37, "mean_probs")
    near(L.grad, g64, g64.abs() * 2 * U24 + 1e-37, "prob_grad")
    near(L.loss[0], l64, l64 * (tol.max().item() + 11 * U24), "loss")
    want, size = ref.router_backward(logits, ids, 0, True, L.dw.cpu(), L.grad.cpu())
    near(L.d_logits, want, want.abs() * U24 + size * 3 * tol + 1e-37, "d_logits")
    dx64, dw64, size = ref.rmsnorm_backward(L.dy.cpu(), h, L.weight.cpu(), L.rstd.cpu(), None)
    near(L.dx, dx64, dx64.abs() * U8 + size * (R_TOL + 8 * U24) + 2.0 ** -133, "dx")
    mag = (L.dy.cpu().double() * h.double() * L.rstd.cpu().double()[:, None]).abs().sum(0)
    near(L.dweight, dw64, mag * (3 + 2 + 10 + 8) * U24, "dweight")  # two rows a workgroup, at most 150 partial sums
