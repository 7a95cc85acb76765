"""The fp64 gradient formulas the GPU tests compare with, against central
differences of the fp64 forward forms."""
import pytest
import torch

import layer_ref as ref

F64 = torch.float64
STEP = 1e-6
# central differences: STEP^2 times a third derivative of order 10 plus
# 2^-53 / STEP of rounding, each below 1e-9 of the values' size here
TOL = 1e-7


def gen(seed):
    return torch.Generator().manual_seed(seed)


def test_norm_gradient():
    g = gen(1)
    M, H, eps = 3, 16, 1e-3
    h = torch.randn(M, H, generator=g, dtype=F64)
    w = torch.randn(H, generator=g, dtype=F64)
    dy = torch.randn(M, H, generator=g, dtype=F64)

    def f(h, w):
        return (h / torch.sqrt((h * h).mean(-1, keepdim=True) + eps) * w * dy).sum()

    r = 1 / torch.sqrt((h * h).mean(-1) + eps)
    dx, dw, _ = ref.rmsnorm_backward(dy, h, w, r, None)
    for i in range(M):
        for j in range(H):
            e = torch.zeros(M, H, dtype=F64)
            e[i, j] = STEP
            assert abs((f(h + e, w) - f(h - e, w)) / (2 * STEP) - dx[i, j]) < TOL
    for j in range(H):
        e = torch.zeros(H, dtype=F64)
        e[j] = STEP
        assert abs((f(h, w + e) - f(h, w - e)) / (2 * STEP) - dw[j]) < TOL


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_router_gradient(sigmoid, renormalize):
    """The choice is held fixed: ids are whole numbers."""
    g = gen(2)
    M, E, k, coef = 5, 9, 3, 0.7
    l = torch.randn(M, E, generator=g, dtype=F64)
    mask = torch.tensor([1, 1, 0, 1, 1], dtype=torch.uint8)
    ids, _ = ref.router_topk(l, k, sigmoid, renormalize, mask=mask)
    dw = torch.randn(M, k, generator=g, dtype=F64)
    dloss = 1.3

    def f(l):
        w = ref.chosen_weights(l, ids, sigmoid, renormalize)
        return (w * dw).sum() + dloss * ref.balance(l, ids, k, sigmoid, coef, mask)[3]

    grad = ref.balance(l, ids, k, sigmoid, coef, mask)[2]
    d, _ = ref.router_backward(l, ids, sigmoid, renormalize, dw, grad, dloss, mask)
    for i in range(M):
        for j in range(E):
            e = torch.zeros(M, E, dtype=F64)
            e[i, j] = STEP
            assert abs((f(l + e) - f(l - e)) / (2 * STEP) - d[i, j]) < TOL, (i, j)


def test_choice_by_hand():
    nan, inf = float("nan"), float("inf")
    l = torch.tensor([[1.0, 3.0, 3.0, 2.0], [-inf, nan, 0.0, -inf], [inf, 0.0, inf, 1.0], [nan, nan, -inf, -inf]])
    ids, w = ref.router_topk(l, 2, False, True)
    assert ids.tolist() == [[1, 2], [2, -1], [0, 2], [-1, -1]]
    assert w.tolist() == [[0.5, 0.5], [1.0, 0.0], [0.5, 0.5], [0.0, 0.0]]


def test_uniform_routing_costs_coef():
    l = torch.zeros(8, 4)
    ids = torch.arange(16).reshape(8, 2) % 4
    counts, mean, grad, loss = ref.balance(l, ids, 2, False, 0.25)
    assert counts.tolist() == [4, 4, 4, 4] and loss.item() == 0.25 and grad.abs().max() == 0
