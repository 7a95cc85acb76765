"""Host-side checks of the operators around the routed experts: every bad
argument is refused with its status before anything is enqueued (run without
a GPU; the placeholder pointers are never dereferenced)."""
import ctypes

import pytest
import torch

import mixture_experts_forward_moe_amd as moe

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3
F = 0x10000
ODD = 0x10001
NAN = float("nan")


def call(name, defaults, **change):
    a = dict(defaults)
    unknown = set(change) - set(a)
    assert not unknown, unknown
    a.update(change)
    return getattr(moe.lib(), name)(*a.values())


NORM = dict(x=F, xs=0, residual=F, rs=0, weight=F, wd=0, eps=1e-6, M=4, H=64, h=F, y=F, elem=0, q=F, sf=F, rstd=F,
            stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(weight=None), INVALID), (dict(y=None, q=None, sf=None), INVALID),
    (dict(sf=None), INVALID), (dict(q=None), INVALID), (dict(residual=None), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=NAN), INVALID), (dict(eps=float("inf")), INVALID), (dict(M=-1), INVALID), (dict(H=0), INVALID),
    (dict(wd=2), INVALID), (dict(elem=2), INVALID), (dict(xs=56), INVALID), (dict(rs=56), INVALID),
    (dict(H=60), UNSUPPORTED), (dict(H=72), UNSUPPORTED), (dict(H=16416), UNSUPPORTED), (dict(xs=68), UNSUPPORTED),
    (dict(rs=68), UNSUPPORTED), (dict(x=ODD), UNSUPPORTED), (dict(residual=ODD), UNSUPPORTED),
    (dict(weight=ODD), UNSUPPORTED), (dict(h=ODD), UNSUPPORTED), (dict(y=ODD), UNSUPPORTED),
    (dict(q=ODD), UNSUPPORTED), (dict(rstd=ODD), UNSUPPORTED), (dict(M=0), OK), (dict(M=0, x=None), OK),
    # written rows over strided ones that other workgroups still read
    (dict(h=F, xs=128, x=F, residual=2 * F, y=None), INVALID), (dict(y=F, x=F, xs=128, h=None), INVALID),
    (dict(h=F, residual=F, rs=128, x=2 * F, y=None), INVALID),
])
def test_norm(change, status):
    assert call("moe_rmsnorm", NORM, **change) == status


BACK = dict(dy=F, h=F, weight=F, wd=1, rstd=F, dh=None, M=4, H=64, dx=F, dweight=F, ws=F, n=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dy=None), INVALID), (dict(h=None), INVALID), (dict(weight=None), INVALID), (dict(rstd=None), INVALID),
    (dict(dx=None), INVALID), (dict(M=-1), INVALID), (dict(H=-8), INVALID), (dict(wd=-1), INVALID),
    (dict(H=60), UNSUPPORTED), (dict(dh=ODD), UNSUPPORTED), (dict(dx=ODD), UNSUPPORTED),
    (dict(dweight=ODD), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=F + 16), WORKSPACE), (dict(n=511), WORKSPACE),
    (dict(M=0, dweight=None, ws=None, n=0), OK),
])
def test_norm_backward(change, status):
    assert call("moe_rmsnorm_backward", BACK, **change) == status


def test_norm_backward_workspace():
    assert moe.rmsnorm_backward_workspace_size(4, 64) == 512
    assert moe.rmsnorm_backward_workspace_size(4, 60) == 0
    assert moe.rmsnorm_backward_workspace_size(-1, 64) == 0
    n = moe.rmsnorm_backward_workspace_size(4096, 6144)
    assert n and call("moe_rmsnorm_backward", BACK, M=4096, H=6144, n=n - 1) == WORKSPACE


TOPK = dict(logits=F, d=1, stride=0, bias=None, mask=None, score=0, renorm=1, M=4, E=16, k=2, ids=F, w=F, coef=0.0,
            counts=None, probs=None, grad=None, loss=None, ws=None, n=0, stream=None)
ALL = dict(counts=F, probs=F, grad=F, loss=F, ws=F, n=1 << 20)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(w=None), INVALID), (dict(d=2), INVALID),
    (dict(score=2), INVALID), (dict(M=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=17), INVALID),
    (dict(stride=15), INVALID), (dict(counts=F), INVALID), (dict(ALL, loss=None), INVALID),
    (dict(ALL, coef=NAN), INVALID), (dict(E=1025), UNSUPPORTED), (dict(E=128, k=65), UNSUPPORTED),
    (dict(M=1 << 30), UNSUPPORTED), (dict(logits=ODD), UNSUPPORTED), (dict(logits=F + 2), UNSUPPORTED),
    (dict(d=0, logits=ODD), UNSUPPORTED), (dict(ids=F + 2), UNSUPPORTED), (dict(w=F + 2), UNSUPPORTED),
    (dict(bias=F + 2), UNSUPPORTED), (dict(ALL, ws=None), WORKSPACE), (dict(ALL, ws=F + 64), WORKSPACE),
    (dict(ALL, counts=F + 2), UNSUPPORTED), (dict(ALL, probs=F + 2), UNSUPPORTED), (dict(ALL, grad=ODD), UNSUPPORTED),
    (dict(ALL, loss=ODD), UNSUPPORTED), (dict(ALL, n=256), WORKSPACE), (dict(M=0), OK), (dict(M=0, logits=None, ids=None, w=None), OK),
])
def test_router_topk(change, status):
    assert call("moe_router_topk", TOPK, **change) == status


LOSS = dict(logits=F, d=1, stride=0, ids=F, mask=None, score=0, M=4, E=16, k=2, coef=1.0, counts=F, probs=F, grad=F,
            loss=F, ws=F, n=1 << 20, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(logits=None), INVALID), (dict(ids=None), INVALID), (dict(counts=None), INVALID), (dict(probs=None), INVALID),
    (dict(grad=None), INVALID), (dict(loss=None), INVALID), (dict(coef=float("inf")), INVALID), (dict(k=17), INVALID),
    (dict(E=1025), UNSUPPORTED), (dict(ids=ODD), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(n=511), WORKSPACE),
    (dict(counts=F + 2), UNSUPPORTED), (dict(loss=ODD), UNSUPPORTED),
])
def test_balance_loss(change, status):
    assert call("moe_balance_loss", LOSS, **change) == status


def test_balance_workspace():
    for M, E in [(0, 1), (1, 1), (17, 60), (65536, 256), (1 << 24, 1024)]:
        n = moe.balance_workspace_size(M, E)
        assert n and n % 256 == 0
        assert call("moe_balance_loss", LOSS, M=M, E=E, k=1, n=n - 1) == WORKSPACE
    assert moe.balance_workspace_size(-1, 8) == 0 and moe.balance_workspace_size(4, 0) == 0
    assert moe.balance_workspace_size(4, 1025) == 0


ROUTER_BACK = dict(logits=F, d=1, stride=0, ids=F, mask=None, score=0, renorm=1, M=4, E=16, k=2, dw=F, grad=F,
                   d_loss=None, out=F, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(dw=None, grad=None), INVALID), (dict(grad=None, d_loss=F), INVALID), (dict(out=None), INVALID),
    (dict(ids=None), INVALID), (dict(logits=None), INVALID), (dict(stride=8), INVALID), (dict(E=2000), UNSUPPORTED),
    (dict(out=F + 2), UNSUPPORTED), (dict(dw=F + 2), UNSUPPORTED), (dict(grad=F + 2), UNSUPPORTED), (dict(M=0), OK),
])
def test_router_backward(change, status):
    assert call("moe_router_backward", ROUTER_BACK, **change) == status


LINEAR = dict(x=F, x_sf=F, elem=0, w=F, w_sf=F, alpha=None, bias=None, M=4, N=16, K=64, acc=0, y=F, d=0, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), INVALID), (dict(x_sf=None), INVALID), (dict(w=None), INVALID), (dict(w_sf=None), INVALID),
    (dict(y=None), INVALID), (dict(elem=2), INVALID), (dict(K=48), INVALID), (dict(K=0), INVALID), (dict(M=-1), INVALID),
    (dict(N=-1), INVALID), (dict(d=2), INVALID), (dict(x=F + 8), UNSUPPORTED), (dict(w=F + 8), UNSUPPORTED),
    (dict(y=ODD), UNSUPPORTED), (dict(d=1, y=F + 2), UNSUPPORTED), (dict(alpha=F + 2), UNSUPPORTED),
    (dict(bias=F + 2), UNSUPPORTED), (dict(K=(1 << 20) + 32), UNSUPPORTED), (dict(M=1 << 26, N=2048), UNSUPPORTED), (dict(N=(1 << 26) + 1), UNSUPPORTED),
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=None, y=None), OK),
])
def test_linear(change, status):
    assert call("moe_linear_mx", LINEAR, **change) == status


def test_binding_refuses_what_does_not_fit():
    """Shapes, element sizes, layouts and devices, before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64)
    with pytest.raises(moe.MoeError, match="on the GPU"):
        moe.moe_rmsnorm(x, w, y=torch.empty_like(x))
    with pytest.raises(moe.MoeError, match="x must be"):
        moe.moe_rmsnorm(x.float(), w, y=x)
    with pytest.raises(moe.MoeError, match="weight must be bf16 or fp32"):
        moe.moe_rmsnorm(x, w.double(), y=x)
    with pytest.raises(moe.MoeError, match="in a row"):
        moe.moe_rmsnorm(torch.zeros(64, 4, dtype=torch.bfloat16).t(), w, y=x)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises(moe.MoeError, match="topk_weights|on the GPU"):
        moe.moe_router_topk(torch.zeros(4, 16), ids, torch.zeros(4, 3))
    with pytest.raises(moe.MoeError, match="type of logits"):
        moe.moe_router_backward(torch.zeros(4, 16), ids, x, prob_grad=w)


def test_binding_refuses_other_element_types():
    """Types of the right size but another meaning."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64)
    f = torch.zeros(4, 16)
    ids = torch.zeros(4, 2, dtype=torch.int32)
    for call_, what in [
        (lambda: moe.moe_rmsnorm(x.half(), w, y=x), "x must be bf16"),
        (lambda: moe.moe_rmsnorm(x, w, y=x.half()), "weight|y must be bf16|on the GPU"),
        (lambda: moe.moe_rmsnorm_backward(x.half(), x, w, w[:4], x), "dy must be bf16"),
        (lambda: moe.moe_linear_mx(x.to(torch.float8_e5m2), w, w, w, x), "x must be bytes|w"),
    ]:
        with pytest.raises(moe.MoeError, match=what):
            call_()
    with pytest.raises(moe.MoeError):
        moe.moe_router_topk(f.half(), ids, f[:, :2])
    # (past the device check the rest is the same function: by itself)
    for t, kind in [(ids, moe._F32), (f, moe._I32), (x.half(), moe._BF16), (f.to(torch.float8_e5m2), moe._BYTE),
                    (f.to(torch.float8_e4m3fnuz), moe._BYTE), (ids.to(torch.int64), moe._I32)]:
        for check in (moe._arg, moe._opt, moe._rows):
            with pytest.raises(moe.MoeError, match=f"must be {kind.name}"):
                check("call", "t", t, tuple(t.shape), kind, 0)


def test_binding_refuses_another_device_than_the_current_one(monkeypatch):
    class OnOne:
        _cuda_getDevice = staticmethod(lambda: 1)
        _cuda_getCurrentRawStream = staticmethod(lambda dev: 7)
    monkeypatch.setattr(moe, "_cuda", OnOne)
    assert moe._raw_stream("call", 1, None) == 7
    with pytest.raises(moe.MoeError, match="not the current device"):
        moe._raw_stream("call", 0, None)


def test_binding_refuses_rows_that_are_not_apart():
    """An expanded row has stride 0, which the library takes for contiguous."""
    row = torch.zeros(1, 64, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError, match="rows apart"):
        moe._rows("call", "x", row.expand(4, 64), (4, 64), moe._BF16, -1)
    over = torch.zeros(4 * 32 + 32).as_strided((4, 64), (32, 1))
    with pytest.raises(moe.MoeError, match="rows apart"):
        moe._rows("call", "x", over, (4, 64), moe._F32, -1)


def test_constants_match_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "moe.h")).read()
    enums = {k: int(v) for k, v in re.findall(r"\b(MOE_[A-Z0-9_]+)\s*=\s*(\d+)", text)}
    assert (enums["MOE_DTYPE_BF16"], enums["MOE_DTYPE_F32"]) == (moe.DTYPE_BF16, moe.DTYPE_F32)
    assert (enums["MOE_SCORE_SOFTMAX"], enums["MOE_SCORE_SIGMOID"]) == (moe.SCORE_SOFTMAX, moe.SCORE_SIGMOID)
