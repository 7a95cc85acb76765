"""Host-side checks of the operators on rows in 8 bits: every bad argument is
refused with its status before anything is enqueued (run without a GPU; the
placeholder pointers are never dereferenced, so each call that is good is one
with nothing to do)."""
import ctypes

import pytest
import torch  # noqa: F401  (before the library, which is loaded below: one HIP runtime for both)

import mixture_experts_forward_moe_amd as moe

OK, INVALID, UNSUPPORTED = 0, 1, 2
F = 0x10000
NAN, INF = float("nan"), float("inf")


def plan(M=64, k=8, El=32, tile=16):
    p = moe.Plan()
    n = moe.lib().moe_plan_workspace_size(M, k, El, tile)
    assert moe.lib().moe_plan_init(ctypes.byref(p), ctypes.c_void_p(F), n, M, k, El, tile) == OK
    return p


def broken(**change):
    p = plan()
    for name, value in change.items():
        setattr(p, name, value)
    return p


def status(name, defaults, change):
    a = dict(defaults)
    unknown = set(change) - set(a)
    assert not unknown, unknown
    a.update(change)
    return getattr(moe.lib(), name)(*(ctypes.byref(v) if isinstance(v, moe.Plan) else v for v in a.values()))


SLOTS = plan().route_slots
EMPTY = plan(M=0)
LOST = [broken(scratch=None), broken(route_slots=SLOTS + 16), broken(tile=24), broken(expert_counts=None),
        broken(expanded_to_permuted=None), None]


def cases(*what):
    return pytest.mark.parametrize("change,want", [(c, s) for c, s in what])


QUANTIZE = dict(x=F, stride=0, rows=4, cols=64, q=F, sf=F, stream=None)


@cases((dict(x=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(rows=-1), INVALID),
       (dict(cols=0), INVALID), (dict(cols=-16), INVALID), (dict(stride=48), INVALID), (dict(stride=-64), INVALID),
       (dict(cols=72), UNSUPPORTED), (dict(stride=68), UNSUPPORTED), (dict(x=F + 8), UNSUPPORTED),
       (dict(q=F + 8), UNSUPPORTED), (dict(rows=(1 << 25) + 1), UNSUPPORTED), (dict(rows=1 << 25, cols=2064), UNSUPPORTED),
       (dict(rows=1 << 62, cols=1 << 30), UNSUPPORTED), (dict(cols=(1 << 30) + 16), UNSUPPORTED), (dict(rows=0), OK),
       (dict(rows=0, x=None, q=None, sf=None), OK), (dict(rows=0, cols=72), UNSUPPORTED))
def test_quantize(change, want):
    assert status("moe_quantize_fp8", QUANTIZE, change) == want


WEIGHT = dict(w=F, batches=2, N=64, K=64, q=F, sf=F, qt=F, sft=F, stream=None)


@cases((dict(w=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(qt=None), INVALID),
       (dict(sft=None), INVALID), (dict(batches=-1), INVALID), (dict(N=-8), INVALID), (dict(K=0), INVALID),
       (dict(K=68), UNSUPPORTED), (dict(N=68), UNSUPPORTED), (dict(w=F + 8), UNSUPPORTED), (dict(q=F + 4), UNSUPPORTED),
       (dict(qt=F + 4), UNSUPPORTED), (dict(sf=F + 2), UNSUPPORTED), (dict(sft=F + 2), UNSUPPORTED),
       (dict(batches=1 << 24), UNSUPPORTED), (dict(N=1 << 24, K=1 << 24), UNSUPPORTED),
       (dict(N=2147483640, K=2147483640, batches=2147483647), UNSUPPORTED), (dict(batches=0), OK), (dict(N=0), OK),
       (dict(N=0, w=None, q=None, sf=None, qt=None, sft=None), OK))
def test_quantize_weight(change, want):
    assert status("moe_quantize_fp8_weight", WEIGHT, change) == want


DISPATCH = dict(x=F, stride=0, plan=plan(), H=64, rows=F, q=F, sf=F, stream=None)


@cases(*((dict(plan=p), INVALID) for p in LOST), (dict(x=None), INVALID), (dict(rows=None, q=None, sf=None), INVALID),
       (dict(q=None), INVALID), (dict(sf=None), INVALID), (dict(H=0), INVALID), (dict(stride=48), INVALID),
       (dict(stride=-64), INVALID), (dict(H=72), UNSUPPORTED), (dict(H=16400), UNSUPPORTED), (dict(stride=68), UNSUPPORTED),
       (dict(x=F + 8), UNSUPPORTED), (dict(rows=F + 8), UNSUPPORTED), (dict(q=F + 8), UNSUPPORTED),
       (dict(plan=plan(M=(1 << 22) + 1, k=1)), UNSUPPORTED), (dict(plan=EMPTY), OK),
       (dict(plan=EMPTY, x=None, rows=None, q=None, sf=None), OK), (dict(plan=EMPTY, q=None), INVALID))
def test_dispatch(change, want):
    assert status("moe_dispatch", DISPATCH, change) == want


BACK = dict(d=F, plan=plan(), H=64, accumulate=0, dx=F, stream=None)


@cases(*((dict(plan=p), INVALID) for p in LOST), (dict(d=None), INVALID), (dict(dx=None), INVALID), (dict(H=-16), INVALID),
       (dict(H=72), UNSUPPORTED), (dict(H=16400), UNSUPPORTED), (dict(d=F + 8), UNSUPPORTED), (dict(dx=F + 8), UNSUPPORTED),
       (dict(plan=plan(M=(1 << 22) + 1, k=1)), UNSUPPORTED), (dict(plan=EMPTY), OK), (dict(plan=EMPTY, d=None, dx=None), OK))
def test_dispatch_backward(change, want):
    assert status("moe_dispatch_backward", BACK, change) == want


FINALIZE = dict(dout=F, y2=F, plan=plan(), w=F, H=64, rsf=1.0, dy2=F, q=F, sf=F, dw=F, stream=None)


@cases(*((dict(plan=p), INVALID) for p in LOST), (dict(dout=None), INVALID), (dict(w=None), INVALID),
       (dict(y2=None), INVALID), (dict(dw=None), INVALID), (dict(q=None), INVALID), (dict(sf=None), INVALID),
       (dict(y2=None, dw=None, dy2=None, q=None, sf=None), INVALID), (dict(rsf=NAN), INVALID), (dict(rsf=INF), INVALID),
       (dict(H=0), INVALID), (dict(H=72), UNSUPPORTED), (dict(H=16400), UNSUPPORTED), (dict(dout=F + 8), UNSUPPORTED),
       (dict(y2=F + 8), UNSUPPORTED), (dict(dy2=F + 8), UNSUPPORTED), (dict(q=F + 8), UNSUPPORTED),
       (dict(w=F + 2), UNSUPPORTED), (dict(dw=F + 2), UNSUPPORTED), (dict(plan=plan(M=(1 << 22) + 1, k=1)), UNSUPPORTED),
       (dict(plan=EMPTY), OK), (dict(plan=EMPTY, dout=None, w=None, y2=None, dw=None), OK))
def test_finalize_backward(change, want):
    assert status("moe_finalize_backward", FINALIZE, change) == want


LINEAR = dict(x=F, x_sf=F, w=F, w_sf=F, bias=F, M=4, N=8, K=64, accumulate=0, y=F, dtype=0, stream=None)


@cases((dict(x=None), INVALID), (dict(x_sf=None), INVALID), (dict(w=None), INVALID), (dict(w_sf=None), INVALID),
       (dict(y=None), INVALID), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(K=0), INVALID), (dict(dtype=2), INVALID),
       (dict(dtype=-1), INVALID), (dict(K=72), UNSUPPORTED), (dict(K=(1 << 20) + 16), UNSUPPORTED),
       (dict(M=(1 << 26) + 1), UNSUPPORTED), (dict(N=(1 << 26) + 1), UNSUPPORTED), (dict(M=1 << 20, N=(1 << 16) + 1), UNSUPPORTED),
       (dict(x=F + 8), UNSUPPORTED), (dict(w=F + 8), UNSUPPORTED), (dict(y=F + 1), UNSUPPORTED),
       (dict(y=F + 2, dtype=1), UNSUPPORTED), (dict(w_sf=F + 2), UNSUPPORTED), (dict(bias=F + 2), UNSUPPORTED),
       (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=None, x_sf=None, w=None, w_sf=None, bias=None, y=None), OK))
def test_linear(change, want):
    assert status("moe_linear_fp8", LINEAR, change) == want


GROUPED = dict(x=F, x_sf=F, plan=plan(), w=F, w_sf=F, N=64, K=64, y=F, stream=None)


@cases(*((dict(plan=p), INVALID) for p in LOST), (dict(x=None), INVALID), (dict(x_sf=None), INVALID), (dict(w=None), INVALID),
       (dict(w_sf=None), INVALID), (dict(y=None), INVALID), (dict(N=-8), INVALID), (dict(K=0), INVALID),
       (dict(N=68), UNSUPPORTED), (dict(K=72), UNSUPPORTED), (dict(N=(1 << 16) + 8), UNSUPPORTED),
       (dict(K=(1 << 16) + 16), UNSUPPORTED), (dict(x=F + 8), UNSUPPORTED), (dict(w=F + 8), UNSUPPORTED),
       (dict(y=F + 8), UNSUPPORTED), (dict(w_sf=F + 2), UNSUPPORTED), (dict(plan=plan(M=1 << 23), N=64), UNSUPPORTED),
       # more threads than a launch has: 2^19 tiles and more of 16 rows
       (dict(plan=plan(M=1 << 20), N=256), UNSUPPORTED),
       (dict(plan=EMPTY), OK), (dict(N=0), OK), (dict(plan=EMPTY, x=None, x_sf=None, w=None, w_sf=None, y=None), OK))
def test_grouped_linear(change, want):
    assert status("moe_grouped_linear_fp8", GROUPED, change) == want


WGRAD = dict(dy=F, x=F, x_sf=F, M=4, N=64, K=64, accumulate=0, dw=F, stream=None)


@cases((dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(x_sf=None), INVALID), (dict(dw=None), INVALID),
       (dict(M=0, dw=None), INVALID), (dict(M=-1), INVALID), (dict(N=-8), INVALID), (dict(K=0), INVALID),
       (dict(N=68), UNSUPPORTED), (dict(K=72), UNSUPPORTED), (dict(N=(1 << 16) + 8), UNSUPPORTED),
       (dict(K=(1 << 16) + 16), UNSUPPORTED), (dict(M=(1 << 26) + 1), UNSUPPORTED), (dict(dy=F + 8), UNSUPPORTED),
       (dict(x=F + 8), UNSUPPORTED), (dict(dw=F + 8), UNSUPPORTED), (dict(N=0), OK),
       (dict(N=0, dy=None, x=None, x_sf=None, dw=None), OK))
def test_wgrad(change, want):
    assert status("moe_linear_fp8_wgrad", WGRAD, change) == want


GWGRAD = dict(dy=F, x=F, x_sf=F, plan=plan(), N=64, K=64, accumulate=0, dw=F, stream=None)


@cases(*((dict(plan=p), INVALID) for p in LOST), (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(x_sf=None), INVALID),
       (dict(dw=None), INVALID), (dict(plan=EMPTY, dw=None), INVALID), (dict(N=-8), INVALID), (dict(K=0), INVALID),
       (dict(N=68), UNSUPPORTED), (dict(K=72), UNSUPPORTED), (dict(N=(1 << 16) + 8), UNSUPPORTED),
       (dict(K=(1 << 16) + 16), UNSUPPORTED), (dict(dy=F + 8), UNSUPPORTED), (dict(x=F + 8), UNSUPPORTED),
       (dict(dw=F + 8), UNSUPPORTED), (dict(plan=plan(El=64), N=1 << 16, K=1 << 16), UNSUPPORTED), (dict(N=0), OK))
def test_grouped_wgrad(change, want):
    assert status("moe_grouped_linear_fp8_wgrad", GWGRAD, change) == want


ACT = dict(h=F, plan=None, rows=4, I=64, act=0, alpha=1.0, beta=0.0, limit=moe.FLT_MAX, y=F, y_sf=F, hq=F, hq_sf=F,
           stream=None)
ACT_BACK = dict(hq=F, hq_sf=F, dy=F, plan=None, rows=4, I=64, act=0, alpha=1.0, beta=0.0, limit=moe.FLT_MAX, dh=F, dq=F,
                dq_sf=F, stream=None)
SHAPE = [*((dict(plan=p, rows=SLOTS), INVALID) for p in LOST[:-1]), (dict(plan=plan(), rows=SLOTS - 16), INVALID),
         (dict(rows=-1), INVALID), (dict(I=0), INVALID), (dict(alpha=NAN), INVALID), (dict(beta=INF), INVALID),
         (dict(limit=NAN), INVALID), (dict(limit=-1.0), INVALID), (dict(act=3), INVALID), (dict(act=-1), INVALID),
         (dict(act=moe.ACT_RELU2), UNSUPPORTED), (dict(act=moe.ACT_GEGLU_TANH, alpha=2.0), INVALID), (dict(I=72), UNSUPPORTED),
         (dict(rows=(1 << 25) + 1), UNSUPPORTED), (dict(rows=1 << 25, I=1040), UNSUPPORTED), (dict(rows=0), OK),
         (dict(rows=0, act=moe.ACT_GEGLU_TANH), OK), (dict(plan=EMPTY, rows=EMPTY.route_slots), OK)]


@cases(*SHAPE, (dict(h=None), INVALID), (dict(y=None), INVALID), (dict(y_sf=None), INVALID), (dict(hq=None), INVALID),
       (dict(hq_sf=None), INVALID), (dict(h=F + 8), UNSUPPORTED), (dict(y=F + 8), UNSUPPORTED), (dict(hq=F + 8), UNSUPPORTED),
       (dict(rows=0, h=None, y=None, y_sf=None, hq=None, hq_sf=None), OK))
def test_act(change, want):
    assert status("moe_gated_act_fp8", ACT, change) == want


@cases(*SHAPE, (dict(hq=None), INVALID), (dict(hq_sf=None), INVALID), (dict(dy=None), INVALID),
       (dict(dh=None, dq=None, dq_sf=None), INVALID), (dict(dq=None), INVALID), (dict(dq_sf=None), INVALID),
       (dict(hq=F + 8), UNSUPPORTED), (dict(dy=F + 8), UNSUPPORTED), (dict(dh=F + 8), UNSUPPORTED), (dict(dq=F + 8), UNSUPPORTED),
       (dict(rows=0, hq=None, hq_sf=None, dy=None, dh=None, dq=None, dq_sf=None), OK))
def test_act_backward(change, want):
    assert status("moe_gated_act_fp8_backward", ACT_BACK, change) == want
