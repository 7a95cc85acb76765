"""What the binding of the operators on rows in 8 bits refuses: each bad
argument among good ones, with an error that names it (no GPU: the last check,
the device, is what good arguments fail here)."""

import pytest
import torch

import mixture_experts_forward_moe_amd as moe

BF16, BYTE, F32 = torch.bfloat16, torch.uint8, torch.float32
M, K_TOP, E, TILE = 12, 2, 4, 16


def plan(device="cpu"):
    p = moe.MoePlan.__new__(moe.MoePlan)
    p.c = moe.Plan()
    p.M, p.top_k, p.num_local_experts, p.tile = M, K_TOP, E, TILE
    p.route_slots, p.max_tiles = 80, 5
    p.workspace = torch.zeros(256, dtype=BYTE)
    return p


def t(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype)


def b(*shape):
    return t(*shape, dtype=BYTE)


def f(*shape):
    return t(*shape, dtype=F32)


S = 80


def good():
    """Arguments of each call that fit together, but for the device."""
    return {
        "moe_quantize_fp8": dict(x=t(4, 192), q=b(4, 192), q_sf=b(4, 2)),
        "moe_quantize_fp8_weight": dict(weight=t(3, 160, 192), q=b(3, 160, 192), sf=f(3, 2, 2), qt=b(3, 192, 160),
                                        sft=f(3, 2, 2)),
        "moe_dispatch": dict(x=t(M, 192), plan=plan(), rows=t(S, 192), q=b(S, 192), q_sf=b(S, 2)),
        "moe_dispatch_backward": dict(d_rows=t(S, 192), plan=plan(), dx=t(M, 192)),
        "moe_finalize_backward": dict(dout=t(M, 192), y2=t(S, 192), plan=plan(), topk_weights=f(M, K_TOP), dy2=t(S, 192),
                                      q=b(S, 192), q_sf=b(S, 2), d_topk_weights=f(M, K_TOP)),
        "moe_linear_fp8": dict(x=b(4, 192), x_sf=b(4, 2), w=b(160, 192), w_sf=f(2, 2), y=t(4, 160), bias=f(160)),
        "moe_grouped_linear_fp8": dict(x=b(S, 192), x_sf=b(S, 2), plan=plan(), w=b(E, 160, 192), w_sf=f(E, 2, 2),
                                       y=t(S, 160)),
        "moe_linear_fp8_wgrad": dict(dy=t(4, 160), x=b(4, 192), x_sf=b(4, 2), dw=f(160, 192)),
        "moe_grouped_linear_fp8_wgrad": dict(dy=t(S, 160), x=b(S, 192), x_sf=b(S, 2), plan=plan(), dw=f(E, 160, 192)),
        "moe_gated_act_fp8": dict(h=t(S, 320), y=b(S, 160), y_sf=b(S, 2), hq=b(S, 320), hq_sf=b(S, 4), plan=plan()),
        "moe_gated_act_fp8_backward": dict(hq=b(S, 320), hq_sf=b(S, 4), dy=t(S, 160), dh=t(S, 320), dq=b(S, 320),
                                           dq_sf=b(S, 4), plan=plan()),
    }


OPTIONAL = {("moe_quantize_fp8_weight", "qt"), ("moe_quantize_fp8_weight", "sft"), ("moe_dispatch", "rows"),
            ("moe_dispatch", "q"), ("moe_dispatch", "q_sf"), ("moe_finalize_backward", "y2"),
            ("moe_finalize_backward", "dy2"), ("moe_finalize_backward", "q"), ("moe_finalize_backward", "q_sf"),
            ("moe_finalize_backward", "d_topk_weights"), ("moe_linear_fp8", "bias"), ("moe_gated_act_fp8", "hq"),
            ("moe_gated_act_fp8", "hq_sf"), ("moe_gated_act_fp8_backward", "dh"), ("moe_gated_act_fp8_backward", "dq"),
            ("moe_gated_act_fp8_backward", "dq_sf")}
# the tensors a call takes its sizes from: of another size, another argument does not fit
SIZES = {("moe_quantize_fp8", "x"), ("moe_quantize_fp8_weight", "weight"), ("moe_dispatch", "x"),
         ("moe_dispatch_backward", "d_rows"), ("moe_finalize_backward", "dout"), ("moe_linear_fp8", "x"),
         ("moe_linear_fp8", "w"), ("moe_grouped_linear_fp8", "x"), ("moe_grouped_linear_fp8", "y"),
         ("moe_linear_fp8_wgrad", "dy"), ("moe_linear_fp8_wgrad", "x"), ("moe_grouped_linear_fp8_wgrad", "dy"),
         ("moe_grouped_linear_fp8_wgrad", "x"), ("moe_gated_act_fp8", "y"), ("moe_gated_act_fp8_backward", "dy")}
# and the one that says which device the call is on
FIRST = {call: name for call, name in SIZES if (call, name) not in {
    ("moe_linear_fp8", "w"), ("moe_grouped_linear_fp8", "y"), ("moe_linear_fp8_wgrad", "x"),
    ("moe_grouped_linear_fp8_wgrad", "x")}}
TENSORS = [(call, name) for call, args in good().items() for name, v in args.items() if isinstance(v, torch.Tensor)]
PLANNED = [call for call, args in good().items() if "plan" in args]


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on device 0: what the checks see."""

    def get_device(self):
        return 0


@pytest.fixture
def calls(monkeypatch):
    """The binding over CPU tensors as if they were on the GPU; what reaches the library."""
    moe._kinds()
    made = []

    class Cuda:
        _cuda_getDevice = staticmethod(lambda: 0)
        _cuda_getCurrentRawStream = staticmethod(lambda dev: 77)

    class Library:
        """Stands in for the library: every call succeeds."""

        def __getattr__(self, name):
            if name == "moe_status_string":
                return lambda s: b""
            return lambda *args: made.append((name, args)) or 0
    library = Library()
    monkeypatch.setattr(moe, "_cuda", Cuda)
    monkeypatch.setattr(moe, "lib", lambda: library)
    return made


def on_gpu(args):
    out = {}
    for k, v in args.items():
        if isinstance(v, torch.Tensor):
            v = v.as_subclass(OnGpu)
        if isinstance(v, moe.MoePlan):
            v.workspace = v.workspace.as_subclass(OnGpu)
        out[k] = v
    return out


@pytest.mark.parametrize("call", list(good()))
def test_good_arguments_pass(calls, call):
    """Each argument in the place that the C function has it: as many as its prototype, and the current stream last."""
    args = on_gpu(good()[call])
    getattr(moe, call)(**args)
    (name, made), = calls
    assert name == call and made[-1] == 77
    pointers = {v.data_ptr() for v in args.values() if isinstance(v, torch.Tensor)}
    assert pointers <= {a for a in made if isinstance(a, int)}


@pytest.mark.parametrize("call", list(good()))
def test_as_many_arguments_as_the_prototype(calls, call, monkeypatch):
    args = on_gpu(good()[call])
    getattr(moe, call)(**args)
    monkeypatch.undo()
    assert len(calls[0][1]) == len(getattr(moe.lib(), call).argtypes)


@pytest.mark.parametrize("call", list(good()))
def test_a_stream_of_the_callers(calls, call):
    class Stream:
        cuda_stream = 4711
        device_index = 0
        device = torch.device("cuda", 0)
    getattr(moe, call)(**on_gpu(good()[call]), stream=Stream())
    assert calls[0][1][-1] == 4711


@pytest.mark.parametrize("call,name", [c for c in TENSORS if c not in OPTIONAL])
def test_required(calls, call, name):
    args = on_gpu(good()[call])
    args[name] = None
    with pytest.raises(moe.MoeError, match=rf"{call}: {name} (is required|must)"):
        getattr(moe, call)(**args)


@pytest.mark.parametrize("call,name", sorted(OPTIONAL))
def test_optional(calls, call, name):
    """What may be left out reaches the library as NULL, which checks what belongs together."""
    args = on_gpu(good()[call])
    args[name] = None
    getattr(moe, call)(**args)
    assert None in calls[0][1]


@pytest.mark.parametrize("call,name", sorted(SIZES))
def test_dimensions(calls, call, name):
    for change in (lambda v: v[None, None], lambda v: v.flatten()):
        args = on_gpu(good()[call])
        args[name] = change(args[name])
        with pytest.raises(moe.MoeError, match=rf"{call}: {name} must have two (or three )?dimensions"):
            getattr(moe, call)(**args)


@pytest.mark.parametrize("call,name", TENSORS)
def test_other_element_types(calls, call, name):
    """Types of the right size but another meaning, and of another size."""
    v = good()[call][name]
    others = {BF16: [torch.float16, torch.int32, torch.float64], F32: [torch.int32, torch.float64, torch.float16],
              BYTE: [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int16]}[v.dtype]
    for dtype in others:
        args = on_gpu(good()[call])
        args[name] = v.to(dtype).as_subclass(OnGpu)
        with pytest.raises(moe.MoeError, match=rf"{call}: {name} must (be (bf16|fp32|int32|bytes)|have the type of)"):
            getattr(moe, call)(**args)


@pytest.mark.parametrize("call,name", TENSORS)
def test_other_shapes_layouts_and_devices(calls, call, name):
    v = good()[call][name]
    bad = {"shape": torch.zeros(*(n + 16 for n in v.shape), dtype=v.dtype).as_subclass(OnGpu), "device": v}
    if v.dim() >= 2:
        bad["layout"] = torch.zeros(*v.shape[:-2], v.shape[-1], v.shape[-2], dtype=v.dtype).transpose(-1, -2).as_subclass(OnGpu)
    else:
        bad["layout"] = torch.zeros(2 * v.numel(), dtype=v.dtype)[::2].as_subclass(OnGpu)
    for what, value in bad.items():
        args = on_gpu(good()[call])
        args[name] = value
        who = name
        if what == "shape" and (call, name) in SIZES or what == "device" and FIRST[call] == name:
            who = r"\w+"
        with pytest.raises(moe.MoeError, match=rf"{call}: {who} must be"):
            getattr(moe, call)(**args)
    assert not calls


@pytest.mark.parametrize("call", PLANNED)
def test_plans(calls, call):
    for value in (object(), moe.Plan(), plan()):  # (the last one on the CPU)
        args = on_gpu(good()[call])
        args["plan"] = value
        with pytest.raises(moe.MoeError, match=rf"{call}: plan must be"):
            getattr(moe, call)(**args)
    if "act" not in call:
        args = on_gpu(good()[call])
        args["plan"] = None
        with pytest.raises(moe.MoeError, match=rf"{call}: plan must be a MoePlan"):
            getattr(moe, call)(**args)
    assert not calls


@pytest.mark.parametrize("call", PLANNED)
def test_rows_that_are_not_the_plans(calls, call):
    """A plan of other sizes than the tensors'."""
    args = on_gpu(good()[call])
    args["plan"].route_slots += 16
    with pytest.raises(moe.MoeError, match=rf"{call}: \w+ must be"):
        getattr(moe, call)(**args)
    assert not calls
