"""What the binding of the operators around the routed experts refuses: each
bad argument among good ones, with an error that names it (no GPU: the last
check, the device, is what good arguments fail here)."""
import pytest
import torch

import mixture_experts_forward_moe_amd as moe

BF16 = torch.bfloat16


def rows(m, n, dtype=torch.float32):
    return torch.zeros(m, n, dtype=dtype)


def good():
    """Arguments of each call that fit together, but for the device."""
    byte, bf, i32 = torch.uint8, BF16, torch.int32
    stats = dict(expert_counts=torch.zeros(16, dtype=i32), mean_probs=torch.zeros(16), prob_grad=torch.zeros(16),
                 loss=torch.zeros(1))
    return {
        "moe_rmsnorm": dict(x=rows(4, 64, bf), weight=torch.zeros(64), y=rows(4, 64, bf), residual=rows(4, 64, bf),
                            residual_out=rows(4, 64, bf), q=rows(4, 64, byte), q_sf=rows(4, 2, byte),
                            rstd=torch.zeros(4)),
        "moe_rmsnorm_backward": dict(dy=rows(4, 64, bf), h=rows(4, 64, bf), weight=torch.zeros(64),
                                     rstd=torch.zeros(4), dx=rows(4, 64, bf), dweight=torch.zeros(64),
                                     dh=rows(4, 64, bf)),
        "moe_router_topk": dict(logits=rows(4, 16), topk_ids=rows(4, 2, i32), topk_weights=rows(4, 2),
                                select_bias=torch.zeros(16), token_mask=torch.zeros(4, dtype=byte), **stats),
        "moe_balance_loss": dict(logits=rows(4, 16), topk_ids=rows(4, 2, i32), coef=1.0, token_mask=torch.zeros(4, dtype=byte),
                                 **stats),
        "moe_router_backward": dict(logits=rows(4, 16), topk_ids=rows(4, 2, i32), d_logits=rows(4, 16),
                                    d_topk_weights=rows(4, 2), prob_grad=torch.zeros(16), d_loss=torch.zeros(1),
                                    token_mask=torch.zeros(4, dtype=byte)),
        "moe_linear_mx": dict(x=rows(4, 64, byte), x_sf=rows(4, 2, byte), w=rows(8, 32, byte), w_sf=rows(8, 2, byte),
                              y=rows(4, 8, bf), alpha=torch.zeros(1), bias=torch.zeros(8)),
    }


REQUIRED = [("moe_rmsnorm", "x"), ("moe_rmsnorm", "weight"), ("moe_rmsnorm_backward", "dy"),
            ("moe_rmsnorm_backward", "weight"), ("moe_router_topk", "logits"), ("moe_router_topk", "topk_ids"),
            ("moe_balance_loss", "logits"), ("moe_balance_loss", "topk_ids"), ("moe_router_backward", "logits"),
            ("moe_router_backward", "topk_ids"), ("moe_router_backward", "d_logits"), ("moe_linear_mx", "x"),
            ("moe_linear_mx", "w"), ("moe_linear_mx", "y")]


@pytest.mark.parametrize("call,name", REQUIRED)
def test_required(call, name):
    args = good()[call]
    args[name] = None
    with pytest.raises(moe.MoeError, match=f"{call}: {name} is required"):
        getattr(moe, call)(**args)


@pytest.mark.parametrize("call,name", [c for c in REQUIRED if c[1] not in ("weight", "y", "d_logits")])
def test_two_dimensions(call, name):
    for change in (lambda t: t[None], lambda t: t[0]):
        args = good()[call]
        args[name] = change(args[name])
        with pytest.raises(moe.MoeError, match=f"{call}: {name} must have two dimensions"):
            getattr(moe, call)(**args)


class OnGpu(torch.Tensor):
    """A CPU tensor that says it is on device 0: what the checks see."""

    def get_device(self):
        return 0


class Library:
    """Stands in for the library: every call succeeds."""

    def __getattr__(self, name):
        return lambda *args: b"" if name == "moe_status_string" else 0


@pytest.fixture
def pretend(monkeypatch):
    """The binding over CPU tensors as if they were on the GPU."""
    moe._kinds()
    # (the binding keeps these: the real ones, before the library is away)
    assert moe.balance_workspace_size(4, 16) and moe.rmsnorm_backward_workspace_size(4, 64)

    class Cuda:
        _cuda_getDevice = staticmethod(lambda: 0)
        _cuda_getCurrentRawStream = staticmethod(lambda dev: 0)
    library = Library()
    monkeypatch.setattr(moe, "_cuda", Cuda)
    monkeypatch.setattr(moe, "lib", lambda: library)
    monkeypatch.setattr(moe, "_alloc", lambda n, device: torch.zeros(n, dtype=torch.uint8))
    yield
    moe.balance_workspace_size.cache_clear()
    moe.rmsnorm_backward_workspace_size.cache_clear()


def on_gpu(args):
    return {k: v.as_subclass(OnGpu) if isinstance(v, torch.Tensor) else v for k, v in args.items()}


TENSORS = [(call, name) for call, args in good().items() for name, v in args.items() if isinstance(v, torch.Tensor)]


@pytest.mark.parametrize("call", list(good()))
def test_good_arguments_pass(pretend, call):
    getattr(moe, call)(**on_gpu(good()[call]))


@pytest.mark.parametrize("call,name", TENSORS)
def test_other_element_types(pretend, call, name):
    """Types of the right size but another meaning, and of another size."""
    t = good()[call][name]
    others = {torch.bfloat16: [torch.float16, torch.int32, torch.float64], torch.float32: [torch.int32, torch.float64, torch.float16],
              torch.int32: [torch.float32, torch.int64, torch.int16],
              torch.uint8: [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.int16]}[t.dtype]
    for dtype in others:
        args = on_gpu(good()[call])
        args[name] = t.to(dtype).as_subclass(OnGpu)
        with pytest.raises(moe.MoeError, match=rf"{call}: {name} must (be (bf16|fp32|int32|bytes)|have the type of)"):
            getattr(moe, call)(**args)


@pytest.mark.parametrize("call,name", TENSORS)
def test_other_shapes_layouts_and_devices(pretend, call, name):
    t = good()[call][name]
    sizes = {("moe_rmsnorm", "x"), ("moe_rmsnorm_backward", "dy"), ("moe_linear_mx", "x"), ("moe_linear_mx", "w")}
    bad = {"shape": torch.zeros(*(n + 1 for n in t.shape), dtype=t.dtype).as_subclass(OnGpu), "device": t}
    if t.dim() == 2:
        bad["layout"] = torch.zeros(*reversed(t.shape), dtype=t.dtype).t().as_subclass(OnGpu)
    else:
        bad["layout"] = torch.zeros(2 * t.numel(), dtype=t.dtype)[::2].as_subclass(OnGpu)
    for what, value in bad.items():
        if what == "layout" and t.numel() == 1:
            continue
        args = on_gpu(good()[call])
        args[name] = value
        # (the sizes of a call come from these: another argument does not fit then;
        # the device that all have to share comes from the first)
        first = next(iter(args))
        who = r"\w+" if what == "shape" and (call, name) in sizes or what in ("shape", "device") and name in (first, "topk_ids") else name
        with pytest.raises(moe.MoeError, match=rf"{call}: {who} must be"):
            getattr(moe, call)(**args)
