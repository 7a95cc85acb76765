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
