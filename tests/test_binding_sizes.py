"""Sizes that an int of the C ABI does not hold are refused by the binding:
ctypes would hand the library their low 32 bits (2^32 + 16 rows as 16).  The
tensors are expanded or without memory; nothing reaches the library."""
import pytest
import torch

import mixture_experts_forward_moe_amd as moe
import test_fp8_binding as fp8
import test_layer_binding as layer
from test_fp8_binding import calls  # noqa: F401  (the fixture)

GOOD = {**fp8.good(), **layer.good()}
# of each call: the tensors a size is taken from, and which of their dimensions
TAKEN = [(call, name, d) for call, name in fp8.SIZES | {
    ("moe_rmsnorm", "x"), ("moe_rmsnorm_backward", "dy"), ("moe_router_topk", "logits"), ("moe_router_topk", "topk_ids"),
    ("moe_balance_loss", "logits"), ("moe_router_backward", "logits"), ("moe_linear_mx", "x"), ("moe_linear_mx", "w")}
    for d in range(-GOOD[call][name].dim(), 0)]
# (sizes that the library takes in 64 bits, or that a plan or another tensor gives)
NOT = {("moe_quantize_fp8", "x", -2), ("moe_dispatch", "x", -2), ("moe_dispatch_backward", "d_rows", -2),
       ("moe_finalize_backward", "dout", -2), ("moe_grouped_linear_fp8", "x", -2), ("moe_grouped_linear_fp8", "y", -2),
       ("moe_linear_fp8_wgrad", "x", -2), ("moe_grouped_linear_fp8_wgrad", "dy", -2), ("moe_linear_fp8", "w", -1),
       ("moe_grouped_linear_fp8_wgrad", "x", -2), ("moe_gated_act_fp8", "y", -2), ("moe_gated_act_fp8_backward", "dy", -2),
       ("moe_router_topk", "topk_ids", -2), ("moe_linear_mx", "x", -1)}


class Large(torch.Tensor):
    """A tensor without memory that says it is on device 0."""

    def get_device(self):
        return 0


def large(t, d, n):
    shape = list(t.shape)
    shape[d] = n
    return torch.empty(shape, dtype=t.dtype, device="meta").as_subclass(Large)


@pytest.mark.parametrize("call,name,d", sorted(set(TAKEN) - NOT))
def test_refused(calls, call, name, d):  # noqa: F811
    for n in (1 << 32) + 16, 1 << 31, 1 << 33:
        args = fp8.on_gpu(GOOD[call])
        args[name] = large(GOOD[call][name], d, n)
        with pytest.raises(moe.MoeError, match=f"{call}: a size is 2\\^31 or more") as e:
            getattr(moe, call)(**args)
        assert e.value.status == moe.ERR_UNSUPPORTED
    assert not calls


def test_every_tensor_may_be_as_large(calls):  # noqa: F811
    """All tensors of a call with 2^32 + 16 rows, which fit together."""
    M, K, N = (1 << 32) + 16, 64, 8
    e = lambda *s, dtype=torch.uint8: torch.empty(s, dtype=dtype, device="meta").as_subclass(Large)  # noqa: E731
    with pytest.raises(moe.MoeError, match="a size is"):
        moe.moe_linear_fp8(e(M, K), e(M, 1), e(N, K), e(1, 1, dtype=torch.float32), e(M, N, dtype=torch.bfloat16))
    assert not calls
    moe.moe_quantize_fp8(e(M, K, dtype=torch.bfloat16), e(M, K), e(M, 1))  # (rows are 64 bits wide)
    assert calls[0][1][2] == M


def test_sort_and_forward(calls):  # noqa: F811
    ids = torch.empty((1 << 32) + 4, 2, dtype=torch.int32, device="meta")
    with pytest.raises(moe.MoeError, match="moe_sort: a size is"):
        moe.moe_sort(ids, 4, 4, 0, 16)
    for call in ("moe_forward", "moe_forward_noalloc"):
        with pytest.raises(moe.MoeError, match=f"{call}: a size is"):
            getattr(moe, call)(None, None, ids, None, None, None, None, None, None, None, 4, 2, 4, 0, moe.W4A16, None, 64, 64)
    assert not calls
