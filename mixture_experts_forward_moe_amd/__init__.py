"""Python binding of libmoe_mi355x.so, the MI355X (gfx950) fused MoE forward.

Argument marshalling only: every step of the forward pass runs in the HIP
kernels behind the C ABI declared in include/moe.h.  torch provides device
memory and the current stream.  There is no fallback: if the library is not
built, every call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe_mi355x.so")

W4A16, W4A4, MXFP8_MXFP4 = 0, 1, 2
FINALIZE_DETERMINISTIC, FINALIZE_ATOMIC = 0, 1
ROUTE_ORDER_AUTO, ROUTE_ORDER_SINGLE, ROUTE_ORDER_SPAN = 0, 1, 2
PATH_AUTO, PATH_DECODE, PATH_TILED = 0, 1, 2   # moe_path_t
OK, ERR_INVALID_ARGUMENT, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_DEVICE, ERR_SCRATCH_TOO_SMALL = range(6)  # moe_status_t
NUM_PHASE_EVENTS = 5
FLT_MAX = 3.4028234663852886e38
NOALLOC_SCRATCH_BYTES = 64 << 20  # MOE_NOALLOC_SCRATCH_BYTES
ACT_SWIGLU, ACT_GEGLU_TANH, ACT_RELU2 = 0, 1, 2   # moe_activation_t (SiTU: ACT_SWIGLU with situ_beta > 0)
DTYPE_BF16, DTYPE_F32 = 0, 1             # moe_dtype_t
SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1      # moe_score_t

EXPORTS = [
    "moe_status_string", "moe_route_slots", "moe_plan_workspace_size", "moe_plan_init", "moe_sort",
    "moe_grouped_gemm1_swiglu", "moe_grouped_gemm1_act", "moe_grouped_gemm2", "moe_grouped_gemm2_bias", "moe_finalize", "moe_opts_init", "moe_default_tile",
    "moe_workspace_size", "moe_forward_plan", "moe_forward", "moe_forward_noalloc", "moe_fc2_input_scale", "moe_nvfp4_global_scale", "moe_quantize_nvfp4", "moe_quantize_mx",
    "moe_rmsnorm", "moe_rmsnorm_backward_workspace_size", "moe_rmsnorm_backward", "moe_router_topk",
    "moe_balance_workspace_size", "moe_balance_loss", "moe_router_backward", "moe_linear_mx",
    "moe_quantize_fp8", "moe_quantize_fp8_weight", "moe_dispatch", "moe_dispatch_backward", "moe_finalize_backward",
    "moe_linear_fp8", "moe_grouped_linear_fp8", "moe_linear_fp8_wgrad", "moe_grouped_linear_fp8_wgrad",
    "moe_gated_act_fp8", "moe_gated_act_fp8_backward",
]


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({status_string(status)})")
        self.status = status


class Plan(ctypes.Structure):
    _fields_ = [
        ("expanded_to_permuted", ctypes.c_void_p), ("permuted_to_expanded", ctypes.c_void_p),
        ("tile_to_expert", ctypes.c_void_p), ("tile_to_mn_limit", ctypes.c_void_p),
        ("num_tiles", ctypes.c_void_p), ("expert_offsets", ctypes.c_void_p), ("expert_counts", ctypes.c_void_p),
        ("scratch", ctypes.c_void_p), ("route_slots", ctypes.c_int64), ("max_tiles", ctypes.c_int32),
        ("tile", ctypes.c_int32), ("M", ctypes.c_int32), ("top_k", ctypes.c_int32),
        ("num_local_experts", ctypes.c_int32), ("max_spans", ctypes.c_int32),
    ]


class Opts(ctypes.Structure):
    _fields_ = [
        ("swiglu_alpha", ctypes.c_float), ("swiglu_beta", ctypes.c_float), ("swiglu_limit", ctypes.c_float),
        ("fc2_input_scale", ctypes.c_void_p), ("routed_scaling_factor", ctypes.c_float),
        ("accumulate", ctypes.c_int), ("finalize_mode", ctypes.c_int), ("route_order", ctypes.c_int),
        ("tile", ctypes.c_int), ("x_row_stride", ctypes.c_int64), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("phase_events", ctypes.c_void_p),
        ("activation", ctypes.c_int), ("situ_beta", ctypes.c_float), ("situ_linear_beta", ctypes.c_float),
        ("w1_alpha_up", ctypes.c_void_p), ("per_token_scale", ctypes.c_void_p),
        ("fc1_bias", ctypes.c_void_p), ("fc2_bias", ctypes.c_void_p), ("path", ctypes.c_int),
    ]


_lib = None


def lib() -> ctypes.CDLL:
    """The native library.  Raises if it has not been built (no fallback)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it first (python -m mixture_experts_forward_moe_amd.build)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        sigs = {
            "moe_status_string": ([I], ctypes.c_char_p),
            "moe_route_slots": ([I, I, I, I], I64),
            "moe_plan_workspace_size": ([I, I, I, I], SZ),
            "moe_plan_init": ([P, P, SZ, I, I, I, I], I),
            "moe_sort": ([P, I, I, I, I, I, I, P, P], I),
            "moe_grouped_gemm1_swiglu": ([I, P, P, I64, P, P, P, P, I, I, F, F, F, P, P, P, P], I),
            "moe_grouped_gemm1_act": ([I, P, P, I64, P, P, P, P, P, I, I, I, F, F, F, F, F, P, P, P, P, P, P], I),
            "moe_grouped_gemm2_bias": ([I, P, P, P, P, P, P, P, I, I, P, P, F, P, P], I),
            "moe_grouped_gemm2": ([I, P, P, P, P, P, P, I, I, P, P, F, P, P], I),
            "moe_finalize": ([P, P, P, I, F, I, P, P], I),
            "moe_opts_init": ([P], None),
            "moe_default_tile": ([I, I, I, I, I], I),
            "moe_workspace_size": ([I, I, I, I, I, I, I, I], SZ),
            "moe_forward_plan": ([P, P, SZ, I, I, I, I], I),
            "moe_forward": ([P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, I, I, I, P, P], I),
            "moe_forward_noalloc": ([P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, P, I, I, I, P, P], I),
            "moe_fc2_input_scale": ([P, P, I64, P, P, P, P, P, I, I, I, F, F, F, F, F, P, P, P, P], I),
            "moe_nvfp4_global_scale": ([P, I64, I64, P, P], I),
            "moe_quantize_nvfp4": ([P, I64, I64, I64, P, P, P, P], I),
            "moe_quantize_mx": ([P, I64, I64, I, P, P, P], I),
            "moe_rmsnorm": ([P, I64, P, I64, P, I, F, I, I, P, P, I, P, P, P, P], I),
            "moe_rmsnorm_backward_workspace_size": ([I, I], SZ),
            "moe_rmsnorm_backward": ([P, P, P, I, P, P, I, I, P, P, P, SZ, P], I),
            "moe_router_topk": ([P, I, I64, P, P, I, I, I, I, I, P, P, F, P, P, P, P, P, SZ, P], I),
            "moe_balance_workspace_size": ([I, I], SZ),
            "moe_balance_loss": ([P, I, I64, P, P, I, I, I, I, F, P, P, P, P, P, SZ, P], I),
            "moe_router_backward": ([P, I, I64, P, P, I, I, I, I, I, P, P, P, P, P], I),
            "moe_linear_mx": ([P, P, I, P, P, P, P, I, I, I, I, P, I, P], I),
            "moe_quantize_fp8": ([P, I64, I64, I, P, P, P], I),
            "moe_quantize_fp8_weight": ([P, I, I, I, P, P, P, P, P], I),
            "moe_dispatch": ([P, I64, P, I, P, P, P, P], I),
            "moe_dispatch_backward": ([P, P, I, I, P, P], I),
            "moe_finalize_backward": ([P, P, P, P, I, F, P, P, P, P, P], I),
            "moe_linear_fp8": ([P, P, P, P, P, I, I, I, I, P, I, P], I),
            "moe_grouped_linear_fp8": ([P, P, P, P, P, I, I, P, P], I),
            "moe_linear_fp8_wgrad": ([P, P, P, I, I, I, I, P, P], I),
            "moe_grouped_linear_fp8_wgrad": ([P, P, P, P, I, I, I, P, P], I),
            "moe_gated_act_fp8": ([P, P, I64, I, I, F, F, F, P, P, P, P, P], I),
            "moe_gated_act_fp8_backward": ([P, P, P, P, I64, I, I, F, F, F, P, P, P, P], I),
        }
        for name, (args, res) in sigs.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = res
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().moe_status_string(status).decode()


def _check(status: int, where: str):
    if status != 0:
        raise MoeError(status, where)


def _ptr(t):
    """device pointer of a tensor (or None)"""
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def route_slots(M: int, top_k: int, num_local_experts: int, tile: int) -> int:
    return lib().moe_route_slots(M, top_k, num_local_experts, tile)


def default_tile(M: int, top_k: int, num_experts: int, num_local_experts: int, mode: int) -> int:
    return lib().moe_default_tile(M, top_k, num_experts, num_local_experts, mode)


def workspace_size(M, H, I, top_k, num_local_experts, tile, mode, finalize_mode=FINALIZE_DETERMINISTIC) -> int:
    return lib().moe_workspace_size(M, H, I, top_k, num_local_experts, tile, mode, finalize_mode)


def _alloc(nbytes: int, device):
    import torch
    # 256-byte alignment: torch's caching allocator aligns blocks to 512 bytes.
    # No initial contents are needed: every piece is written before it is read.
    t = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    assert t.data_ptr() % 256 == 0
    return t


class MoePlan:
    """A routing plan with its device workspace (torch-owned).  With
    `forward_workspace`, a view of the plan a moe_forward built in that
    workspace (moe_forward_plan) instead of a workspace of its own."""

    def __init__(self, M: int, top_k: int, num_local_experts: int, tile: int, device="cuda",
                 forward_workspace=None):
        self.c = Plan()
        if forward_workspace is not None:
            self.workspace = forward_workspace
            _check(lib().moe_forward_plan(ctypes.byref(self.c), _ptr(forward_workspace), forward_workspace.numel(),
                                          M, top_k, num_local_experts, tile), "moe_forward_plan")
        else:
            n = lib().moe_plan_workspace_size(M, top_k, num_local_experts, tile)
            if n == 0:
                raise MoeError(1, "moe_plan_workspace_size")
            self.workspace = _alloc(n, device)
            _check(lib().moe_plan_init(ctypes.byref(self.c), _ptr(self.workspace), n, M, top_k, num_local_experts,
                                       tile), "moe_plan_init")
        self.M, self.top_k, self.num_local_experts, self.tile = M, top_k, num_local_experts, tile
        self.route_slots = self.c.route_slots
        self.max_tiles = self.c.max_tiles

    def _view(self, field, n):
        import torch
        off = getattr(self.c, field) - self.workspace.data_ptr()
        return self.workspace[off:off + 4 * n].view(torch.int32)

    @property
    def expanded_to_permuted(self):
        return self._view("expanded_to_permuted", self.M * self.top_k)

    @property
    def permuted_to_expanded(self):
        return self._view("permuted_to_expanded", self.route_slots)

    @property
    def tile_to_expert(self):
        return self._view("tile_to_expert", self.max_tiles)

    @property
    def tile_to_mn_limit(self):
        return self._view("tile_to_mn_limit", self.max_tiles)

    @property
    def num_tiles(self):
        return self._view("num_tiles", 1)

    @property
    def expert_offsets(self):
        return self._view("expert_offsets", self.num_local_experts + 1)

    @property
    def expert_counts(self):
        return self._view("expert_counts", self.num_local_experts)


def moe_sort(topk_ids, num_experts: int, num_local_experts: int, local_expert_offset: int, tile: int,
             route_order: int = ROUTE_ORDER_AUTO, plan: MoePlan | None = None, stream=None) -> MoePlan:
    M, top_k = topk_ids.shape
    _below_2_31("moe_sort", M | top_k)
    if plan is None:
        plan = MoePlan(M, top_k, num_local_experts, tile, topk_ids.device)
    _check(lib().moe_sort(_ptr(topk_ids), M, top_k, num_experts, num_local_experts, local_expert_offset, route_order,
                          ctypes.byref(plan.c), _stream(stream)), "moe_sort")
    return plan


def moe_grouped_gemm1_swiglu(mode, x, x_sf, plan: MoePlan, w1, w1_sf, w1_alpha, H, I, y1, y1_sf=None,
                             swiglu_alpha=1.0, swiglu_beta=0.0, swiglu_limit=FLT_MAX, fc2_input_scale=None,
                             x_row_stride=0, stream=None):
    _check(lib().moe_grouped_gemm1_swiglu(mode, _ptr(x), _ptr(x_sf), x_row_stride, ctypes.byref(plan.c), _ptr(w1),
                                          _ptr(w1_sf), _ptr(w1_alpha), H, I, swiglu_alpha, swiglu_beta, swiglu_limit,
                                          _ptr(fc2_input_scale), _ptr(y1), _ptr(y1_sf), _stream(stream)),
           "moe_grouped_gemm1_swiglu")


def moe_grouped_gemm1_act(mode, x, x_sf, plan: MoePlan, w1, w1_sf, w1_alpha, H, I, y1, y1_sf=None,
                          activation=ACT_SWIGLU, swiglu_alpha=1.0, swiglu_beta=0.0, swiglu_limit=FLT_MAX,
                          situ_beta=0.0, situ_linear_beta=0.0, fc2_input_scale=None, x_row_stride=0, stream=None,
                          w1_alpha_up=None, per_token_scale=None, fc1_bias=None):
    _check(lib().moe_grouped_gemm1_act(mode, _ptr(x), _ptr(x_sf), x_row_stride, ctypes.byref(plan.c), _ptr(w1),
                                       _ptr(w1_sf), _ptr(w1_alpha), _ptr(w1_alpha_up), H, I, activation,
                                       swiglu_alpha, swiglu_beta, swiglu_limit, situ_beta, situ_linear_beta,
                                       _ptr(fc2_input_scale), _ptr(per_token_scale), _ptr(fc1_bias), _ptr(y1),
                                       _ptr(y1_sf),
                                       _stream(stream)), "moe_grouped_gemm1_act")


def moe_grouped_gemm2(mode, y1, y1_sf, plan: MoePlan, w2, w2_sf, w2_alpha, H, I, y2=None, topk_weights=None,
                      routed_scaling_factor=1.0, out=None, stream=None, fc2_bias=None):
    if fc2_bias is None:
        _check(lib().moe_grouped_gemm2(mode, _ptr(y1), _ptr(y1_sf), ctypes.byref(plan.c), _ptr(w2), _ptr(w2_sf),
                                       _ptr(w2_alpha), H, I, _ptr(y2), _ptr(topk_weights), routed_scaling_factor,
                                       _ptr(out), _stream(stream)), "moe_grouped_gemm2")
    else:
        _check(lib().moe_grouped_gemm2_bias(mode, _ptr(y1), _ptr(y1_sf), ctypes.byref(plan.c), _ptr(w2),
                                            _ptr(w2_sf), _ptr(w2_alpha), _ptr(fc2_bias), H, I, _ptr(y2),
                                            _ptr(topk_weights), routed_scaling_factor, _ptr(out), _stream(stream)),
               "moe_grouped_gemm2_bias")


def moe_finalize(y2, plan: MoePlan, topk_weights, H, out, routed_scaling_factor=1.0, accumulate=False, stream=None):
    _check(lib().moe_finalize(_ptr(y2), ctypes.byref(plan.c), _ptr(topk_weights), H, routed_scaling_factor,
                              int(bool(accumulate)), _ptr(out), _stream(stream)), "moe_finalize")


def make_opts(workspace=None, swiglu_alpha=1.0, swiglu_beta=0.0, swiglu_limit=FLT_MAX, fc2_input_scale=None,
              routed_scaling_factor=1.0, accumulate=False, finalize_mode=FINALIZE_DETERMINISTIC,
              route_order=ROUTE_ORDER_AUTO, tile=0, x_row_stride=0, phase_events=None, activation=ACT_SWIGLU,
              situ_beta=0.0, situ_linear_beta=0.0, w1_alpha_up=None, per_token_scale=None, fc1_bias=None,
              fc2_bias=None, path=PATH_AUTO) -> Opts:
    o = Opts()
    lib().moe_opts_init(ctypes.byref(o))
    o.swiglu_alpha, o.swiglu_beta, o.swiglu_limit = swiglu_alpha, swiglu_beta, swiglu_limit
    o.activation, o.situ_beta, o.situ_linear_beta = activation, situ_beta, situ_linear_beta
    o.w1_alpha_up = None if w1_alpha_up is None else w1_alpha_up.data_ptr()
    o.per_token_scale = None if per_token_scale is None else per_token_scale.data_ptr()
    o.fc1_bias = None if fc1_bias is None else fc1_bias.data_ptr()
    o.fc2_bias = None if fc2_bias is None else fc2_bias.data_ptr()
    o.fc2_input_scale = None if fc2_input_scale is None else fc2_input_scale.data_ptr()
    o.routed_scaling_factor = routed_scaling_factor
    o.accumulate = int(bool(accumulate))
    o.finalize_mode = finalize_mode
    o.route_order = route_order
    o.tile = tile
    o.x_row_stride = x_row_stride
    o.path = path
    if workspace is not None:
        o.workspace = workspace.data_ptr()
        o.workspace_bytes = workspace.numel() * workspace.element_size()
    if phase_events is not None:
        arr = (ctypes.c_void_p * NUM_PHASE_EVENTS)(*[None if e is None else e.cuda_event for e in phase_events])
        o._events = arr
        o.phase_events = ctypes.cast(arr, ctypes.c_void_p)
    return o


def moe_forward(x, x_sf, topk_ids, topk_weights, w1, w1_sf, w1_alpha, w2, w2_sf, w2_alpha, num_experts: int,
                top_k: int, num_local_experts: int, local_expert_offset: int, quant_mode: int, out, H: int, I: int,
                opts: Opts | None = None, workspace=None, stream=None, **kw):
    """The whole forward pass into `out` (bf16 [M, H]).  A workspace is taken
    from `workspace`, or allocated here (outside the library) when None."""
    M = topk_ids.shape[0]
    _below_2_31("moe_forward", M)
    if opts is None:
        tile = kw.pop("tile", 0) or default_tile(M, top_k, num_experts, num_local_experts, quant_mode)
        fm = kw.get("finalize_mode", FINALIZE_DETERMINISTIC)
        if workspace is None:
            workspace = _alloc(workspace_size(M, H, I, top_k, num_local_experts, tile, quant_mode, fm), x.device)
        opts = make_opts(workspace=workspace, tile=tile, **kw)
    _check(lib().moe_forward(_ptr(x), _ptr(x_sf), _ptr(topk_ids), _ptr(topk_weights), _ptr(w1), _ptr(w1_sf),
                             _ptr(w1_alpha), _ptr(w2), _ptr(w2_sf), _ptr(w2_alpha), num_experts, top_k,
                             num_local_experts, local_expert_offset, quant_mode, _ptr(out), M, H, I,
                             ctypes.byref(opts), _stream(stream)), "moe_forward")
    return out


def moe_forward_noalloc(x, x_sf, topk_ids, topk_weights, w1, w1_sf, w1_alpha, w2, w2_sf, w2_alpha, num_experts: int,
                        top_k: int, num_local_experts: int, local_expert_offset: int, quant_mode: int, out, H: int,
                        I: int, stream=None, **kw):
    """moe_forward with the library's own fixed scratch array as workspace
    (nothing is allocated, here or in the library)."""
    M = topk_ids.shape[0]
    _below_2_31("moe_forward_noalloc", M)
    opts = make_opts(**kw)
    _check(lib().moe_forward_noalloc(_ptr(x), _ptr(x_sf), _ptr(topk_ids), _ptr(topk_weights), _ptr(w1), _ptr(w1_sf),
                                     _ptr(w1_alpha), _ptr(w2), _ptr(w2_sf), _ptr(w2_alpha), num_experts, top_k,
                                     num_local_experts, local_expert_offset, quant_mode, _ptr(out), M, H, I,
                                     ctypes.byref(opts), _stream(stream)), "moe_forward_noalloc")
    return out


def moe_fc2_input_scale(x, x_sf, plan: MoePlan, w1, w1_sf, w1_alpha, H, I, fc2_input_scale, activation=ACT_SWIGLU,
                        swiglu_alpha=1.0, swiglu_beta=0.0, swiglu_limit=FLT_MAX, situ_beta=0.0, situ_linear_beta=0.0,
                        x_row_stride=0, w1_alpha_up=None, per_token_scale=None, fc1_bias=None, stream=None):
    """W4A4: fc2_input_scale (device fp32 [1]) = max |y1| / (6 * 448) over the plan's routes."""
    _check(lib().moe_fc2_input_scale(_ptr(x), _ptr(x_sf), x_row_stride, ctypes.byref(plan.c), _ptr(w1), _ptr(w1_sf),
                                     _ptr(w1_alpha), _ptr(w1_alpha_up), H, I, activation, swiglu_alpha, swiglu_beta,
                                     swiglu_limit, situ_beta, situ_linear_beta, _ptr(per_token_scale),
                                     _ptr(fc1_bias), _ptr(fc2_input_scale), _stream(stream)), "moe_fc2_input_scale")


def moe_nvfp4_global_scale(x, batches: int, gscale, stream=None):
    _check(lib().moe_nvfp4_global_scale(_ptr(x), batches, x.numel() // max(batches, 1), _ptr(gscale),
                                        _stream(stream)), "moe_nvfp4_global_scale")


def moe_quantize_nvfp4(x, batches: int, rows: int, cols: int, gscale, q, sf, stream=None):
    _check(lib().moe_quantize_nvfp4(_ptr(x), batches, rows, cols, _ptr(gscale), _ptr(q), _ptr(sf), _stream(stream)),
           "moe_quantize_nvfp4")


def moe_quantize_mx(x, rows: int, cols: int, elem: int, q, sf, stream=None):
    _check(lib().moe_quantize_mx(_ptr(x), rows, cols, elem, _ptr(q), _ptr(sf), _stream(stream)), "moe_quantize_mx")


# ---- around the routed experts: norm, router, balance loss, linear ----------

class _Kind(list):
    """The element types an argument may come in: filled in when first used, so
    that this module imports without torch."""

    def __init__(self, name, *types):
        self.name, self.types = name, types


_BF16 = _Kind("bf16", "bfloat16", "int16", "uint16")  # also as its 16 bits
_F32 = _Kind("fp32", "float32")
_I32 = _Kind("int32", "int32", "uint32")
_BYTE = _Kind("bytes", "uint8", "int8", "bool", "float8_e4m3fn", "float8_e8m0fnu", "float4_e2m1fn_x2")
_cuda = None  # torch._C


def _kinds():
    global _cuda
    import torch
    _cuda = torch._C
    for kind in (_BF16, _F32, _I32, _BYTE):
        kind[:] = [getattr(torch, n) for n in kind.types if hasattr(torch, n)]


def _refuse(where, name, t, shape, kind, strided):
    if t is None:
        what = "is required"
    elif t.shape != shape or t.dtype not in kind:
        what = f"must be {kind.name} {shape}, is {t.dtype} {tuple(t.shape)}"
    elif not (t.is_contiguous() or strided and t.stride(-1) == 1 and t.stride(0) >= shape[1]):
        what = "must be contiguous" + (" in a row, and its rows apart" if strided else "")
    else:
        what = "must be on the GPU, with the call's other tensors"
    raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: {name} {what}")


def _arg(where: str, name: str, t, shape, kind: _Kind, dev: int):
    """The device address of tensor `t`, checked against the shape, the element
    type and the device that the call takes it with."""
    if not kind:
        _kinds()
    if t is None or t.shape != shape or t.dtype not in kind or t.get_device() != dev or dev < 0 \
            or not t.is_contiguous():
        _refuse(where, name, t, shape, kind, False)
    return t.data_ptr()


def _opt(where, name, t, shape, kind, dev):
    """The same of a tensor that may be None."""
    if t is None:
        return None
    if not kind:
        _kinds()
    if t.shape != shape or t.dtype not in kind or t.get_device() != dev or dev < 0 or not t.is_contiguous():
        _refuse(where, name, t, shape, kind, False)
    return t.data_ptr()


def _rows(where, name, t, shape, kind, dev):
    """(address, row stride in elements; 0: contiguous) of a [rows, columns]
    tensor whose rows may be apart."""
    if not kind:
        _kinds()
    if t is not None and t.shape == shape and t.dtype in kind and t.get_device() == dev and dev >= 0:
        if t.is_contiguous():
            return t.data_ptr(), 0
        # (rows of an expanded tensor are not apart: their stride is 0)
        if (t.stride(1) == 1 or shape[1] == 1) and t.stride(0) >= shape[1]:
            return t.data_ptr(), t.stride(0)
    _refuse(where, name, t, shape, kind, True)


def _shapes(where, **given):
    """What a call says whose sizes could not be taken from these tensors."""
    for name, t in given.items():
        if t is None or t.dim() != 2:
            what = "is required" if t is None else f"must have two dimensions, has {t.dim()}"
            raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: {name} {what}")


def _below_2_31(where: str, sizes: int):
    """Refuses a tensor's sizes (or-ed together) that an int of the C ABI does
    not hold: ctypes would cut them off."""
    if sizes >> 31:
        raise MoeError(ERR_UNSUPPORTED, f"{where}: a size is 2^31 or more")


def _dtype(where: str, name: str, t) -> int:
    """moe_dtype_t of a floating tensor (bf16 also as 16-bit integers)."""
    if not _F32:
        _kinds()
    if t is None:
        raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: {name} is required")
    if t.dtype in _F32:
        return DTYPE_F32
    if t.dtype in _BF16:
        return DTYPE_BF16
    raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: {name} must be bf16 or fp32, is {t.dtype}")


def _raw_stream(where, dev, stream):
    """The stream of a call on device `dev`, which must be the current one.
    (After the arguments' checks: they are on a GPU, so torch has set it up.)"""
    if _cuda._cuda_getDevice() != dev:
        raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: the tensors are on cuda:{dev}, which is not the current device")
    return _cuda._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _workspace(where, nbytes: int, given, t, stream):
    """(tensor, address, bytes): the caller's workspace, or one from torch's
    allocator: from the memory of the call's stream, whose blocks other work on
    that stream alone has used and will use."""
    if given is not None:
        if given.get_device() != t.get_device() or not given.is_contiguous():
            raise MoeError(ERR_INVALID_ARGUMENT,
                           f"{where}: workspace must be contiguous, with the call's other tensors")
        return given, given.data_ptr(), given.numel() * given.element_size()
    if stream is None:
        given = _alloc(nbytes, t.device)
    else:
        import torch
        with torch.cuda.stream(stream):
            given = _alloc(nbytes, t.device)
    return given, given.data_ptr(), nbytes


def moe_rmsnorm(x, weight, y=None, residual=None, residual_out=None, q=None, q_sf=None, elem=0, rstd=None, eps=1e-6,
                stream=None):
    """h = bf16(x + residual), y = bf16(h * rsqrt(mean(h^2) + eps) * weight),
    and y's MX codes, in one pass (see moe_rmsnorm in moe.h).  x, residual
    bf16 [M, H], rows may be strided; weight bf16 or fp32 [H]."""
    w = "moe_rmsnorm"
    try:
        M, H = shape = x.shape
    except (AttributeError, ValueError):
        _shapes(w, x=x)
        raise
    _below_2_31(w, M | H)
    dev = x.get_device()
    wd = _dtype(w, "weight", weight)
    xp, xs = _rows(w, "x", x, shape, _BF16, dev)
    rp, rs = (None, 0) if residual is None else _rows(w, "residual", residual, shape, _BF16, dev)
    _check(lib().moe_rmsnorm(
        xp, xs, rp, rs, _arg(w, "weight", weight, (H,), _F32 if wd else _BF16, dev), wd, eps, M, H,
        _opt(w, "residual_out", residual_out, shape, _BF16, dev), _opt(w, "y", y, shape, _BF16, dev), elem,
        _opt(w, "q", q, (M, H if elem == 0 else H // 2), _BYTE, dev), _opt(w, "q_sf", q_sf, (M, H // 32), _BYTE, dev),
        _opt(w, "rstd", rstd, (M,), _F32, dev), _raw_stream(w, dev, stream)), w)


@functools.lru_cache
def rmsnorm_backward_workspace_size(M: int, H: int) -> int:
    return lib().moe_rmsnorm_backward_workspace_size(M, H)


def moe_rmsnorm_backward(dy, h, weight, rstd, dx, dweight=None, dh=None, workspace=None, stream=None):
    """Gradients of moe_rmsnorm's rows and weight.  A workspace (only with
    dweight) is taken from `workspace`, or allocated here when None."""
    w = "moe_rmsnorm_backward"
    try:
        M, H = shape = dy.shape
    except (AttributeError, ValueError):
        _shapes(w, dy=dy)
        raise
    _below_2_31(w, M | H)
    dev = dy.get_device()
    wd = _dtype(w, "weight", weight)
    args = (_arg(w, "dy", dy, shape, _BF16, dev), _arg(w, "h", h, shape, _BF16, dev),
            _arg(w, "weight", weight, (H,), _F32 if wd else _BF16, dev), wd, _arg(w, "rstd", rstd, (M,), _F32, dev),
            _opt(w, "dh", dh, shape, _BF16, dev), M, H, _arg(w, "dx", dx, shape, _BF16, dev),
            _opt(w, "dweight", dweight, (H,), _F32, dev))
    st = _raw_stream(w, dev, stream)
    wp, nbytes = None, 0
    if dweight is not None:
        workspace, wp, nbytes = _workspace(w, rmsnorm_backward_workspace_size(M, H), workspace, dy, stream)
    _check(lib().moe_rmsnorm_backward(*args, wp, nbytes, st), w)


@functools.lru_cache
def balance_workspace_size(M: int, E: int) -> int:
    return lib().moe_balance_workspace_size(M, E)


def _balance_args(w, E, dev, expert_counts, mean_probs, prob_grad, loss):
    return (_arg(w, "expert_counts", expert_counts, (E,), _I32, dev),
            _arg(w, "mean_probs", mean_probs, (E,), _F32, dev), _arg(w, "prob_grad", prob_grad, (E,), _F32, dev),
            _arg(w, "loss", loss, (1,), _F32, dev))


def moe_router_topk(logits, topk_ids, topk_weights, score=SCORE_SOFTMAX, renormalize=True, select_bias=None,
                    token_mask=None, coef=0.0, expert_counts=None, mean_probs=None, prob_grad=None, loss=None,
                    workspace=None, stream=None):
    """Experts (int32 [M, top_k]) and routing weights (fp32 [M, top_k]) of
    router logits [M, E], as moe_forward takes them.  With expert_counts,
    mean_probs, prob_grad and loss (all four) also the balance loss of that
    choice, from the same reading of the logits."""
    w = "moe_router_topk"
    try:
        (M, E), (_, k) = logits.shape, topk_ids.shape
    except (AttributeError, ValueError):
        _shapes(w, logits=logits, topk_ids=topk_ids)
        raise
    _below_2_31(w, M | E | k)
    dev = logits.get_device()
    d = _dtype(w, "logits", logits)
    lp, ls = _rows(w, "logits", logits, (M, E), _F32 if d else _BF16, dev)
    args = (lp, d, ls, _opt(w, "select_bias", select_bias, (E,), _F32, dev),
            _opt(w, "token_mask", token_mask, (M,), _BYTE, dev), score, 1 if renormalize else 0, M, E, k,
            _arg(w, "topk_ids", topk_ids, (M, k), _I32, dev),
            _arg(w, "topk_weights", topk_weights, (M, k), _F32, dev), coef)
    st = _raw_stream(w, dev, stream)
    if expert_counts is None and mean_probs is None and prob_grad is None and loss is None:
        _check(lib().moe_router_topk(*args, None, None, None, None, None, 0, st), w)
        return
    balance = _balance_args(w, E, dev, expert_counts, mean_probs, prob_grad, loss)
    workspace, wp, nbytes = _workspace(w, balance_workspace_size(M, E), workspace, logits, stream)
    _check(lib().moe_router_topk(*args, *balance, wp, nbytes, st), w)


def moe_balance_loss(logits, topk_ids, coef, expert_counts, mean_probs, prob_grad, loss, score=SCORE_SOFTMAX,
                     token_mask=None, workspace=None, stream=None):
    """Per-expert counts, mean probabilities and the load-balancing loss of
    given expert ids, and the loss's gradient in the probabilities."""
    w = "moe_balance_loss"
    try:
        (M, E), (_, k) = logits.shape, topk_ids.shape
    except (AttributeError, ValueError):
        _shapes(w, logits=logits, topk_ids=topk_ids)
        raise
    _below_2_31(w, M | E | k)
    dev = logits.get_device()
    d = _dtype(w, "logits", logits)
    lp, ls = _rows(w, "logits", logits, (M, E), _F32 if d else _BF16, dev)
    args = (lp, d, ls, _arg(w, "topk_ids", topk_ids, (M, k), _I32, dev),
            _opt(w, "token_mask", token_mask, (M,), _BYTE, dev), score, M, E, k, coef,
            *_balance_args(w, E, dev, expert_counts, mean_probs, prob_grad, loss))
    st = _raw_stream(w, dev, stream)
    workspace, wp, nbytes = _workspace(w, balance_workspace_size(M, E), workspace, logits, stream)
    _check(lib().moe_balance_loss(*args, wp, nbytes, st), w)


def moe_router_backward(logits, topk_ids, d_logits, d_topk_weights=None, prob_grad=None, d_loss=None,
                        score=SCORE_SOFTMAX, renormalize=True, token_mask=None, stream=None):
    """The gradient of the logits, in their type, from that of the routing
    weights and / or of the balance loss (a device scalar; None: 1)."""
    w = "moe_router_backward"
    try:
        (M, E), (_, k) = logits.shape, topk_ids.shape
    except (AttributeError, ValueError):
        _shapes(w, logits=logits, topk_ids=topk_ids)
        raise
    _below_2_31(w, M | E | k)
    dev = logits.get_device()
    d = _dtype(w, "logits", logits)
    if _dtype(w, "d_logits", d_logits) != d:
        raise MoeError(ERR_INVALID_ARGUMENT, f"{w}: d_logits must have the type of logits")
    kind = _F32 if d else _BF16
    lp, ls = _rows(w, "logits", logits, (M, E), kind, dev)
    _check(lib().moe_router_backward(
        lp, d, ls, _arg(w, "topk_ids", topk_ids, (M, k), _I32, dev),
        _opt(w, "token_mask", token_mask, (M,), _BYTE, dev), score, 1 if renormalize else 0, M, E, k,
        _opt(w, "d_topk_weights", d_topk_weights, (M, k), _F32, dev),
        _opt(w, "prob_grad", prob_grad, (E,), _F32, dev), _opt(w, "d_loss", d_loss, (1,), _F32, dev),
        _arg(w, "d_logits", d_logits, (M, E), kind, dev), _raw_stream(w, dev, stream)), w)


def moe_linear_mx(x, x_sf, w, w_sf, y, x_elem=0, alpha=None, bias=None, accumulate=False, stream=None):
    """y = alpha * x w^T + bias (+ y) of MX operands: x E4M3 [M, K] (x_elem 0)
    or packed E2M1 [M, K/2] (1) with E8M0 x_sf [M, K/32]; w packed E2M1
    [N, K/2] with w_sf [N, K/32]; y bf16 or fp32 [M, N].  Sums are fp32; E4M3
    products keep 13 bits below the largest of 8 neighbours (see moe.h)."""
    f = "moe_linear_mx"
    try:
        (M, _), (N, K) = x.shape, w.shape
    except (AttributeError, ValueError):
        _shapes(f, x=x, w=w)
        raise
    K *= 2
    _below_2_31(f, M | N | K)
    dev = x.get_device()
    d = _dtype(f, "y", y)
    _check(lib().moe_linear_mx(
        _arg(f, "x", x, (M, K if x_elem == 0 else K // 2), _BYTE, dev),
        _arg(f, "x_sf", x_sf, (M, K // 32), _BYTE, dev), x_elem, _arg(f, "w", w, (N, K // 2), _BYTE, dev),
        _arg(f, "w_sf", w_sf, (N, K // 32), _BYTE, dev),
        _opt(f, "alpha", alpha, (1,), _F32, dev), _opt(f, "bias", bias, (N,), _F32, dev), M, N, K,
        1 if accumulate else 0, _arg(f, "y", y, (M, N), _F32 if d else _BF16, dev), d,
        _raw_stream(f, dev, stream)), f)


# ---- rows in 8 bits: training and serving the experts in E4M3 ---------------

def _nb(cols: int) -> int:
    return (cols + 127) // 128


def _two(where, name, t):
    """The two sizes of a tensor."""
    try:
        a, b = t.shape
        return a, b
    except (AttributeError, ValueError):
        _shapes(where, **{name: t})
        raise


def _plan_arg(where, plan, dev):
    """The plan's C struct, checked to be on the call's device."""
    if not isinstance(plan, MoePlan):
        raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: plan must be a MoePlan, is {type(plan).__name__}")
    if plan.workspace.get_device() != dev:
        raise MoeError(ERR_INVALID_ARGUMENT, f"{where}: plan must be on the GPU, with the call's other tensors")
    return ctypes.byref(plan.c)


def moe_quantize_fp8(x, q, q_sf, stream=None):
    """E4M3 codes q [rows, cols] and E8M0 scales q_sf [rows, ceil(cols / 128)]
    of bf16 rows x, which may be strided."""
    w = "moe_quantize_fp8"
    rows, cols = _two(w, "x", x)
    _below_2_31(w, cols)
    dev = x.get_device()
    xp, xs = _rows(w, "x", x, (rows, cols), _BF16, dev)
    _check(lib().moe_quantize_fp8(xp, xs, rows, cols, _arg(w, "q", q, (rows, cols), _BYTE, dev),
                                  _arg(w, "q_sf", q_sf, (rows, _nb(cols)), _BYTE, dev),
                                  _raw_stream(w, dev, stream)), w)


def moe_quantize_fp8_weight(weight, q, sf, qt=None, sft=None, stream=None):
    """E4M3 codes and fp32 scales for blocks of 128 x 128 of bf16 weights
    [N, K] or [batches, N, K]; qt and sft the same transposed (for
    the gradient of a product's rows)."""
    w = "moe_quantize_fp8_weight"
    if weight is None or weight.dim() not in (2, 3):
        raise MoeError(ERR_INVALID_ARGUMENT, f"{w}: weight must have two or three dimensions")
    lead, (N, K) = tuple(weight.shape[:-2]), weight.shape[-2:]
    _below_2_31(w, N | K | (lead[0] if lead else 1))
    dev = weight.get_device()
    _check(lib().moe_quantize_fp8_weight(
        _arg(w, "weight", weight, (*lead, N, K), _BF16, dev), lead[0] if lead else 1, N, K,
        _arg(w, "q", q, (*lead, N, K), _BYTE, dev), _arg(w, "sf", sf, (*lead, _nb(N), _nb(K)), _F32, dev),
        _opt(w, "qt", qt, (*lead, K, N), _BYTE, dev), _opt(w, "sft", sft, (*lead, _nb(K), _nb(N)), _F32, dev),
        _raw_stream(w, dev, stream)), w)


def moe_dispatch(x, plan: MoePlan, rows=None, q=None, q_sf=None, stream=None):
    """Each token's bf16 row x [M, H] (rows may be strided) at the slots of its
    routes: as bf16 rows [route_slots, H], and / or quantised, q [route_slots,
    H] with q_sf [route_slots, ceil(H / 128)]."""
    w = "moe_dispatch"
    H = _two(w, "x", x)[1]
    _below_2_31(w, H)
    dev = x.get_device()
    p = _plan_arg(w, plan, dev)
    n = plan.route_slots
    xp, xs = _rows(w, "x", x, (plan.M, H), _BF16, dev)
    _check(lib().moe_dispatch(xp, xs, p, H, _opt(w, "rows", rows, (n, H), _BF16, dev),
                              _opt(w, "q", q, (n, H), _BYTE, dev), _opt(w, "q_sf", q_sf, (n, _nb(H)), _BYTE, dev),
                              _raw_stream(w, dev, stream)), w)


def moe_dispatch_backward(d_rows, plan: MoePlan, dx, accumulate=False, stream=None):
    """dx [M, H] = (dx +) the sum of d_rows [route_slots, H] over each token's
    routes."""
    w = "moe_dispatch_backward"
    H = _two(w, "d_rows", d_rows)[1]
    _below_2_31(w, H)
    dev = d_rows.get_device()
    p = _plan_arg(w, plan, dev)
    _check(lib().moe_dispatch_backward(_arg(w, "d_rows", d_rows, (plan.route_slots, H), _BF16, dev), p, H,
                                       1 if accumulate else 0, _arg(w, "dx", dx, (plan.M, H), _BF16, dev),
                                       _raw_stream(w, dev, stream)), w)


def moe_finalize_backward(dout, y2, plan: MoePlan, topk_weights, dy2=None, q=None, q_sf=None, d_topk_weights=None,
                          routed_scaling_factor=1.0, stream=None):
    """The gradients of moe_finalize: of its rows (dy2 bf16 [route_slots, H],
    and / or quantised in q, q_sf) and, with y2, of the routing weights."""
    w = "moe_finalize_backward"
    H = _two(w, "dout", dout)[1]
    _below_2_31(w, H)
    dev = dout.get_device()
    p = _plan_arg(w, plan, dev)
    n = plan.route_slots
    _check(lib().moe_finalize_backward(
        _arg(w, "dout", dout, (plan.M, H), _BF16, dev), _opt(w, "y2", y2, (n, H), _BF16, dev), p,
        _arg(w, "topk_weights", topk_weights, (plan.M, plan.top_k), _F32, dev), H, routed_scaling_factor,
        _opt(w, "dy2", dy2, (n, H), _BF16, dev), _opt(w, "q", q, (n, H), _BYTE, dev),
        _opt(w, "q_sf", q_sf, (n, _nb(H)), _BYTE, dev),
        _opt(w, "d_topk_weights", d_topk_weights, (plan.M, plan.top_k), _F32, dev), _raw_stream(w, dev, stream)), w)


def moe_linear_fp8(x, x_sf, w, w_sf, y, bias=None, accumulate=False, stream=None):
    """y = x w^T + bias (+ y): x E4M3 [M, K] with E8M0 x_sf [M, ceil(K / 128)],
    w E4M3 [N, K] with fp32 w_sf [ceil(N / 128), ceil(K / 128)], y bf16 or fp32
    [M, N].  What the matrix instruction keeps of a product stands in moe.h."""
    f = "moe_linear_fp8"
    M, K = _two(f, "x", x)
    N = _two(f, "w", w)[0]
    _below_2_31(f, M | N | K)
    dev = x.get_device()
    d = _dtype(f, "y", y)
    _check(lib().moe_linear_fp8(
        _arg(f, "x", x, (M, K), _BYTE, dev), _arg(f, "x_sf", x_sf, (M, _nb(K)), _BYTE, dev),
        _arg(f, "w", w, (N, K), _BYTE, dev), _arg(f, "w_sf", w_sf, (_nb(N), _nb(K)), _F32, dev),
        _opt(f, "bias", bias, (N,), _F32, dev), M, N, K, 1 if accumulate else 0,
        _arg(f, "y", y, (M, N), _F32 if d else _BF16, dev), d, _raw_stream(f, dev, stream)), f)


def moe_grouped_linear_fp8(x, x_sf, plan: MoePlan, w, w_sf, y, stream=None):
    """y[s] = bf16(x[s] w[e]^T) for every valid slot s of expert e: x E4M3
    [route_slots, K], w E4M3 [E_l, N, K] with w_sf [E_l, ceil(N / 128),
    ceil(K / 128)], y bf16 [route_slots, N]."""
    f = "moe_grouped_linear_fp8"
    K, N = _two(f, "x", x)[1], _two(f, "y", y)[1]
    _below_2_31(f, N | K)
    dev = x.get_device()
    p = _plan_arg(f, plan, dev)
    n, E = plan.route_slots, plan.num_local_experts
    _check(lib().moe_grouped_linear_fp8(
        _arg(f, "x", x, (n, K), _BYTE, dev), _arg(f, "x_sf", x_sf, (n, _nb(K)), _BYTE, dev), p,
        _arg(f, "w", w, (E, N, K), _BYTE, dev), _arg(f, "w_sf", w_sf, (E, _nb(N), _nb(K)), _F32, dev), N, K,
        _arg(f, "y", y, (n, N), _BF16, dev), _raw_stream(f, dev, stream)), f)


def moe_linear_fp8_wgrad(dy, x, x_sf, dw, accumulate=False, stream=None):
    """dw [N, K] = dy^T x (+ dw) in fp32, from bf16 dy [M, N] and the product's
    rows in 8 bits, x E4M3 [M, K] with x_sf."""
    f = "moe_linear_fp8_wgrad"
    M, N = _two(f, "dy", dy)
    K = _two(f, "x", x)[1]
    _below_2_31(f, M | N | K)
    dev = dy.get_device()
    _check(lib().moe_linear_fp8_wgrad(
        _arg(f, "dy", dy, (M, N), _BF16, dev), _arg(f, "x", x, (M, K), _BYTE, dev),
        _arg(f, "x_sf", x_sf, (M, _nb(K)), _BYTE, dev), M, N, K, 1 if accumulate else 0,
        _arg(f, "dw", dw, (N, K), _F32, dev), _raw_stream(f, dev, stream)), f)


def moe_grouped_linear_fp8_wgrad(dy, x, x_sf, plan: MoePlan, dw, accumulate=False, stream=None):
    """The same of every expert, dw [E_l, N, K], from the valid slots of its
    range: dy bf16 [route_slots, N], x E4M3 [route_slots, K]."""
    f = "moe_grouped_linear_fp8_wgrad"
    N, K = _two(f, "dy", dy)[1], _two(f, "x", x)[1]
    _below_2_31(f, N | K)
    dev = dy.get_device()
    p = _plan_arg(f, plan, dev)
    n, E = plan.route_slots, plan.num_local_experts
    _check(lib().moe_grouped_linear_fp8_wgrad(
        _arg(f, "dy", dy, (n, N), _BF16, dev), _arg(f, "x", x, (n, K), _BYTE, dev),
        _arg(f, "x_sf", x_sf, (n, _nb(K)), _BYTE, dev), p, N, K, 1 if accumulate else 0,
        _arg(f, "dw", dw, (E, N, K), _F32, dev), _raw_stream(f, dev, stream)), f)


def moe_gated_act_fp8(h, y, y_sf, hq=None, hq_sf=None, plan: MoePlan | None = None, activation=ACT_SWIGLU,
                      swiglu_alpha=1.0, swiglu_beta=0.0, swiglu_limit=FLT_MAX, stream=None):
    """The gated activation of bf16 rows h = (gate, up) [rows, 2I], quantised (y
    [rows, I], y_sf [rows, ceil(I / 128)]), and h kept in 8 bits for the
    backward pass (hq [rows, 2I], hq_sf [rows, 2 ceil(I / 128)]).  With a plan
    its valid slots are the rows."""
    w = "moe_gated_act_fp8"
    rows, I = _two(w, "y", y)
    _below_2_31(w, 2 * I)
    dev = y.get_device()
    p = None if plan is None else _plan_arg(w, plan, dev)
    if plan is not None:
        rows = plan.route_slots
    _check(lib().moe_gated_act_fp8(
        _arg(w, "h", h, (rows, 2 * I), _BF16, dev), p, rows, I, activation, swiglu_alpha, swiglu_beta, swiglu_limit,
        _arg(w, "y", y, (rows, I), _BYTE, dev), _arg(w, "y_sf", y_sf, (rows, _nb(I)), _BYTE, dev),
        _opt(w, "hq", hq, (rows, 2 * I), _BYTE, dev), _opt(w, "hq_sf", hq_sf, (rows, 2 * _nb(I)), _BYTE, dev),
        _raw_stream(w, dev, stream)), w)


def moe_gated_act_fp8_backward(hq, hq_sf, dy, dh=None, dq=None, dq_sf=None, plan: MoePlan | None = None,
                               activation=ACT_SWIGLU, swiglu_alpha=1.0, swiglu_beta=0.0, swiglu_limit=FLT_MAX,
                               stream=None):
    """The gradient of moe_gated_act_fp8's h at the h it kept, from dy bf16
    [rows, I]: dh bf16 [rows, 2I] and / or quantised, dq [rows, 2I] with dq_sf
    [rows, 2 ceil(I / 128)]."""
    w = "moe_gated_act_fp8_backward"
    rows, I = _two(w, "dy", dy)
    _below_2_31(w, 2 * I)
    dev = dy.get_device()
    p = None if plan is None else _plan_arg(w, plan, dev)
    if plan is not None:
        rows = plan.route_slots
    _check(lib().moe_gated_act_fp8_backward(
        _arg(w, "hq", hq, (rows, 2 * I), _BYTE, dev), _arg(w, "hq_sf", hq_sf, (rows, 2 * _nb(I)), _BYTE, dev),
        _arg(w, "dy", dy, (rows, I), _BF16, dev), p, rows, I, activation, swiglu_alpha, swiglu_beta, swiglu_limit,
        _opt(w, "dh", dh, (rows, 2 * I), _BF16, dev), _opt(w, "dq", dq, (rows, 2 * I), _BYTE, dev),
        _opt(w, "dq_sf", dq_sf, (rows, 2 * _nb(I)), _BYTE, dev), _raw_stream(w, dev, stream)), w)
