"""Python binding of libmoe_fp8.so, the MI355X (gfx950) routed FP8 W8A8
block-scale MoE expert path.

Argument marshalling only: every step runs in the library's HIP kernels.
Tensors are torch tensors used for their device memory (``data_ptr()``) and
the current HIP stream; nothing here computes any part of the path.  The
functions carry the C ABI's names (see include/moe_fp8.h) and raise
``MoeError`` on a non-OK status.  If the shared library has not been built,
importing this package raises -- there is no fallback.
"""

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_fp8.so")

MOE_OK = 0
MOE_ERR_NULL, MOE_ERR_SHAPE, MOE_ERR_ALIGN, MOE_ERR_CAPACITY, MOE_ERR_UNSUPPORTED, MOE_ERR_HIP = \
    1, 2, 3, 4, 5, 6
MOE_IDS_I32, MOE_IDS_I64 = 0, 1
MOE_SCALE_FP32, MOE_SCALE_UE8M0 = 0, 1
MOE_F_INTER_UE8M0 = 1
MOE_F_MMA_E8M0 = 2
MOE_F_FP8_GATEUP = 4
MOE_F_SPLITK_SHIFT = 8
MOE_F_GATEUP_PATH_SHIFT = 16
MOE_F_DOWN_PATH_SHIFT = 18
MOE_PATH_AUTO, MOE_PATH_STREAM, MOE_PATH_PERSISTENT, MOE_PATH_COLUMNS = 0, 1, 2, 3
MOE_F_FUSE_SHIFT = 20
MOE_F_W13_PACKED = 0x400000
MOE_FUSE_AUTO, MOE_FUSE_OFF, MOE_FUSE_ON = 0, 1, 2
MOE_DT_BF16, MOE_DT_F16, MOE_DT_F32 = 0, 1, 2
MOE_GMM_FWD, MOE_GMM_DX, MOE_GMM_DW = 0, 1, 2
MOE_ACT_NONE, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_SWIGLU = 0, 1, 2, 3
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1

STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_NULL", 2: "MOE_ERR_SHAPE", 3: "MOE_ERR_ALIGN",
                4: "MOE_ERR_CAPACITY", 5: "MOE_ERR_UNSUPPORTED", 6: "MOE_ERR_HIP"}

EXPORTED = ("moe_plan_capacity", "moe_plan_workspace_size", "moe_plan", "moe_quant_act",
            "moe_plan_quant",
            "moe_fp8_experts_workspace_size", "moe_fp8_experts_workspace_layout",
            "moe_fp8_experts_schedule",
            "moe_fp8_experts", "moe_fp8_gate_up", "moe_fp8_down_reduce", "moe_status_str",
            "moe_last_hip_error", "moe_last_error", "moe_debug_e4m3_encode",
            "moe_debug_count_non_pow2", "moe_fp8_experts_noalloc", "moe_route_plan",
            "moe_w4a8_experts_workspace_size", "moe_w4a8_experts", "moe_prepack_w13_size",
            "moe_prepack_w13", "moe_fp8_layer", "moe_group_mm_workspace_size", "moe_group_mm",
            "moe_group_mm_dx", "moe_group_mm_dw", "moe_fp8_linear_workspace_size",
            "moe_fp8_linear", "moe_route_scored", "moe_route_scored_bwd", "moe_combine", "moe_combine_bwd",
            "moe_quant_i8", "moe_i8_linear_workspace_size", "moe_i8_linear",
            "moe_i8_group_mm_workspace_size", "moe_i8_group_mm", "moe_debug_i8_schedule")

MOE_NOALLOC_SCRATCH_BYTES = 64 << 20


class MoeError(RuntimeError):
    def __init__(self, status, where, detail):
        self.status = status
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run __graft_entry__.build() "
                      "(or python fp8_block_scale_amd/build.py)")

_lib = ctypes.CDLL(LIB_PATH)

_i32, _i64, _u32, _sz, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint32, ctypes.c_size_t, ctypes.c_void_p
_pi64, _psz = ctypes.POINTER(ctypes.c_int64), ctypes.POINTER(ctypes.c_size_t)


def _proto(name, res, *args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = list(args)
    return f


_c = {
    "moe_plan_capacity": _proto("moe_plan_capacity", _i32, _i64, _i32, _i32, _i32, _pi64, _pi64),
    "moe_plan_workspace_size": _proto("moe_plan_workspace_size", _sz, _i64, _i32, _i32, _i32),
    "moe_plan": _proto("moe_plan", _i32, _vp, _i32, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _i64,
                       _vp, _vp, _sz, _vp),
    "moe_quant_act": _proto("moe_quant_act", _i32, _vp, _i64, _i64, _i64, _vp, _vp, _i32, _vp),
    "moe_route_plan": _proto("moe_route_plan", _i32, _vp, _i64, _i32, _i32, _i32, ctypes.c_float, _i32,
                             _vp, _vp, _vp, _i64, _vp, _i64, _vp, _vp, _sz, _vp, _i64, _i64, _vp,
                             _vp, _i32, _vp),
    "moe_plan_quant": _proto("moe_plan_quant", _i32, _vp, _i32, _i64, _i32, _i32, _i32, _vp, _i64, _vp,
                             _i64, _vp, _vp, _sz, _vp, _i64, _i64, _vp, _vp, _i32, _vp),
    "moe_fp8_experts_workspace_size": _proto("moe_fp8_experts_workspace_size", _sz, _i64, _i64,
                                             _i64, _i32, _i32, _i32, _i64, _u32),
    "moe_fp8_experts_workspace_layout": _proto("moe_fp8_experts_workspace_layout", _i32, _i64, _i64,
                                               _i64, _i32, _i32, _i32, _i64, _u32, _psz, _psz),
    "moe_fp8_experts_schedule": _proto("moe_fp8_experts_schedule", _i32, _i64, _i64, _i64, _i32,
                                       _i32, _i32, _i64, _u32, _vp),
    "moe_fp8_experts": _proto("moe_fp8_experts", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                              _vp, _i64, _i64, _i64, _i32, _i32, _i32, _i64, _u32, _vp, _vp, _sz,
                              _vp),
    "moe_fp8_layer": _proto("moe_fp8_layer", _i32, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _vp,
                            _vp, _i64, _i64, _i64, _i32, _i32, _i32, _vp, _i64, _vp, _i64, _vp,
                            _vp, _vp, _vp, _sz, _u32, _vp, _vp, _sz, _vp),
    "moe_fp8_gate_up": _proto("moe_fp8_gate_up", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                              _i64, _i32, _i32, _i32, _i64, _u32, _vp, _sz, _vp),
    "moe_fp8_down_reduce": _proto("moe_fp8_down_reduce", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                                  _i64, _i64, _i32, _i32, _i32, _i64, _u32, _vp, _vp, _sz, _vp),
    "moe_fp8_experts_noalloc": _proto("moe_fp8_experts_noalloc", _i32, _vp, _vp, _vp, _vp, _vp,
                                      _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i32, _i32,
                                      _i32, _i64, _u32, _vp, _vp),
    "moe_w4a8_experts_workspace_size": _proto("moe_w4a8_experts_workspace_size", _sz, _i64, _i64,
                                              _i64, _i32, _i32, _i32, _i64, _u32),
    "moe_w4a8_experts": _proto("moe_w4a8_experts", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp,
                               _vp, _vp, _i64, _i64, _i64, _i32, _i32, _i32, _i64, _u32, _vp, _vp,
                               _sz, _vp),
    "moe_prepack_w13_size": _proto("moe_prepack_w13_size", _sz, _i64, _i64, _i64),
    "moe_prepack_w13": _proto("moe_prepack_w13", _i32, _vp, _i64, _i64, _i64, _vp, _vp),
    "moe_group_mm_workspace_size": _proto("moe_group_mm_workspace_size", _sz, _i32, _i64, _i64, _i64,
                                          _i32, _i32, _i32, _i64, _i32),
    "moe_group_mm": _proto("moe_group_mm", _i32, _vp, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _i64, _i64,
                           _i64, _i32, _i32, _i32, _i64, _vp, _i64, _vp, _sz, _vp),
    "moe_group_mm_dx": _proto("moe_group_mm_dx", _i32, _vp, _i64, _vp, _i32, _vp, _vp, _vp, _i64, _i64,
                              _i64, _i32, _i32, _i32, _i64, _vp, _i64, _i32, _vp, _sz, _vp),
    "moe_group_mm_dw": _proto("moe_group_mm_dw", _i32, _vp, _i64, _vp, _i64, _i32, _i32, _vp, _vp, _vp,
                              _i64, _i64, _i64, _i32, _i32, _i32, _i64, _vp, _i32, _i32, _vp, _sz,
                              _vp),
    "moe_fp8_linear_workspace_size": _proto("moe_fp8_linear_workspace_size", _sz, _i64, _i64, _i64,
                                            _i32),
    "moe_fp8_linear": _proto("moe_fp8_linear", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64,
                             _i64, _i32, _vp, _i64, _vp, _sz, _vp),
    "moe_route_scored": _proto("moe_route_scored", _i32, _vp, _i32, _i64, _i64, _i32, _i32, _i32, _vp, _i32,
                               _i32, _i32, _i32, ctypes.c_float, _i32, _vp, _vp, _vp),
    "moe_route_scored_bwd": _proto("moe_route_scored_bwd", _i32, _vp, _i32, _i64, _i64, _i32, _i32, _i32, _i32,
                                   ctypes.c_float, _vp, _vp, _vp, _i64, _vp),
    "moe_combine": _proto("moe_combine", _i32, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _vp, _i64, _i64, _i64,
                          _i32, _vp, _i64, _vp),
    "moe_combine_bwd": _proto("moe_combine_bwd", _i32, _vp, _i64, _vp, _i64, _i32, _vp, _vp, _i32, _i32, _i64,
                              _i64, _i32, _vp, _i64, _vp, _vp),
    "moe_quant_i8": _proto("moe_quant_i8", _i32, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp),
    "moe_i8_linear_workspace_size": _proto("moe_i8_linear_workspace_size", _sz, _i64, _i64, _i64, _i32),
    "moe_i8_linear": _proto("moe_i8_linear", _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i32,
                            _vp, _i32, _i64, _vp, _sz, _vp),
    "moe_i8_group_mm_workspace_size": _proto("moe_i8_group_mm_workspace_size", _sz, _i64, _i64, _i64, _i32,
                                             _i32, _i32, _i64, _i32, _i32),
    "moe_i8_group_mm": _proto("moe_i8_group_mm", _i32, _vp, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _i64,
                              _i64, _i64, _i32, _i32, _i32, _i64, _i32, _vp, _i32, _i64, _vp, _sz, _vp),
    "moe_debug_i8_schedule": _proto("moe_debug_i8_schedule", _i32, _i64, _i64, _i64, _i32, _i32, _i32, _i64, _i32,
                                    _vp),
    "moe_status_str": _proto("moe_status_str", ctypes.c_char_p, _i32),
    "moe_last_hip_error": _proto("moe_last_hip_error", ctypes.c_char_p),
    "moe_last_error": _proto("moe_last_error", ctypes.c_char_p),
    "moe_debug_e4m3_encode": _proto("moe_debug_e4m3_encode", _i32, _vp, _vp, _i64, _vp),
    "moe_debug_count_non_pow2": _proto("moe_debug_count_non_pow2", _i32, _vp, _i64, _vp, _vp),
}


def _check(st, where):
    if st != MOE_OK:
        raise MoeError(st, where, _c["moe_last_hip_error"]().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


# ------------------------------------------------------------------ plan --

def moe_plan_capacity(M, top_k, E, block_m):
    sc, bc = ctypes.c_int64(), ctypes.c_int64()
    _check(_c["moe_plan_capacity"](M, top_k, E, block_m, ctypes.byref(sc), ctypes.byref(bc)),
           "moe_plan_capacity")
    return sc.value, bc.value


def moe_plan_workspace_size(M, top_k, E, block_m):
    return _c["moe_plan_workspace_size"](M, top_k, E, block_m)


def _plan_args(topk_ids, E, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded,
               workspace):
    M, top_k = topk_ids.shape
    if topk_ids.dtype == torch.int32:
        dt = MOE_IDS_I32
    elif topk_ids.dtype == torch.int64:
        dt = MOE_IDS_I64
    else:
        raise TypeError("topk_ids must be int32 or int64")
    assert topk_ids.is_contiguous() and sorted_token_ids.dtype == torch.int32
    assert expert_ids.dtype == torch.int32 and num_tokens_post_padded.dtype == torch.int32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    return (_ptr(topk_ids), dt, M, top_k, E, block_m, _ptr(sorted_token_ids), sorted_token_ids.numel(),
            _ptr(expert_ids), expert_ids.numel(), _ptr(num_tokens_post_padded), _ptr(workspace),
            ws_bytes)


def _quant_args(x_bf16, x_q, x_s):
    assert x_bf16.dtype == torch.bfloat16 and x_bf16.dim() == 2 and x_bf16.stride(1) == 1
    M, K = x_bf16.shape
    assert x_q.dtype == torch.uint8 and x_q.is_contiguous() and tuple(x_q.shape) == (M, K)
    assert x_s.dtype == torch.float32 and x_s.is_contiguous() and tuple(x_s.shape) == (M, K // 128)
    return M, K, x_bf16.stride(0)


def moe_plan(topk_ids, E, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded,
             workspace=None, stream=None):
    """topk_ids [M, top_k] int32/int64 (device); outputs are preallocated int32 tensors."""
    args = _plan_args(topk_ids, E, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded,
                      workspace)
    _check(_c["moe_plan"](*args, _stream(stream)), "moe_plan")


def moe_plan_quant(topk_ids, E, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded,
                   x_bf16, x_q, x_s, scale_mode=MOE_SCALE_FP32, workspace=None, stream=None):
    """moe_plan and moe_quant_act in one call (one launch fewer); same outputs."""
    args = _plan_args(topk_ids, E, block_m, sorted_token_ids, expert_ids, num_tokens_post_padded,
                      workspace)
    M, K, ld = _quant_args(x_bf16, x_q, x_s)
    assert M == topk_ids.shape[0], "x_bf16 and topk_ids disagree on M"
    _check(_c["moe_plan_quant"](*args, _ptr(x_bf16), K, ld, _ptr(x_q), _ptr(x_s), scale_mode,
                                _stream(stream)), "moe_plan_quant")


def moe_route_plan(router_logits, top_k, n_shared, routed_scaling, block_m, topk_ids,
                   topk_weights, sorted_token_ids, expert_ids, num_tokens_post_padded,
                   workspace=None, x_bf16=None, x_q=None, x_s=None, scale_mode=MOE_SCALE_FP32,
                   stream=None):
    """Router (softmax top-k, routed scaling, optional shared expert) and the
    plan in the plan's launches; with x_bf16 also the activation quantisation.
    router_logits [M, E_routed] fp32; topk_ids int32 / topk_weights fp32
    [M, top_k + n_shared] out; the plan buffers sized for E_routed + n_shared
    experts and top_k + n_shared routes per token."""
    assert router_logits.dtype == torch.float32 and router_logits.is_contiguous()
    M, Er = router_logits.shape
    kk = top_k + n_shared
    assert topk_ids.dtype == torch.int32 and topk_ids.is_contiguous() and tuple(topk_ids.shape) == (M, kk)
    assert topk_weights.dtype == torch.float32 and topk_weights.is_contiguous()
    assert tuple(topk_weights.shape) == (M, kk)
    assert sorted_token_ids.dtype == torch.int32 and expert_ids.dtype == torch.int32
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    if x_bf16 is not None:
        Mx, K, ld = _quant_args(x_bf16, x_q, x_s)
        assert Mx == M, "x_bf16 and router_logits disagree on M"
    else:
        K, ld = 0, 0
    _check(_c["moe_route_plan"](_ptr(router_logits), M, Er, top_k, n_shared, routed_scaling, block_m,
                                _ptr(topk_ids), _ptr(topk_weights), _ptr(sorted_token_ids),
                                sorted_token_ids.numel(), _ptr(expert_ids), expert_ids.numel(),
                                _ptr(num_tokens_post_padded), _ptr(workspace), ws_bytes,
                                _ptr(x_bf16), K, ld, _ptr(x_q), _ptr(x_s), scale_mode,
                                _stream(stream)), "moe_route_plan")


# ------------------------------------------------------------- quant act --

def moe_quant_act(x_bf16, x_q, x_s, scale_mode=MOE_SCALE_FP32, stream=None):
    """x_bf16 [M, K] bf16 (row stride may exceed K); x_q uint8 [M, K]; x_s fp32 [M, K/128]."""
    M, K, ld = _quant_args(x_bf16, x_q, x_s)
    _check(_c["moe_quant_act"](_ptr(x_bf16), M, K, ld, _ptr(x_q), _ptr(x_s), scale_mode,
                               _stream(stream)), "moe_quant_act")


def moe_debug_e4m3_encode(inp, out, stream=None):
    assert inp.dtype == torch.float32 and out.dtype == torch.uint8 and inp.numel() == out.numel()
    _check(_c["moe_debug_e4m3_encode"](_ptr(inp), _ptr(out), inp.numel(), _stream(stream)),
           "moe_debug_e4m3_encode")


def moe_debug_count_non_pow2(scales, count, stream=None):
    """count[0] = how many of `scales` (FP32, device) are not powers of two in
    [2^-126, 2^127] -- the values MOE_F_MMA_E8M0 cannot take as they are."""
    assert scales.dtype == torch.float32 and scales.is_contiguous()
    assert count.dtype in (torch.int32, torch.uint32) and count.numel() >= 1
    _check(_c["moe_debug_count_non_pow2"](_ptr(scales), scales.numel(), _ptr(count), _stream(stream)),
           "moe_debug_count_non_pow2")


# --------------------------------------------------------------- experts --

def moe_fp8_experts_workspace_size(M, K, I, E, top_k, block_m, sorted_cap, flags=0):
    return _c["moe_fp8_experts_workspace_size"](M, K, I, E, top_k, block_m, sorted_cap, flags)


def moe_fp8_experts_workspace_layout(M, K, I, E, top_k, block_m, sorted_cap, flags=0):
    a, b = ctypes.c_size_t(), ctypes.c_size_t()
    _check(_c["moe_fp8_experts_workspace_layout"](M, K, I, E, top_k, block_m, sorted_cap, flags,
                                                  ctypes.byref(a), ctypes.byref(b)),
           "moe_fp8_experts_workspace_layout")
    return a.value, b.value


def moe_fp8_experts_schedule(M, K, I, E, top_k, block_m, sorted_cap, flags=0):
    """(gate/up kernel (0 per block, 1 persistent, 2 split over intermediate-column
    slices), down kernel (0 per block, 1 persistent, 2 split over output columns),
    split-K factor, K-blocks per split, steps 3-5 as one launch)."""
    info = (ctypes.c_int32 * 5)()
    _check(_c["moe_fp8_experts_schedule"](M, K, I, E, top_k, block_m, sorted_cap, flags, info),
           "moe_fp8_experts_schedule")
    return int(info[0]), int(info[1]), int(info[2]), int(info[3]), bool(info[4])


def moe_fp8_layer(x_bf16, topk_ids, topk_weights, w13, w13_s, w2, w2_s, block_m, sorted_token_ids,
                  expert_ids, num_tokens_post_padded, x_q, x_s, out_bf16, workspace, flags=0,
                  scale_mode=MOE_SCALE_FP32, plan_workspace=None, stream=None):
    """All five steps (moe_plan_quant then moe_fp8_experts) in one call, with
    one launch fewer at decode sizes; same outputs."""
    pa = _plan_args(topk_ids, w13.shape[0], block_m, sorted_token_ids, expert_ids,
                    num_tokens_post_padded, plan_workspace)
    ids_ptr, dt, M, top_k, E, _, s_ptr, s_cap, e_ptr, e_cap, n_ptr, pw_ptr, pw_bytes = pa
    Mx, K, ld = _quant_args(x_bf16, x_q, x_s)
    assert Mx == M, "x_bf16 and topk_ids disagree on M"
    I = w13.shape[1] // 2
    for t in (w13, w13_s, w2, w2_s, topk_weights, out_bf16, workspace):
        assert t.is_contiguous()
    assert out_bf16.dtype == torch.bfloat16 and topk_weights.dtype == torch.float32
    _check(_c["moe_fp8_layer"](_ptr(x_bf16), ld, scale_mode, ids_ptr, dt, _ptr(topk_weights),
                               _ptr(w13), _ptr(w13_s), _ptr(w2), _ptr(w2_s), M, K, I, E, top_k,
                               block_m, s_ptr, s_cap, e_ptr, e_cap, n_ptr, _ptr(x_q), _ptr(x_s),
                               pw_ptr, pw_bytes, flags, _ptr(out_bf16), _ptr(workspace),
                               workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_fp8_layer")


def moe_fp8_experts(x_q, x_s, w13, w13_s, w2, w2_s, topk_weights, sorted_token_ids, expert_ids,
                    num_tokens_post_padded, top_k, block_m, out_bf16, workspace, flags=0,
                    stream=None):
    """Steps 3-5; accumulates into out_bf16 [M, K]."""
    M, K = x_q.shape
    E, twoI, _ = w13.shape
    I = twoI // 2
    for t in (x_q, x_s, w13, w13_s, w2, w2_s, topk_weights, sorted_token_ids, expert_ids,
              out_bf16, workspace):
        assert t.is_contiguous()
    assert out_bf16.dtype == torch.bfloat16 and topk_weights.dtype == torch.float32
    # the kernels read expert ids of blocks below P only; P / block_m is at
    # most the plan's block capacity and at most sorted_cap / block_m
    assert expert_ids.numel() >= min(moe_plan_capacity(M, top_k, E, block_m)[1],
                                     sorted_token_ids.numel() // block_m), \
        "expert_ids shorter than the plan can need"
    _check(_c["moe_fp8_experts"](_ptr(x_q), _ptr(x_s), _ptr(w13), _ptr(w13_s), _ptr(w2),
                                 _ptr(w2_s), _ptr(topk_weights), _ptr(sorted_token_ids),
                                 _ptr(expert_ids), _ptr(num_tokens_post_padded), M, K, I, E, top_k,
                                 block_m, sorted_token_ids.numel(), flags, _ptr(out_bf16),
                                 _ptr(workspace), workspace.numel() * workspace.element_size(),
                                 _stream(stream)),
           "moe_fp8_experts")


def moe_prepack_w13_size(E, I, K):
    return _c["moe_prepack_w13_size"](E, I, K)


def moe_prepack_w13(w13, out=None, stream=None):
    """W13 [E, 2I, K] uint8 -> its packed tile layout (a new uint8 tensor of
    the same size unless `out` is given); pass MOE_F_W13_PACKED with it."""
    E, twoI, K = w13.shape
    assert w13.dtype == torch.uint8 and w13.is_contiguous()
    if out is None:
        out = torch.empty(moe_prepack_w13_size(E, twoI // 2, K), dtype=torch.uint8,
                          device=w13.device)
    assert out.is_contiguous() and out.numel() == moe_prepack_w13_size(E, twoI // 2, K)
    _check(_c["moe_prepack_w13"](_ptr(w13), E, twoI // 2, K, _ptr(out), _stream(stream)),
           "moe_prepack_w13")
    return out.view(E, twoI, K)


def moe_w4a8_experts_workspace_size(M, K, I, E, top_k, block_m, sorted_cap, flags=0):
    return _c["moe_w4a8_experts_workspace_size"](M, K, I, E, top_k, block_m, sorted_cap, flags)


def moe_w4a8_experts(x_q, x_s, w13, w13_e, w2, w2_e, topk_weights, sorted_token_ids, expert_ids,
                     num_tokens_post_padded, top_k, block_m, out_bf16, workspace, flags=0,
                     stream=None):
    """Steps 3-5 with E2M1 weights (w13 [E, 2I, K/2], w13_e [E, 2I, K/32],
    w2 [E, K, I/2], w2_e [E, K, I/32], all uint8); accumulates into
    out_bf16 [M, K]."""
    M, K = x_q.shape
    E, twoI, half = w13.shape
    I = twoI // 2
    assert 2 * half == K and w2.shape == (E, K, I // 2)
    assert w13_e.shape == (E, twoI, K // 32) and w2_e.shape == (E, K, I // 32)
    for t in (x_q, x_s, w13, w13_e, w2, w2_e, topk_weights, sorted_token_ids, expert_ids,
              out_bf16, workspace):
        assert t.is_contiguous()
    assert w13.dtype == w13_e.dtype == w2.dtype == w2_e.dtype == torch.uint8
    assert out_bf16.dtype == torch.bfloat16 and topk_weights.dtype == torch.float32
    assert expert_ids.numel() >= min(moe_plan_capacity(M, top_k, E, block_m)[1],
                                     sorted_token_ids.numel() // block_m), \
        "expert_ids shorter than the plan can need"
    _check(_c["moe_w4a8_experts"](_ptr(x_q), _ptr(x_s), _ptr(w13), _ptr(w13_e), _ptr(w2),
                                  _ptr(w2_e), _ptr(topk_weights), _ptr(sorted_token_ids),
                                  _ptr(expert_ids), _ptr(num_tokens_post_padded), M, K, I, E, top_k,
                                  block_m, sorted_token_ids.numel(), flags, _ptr(out_bf16),
                                  _ptr(workspace), workspace.numel() * workspace.element_size(),
                                  _stream(stream)),
           "moe_w4a8_experts")


def moe_fp8_experts_noalloc(x_q, x_s, w13, w13_s, w2, w2_s, topk_weights, sorted_token_ids,
                            expert_ids, num_tokens_post_padded, top_k, block_m, out_bf16, flags=0,
                            stream=None):
    """moe_fp8_experts with the library's static per-device scratch as the
    workspace (no allocation anywhere); raises MoeError (MOE_ERR_CAPACITY)
    for sizes whose workspace exceeds MOE_NOALLOC_SCRATCH_BYTES."""
    M, K = x_q.shape
    E, twoI, _ = w13.shape
    for t in (x_q, x_s, w13, w13_s, w2, w2_s, topk_weights, sorted_token_ids, expert_ids,
              out_bf16):
        assert t.is_contiguous()
    assert out_bf16.dtype == torch.bfloat16 and topk_weights.dtype == torch.float32
    _check(_c["moe_fp8_experts_noalloc"](_ptr(x_q), _ptr(x_s), _ptr(w13), _ptr(w13_s), _ptr(w2),
                                         _ptr(w2_s), _ptr(topk_weights), _ptr(sorted_token_ids),
                                         _ptr(expert_ids), _ptr(num_tokens_post_padded), M, K,
                                         twoI // 2, E, top_k, block_m, sorted_token_ids.numel(),
                                         flags, _ptr(out_bf16), _stream(stream)),
           "moe_fp8_experts_noalloc")


def moe_fp8_gate_up(x_q, x_s, w13, w13_s, sorted_token_ids, expert_ids, num_tokens_post_padded,
                    top_k, block_m, workspace, flags=0, stream=None):
    """Steps 3-4 into the workspace (see MoeLayerBuffers.intermediate)."""
    M, K = x_q.shape
    E, twoI, _ = w13.shape
    _check(_c["moe_fp8_gate_up"](_ptr(x_q), _ptr(x_s), _ptr(w13), _ptr(w13_s), _ptr(sorted_token_ids),
                                 _ptr(expert_ids), _ptr(num_tokens_post_padded), M, K, twoI // 2, E,
                                 top_k, block_m, sorted_token_ids.numel(), flags, _ptr(workspace),
                                 workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_fp8_gate_up")


def moe_fp8_down_reduce(w2, w2_s, topk_weights, sorted_token_ids, expert_ids,
                        num_tokens_post_padded, top_k, block_m, out_bf16, workspace, flags=0,
                        stream=None):
    """Step 5: out_bf16 += weighted down projections of the workspace rows."""
    E, K, I = w2.shape
    M = out_bf16.shape[0]
    _check(_c["moe_fp8_down_reduce"](_ptr(w2), _ptr(w2_s), _ptr(topk_weights), _ptr(sorted_token_ids),
                                     _ptr(expert_ids), _ptr(num_tokens_post_padded), M, K, I, E,
                                     top_k, block_m, sorted_token_ids.numel(), flags,
                                     _ptr(out_bf16), _ptr(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_fp8_down_reduce")


# ------------------------------------------------- 16-bit grouped products --

_DT = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16, torch.float32: MOE_DT_F32}
_DT16 = {torch.bfloat16: MOE_DT_BF16, torch.float16: MOE_DT_F16}


def _need(cond, where, what):
    """Argument check of the entry points below: raises as the library does
    for the sizes it sees (these are the ones it cannot see)."""
    if not cond:
        raise MoeError(MOE_ERR_SHAPE, where, what)


# The handle of a device's current stream; torch's own accessor of the handle
# where it has one (0.1 against 1.1 us for the stream object, which counts in a
# call of a few microseconds).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(where, stream, tensors, *args):
    """Calls the entry point on the stream given (default: the current one of
    the tensors' device) after a check that all tensors (None: absent) and the
    stream are on one GPU; that GPU is the current device during the call."""
    dev = tensors[0].get_device()
    if dev < 0:
        raise MoeError(MOE_ERR_SHAPE, where, "tensors must be on a GPU")
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise MoeError(MOE_ERR_SHAPE, where, "tensors are on different devices")
    if stream is None:
        raw = _raw_stream(dev)
    else:
        if stream.device_index != dev:
            raise MoeError(MOE_ERR_SHAPE, where, "the stream is on another device than the tensors")
        raw = stream.cuda_stream
    if _current_device() == dev:
        st = _c[where](*args, raw)
    else:
        with torch.cuda.device(dev):
            st = _c[where](*args, raw)
    if st != MOE_OK:
        _check(st, where)


def _rows_arg(where, name, t, dtype, cols):
    """A 2-d operand with unit column stride: (pointer, leading dimension)."""
    if t.dim() != 2 or t.dtype != dtype:
        raise MoeError(MOE_ERR_SHAPE, where, f"{name} must be a 2-d {dtype} tensor")
    rows, n = t.shape
    if n != cols:
        raise MoeError(MOE_ERR_SHAPE, where, f"{name} must have {cols} columns")
    ld, unit = t.stride()
    if unit != 1 and n != 1:
        raise MoeError(MOE_ERR_SHAPE, where, f"{name} must have unit column stride")
    if rows <= 1:                       # a single row may carry any stride
        return t.data_ptr(), n
    if ld < n:
        raise MoeError(MOE_ERR_SHAPE, where, f"rows of {name} overlap")
    return t.data_ptr(), ld


def _group_plan(where, sorted_token_ids, expert_ids, num_tokens_post_padded, R, top_k, E, block_m):
    """The plan's pointers and the length that the kernels may trust."""
    for t in (sorted_token_ids, expert_ids, num_tokens_post_padded):
        if t.dtype is not torch.int32 or not t.is_contiguous():
            raise MoeError(MOE_ERR_SHAPE, where, "the plan must be contiguous int32")
    if num_tokens_post_padded.numel() < 1:
        raise MoeError(MOE_ERR_SHAPE, where, "num_tokens_post_padded is empty")
    if top_k < 1 or R % top_k != 0:
        raise MoeError(MOE_ERR_SHAPE, where, "the routes are no multiple of top_k")
    # A block's expert is read wherever the device's plan length says there is
    # one, within sorted_cap: so that is cut to the blocks that expert_ids has.
    # No plan is longer than any routing of these routes needs.
    cap = sorted_token_ids.numel()
    if block_m > 0 and cap % block_m == 0:
        have = expert_ids.numel()
        if have < min(cap // block_m, -(-(R + min(E, R) * (block_m - 1)) // block_m)):
            raise MoeError(MOE_ERR_SHAPE, where, "expert_ids shorter than the plan can need")
        cap = min(cap, have * block_m)
    return (sorted_token_ids.data_ptr(), expert_ids.data_ptr(), num_tokens_post_padded.data_ptr()), cap


def _x_rows(where, name, t, R, top_k, per_route):
    """Whether x / dx has one row per route (else one per token): as told, or
    (None) as its rows say, one per token if top_k is 1."""
    rows = t.shape[0]
    if per_route is None:
        per_route = rows * top_k != R
    if rows != (R if per_route else R // top_k):
        raise MoeError(MOE_ERR_SHAPE, where, name + " must have one row per token or per route")
    return 1 if per_route else 0


def _ws(where, workspace):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise MoeError(MOE_ERR_SHAPE, where, "workspace must be contiguous")
    return workspace.data_ptr(), workspace.nbytes


def moe_group_mm_workspace_size(op, M, K, N, E, top_k, block_m, sorted_cap, x_per_route=False):
    return _c["moe_group_mm_workspace_size"](op, M, K, N, E, top_k, block_m, sorted_cap,
                                             int(bool(x_per_route)))


def moe_group_mm(x, w, sorted_token_ids, expert_ids, num_tokens_post_padded, top_k, block_m, out,
                 workspace=None, stream=None, x_per_route=None):
    """out[r] = x[t(r)] @ w[e(r)]^T for every route r of the plan.  w [E, N, K]
    bf16 or fp16; out [M * top_k, N]; x [M, K] (t(r) = r // top_k) or
    [M * top_k, K] (t(r) = r), all of w's type; x_per_route tells which (None:
    by x's rows).  Rows of masked routes are left as they were."""
    where = "moe_group_mm"
    _need(w.dim() == 3 and w.is_contiguous() and w.dtype in (torch.bfloat16, torch.float16), where,
          "w must be a contiguous 3-d bf16 or fp16 tensor")
    E, N, K = w.shape
    xp, ld_x = _rows_arg(where, "x", x, w.dtype, K)
    yp, ld_y = _rows_arg(where, "out", out, w.dtype, N)
    R = out.shape[0]
    plan, cap = _group_plan(where, sorted_token_ids, expert_ids, num_tokens_post_padded, R, top_k, E, block_m)
    per_route = _x_rows(where, "x", x, R, top_k, x_per_route)
    _launch(where, stream, (x, w, out, sorted_token_ids, expert_ids, num_tokens_post_padded, workspace),
            xp, ld_x, per_route, w.data_ptr(), _DT[w.dtype], *plan, R // top_k, K, N, E, top_k, block_m,
            cap, yp, ld_y, *_ws(where, workspace))


def moe_group_mm_dx(dy, w, sorted_token_ids, expert_ids, num_tokens_post_padded, top_k, block_m, dx,
                    workspace=None, stream=None, x_per_route=None):
    """The gradient of moe_group_mm by x: dx [M, K] (the gradients of a
    token's routes added) or [M * top_k, K] (one row per route; rows of masked
    routes left as they were) from dy [M * top_k, N] and w [E, N, K]."""
    where = "moe_group_mm_dx"
    _need(w.dim() == 3 and w.is_contiguous() and w.dtype in (torch.bfloat16, torch.float16), where,
          "w must be a contiguous 3-d bf16 or fp16 tensor")
    E, N, K = w.shape
    yp, ld_y = _rows_arg(where, "dy", dy, w.dtype, N)
    xp, ld_x = _rows_arg(where, "dx", dx, w.dtype, K)
    R = dy.shape[0]
    plan, cap = _group_plan(where, sorted_token_ids, expert_ids, num_tokens_post_padded, R, top_k, E, block_m)
    per_route = _x_rows(where, "dx", dx, R, top_k, x_per_route)
    _launch(where, stream, (dy, w, dx, sorted_token_ids, expert_ids, num_tokens_post_padded, workspace),
            yp, ld_y, w.data_ptr(), _DT[w.dtype], *plan, R // top_k, K, N, E, top_k, block_m,
            cap, xp, ld_x, per_route, *_ws(where, workspace))


def moe_group_mm_dw(dy, x, sorted_token_ids, expert_ids, num_tokens_post_padded, top_k, block_m, dw,
                    workspace=None, accumulate=False, stream=None, x_per_route=None):
    """The gradient of moe_group_mm by w: dw [E, N, K] (of dy's type or fp32)
    from dy [M * top_k, N] and x [M, K] or [M * top_k, K]; accumulate adds to
    dw instead of overwriting it."""
    where = "moe_group_mm_dw"
    _need(dy.dtype in (torch.bfloat16, torch.float16), where, "dy must be bf16 or fp16")
    _need(dw.dim() == 3 and dw.is_contiguous() and dw.dtype in (dy.dtype, torch.float32), where,
          "dw must be a contiguous 3-d tensor of dy's type or fp32")
    E, N, K = dw.shape
    yp, ld_y = _rows_arg(where, "dy", dy, dy.dtype, N)
    xp, ld_x = _rows_arg(where, "x", x, dy.dtype, K)
    R = dy.shape[0]
    plan, cap = _group_plan(where, sorted_token_ids, expert_ids, num_tokens_post_padded, R, top_k, E, block_m)
    per_route = _x_rows(where, "x", x, R, top_k, x_per_route)
    _launch(where, stream, (dy, x, dw, sorted_token_ids, expert_ids, num_tokens_post_padded, workspace),
            yp, ld_y, xp, ld_x, per_route, _DT[dy.dtype], *plan, R // top_k, K, N, E, top_k, block_m,
            cap, dw.data_ptr(), _DT[dw.dtype], int(bool(accumulate)),
            *_ws(where, workspace))


# --------------------------------------------------------- dense product --

def moe_fp8_linear_workspace_size(M, N, K, act=MOE_ACT_NONE):
    return _c["moe_fp8_linear_workspace_size"](M, N, K, act)


def moe_fp8_linear(x_q, x_s, w, w_s, out, bias=None, residual=None, act=MOE_ACT_NONE, workspace=None,
                   stream=None):
    """out = act(x w^T + bias) + residual from FP8 block-scaled codes: x_q
    [M, K] uint8 with x_s [M, K/128] fp32 (moe_quant_act's), w [N, K] uint8
    with w_s [ceil(N/128), K/128] fp32, bias [N] fp32, residual and out bf16
    [M, N] -- [M, N/2] with MOE_ACT_SWIGLU, whose w holds the gate rows, then
    the up rows.  residual may be out itself."""
    where = "moe_fp8_linear"
    for n, t, dt in (("x_q", x_q, torch.uint8), ("x_s", x_s, torch.float32), ("w", w, torch.uint8),
                     ("w_s", w_s, torch.float32)):
        if t.dim() != 2 or t.dtype != dt or not t.is_contiguous():
            raise MoeError(MOE_ERR_SHAPE, where, f"{n} must be a contiguous 2-d {dt} tensor")
    M, K = x_q.shape
    N = w.shape[0]
    _need(w.shape[1] == K, where, "w and x_q disagree on K")
    _need(K % 128 == 0 and tuple(x_s.shape) == (M, K // 128), where, "x_s must be [M, K / 128]")
    _need(tuple(w_s.shape) == ((N + 127) // 128, K // 128), where, "w_s must be [ceil(N / 128), K / 128]")
    _need(bias is None or (bias.dtype == torch.float32 and bias.is_contiguous()
                           and tuple(bias.shape) == (N,)), where, "bias must be contiguous fp32 [N]")
    n_out = N // 2 if act == MOE_ACT_SWIGLU else N
    op, ld_out = _rows_arg(where, "out", out, torch.bfloat16, n_out)
    _need(out.shape[0] == M, where, "out and x_q disagree on M")
    rp, ld_res = None, 0
    if residual is not None:
        rp, ld_res = _rows_arg(where, "residual", residual, torch.bfloat16, n_out)
        _need(residual.shape[0] == M, where, "residual and x_q disagree on M")
    _launch(where, stream, (x_q, x_s, w, w_s, out, bias, residual, workspace), x_q.data_ptr(),
            x_s.data_ptr(), w.data_ptr(), w_s.data_ptr(), None if bias is None else bias.data_ptr(), rp,
            ld_res, M, N, K, act, op, ld_out, *_ws(where, workspace))


# ------------------------------------------------------ routing by scores --

def _slots(where, name, t, dtype, shape):
    """The pointer of a dense operand of this type and shape."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise MoeError(MOE_ERR_SHAPE, where, f"{name} must be a contiguous {dtype} tensor of shape {shape}")
    return t.data_ptr()


def _16bit(where, name, t):
    """(rows, columns, pointer, leading dimension) of a bf16 or fp16 operand."""
    if t.dim() != 2 or t.dtype not in _DT16:
        raise MoeError(MOE_ERR_SHAPE, where, f"{name} must be a 2-d bf16 or fp16 tensor")
    rows, cols = t.shape
    return rows, cols, *_rows_arg(where, name, t, t.dtype, cols)


def moe_route_scored(router_logits, top_k, topk_ids, topk_weights, score=MOE_SCORE_SIGMOID, bias=None,
                     n_group=1, topk_group=1, group_top=2, renorm=True, routed_scaling=1.0, n_shared=0,
                     stream=None):
    """Experts by scores: router_logits [M, E_routed] fp32, bf16 or fp16 ->
    topk_ids int32 and topk_weights fp32 [M, top_k + n_shared].  Scores are the
    logits' sigmoids or softmax; score + bias [E_routed] fp32 decides who is
    chosen, within the topk_group of n_group groups with the largest sums of
    group_top scores; weights are the chosen scores, divided by their sum
    (renorm), times routed_scaling; a shared expert follows with weight 1.
    Slots that no expert is left for (logits of -infinity) hold id -1."""
    where = "moe_route_scored"
    _need(router_logits.dim() == 2 and router_logits.dtype in _DT, where,
          "router_logits must be a 2-d fp32, bf16 or fp16 tensor")
    M, E = router_logits.shape
    lp, ld = _rows_arg(where, "router_logits", router_logits, router_logits.dtype, E)
    shape = (M, top_k + n_shared)
    bp = None if bias is None else _slots(where, "bias", bias, torch.float32, (E,))
    ip = _slots(where, "topk_ids", topk_ids, torch.int32, shape)
    wp = _slots(where, "topk_weights", topk_weights, torch.float32, shape)
    _launch(where, stream, (router_logits, bias, topk_ids, topk_weights), lp, _DT[router_logits.dtype], M, ld,
            E, top_k, score, bp, n_group, topk_group, group_top, int(bool(renorm)), routed_scaling, n_shared,
            ip, wp)


def moe_route_scored_bwd(router_logits, topk_ids, d_weights, d_logits, score=MOE_SCORE_SIGMOID, renorm=True,
                         routed_scaling=1.0, stream=None):
    """The gradient of moe_route_scored's weights by the logits, the choice
    taken as fixed: d_logits [M, E_routed] of the logits' type from topk_ids
    int32 and d_weights fp32 [M, top_k + n_shared]."""
    where = "moe_route_scored_bwd"
    _need(router_logits.dim() == 2 and router_logits.dtype in _DT, where,
          "router_logits must be a 2-d fp32, bf16 or fp16 tensor")
    M, E = router_logits.shape
    lp, ld = _rows_arg(where, "router_logits", router_logits, router_logits.dtype, E)
    dp, ld_d = _rows_arg(where, "d_logits", d_logits, router_logits.dtype, E)
    _need(d_logits.shape[0] == M and topk_ids.dim() == 2 and topk_ids.shape[0] == M, where,
          "router_logits, topk_ids and d_logits disagree on M")
    shape = tuple(topk_ids.shape)
    ip = _slots(where, "topk_ids", topk_ids, torch.int32, shape)
    wp = _slots(where, "d_weights", d_weights, torch.float32, shape)
    _launch(where, stream, (router_logits, topk_ids, d_weights, d_logits), lp, _DT[router_logits.dtype], M, ld,
            E, shape[1], score, int(bool(renorm)), routed_scaling, ip, wp, dp, ld_d)


# ------------------------------------------------- weighted sum of routes --

_IDS = {torch.int32: MOE_IDS_I32, torch.int64: MOE_IDS_I64}


def _combine_args(where, y, topk_weights, topk_ids, E):
    """(M, top_k, K, y's pointer and leading dimension, ids' pointer and type)"""
    R, K, yp, ld_y = _16bit(where, "y", y)
    _need(topk_weights.dim() == 2, where, "topk_weights must be [M, top_k]")
    M, k = topk_weights.shape
    _need(R == M * k, where, "y must have one row per route")
    ip, dt = None, MOE_IDS_I32
    if topk_ids is not None:
        dt = _IDS.get(topk_ids.dtype)
        _need(dt is not None, where, "topk_ids must be int32 or int64")
        _need(E is not None, where, "topk_ids need E")
        ip = _slots(where, "topk_ids", topk_ids, topk_ids.dtype, (M, k))
    return M, k, K, yp, ld_y, ip, dt


def moe_combine(y, topk_weights, out, topk_ids=None, E=None, residual=None, stream=None):
    """out[t] = residual[t] + sum_j topk_weights[t, j] y[t * top_k + j]: y
    [M * top_k, K] bf16 or fp16 (moe_group_mm's or moe_i8_group_mm's rows),
    topk_weights [M, top_k] fp32, out and residual [M, K] of y's type (residual
    may be out).  Routes whose topk_ids lie outside [0, E) are masked; without
    topk_ids every route counts."""
    where = "moe_combine"
    M, k, K, yp, ld_y, ip, dt = _combine_args(where, y, topk_weights, topk_ids, E)
    wp = _slots(where, "topk_weights", topk_weights, torch.float32, (M, k))
    op, ld_out = _rows_arg(where, "out", out, y.dtype, K)
    _need(out.shape[0] == M, where, "out and topk_weights disagree on M")
    rp, ld_res = None, 0
    if residual is not None:
        rp, ld_res = _rows_arg(where, "residual", residual, y.dtype, K)
        _need(residual.shape[0] == M, where, "residual and topk_weights disagree on M")
    _launch(where, stream, (y, topk_weights, out, topk_ids, residual), yp, ld_y, _DT[y.dtype], wp, ip, dt,
            0 if E is None else E, rp, ld_res, M, K, k, op, ld_out)


def moe_combine_bwd(dout, y, topk_weights, dy, d_weights, topk_ids=None, E=None, stream=None):
    """The gradient of moe_combine: dy [M * top_k, K] = topk_weights * dout
    (rows of masked routes left as they were) and d_weights [M, top_k] fp32 =
    the products of dout's and y's rows (0 for masked routes)."""
    where = "moe_combine_bwd"
    M, k, K, yp, ld_y, ip, dt = _combine_args(where, y, topk_weights, topk_ids, E)
    wp = _slots(where, "topk_weights", topk_weights, torch.float32, (M, k))
    gp = _slots(where, "d_weights", d_weights, torch.float32, (M, k))
    op, ld_out = _rows_arg(where, "dout", dout, y.dtype, K)
    dp, ld_dy = _rows_arg(where, "dy", dy, y.dtype, K)
    _need(dout.shape[0] == M and dy.shape[0] == M * k, where, "dout, dy and topk_weights disagree on rows")
    _launch(where, stream, (dout, y, topk_weights, dy, d_weights, topk_ids), op, ld_out, yp, ld_y, _DT[y.dtype],
            wp, ip, dt, 0 if E is None else E, M, K, k, dp, ld_dy, gp)


# ------------------------------------------------- 8-bit integer products --

def moe_quant_i8(x, x_q, x_s, stream=None):
    """x [M, K] bf16 or fp16 (row stride may exceed K) -> x_q int8 [M, K] and
    one scale a row, x_s fp32 [M]: s = max(amax / 127, 2^-126), codes rounded
    to nearest even.  Activations by token, or weights [N, K] by channel."""
    where = "moe_quant_i8"
    M, K, xp, ld = _16bit(where, "x", x)
    qp = _slots(where, "x_q", x_q, torch.int8, (M, K))
    sp = _slots(where, "x_s", x_s, torch.float32, (M,))
    _launch(where, stream, (x, x_q, x_s), xp, _DT[x.dtype], M, K, ld, qp, sp)


def moe_i8_linear_workspace_size(M, N, K, act=MOE_ACT_NONE):
    return _c["moe_i8_linear_workspace_size"](M, N, K, act)


def moe_i8_linear(x_q, x_s, w, w_s, out, bias=None, residual=None, act=MOE_ACT_NONE, workspace=None,
                  stream=None):
    """out = act(x_s w_s (x_q w^T) + bias) + residual: x_q [M, K] and w [N, K]
    int8 with scales x_s [M] and w_s [N] fp32, bias [N] fp32, residual and out
    bf16 or fp16 [M, N] -- [M, N/2] with MOE_ACT_SWIGLU, whose w holds the gate
    rows, then the up rows.  residual may be out itself."""
    where = "moe_i8_linear"
    _need(x_q.dim() == 2 and w.dim() == 2, where, "x_q and w must be 2-d")
    M, K = x_q.shape
    N = w.shape[0]
    ot = out.dtype
    qp = _slots(where, "x_q", x_q, torch.int8, (M, K))
    wp = _slots(where, "w", w, torch.int8, (N, K))
    xsp = _slots(where, "x_s", x_s, torch.float32, (M,))
    wsp = _slots(where, "w_s", w_s, torch.float32, (N,))
    bp = None if bias is None else _slots(where, "bias", bias, torch.float32, (N,))
    _need(ot in _DT16, where, "out must be bf16 or fp16")
    n_out = N // 2 if act == MOE_ACT_SWIGLU else N
    op, ld_out = _rows_arg(where, "out", out, ot, n_out)
    _need(out.shape[0] == M, where, "out and x_q disagree on M")
    rp, ld_res = None, 0
    if residual is not None:
        rp, ld_res = _rows_arg(where, "residual", residual, ot, n_out)
        _need(residual.shape[0] == M, where, "residual and x_q disagree on M")
    _launch(where, stream, (x_q, x_s, w, w_s, out, bias, residual, workspace), qp, xsp, wp, wsp, bp, rp, ld_res,
            M, N, K, act, op, _DT16[ot], ld_out, *_ws(where, workspace))


def moe_i8_group_mm_workspace_size(M, K, N, E, top_k, block_m, sorted_cap, act=MOE_ACT_NONE,
                                   x_per_route=False):
    return _c["moe_i8_group_mm_workspace_size"](M, K, N, E, top_k, block_m, sorted_cap, act,
                                                int(bool(x_per_route)))


def moe_i8_group_mm(x_q, x_s, w, w_s, sorted_token_ids, expert_ids, num_tokens_post_padded, top_k, block_m,
                    out, bias=None, act=MOE_ACT_NONE, workspace=None, stream=None, x_per_route=None):
    """out[r] = act(x_s[t(r)] w_s[e(r)] (x_q[t(r)] w[e(r)]^T) + bias[e(r)]) for
    every route r of the plan: w [E, N, K] int8 with w_s [E, N] fp32, bias
    [E, N] fp32, x_q [M, K] (t(r) = r // top_k) or [M * top_k, K] (t(r) = r)
    int8 with x_s fp32, out [M * top_k, N] bf16 or fp16 (N/2 columns with
    MOE_ACT_SWIGLU); x_per_route tells which rows x_q has (None: by their
    number).  Rows of masked routes are left as they were."""
    where = "moe_i8_group_mm"
    _need(w.dim() == 3 and x_q.dim() == 2, where, "w must be 3-d, x_q 2-d")
    E, N, K = w.shape
    wp = _slots(where, "w", w, torch.int8, (E, N, K))
    wsp = _slots(where, "w_s", w_s, torch.float32, (E, N))
    bp = None if bias is None else _slots(where, "bias", bias, torch.float32, (E, N))
    rows = x_q.shape[0]
    qp = _slots(where, "x_q", x_q, torch.int8, (rows, K))
    xsp = _slots(where, "x_s", x_s, torch.float32, (rows,))
    ot = out.dtype
    _need(ot in _DT16, where, "out must be bf16 or fp16")
    op, ld_out = _rows_arg(where, "out", out, ot, N // 2 if act == MOE_ACT_SWIGLU else N)
    R = out.shape[0]
    plan, cap = _group_plan(where, sorted_token_ids, expert_ids, num_tokens_post_padded, R, top_k, E, block_m)
    per_route = _x_rows(where, "x_q", x_q, R, top_k, x_per_route)
    _launch(where, stream, (x_q, x_s, w, w_s, out, bias, sorted_token_ids, expert_ids, num_tokens_post_padded,
                            workspace), qp, xsp, per_route, wp, wsp, bp, *plan, R // top_k, K, N, E, top_k,
            block_m, cap, act, op, _DT16[ot], ld_out, *_ws(where, workspace))


def moe_debug_i8_schedule(M, K, N, E=0, top_k=1, block_m=8, sorted_cap=0, act=MOE_ACT_NONE):
    """The kernel of moe_i8_linear (E = 0) or moe_i8_group_mm at these sizes: (the
    few-rows kernel's rows per pass or 0, a tile's rows, its weight rows)."""
    info = (ctypes.c_int32 * 3)()
    _check(_c["moe_debug_i8_schedule"](M, K, N, E, top_k, block_m, sorted_cap, act, info), "moe_debug_i8_schedule")
    return tuple(info)


def moe_status_str(status):
    return _c["moe_status_str"](status).decode()


def moe_last_hip_error():
    return _c["moe_last_hip_error"]().decode()


moe_last_error = moe_last_hip_error


# ------------------------------------------------------------- a layer --

class MoeLayerBuffers:
    """Device buffers for one call of the whole path at a given geometry
    (allocated once with torch; reused across calls)."""

    def __init__(self, M, K, I, E, top_k, block_m, flags=0, device="cuda", w4a8=False):
        self.M, self.K, self.I, self.E, self.top_k, self.block_m = M, K, I, E, top_k, block_m
        self.flags = flags
        self.w4a8 = w4a8
        self.sorted_cap, self.blocks_cap = moe_plan_capacity(M, top_k, E, block_m)
        dev = torch.device(device)
        self.sorted_ids = torch.empty(self.sorted_cap, dtype=torch.int32, device=dev)
        self.expert_ids = torch.empty(self.blocks_cap, dtype=torch.int32, device=dev)
        self.ntp = torch.empty(1, dtype=torch.int32, device=dev)
        self.x_q = torch.empty((M, K), dtype=torch.uint8, device=dev)
        self.x_s = torch.empty((M, K // 128), dtype=torch.float32, device=dev)
        size = moe_w4a8_experts_workspace_size if w4a8 else moe_fp8_experts_workspace_size
        ws = size(M, K, I, E, top_k, block_m, self.sorted_cap, flags)
        if w4a8 and M > 0 and ws == 0:
            raise MoeError(MOE_ERR_SHAPE, "moe_w4a8_experts_workspace_size", moe_last_hip_error())
        self.workspace = torch.empty(max(ws, 256), dtype=torch.uint8, device=dev)
        pws = moe_plan_workspace_size(M, top_k, E, block_m)
        self.plan_ws = torch.empty(pws, dtype=torch.uint8, device=dev) if pws else None
        self.h_q_off, self.h_s_off = moe_fp8_experts_workspace_layout(
            M, K, I, E, top_k, block_m, self.sorted_cap, flags)

    def intermediate(self):
        """(h_q [sorted_cap, I] uint8, h_s [sorted_cap, I/128] fp32) views of the workspace."""
        n_q = self.sorted_cap * self.I
        n_s = self.sorted_cap * (self.I // 128)
        hq = self.workspace[self.h_q_off:self.h_q_off + n_q].view(self.sorted_cap, self.I)
        hs = self.workspace[self.h_s_off:self.h_s_off + 4 * n_s].view(torch.float32)
        return hq, hs.view(self.sorted_cap, self.I // 128)


def moe_layer(bufs, x_bf16, topk_ids, topk_weights, w13, w13_s, w2, w2_s, out_bf16,
              act_scale_mode=MOE_SCALE_FP32, stream=None):
    """All five steps on one stream (moe_fp8_layer: plan with activation
    quantisation, experts)."""
    moe_fp8_layer(x_bf16, topk_ids, topk_weights, w13, w13_s, w2, w2_s, bufs.block_m,
                  bufs.sorted_ids, bufs.expert_ids, bufs.ntp, bufs.x_q, bufs.x_s, out_bf16,
                  bufs.workspace, bufs.flags, act_scale_mode, bufs.plan_ws, stream)
