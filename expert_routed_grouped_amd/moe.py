"""Thin ctypes binding of ``libmoe.so`` (declared in ``include/moe.h``).

Argument marshalling only: torch tensors in, raw device pointers and sizes to
the C ABI, every step runs in the library's HIP kernels on the tensor's
current stream.  There is no fallback: without the built library every call
raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmoe.so")

MOE_F32, MOE_BF16, MOE_FP8_E4M3, MOE_MXFP8, MOE_F32_ROUTER_PACKED = 0, 1, 2, 3, 4
MOE_MXFP4 = 5
MOE_FFN_GATHER, MOE_FFN_ZERO_Y, MOE_FFN_ONLY_GATE_UP, MOE_FFN_ONLY_DOWN = 1, 2, 4, 8
MOE_FFN_PACKED_WEIGHTS = 16
STATUS = {0: "MOE_OK", -1: "MOE_ERR_NULL", -2: "MOE_ERR_SHAPE", -3: "MOE_ERR_DTYPE", -4: "MOE_ERR_WORKSPACE",
          -5: "MOE_ERR_HIP", -6: "MOE_ERR_ALIGN"}

# Every symbol moe.h declares (checked by the CPU test suite).
EXPORTS = ("moe_version", "moe_status_str", "moe_route", "moe_permute", "moe_permute_workspace_size",
           "moe_ffn_workspace_size", "moe_grouped_ffn", "moe_combine", "moe_quantize_mx", "moe_ffn_mx_workspace_size",
           "moe_grouped_ffn_mx", "moe_shared_workspace_size", "moe_shared_expert", "moe_route_dispatch_workspace_size",
           "moe_route_dispatch", "moe_pack_weights", "moe_pack_router", "moe_grouped_ffn_noalloc",
           "moe_decode_layer_workspace_size", "moe_decode_layer", "moe_workspace_size", "moe_quantize_mx4",
           "moe_dequantize_mx", "moe_mx4_packed_scale_bytes", "moe_pack_mx4", "moe_ffn_mx4_workspace_size",
           "moe_grouped_ffn_mx4", "moe_decode_layer_mx4_workspace_size", "moe_decode_layer_mx4", "moe_grouped_mm",
           "moe_grouped_wgrad_workspace_size", "moe_grouped_wgrad", "moe_swiglu", "moe_swiglu_backward",
           "moe_route_backward", "moe_block_norm",
           "moe_block_norm_backward_workspace_size", "moe_block_norm_backward")
MOE_MM_TRANSPOSED, MOE_WGRAD_ADD = 1, 1
MOE_GATE_NONE, MOE_GATE_CHANNEL, MOE_GATE_TOKEN = 0, 1, 2
MOE_OP_PERMUTE, MOE_OP_GROUPED_FFN, MOE_OP_GROUPED_FFN_F32, MOE_OP_GROUPED_FFN_MX = 0, 1, 2, 3
MOE_OP_ROUTE_DISPATCH, MOE_OP_DECODE_LAYER, MOE_OP_SHARED_EXPERT, MOE_OP_SHARED_EXPERT_F32 = 4, 5, 6, 7
MOE_OP_GROUPED_FFN_MX4, MOE_OP_DECODE_LAYER_MX4 = 8, 9
MOE_NOALLOC_SCRATCH_BYTES = 32 << 20


class MoEError(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed: {STATUS.get(status, status)} ({text})")
        self.status = status


_lib = None


def lib():
    """Load libmoe.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m expert_routed_grouped_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.moe_version.restype = I
        L.moe_version.argtypes = []
        L.moe_status_str.restype = ctypes.c_char_p
        L.moe_status_str.argtypes = [I]
        L.moe_route.restype = I
        L.moe_route.argtypes = [P, I, P, I, P, I, I, I, I, P, P, P]
        L.moe_permute.restype = I
        L.moe_permute.argtypes = [P, P, I, I, I, I, I, P, P, P, P, P, P, I, I, P, P, Z, P]
        L.moe_permute_workspace_size.restype = Z
        L.moe_permute_workspace_size.argtypes = [I, I, I]
        L.moe_ffn_workspace_size.restype = Z
        L.moe_ffn_workspace_size.argtypes = [I, I, I, I, I]
        L.moe_grouped_ffn.restype = I
        L.moe_grouped_ffn.argtypes = [P, I, P, P, P, I, I, I, I, I, P, P, I, P, P, P, P, P, Z, ctypes.c_uint, P]
        L.moe_grouped_ffn_noalloc.restype = I
        L.moe_grouped_ffn_noalloc.argtypes = [P, I, P, P, P, I, I, I, I, I, P, P, I, P, P, P, P, ctypes.c_uint, P]
        L.moe_workspace_size.restype = Z
        L.moe_workspace_size.argtypes = [I, I, I, I, I, I]
        L.moe_decode_layer_workspace_size.restype = Z
        L.moe_decode_layer_workspace_size.argtypes = [I, I, I, I]
        L.moe_decode_layer.restype = I
        L.moe_decode_layer.argtypes = [P, I, P, I, P, I, I, I, I, I, I, I, P, P, I, P, P, P, P, P, P, P, P, P, P, P,
                                       Z, ctypes.c_uint, P]
        L.moe_combine.restype = I
        L.moe_combine.argtypes = [P, P, P, I, I, I, P, P]
        L.moe_quantize_mx.restype = I
        L.moe_quantize_mx.argtypes = [P, I, I, I, P, P, P]
        L.moe_ffn_mx_workspace_size.restype = Z
        L.moe_ffn_mx_workspace_size.argtypes = [I, I]
        L.moe_grouped_ffn_mx.restype = I
        L.moe_grouped_ffn_mx.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P, P, P, P, P, P, Z, ctypes.c_uint, P]
        L.moe_shared_workspace_size.restype = Z
        L.moe_shared_workspace_size.argtypes = [I, I, I]
        L.moe_shared_expert.restype = I
        L.moe_shared_expert.argtypes = [P, I, I, I, I, P, P, I, P, P, P, P, Z, ctypes.c_uint, P]
        L.moe_route_dispatch_workspace_size.restype = Z
        L.moe_route_dispatch_workspace_size.argtypes = []
        L.moe_route_dispatch.restype = I
        L.moe_route_dispatch.argtypes = [P, I, P, I, P, I, I, I, I, I, I, P, P, P, P, P, P, P, P, P, Z, P]
        L.moe_pack_weights.restype = I
        L.moe_pack_weights.argtypes = [P, I, I, I, I, P, P]
        L.moe_pack_router.restype = I
        L.moe_pack_router.argtypes = [P, I, I, I, P, P]
        L64 = ctypes.c_int64
        L.moe_quantize_mx4.restype = I
        L.moe_quantize_mx4.argtypes = [P, I, L64, I, P, P, P]
        L.moe_dequantize_mx.restype = I
        L.moe_dequantize_mx.argtypes = [P, P, I, L64, I, P, I, P]
        L.moe_mx4_packed_scale_bytes.restype = Z
        L.moe_mx4_packed_scale_bytes.argtypes = [L64, I]
        L.moe_pack_mx4.restype = I
        L.moe_pack_mx4.argtypes = [P, P, L64, I, P, P, P]
        L.moe_ffn_mx4_workspace_size.restype = Z
        L.moe_ffn_mx4_workspace_size.argtypes = [I, I, I, I, I, I]
        L.moe_grouped_ffn_mx4.restype = I
        L.moe_grouped_ffn_mx4.argtypes = [P, P, I, P, P, P, P, I, I, I, I, I, P, P, P, P, P, I, P, Z, P]
        L.moe_decode_layer_mx4_workspace_size.restype = Z
        L.moe_decode_layer_mx4_workspace_size.argtypes = [I, I, I, I, I]
        L.moe_decode_layer_mx4.restype = I
        L.moe_decode_layer_mx4.argtypes = [P, P, P, I, I, I, I, I, I, I, P, P, P, P, P, P, P, I, P, Z, P]
        U, F = ctypes.c_uint, ctypes.c_float
        L.moe_grouped_mm.restype = I
        L.moe_grouped_mm.argtypes = [P, P, I, P, I, P, I, I, I, I, P, I, U, P]
        L.moe_grouped_wgrad_workspace_size.restype = Z
        L.moe_grouped_wgrad_workspace_size.argtypes = [I, I, I, I, I]
        L.moe_grouped_wgrad.restype = I
        L.moe_grouped_wgrad.argtypes = [P, P, I, P, P, I, I, P, I, I, I, I, P, I, P, Z, U, P]
        L.moe_swiglu.restype = I
        L.moe_swiglu.argtypes = [P, I, P, P, I, I, I, P, P]
        L.moe_swiglu_backward.restype = I
        L.moe_swiglu_backward.argtypes = [P, P, I, P, P, I, I, I, P, P, P, P]
        L.moe_route_backward.restype = I
        L.moe_route_backward.argtypes = [P, P, P, I, I, I, I, P, P, I, P, P, P, I, P, I, P, I, P, P, P]
        L.moe_block_norm.restype = I
        L.moe_block_norm.argtypes = [P, I, P, I, P, P, P, I, I, F, F, I, I, P, P, P, P, P]
        L.moe_block_norm_backward_workspace_size.restype = Z
        L.moe_block_norm_backward_workspace_size.argtypes = [I, I]
        L.moe_block_norm_backward.restype = I
        L.moe_block_norm_backward.argtypes = [P, I, P, I, P, P, P, I, I, F, P, P, P, P, I, I, P, P, I, P, P, P, P, Z, P]
        _lib = L
    return _lib


def _check(fn: str, status: int):
    if status != 0:
        raise MoEError(fn, status, lib().moe_status_str(status).decode())


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the MoE library must be contiguous")
    if not t.is_cuda:  # every array of the ABI is device memory; a host pointer would fault the GPU
        raise ValueError("tensors passed to the MoE library must be on the GPU")
    return ctypes.c_void_p(t.data_ptr())


def _dtype(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return MOE_F32
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype in (torch.uint8, torch.float8_e4m3fn):
        return MOE_FP8_E4M3
    raise TypeError(f"unsupported dtype {t.dtype}")


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def torch_stream(stream, device):
    """``stream`` (a stream, its raw address or None: the device's current one) as a torch stream."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if hasattr(stream, "wait_event"):
        return stream
    return torch.cuda.ExternalStream(int(getattr(stream, "cuda_stream", stream)), device=device)


def _new(shape, dtype, device, stream) -> torch.Tensor:
    """What a call allocates itself comes from the pool of the stream it runs on: memory of another stream's pool may
    have work of that stream ahead of it, or be handed out again while this call still runs."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(torch_stream(stream, device)):
        return torch.empty(shape, dtype=dtype, device=device)


def moe_version() -> int:
    return lib().moe_version()


def moe_route(x: torch.Tensor, w_router: torch.Tensor, bias: Optional[torch.Tensor], k: int,
              topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None, stream=None):
    """Router logits (canonical fp32 FMA chain), top-k, renormalised gates -> (topk_ids, topk_w)."""
    T, H = x.shape
    E = w_router.shape[0]
    if topk_ids is None:
        topk_ids = _new((T, k), torch.int32, x.device, stream)
    if topk_w is None:
        topk_w = _new((T, k), torch.float32, x.device, stream)
    _check("moe_route", lib().moe_route(_ptr(x), _dtype(x), _ptr(w_router), _dtype(w_router), _ptr(bias), T, H, E, k,
                                        _ptr(topk_ids), _ptr(topk_w), _stream(stream)))
    return topk_ids, topk_w


def moe_permute(topk_ids: torch.Tensor, topk_w: torch.Tensor, E: int, e_begin: int, e_end: int,
                x: Optional[torch.Tensor] = None, x_perm: Optional[torch.Tensor] = None, out: Optional[dict] = None,
                stream=None) -> dict:
    """Counts, offsets and the stable by-expert grouping of the local assignments.

    Returns dict(counts, offsets, row_token, row_w, token_row[, x_perm]); row
    buffers have R_cap = T*min(k, E_loc) entries, the first offsets[-1] are valid."""
    T, k = topk_ids.shape
    El = e_end - e_begin
    R_cap = T * min(k, El)
    dev = topk_ids.device
    o = dict(out) if out else {}
    for name, shape, dtype in (("counts", (El,), torch.int32), ("offsets", (El + 1,), torch.int32),
                               ("row_token", (max(R_cap, 1),), torch.int32), ("row_w", (max(R_cap, 1),), torch.float32),
                               ("token_row", (T, k), torch.int32),
                               ("workspace", (max(moe_permute_workspace_size(T, k, El), 256),), torch.uint8)):
        if name not in o:
            o[name] = _new(shape, dtype, dev, stream)
    H = 0
    xdt = MOE_BF16
    if x is not None:
        H = x.shape[1]
        xdt = _dtype(x)
        if x_perm is None:
            x_perm = _new((max(R_cap, 1), H), x.dtype, dev, stream)
        o["x_perm"] = x_perm
    _check("moe_permute", lib().moe_permute(_ptr(topk_ids), _ptr(topk_w), T, k, E, e_begin, e_end,
                                            _ptr(o["counts"]), _ptr(o["offsets"]), _ptr(o["row_token"]),
                                            _ptr(o["row_w"]), _ptr(o["token_row"]), _ptr(x), xdt, H,
                                            _ptr(x_perm), _ptr(o["workspace"]),
                                            o["workspace"].numel() * o["workspace"].element_size(), _stream(stream)))
    o["R_cap"] = R_cap
    return o


def moe_workspace_size(op: int, T: int, k: int, E_loc: int, H: int, I: int) -> int:
    """Bytes of workspace one call of ``op`` (MOE_OP_*) needs."""
    return int(lib().moe_workspace_size(op, T, k, E_loc, H, I))


def moe_permute_workspace_size(T: int, k: int, E_loc: int) -> int:
    return int(lib().moe_permute_workspace_size(T, k, E_loc))


def moe_ffn_workspace_size(R_cap: int, E_loc: int, H: int, I: int, a_dtype: int) -> int:
    return int(lib().moe_ffn_workspace_size(R_cap, E_loc, H, I, a_dtype))


def moe_grouped_ffn(a: torch.Tensor, offsets: torch.Tensor, row_token: torch.Tensor, row_w: torch.Tensor, T: int,
                    R_cap: int, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                    s_gate_up: Optional[torch.Tensor] = None, s_down: Optional[torch.Tensor] = None,
                    y: Optional[torch.Tensor] = None, y_perm: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, gather: bool = True, zero_y: bool = True,
                    phase: str = "both", packed: bool = False, stream=None):
    """SwiGLU expert FFN over the grouped rows.  With ``y`` the gate-weighted combine is
    fused (y accumulates; zeroed first when ``zero_y``); otherwise writes ``y_perm``.
    ``phase``: "both", "gate_up" or "down" (the two halves, same arguments and workspace).
    ``packed``: both weight tensors come from moe_pack_weights."""
    El, twoI, H = w_gate_up.shape
    I = twoI // 2
    adt = _dtype(a)
    need = moe_ffn_workspace_size(R_cap, El, H, I, adt)
    if workspace is None:
        workspace = _new((need,), torch.uint8, a.device, stream)
    flags = (MOE_FFN_GATHER if gather else 0) | (MOE_FFN_ZERO_Y if zero_y else 0)
    flags |= {"both": 0, "gate_up": MOE_FFN_ONLY_GATE_UP, "down": MOE_FFN_ONLY_DOWN}[phase]
    flags |= MOE_FFN_PACKED_WEIGHTS if packed else 0
    _check("moe_grouped_ffn", lib().moe_grouped_ffn(
        _ptr(a), adt, _ptr(offsets), _ptr(row_token), _ptr(row_w), El, T, R_cap, H, I, _ptr(w_gate_up),
        _ptr(w_down), _dtype(w_gate_up), _ptr(s_gate_up), _ptr(s_down), _ptr(y), _ptr(y_perm), _ptr(workspace),
        workspace.numel() * workspace.element_size(), flags, _stream(stream)))
    return y if y is not None else y_perm


def moe_grouped_ffn_noalloc(a: torch.Tensor, offsets: torch.Tensor, row_token: torch.Tensor, row_w: torch.Tensor,
                            T: int, R_cap: int, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                            s_gate_up: Optional[torch.Tensor] = None, s_down: Optional[torch.Tensor] = None,
                            y: Optional[torch.Tensor] = None, y_perm: Optional[torch.Tensor] = None,
                            gather: bool = True, zero_y: bool = True, phase: str = "both", packed: bool = False,
                            stream=None):
    """moe_grouped_ffn with its intermediate in the library's static per-GPU scratch array (no
    workspace argument, nothing allocated by the call).  Calls on one GPU must not overlap."""
    El, twoI, H = w_gate_up.shape
    I = twoI // 2
    flags = (MOE_FFN_GATHER if gather else 0) | (MOE_FFN_ZERO_Y if zero_y else 0)
    flags |= {"both": 0, "gate_up": MOE_FFN_ONLY_GATE_UP, "down": MOE_FFN_ONLY_DOWN}[phase]
    flags |= MOE_FFN_PACKED_WEIGHTS if packed else 0
    _check("moe_grouped_ffn_noalloc", lib().moe_grouped_ffn_noalloc(
        _ptr(a), _dtype(a), _ptr(offsets), _ptr(row_token), _ptr(row_w), El, T, R_cap, H, I, _ptr(w_gate_up),
        _ptr(w_down), _dtype(w_gate_up), _ptr(s_gate_up), _ptr(s_down), _ptr(y), _ptr(y_perm), flags,
        _stream(stream)))
    return y if y is not None else y_perm


def moe_quantize_mx(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                    stream=None):
    """MXFP8 quantisation of a [rows, K] fp32/bf16 tensor -> (codes uint8 [rows, K], scales uint8 [rows, K/32])."""
    rows, K = x.shape
    if codes is None:
        codes = _new((rows, K), torch.uint8, x.device, stream)
    if scales is None:
        scales = _new((rows, K // 32), torch.uint8, x.device, stream)
    _check("moe_quantize_mx", lib().moe_quantize_mx(_ptr(x), _dtype(x), rows, K, _ptr(codes), _ptr(scales),
                                                    _stream(stream)))
    return codes, scales


def moe_ffn_mx_workspace_size(R_cap: int, I: int) -> int:
    return int(lib().moe_ffn_mx_workspace_size(R_cap, I))


def moe_grouped_ffn_mx(a_codes: torch.Tensor, a_scales: torch.Tensor, offsets: torch.Tensor, row_token: torch.Tensor,
                       row_w: torch.Tensor, T: int, R_cap: int, wgu_codes: torch.Tensor, wgu_scales: torch.Tensor,
                       wd_codes: torch.Tensor, wd_scales: torch.Tensor, y: Optional[torch.Tensor] = None,
                       y_perm: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       gather: bool = True, zero_y: bool = True, phase: str = "both", packed: bool = False,
                       stream=None):
    """W8A8 MXFP8 SwiGLU expert FFN (activations and weights as MX codes + E8M0 scales).  ``packed``:
    the weight codes are in the packed block layout (moe_pack_weights); scales stay row-major."""
    El, twoI, H = wgu_codes.shape
    I = twoI // 2
    need = moe_ffn_mx_workspace_size(R_cap, I)
    if workspace is None:
        workspace = _new((need,), torch.uint8, a_codes.device, stream)
    flags = (MOE_FFN_GATHER if gather else 0) | (MOE_FFN_ZERO_Y if zero_y else 0)
    flags |= {"both": 0, "gate_up": MOE_FFN_ONLY_GATE_UP, "down": MOE_FFN_ONLY_DOWN}[phase]
    flags |= MOE_FFN_PACKED_WEIGHTS if packed else 0
    _check("moe_grouped_ffn_mx", lib().moe_grouped_ffn_mx(
        _ptr(a_codes), _ptr(a_scales), _ptr(offsets), _ptr(row_token), _ptr(row_w), El, T, R_cap, H, I,
        _ptr(wgu_codes), _ptr(wgu_scales), _ptr(wd_codes), _ptr(wd_scales), _ptr(y), _ptr(y_perm), _ptr(workspace),
        workspace.numel() * workspace.element_size(), flags, _stream(stream)))
    return y if y is not None else y_perm


def moe_combine(y_perm: torch.Tensor, token_row: torch.Tensor, topk_w: torch.Tensor, y: Optional[torch.Tensor] = None,
                stream=None) -> torch.Tensor:
    T, k = token_row.shape
    H = y_perm.shape[1]
    if y is None:
        y = _new((T, H), torch.float32, y_perm.device, stream)
    _check("moe_combine", lib().moe_combine(_ptr(y_perm), _ptr(token_row), _ptr(topk_w), T, k, H, _ptr(y),
                                            _stream(stream)))
    return y


def moe_shared_workspace_size(T: int, I_s: int, x_dtype: int) -> int:
    return int(lib().moe_shared_workspace_size(T, I_s, x_dtype))


def moe_shared_expert(x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, y: torch.Tensor,
                      s_gate_up: Optional[torch.Tensor] = None, s_down: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, zero_y: bool = False, packed: bool = False,
                      stream=None):
    """y += shared-expert SwiGLU FFN of x (every token, weight 1); ``zero_y`` zeroes y first;
    ``packed``: both weight tensors come from moe_pack_weights."""
    T, H = x.shape
    I_s = w_gate_up.shape[0] // 2
    xdt = _dtype(x)
    need = moe_shared_workspace_size(T, I_s, xdt)
    if workspace is None:
        workspace = _new((need,), torch.uint8, x.device, stream)
    _check("moe_shared_expert", lib().moe_shared_expert(
        _ptr(x), xdt, T, H, I_s, _ptr(w_gate_up), _ptr(w_down), _dtype(w_gate_up), _ptr(s_gate_up), _ptr(s_down),
        _ptr(y), _ptr(workspace), workspace.numel() * workspace.element_size(),
        (MOE_FFN_ZERO_Y if zero_y else 0) | (MOE_FFN_PACKED_WEIGHTS if packed else 0), _stream(stream)))
    return y


def moe_pack_weights(w: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Weights [E, N, K] (or [N, K], one expert) in the packed block layout, as a tensor of the
    same shape and dtype (pass it with ``packed=True``)."""
    E, N, K = (1, *w.shape) if w.dim() == 2 else w.shape
    if out is None:
        out = _new(w.shape, w.dtype, w.device, stream)
    if out.shape != w.shape or out.dtype != w.dtype:
        raise ValueError("out must have the shape and dtype of w")
    _check("moe_pack_weights", lib().moe_pack_weights(_ptr(w), _dtype(w), E, N, K, _ptr(out), _stream(stream)))
    return out


def moe_route_dispatch_workspace(device="cuda") -> torch.Tensor:
    """A zeroed workspace for moe_route_dispatch (its ticket counter starts at zero)."""
    return torch.zeros(int(lib().moe_route_dispatch_workspace_size()), dtype=torch.uint8, device=device)


def moe_pack_router(w_router: torch.Tensor, stream=None) -> torch.Tensor:
    """The router weight [E, H] (bf16 or fp32) as exact fp32 in the layout of moe_pack_router,
    [H/4, E, 4]; pass it to moe_route_dispatch with ``router_packed=True``."""
    E, H = w_router.shape
    out = _new((H // 4, E, 4), torch.float32, w_router.device, stream)
    _check("moe_pack_router", lib().moe_pack_router(_ptr(w_router), _dtype(w_router), E, H, _ptr(out),
                                                    _stream(stream)))
    return out


def moe_route_dispatch(x: torch.Tensor, w_router: torch.Tensor, bias: Optional[torch.Tensor], k: int, E: int,
                       e_begin: int, e_end: int, workspace: torch.Tensor, topk_ids: torch.Tensor, topk_w: torch.Tensor,
                       out: dict, y_zero: Optional[torch.Tensor] = None, router_packed: bool = False,
                       stream=None) -> dict:
    """Route + local dispatch of a decode batch in one launch; ``out`` holds counts, offsets,
    row_token, row_w, token_row (as from moe_permute); zeroes ``y_zero`` when given.
    ``router_packed``: ``w_router`` is the fp32 [H/4, E, 4] tensor of moe_pack_router (the C ABI
    cannot see buffer sizes, so the layout is checked here: a raw [E, H] weight passed as packed
    would be read past its end)."""
    T, H = x.shape
    if router_packed:
        if w_router.dtype != torch.float32 or tuple(w_router.shape) != (H // 4, E, 4) or H % 4 != 0:
            raise ValueError(f"router_packed needs the fp32 [H/4, E, 4] = {(H // 4, E, 4)} tensor of moe_pack_router, "
                             f"got {w_router.dtype} {tuple(w_router.shape)}")
    elif tuple(w_router.shape) != (E, H):
        raise ValueError(f"w_router must be [E, H] = {(E, H)}, got {tuple(w_router.shape)}")
    _check("moe_route_dispatch", lib().moe_route_dispatch(
        _ptr(x), _dtype(x), _ptr(w_router), MOE_F32_ROUTER_PACKED if router_packed else _dtype(w_router), _ptr(bias),
        T, H, E, k, e_begin, e_end, _ptr(topk_ids),
        _ptr(topk_w), _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["row_token"]), _ptr(out["row_w"]),
        _ptr(out["token_row"]), _ptr(y_zero), _ptr(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


def moe_decode_layer_workspace(T: int, k: int, E_loc: int, I: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for moe_decode_layer (its control words must start at zero)."""
    return torch.zeros(int(lib().moe_decode_layer_workspace_size(T, k, E_loc, I)), dtype=torch.uint8, device=device)


def moe_decode_layer(x: torch.Tensor, w_router: torch.Tensor, bias: Optional[torch.Tensor], k: int, E: int,
                     e_begin: int, e_end: int, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                     s_gate_up: Optional[torch.Tensor], s_down: Optional[torch.Tensor], workspace: torch.Tensor,
                     topk_ids: torch.Tensor, topk_w: torch.Tensor, out: dict, y: torch.Tensor,
                     router_packed: bool = False, packed: bool = False, stream=None) -> torch.Tensor:
    """The whole decode layer in one launch: routing into ``topk_ids``/``topk_w``, the grouping into
    ``out`` (counts, offsets, row_token, row_w, token_row as from moe_permute) and y [T, H]
    (overwritten).  ``router_packed``: ``w_router`` is the moe_pack_router tensor; ``packed``: the
    expert weights come from moe_pack_weights."""
    T, H = x.shape
    El, twoI, _ = w_gate_up.shape
    if router_packed:
        if w_router.dtype != torch.float32 or tuple(w_router.shape) != (H // 4, E, 4):
            raise ValueError(f"router_packed needs the fp32 [H/4, E, 4] = {(H // 4, E, 4)} tensor of moe_pack_router, "
                             f"got {w_router.dtype} {tuple(w_router.shape)}")
    elif tuple(w_router.shape) != (E, H):
        raise ValueError(f"w_router must be [E, H] = {(E, H)}, got {tuple(w_router.shape)}")
    if El != e_end - e_begin or tuple(w_down.shape) != (El, H, twoI // 2):
        raise ValueError("expert weights must be [E_loc, 2I, H] and [E_loc, H, I]")
    _check("moe_decode_layer", lib().moe_decode_layer(
        _ptr(x), _dtype(x), _ptr(w_router), MOE_F32_ROUTER_PACKED if router_packed else _dtype(w_router), _ptr(bias),
        T, H, E, k, e_begin, e_end, twoI // 2, _ptr(w_gate_up), _ptr(w_down), _dtype(w_gate_up), _ptr(s_gate_up),
        _ptr(s_down), _ptr(topk_ids), _ptr(topk_w), _ptr(out["counts"]), _ptr(out["offsets"]), _ptr(out["row_token"]),
        _ptr(out["row_w"]), _ptr(out["token_row"]), _ptr(y), _ptr(workspace), workspace.numel() * workspace.element_size(),
        MOE_FFN_PACKED_WEIGHTS if packed else 0, _stream(stream)))
    return y


def decode_layer_error_word(workspace: torch.Tensor) -> int:
    """The diagnostic word of a moe_decode_layer workspace (nonzero: a wait in the kernel gave up)."""
    return int(workspace[16:20].view(torch.int32).item())


# ---- MXFP4 (include/moe.h, the *_mx4 calls) ----
# The C ABI cannot see buffer sizes, so the shape, type and device of every tensor are checked here.  A call is short
# next to what Python adds to it: one pass over each argument, raw addresses and streams.
def _arg(t: Optional[torch.Tensor], name: str, dtype, shape, device):
    """Address of a contiguous GPU tensor of this type, shape and device (None stays None)."""
    if t is None:
        return None
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


class _On:
    """``device`` as the current one (if it is not), so that a call runs there, on its current stream."""

    def __init__(self, device: torch.device):
        if device.type != "cuda":
            raise ValueError("tensors passed to the MoE library must be on the GPU")
        self.index = device.index
        self.other = None

    def __enter__(self):
        if torch.cuda.current_device() != self.index:
            self.other = torch.cuda.device(self.index)
            self.other.__enter__()
        return self

    def __exit__(self, *exc):
        if self.other is not None:
            self.other.__exit__(*exc)

    def stream(self, stream) -> int:
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.index)
        if getattr(stream, "device", None) not in (None, torch.device("cuda", self.index)):
            raise ValueError(f"stream is on {stream.device}, the tensors on cuda:{self.index}")
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _out_dtype(dtype) -> int:
    if dtype == torch.bfloat16:
        return MOE_BF16
    if dtype == torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported output dtype {dtype}")


def moe_quantize_mx4(x: torch.Tensor, codes: Optional[torch.Tensor] = None, scales: Optional[torch.Tensor] = None,
                     stream=None):
    """MXFP4 quantisation of a [rows, K] fp32/bf16 tensor -> (codes uint8 [rows, K/2], scales uint8 [rows, K/32])."""
    rows, K = x.shape
    dt, dev, u8 = _out_dtype(x.dtype), x.device, torch.uint8
    if codes is None:
        codes = _new((rows, K // 2), u8, dev, stream)
    if scales is None:
        scales = _new((rows, K // 32), u8, dev, stream)
    args = (_arg(x, "x", x.dtype, (rows, K), dev), dt, rows, K, _arg(codes, "codes", u8, (rows, K // 2), dev),
            _arg(scales, "scales", u8, (rows, K // 32), dev))
    with _On(dev) as on:
        _check("moe_quantize_mx4", lib().moe_quantize_mx4(*args, on.stream(stream)))
    return codes, scales


def moe_dequantize_mx(codes: torch.Tensor, scales: torch.Tensor, out: Optional[torch.Tensor] = None,
                      dtype=torch.float32, stream=None) -> torch.Tensor:
    """The values of MXFP4 codes [rows, K/2] or MXFP8 codes [rows, K] with scales [rows, K/32] (which of the two
    follows from the widths) -> [rows, K] of ``dtype`` (fp32 or bf16)."""
    rows, K, dev, u8 = codes.shape[0], scales.shape[1] * 32, codes.device, torch.uint8
    if codes.shape[1] not in (K, K // 2):
        raise ValueError(f"codes {tuple(codes.shape)} and scales {tuple(scales.shape)} are no MXFP4 or MXFP8 pair")
    fp4 = codes.shape[1] == K // 2
    if out is None:
        _out_dtype(dtype)
        out = _new((rows, K), dtype, dev, stream)
    args = (_arg(codes, "codes", u8, (rows, K // 2 if fp4 else K), dev),
            _arg(scales, "scales", u8, (rows, K // 32), dev), MOE_MXFP4 if fp4 else MOE_MXFP8, rows, K,
            _arg(out, "out", out.dtype, (rows, K), dev), _out_dtype(out.dtype))
    with _On(dev) as on:
        _check("moe_dequantize_mx", lib().moe_dequantize_mx(*args, on.stream(stream)))
    return out


def moe_pack_mx4(codes: torch.Tensor, scales: torch.Tensor, stream=None):
    """MXFP4 weights [E, N, K/2] (or [N, K/2]) with scales [E, N, K/32] in the layout of moe_pack_mx4:
    (codes uint8 [E, N/16, K/128, 1024], scales uint8 [E, N/16, ceil(K/512), 256]); without E for 2-D weights."""
    if codes.dim() not in (2, 3) or scales.dim() != codes.dim():
        raise ValueError("codes and scales must both be [E, N, ...] or [N, ...]")
    lead, N, K, dev, u8 = codes.shape[:-2], codes.shape[-2], codes.shape[-1] * 2, codes.device, torch.uint8
    pcodes, pscales = (_arg(codes, "codes", u8, (*lead, N, K // 2), dev),
                       _arg(scales, "scales", u8, (*lead, N, K // 32), dev))
    if N % 16 != 0 or K % 128 != 0:
        raise MoEError("moe_pack_mx4", -2, "N must be a multiple of 16 and K of 128")
    pc = _new((*lead, N // 16, K // 128, 1024), u8, dev, stream)
    ps = _new((*lead, N // 16, (K + 511) // 512, 256), u8, dev, stream)
    with _On(dev) as on:
        _check("moe_pack_mx4", lib().moe_pack_mx4(pcodes, pscales, (lead[0] if lead else 1) * N, K, pc.data_ptr(),
                                                  ps.data_ptr(), on.stream(stream)))
    return pc, ps


def _mx4_weights(wgu, wd, dev):
    """Sizes (E_loc, H, I) and addresses of packed gate/up and down weights, each a (codes, scales) pair of
    moe_pack_mx4."""
    (gc, gs), (dc, ds) = wgu, wd
    if gc.dim() != 4 or dc.dim() != 4 or gc.shape[1] % 2 != 0:
        raise ValueError("weights must be the (codes, scales) pairs of moe_pack_mx4, with experts in front")
    El, gI, hb, _ = gc.shape
    H, I, u8 = hb * 128, gI * 8, torch.uint8
    return El, H, I, (_arg(gc, "w_gate_up codes", u8, (El, gI, hb, 1024), dev),
                      _arg(gs, "w_gate_up scales", u8, (El, gI, (H + 511) // 512, 256), dev),
                      _arg(dc, "w_down codes", u8, (El, H // 16, I // 128, 1024), dev),
                      _arg(ds, "w_down scales", u8, (El, H // 16, (I + 511) // 512, 256), dev))


def moe_ffn_mx4_workspace_size(T: int, k: int, E_loc: int, H: int, I: int, y_dtype: int = MOE_F32) -> int:
    return int(lib().moe_ffn_mx4_workspace_size(T, k, E_loc, H, I, y_dtype))


def moe_ffn_mx4_workspace(T: int, k: int, E_loc: int, H: int, I: int, dtype=torch.bfloat16,
                          device="cuda") -> torch.Tensor:
    """A workspace for moe_grouped_ffn_mx4 with output of ``dtype``."""
    return torch.empty(moe_ffn_mx4_workspace_size(T, k, E_loc, H, I, _out_dtype(dtype)), dtype=torch.uint8,
                       device=device)


def moe_grouped_ffn_mx4(a_codes: torch.Tensor, a_scales: torch.Tensor, offsets: torch.Tensor, row_token: torch.Tensor,
                        row_w: torch.Tensor, token_row: torch.Tensor, wgu, wd, y: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, dtype=torch.bfloat16, stream=None) -> torch.Tensor:
    """SwiGLU expert FFN with MXFP4 weights and the gate-weighted sum to token order -> y [T, H] of ``dtype``
    (overwritten).  Activations MXFP8 or MXFP4 (from the width of ``a_codes``); ``wgu`` and ``wd`` are the
    (codes, scales) pairs of moe_pack_mx4; the maps are those of moe_permute."""
    dev, u8, i32 = a_codes.device, torch.uint8, torch.int32
    El, H, I, w = _mx4_weights(wgu, wd, dev)
    T, k = token_row.shape
    fp4 = a_codes.shape[1] == H // 2
    if row_token.numel() < T * min(k, El) or row_w.numel() < T * min(k, El):
        raise ValueError(f"row_token and row_w must hold T * min(k, E_loc) = {T * min(k, El)} entries")
    if y is None:
        _out_dtype(dtype)
        y = _new((T, H), dtype, dev, stream)
    ydt = _out_dtype(y.dtype)
    if workspace is None:
        workspace = _new((moe_ffn_mx4_workspace_size(T, k, El, H, I, ydt),), u8, dev, stream)
    args = (_arg(a_codes, "a_codes", u8, (T, H // 2 if fp4 else H), dev), _arg(a_scales, "a_scales", u8, (T, H // 32), dev),
            MOE_MXFP4 if fp4 else MOE_MXFP8, _arg(offsets, "offsets", i32, (El + 1,), dev),
            _arg(row_token, "row_token", i32, row_token.shape, dev), _arg(row_w, "row_w", torch.float32, row_w.shape, dev),
            _arg(token_row, "token_row", i32, (T, k), dev), El, T, k, H, I, *w, _arg(y, "y", y.dtype, (T, H), dev), ydt,
            _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev), workspace.nbytes)
    with _On(dev) as on:
        _check("moe_grouped_ffn_mx4", lib().moe_grouped_ffn_mx4(*args, on.stream(stream)))
    return y


def moe_decode_layer_mx4_workspace(T: int, k: int, E_loc: int, H: int, I: int, device="cuda") -> torch.Tensor:
    """A zeroed workspace for moe_decode_layer_mx4 (its control words must start at zero)."""
    return torch.zeros(int(lib().moe_decode_layer_mx4_workspace_size(T, k, E_loc, H, I)), dtype=torch.uint8,
                       device=device)


def moe_decode_layer_mx4(x: torch.Tensor, w_router_packed: torch.Tensor, bias: Optional[torch.Tensor], k: int,
                         e_begin: int, e_end: int, wgu, wd, workspace: torch.Tensor,
                         topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None,
                         y: Optional[torch.Tensor] = None, dtype=torch.bfloat16, stream=None):
    """The whole MoE layer of up to 64 tokens with MXFP4 experts -> (y [T, H] of ``dtype``, topk_ids, topk_w).
    ``w_router_packed`` is the fp32 [H/4, E, 4] tensor of moe_pack_router, ``wgu`` and ``wd`` the (codes, scales)
    pairs of moe_pack_mx4 for the experts [e_begin, e_end), ``workspace`` starts zeroed
    (moe_decode_layer_mx4_workspace; decode_layer_error_word reads its diagnostic)."""
    dev, f32 = x.device, torch.float32
    El, H, I, w = _mx4_weights(wgu, wd, dev)
    T = x.shape[0]
    if w_router_packed.dim() != 3:
        raise ValueError("w_router_packed must be the [H/4, E, 4] tensor of moe_pack_router")
    E = w_router_packed.shape[1]
    if El != e_end - e_begin:
        raise ValueError(f"weights hold {El} experts, [{e_begin}, {e_end}) has {e_end - e_begin}")
    if topk_ids is None:
        topk_ids = _new((T, k), torch.int32, dev, stream)
    if topk_w is None:
        topk_w = _new((T, k), f32, dev, stream)
    if y is None:
        _out_dtype(dtype)
        y = _new((T, H), dtype, dev, stream)
    args = (_arg(x, "x", torch.bfloat16, (T, H), dev), _arg(w_router_packed, "w_router_packed", f32, (H // 4, E, 4), dev),
            _arg(bias, "bias", f32, (E,), dev), T, H, E, k, e_begin, e_end, I, *w,
            _arg(topk_ids, "topk_ids", torch.int32, (T, k), dev), _arg(topk_w, "topk_w", f32, (T, k), dev),
            _arg(y, "y", y.dtype, (T, H), dev), _out_dtype(y.dtype),
            _arg(workspace, "workspace", torch.uint8, workspace.shape, dev), workspace.nbytes)
    with _On(dev) as on:
        _check("moe_decode_layer_mx4", lib().moe_decode_layer_mx4(*args, on.stream(stream)))
    return y, topk_ids, topk_w


def _space(workspace: Optional[torch.Tensor], need: int, dev, stream):
    """(address, bytes) of a call's workspace, made here where the caller gives none; and the tensor to keep."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _new((need,), torch.uint8, dev, stream)
    return _arg(workspace, "workspace", workspace.dtype, workspace.shape, dev), workspace.nbytes, workspace


def _index(t: Optional[torch.Tensor], name: str, dev):
    """Address of a row index of any length (None stays None)."""
    return None if t is None else _arg(t, name, torch.int32, (t.shape[0],), dev)


def moe_grouped_mm(a: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, row_index: Optional[torch.Tensor] = None,
                   transposed: bool = False, out: Optional[torch.Tensor] = None, dtype=None, stream=None) -> torch.Tensor:
    """Rows grouped by expert times their expert's matrix -> out [R_cap, N] of ``dtype`` (default: a's).

    ``w`` is [E_loc, N, K] (a projection), or [E_loc, K, N] with ``transposed`` (the gradient of its input).  Row r reads
    a[row_index[r]], or a[r].  R_cap is the length of ``row_index``, of ``out``, or of ``a``; rows behind offsets[-1]
    are left as they were."""
    dev, i32 = a.device, torch.int32
    if a.dim() != 2 or w.dim() != 3:
        raise ValueError("a must be [rows, K], w [E_loc, N, K] (transposed: [E_loc, K, N])")
    El, N, K = w.shape
    if transposed:
        N, K = K, N
    R = out.shape[0] if out is not None else (row_index if row_index is not None else a).shape[0]
    if row_index is not None and row_index.shape[0] < R:
        raise ValueError(f"row_index has {row_index.shape[0]} entries for {R} rows")
    if out is None:
        _out_dtype(a.dtype if dtype is None else dtype)
        out = _new((R, N), a.dtype if dtype is None else dtype, dev, stream)
    args = (_arg(a, "a", a.dtype, (a.shape[0], K), dev),
            _index(row_index, "row_index", dev), a.shape[0],
            _arg(w, "w", a.dtype, w.shape, dev), _out_dtype(a.dtype), _arg(offsets, "offsets", i32, (El + 1,), dev), El, R, N,
            K, _arg(out, "out", out.dtype, (R, N), dev), _out_dtype(out.dtype), MOE_MM_TRANSPOSED if transposed else 0)
    with _On(dev) as on:
        _check("moe_grouped_mm", lib().moe_grouped_mm(*args, on.stream(stream)))
    return out


def moe_grouped_wgrad_workspace_size(E_loc: int, R_cap: int, M: int, N: int, dtype=torch.bfloat16) -> int:
    return int(lib().moe_grouped_wgrad_workspace_size(E_loc, R_cap, M, N, _out_dtype(dtype)))


def moe_grouped_wgrad(a: torch.Tensor, b: torch.Tensor, offsets: torch.Tensor, a_index: Optional[torch.Tensor] = None,
                      b_index: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None, add: bool = False,
                      dtype=None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Weight gradient of a grouped product: out[e] = (out[e] if add) + sum over e's rows of a_r b_r^T -> [E_loc, M, N]
    of ``dtype`` (default: a's).  ``a`` [rows, M] is the gradient of the product, ``b`` [rows, N] its input; either may
    be gathered by an index of its rows."""
    dev, i32 = a.device, torch.int32
    if a.dim() != 2 or b.dim() != 2:
        raise ValueError("a must be [rows, M] and b [rows, N]")
    El, M, N = offsets.shape[0] - 1, a.shape[1], b.shape[1]
    R = min((t if i is None else i).shape[0] for t, i in ((a, a_index), (b, b_index)))
    if out is None:
        if add:
            raise ValueError("add needs out")
        _out_dtype(a.dtype if dtype is None else dtype)
        out = _new((El, M, N), a.dtype if dtype is None else dtype, dev, stream)
    dt = _out_dtype(a.dtype)
    ws, nws, workspace = _space(workspace, int(lib().moe_grouped_wgrad_workspace_size(El, R, M, N, dt)), dev, stream)
    args = (_arg(a, "a", a.dtype, a.shape, dev),
            _index(a_index, "a_index", dev), a.shape[0],
            _arg(b, "b", a.dtype, b.shape, dev),
            _index(b_index, "b_index", dev), b.shape[0], dt,
            _arg(offsets, "offsets", i32, (El + 1,), dev), El, R, M, N, _arg(out, "out", out.dtype, (El, M, N), dev),
            _out_dtype(out.dtype), ws, nws, MOE_WGRAD_ADD if add else 0)
    with _On(dev) as on:
        _check("moe_grouped_wgrad", lib().moe_grouped_wgrad(*args, on.stream(stream)))
    return out


def _rows_of(offsets: Optional[torch.Tensor], dev):
    """(address of the offsets or None, experts)."""
    if offsets is None:
        return None, 1
    return _arg(offsets, "offsets", torch.int32, (offsets.shape[0],), dev), offsets.shape[0] - 1


def moe_swiglu(gu: torch.Tensor, offsets: Optional[torch.Tensor] = None, row_w: Optional[torch.Tensor] = None,
               h: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """h[r] = row_w[r] silu(gu[r, :I]) gu[r, I:] -> [R_cap, I] of gu's type.  Without ``offsets`` all rows are computed,
    with them those below offsets[-1]."""
    R, I2 = gu.shape
    dev, I = gu.device, I2 // 2
    if h is None:
        h = _new((R, I), gu.dtype, dev, stream)
    off, El = _rows_of(offsets, dev)
    args = (_arg(gu, "gu", gu.dtype, (R, 2 * I), dev), _out_dtype(gu.dtype), off,
            _arg(row_w, "row_w", torch.float32, (R,), dev), El, R, I,
            _arg(h, "h", gu.dtype, (R, I), dev))
    with _On(dev) as on:
        _check("moe_swiglu", lib().moe_swiglu(*args, on.stream(stream)))
    return h


def moe_swiglu_backward(gu: torch.Tensor, dh: torch.Tensor, offsets: Optional[torch.Tensor] = None,
                        row_w: Optional[torch.Tensor] = None, dgu: Optional[torch.Tensor] = None,
                        h: Optional[torch.Tensor] = None, d_row_w: Optional[torch.Tensor] = None, stream=None):
    """Gradient of moe_swiglu -> (dgu [R_cap, 2I], h [R_cap, I] as the forward call gives it, d_row_w [R_cap] or None
    without ``row_w``).  ``dgu`` may be ``gu`` and ``h`` may be ``dh``."""
    R, I2 = gu.shape
    dev, I, f32 = gu.device, I2 // 2, torch.float32
    if dgu is None:
        dgu = _new((R, 2 * I), gu.dtype, dev, stream)
    if h is None:
        h = _new((R, I), gu.dtype, dev, stream)
    if d_row_w is None and row_w is not None:
        d_row_w = _new((R,), f32, dev, stream)
    off, El = _rows_of(offsets, dev)
    args = (_arg(gu, "gu", gu.dtype, (R, 2 * I), dev), _arg(dh, "dh", gu.dtype, (R, I), dev), _out_dtype(gu.dtype), off,
            _arg(row_w, "row_w", f32, (R,), dev), El, R, I,
            _arg(dgu, "dgu", gu.dtype, (R, 2 * I), dev), _arg(h, "h", gu.dtype, (R, I), dev),
            _arg(d_row_w, "d_row_w", f32, (R,), dev))
    with _On(dev) as on:
        _check("moe_swiglu_backward", lib().moe_swiglu_backward(*args, on.stream(stream)))
    return dgu, h, d_row_w


def moe_route_backward(topk_ids: torch.Tensor, topk_w: torch.Tensor, d_topk_w: torch.Tensor, x: torch.Tensor,
                       w_router: torch.Tensor, perm: dict, rows: Optional[torch.Tensor] = None,
                       token_row: Optional[torch.Tensor] = None, dx: Optional[torch.Tensor] = None, dtype=None,
                       dw_router: Optional[torch.Tensor] = None, d_bias: Optional[torch.Tensor] = None, stream=None):
    """Gradients of the router weight [E, H] and bias [E] (fp32) and of the layer's input [T, H] (``dtype``, default x's)
    from that of the gates -> (dx, dw_router, d_bias).

    ``perm`` is moe_permute's over all E experts.  ``rows`` [R_cap, H] are the input gradients of the local experts' rows,
    which dx sums too; ``token_row`` [T, k] says which (default: perm's, for a layer that holds every expert)."""
    (T, k), (E, H) = topk_ids.shape, w_router.shape
    dev, i32, f32 = x.device, torch.int32, torch.float32
    if dx is None:
        _out_dtype(x.dtype if dtype is None else dtype)
        dx = _new((T, H), x.dtype if dtype is None else dtype, dev, stream)
    if dw_router is None:
        dw_router = _new((E, H), f32, dev, stream)
    if d_bias is None:
        d_bias = _new((E,), f32, dev, stream)
    if rows is not None and token_row is None:
        token_row = perm["token_row"]
    row_token = perm["row_token"]
    if row_token.dim() != 1 or row_token.shape[0] < T * k:
        raise ValueError(f"perm must be over all experts: row_token needs T * k = {T * k} entries")
    args = (_arg(topk_ids, "topk_ids", i32, (T, k), dev), _arg(topk_w, "topk_w", f32, (T, k), dev),
            _arg(d_topk_w, "d_topk_w", f32, (T, k), dev), T, k, E, H, _arg(x, "x", x.dtype, (T, H), dev),
            _arg(w_router, "w_router", x.dtype, (E, H), dev), _out_dtype(x.dtype),
            _arg(perm["offsets"], "perm offsets", i32, (E + 1,), dev),
            _arg(row_token, "perm row_token", i32, row_token.shape, dev),
            None if rows is None else _arg(rows, "rows", rows.dtype, (rows.shape[0], H), dev),
            MOE_F32 if rows is None else _out_dtype(rows.dtype),
            None if rows is None else _arg(token_row, "token_row", i32, (T, k), dev),
            0 if rows is None else rows.shape[0], _arg(dx, "dx", dx.dtype, (T, H), dev), _out_dtype(dx.dtype),
            _arg(dw_router, "dw_router", f32, (E, H), dev), _arg(d_bias, "d_bias", f32, (E,), dev))
    with _On(dev) as on:
        _check("moe_route_backward", lib().moe_route_backward(*args, on.stream(stream)))
    return dx, dw_router, d_bias


def _norm_weights(T, H, dev, w_next, w_post, gate):
    """MOE_* type and gate kind of the norms' weights and gate, and their addresses; all of one type."""
    first = w_next if w_next is not None else w_post if w_post is not None else gate
    if first is None:
        return MOE_F32, MOE_GATE_NONE, None, None, None
    dt, kind, row = first.dtype, MOE_GATE_NONE, (H,)
    if gate is not None:
        kind = MOE_GATE_CHANNEL if gate.dim() == 1 else MOE_GATE_TOKEN
    return (_out_dtype(dt), kind, _arg(w_next, "w_next", dt, row, dev), _arg(w_post, "w_post", dt, row, dev),
            _arg(gate, "gate", dt, row if kind == MOE_GATE_CHANNEL else (T, 1), dev))


def moe_block_norm(x: torch.Tensor, w_next: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                   w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, scale: float = 1.0,
                   eps: float = 1e-6, x_out: Optional[torch.Tensor] = None, n: Optional[torch.Tensor] = None,
                   stats: bool = False, stream=None):
    """The residual around a block with the RMS norms after it and before the next one ->
    (x_out, n, rstd_next, rstd_post):

    x_out = scale x + gate rms(y) w_post (without ``w_post``: scale x + gate y), n = rms(x_out) w_next.  ``gate`` is [H]
    (per channel) or [T, 1] (per token).  Without ``y``: n = rms(x) w_next alone, x_out None.  Without ``w_next``: n None.
    With ``stats`` the reciprocal roots [T] that the backward pass needs are returned too, else None.  ``x_out`` may be
    ``x`` itself."""
    T, H = x.shape
    dev, f32 = x.device, torch.float32
    if y is not None and x_out is None:
        x_out = _new((T, H), x.dtype, dev, stream)
    if w_next is not None and n is None:
        n = _new((T, H), x.dtype, dev, stream)
    rn = _new((T,), f32, dev, stream) if stats and w_next is not None else None
    rp = _new((T,), f32, dev, stream) if stats and w_post is not None else None
    wdt, kind, wn, wp, g = _norm_weights(T, H, dev, w_next, w_post, gate)
    xdt, all_ = x.dtype, (T, H)
    yp, ydt = (None, MOE_F32) if y is None else (_arg(y, "y", y.dtype, all_, dev), _out_dtype(y.dtype))
    args = (_arg(x, "x", xdt, all_, dev), _out_dtype(xdt), yp, ydt, wn, wp, g, wdt, kind, scale, eps, T, H,
            _arg(x_out, "x_out", xdt, all_, dev), _arg(n, "n", xdt, all_, dev), None if rn is None else rn.data_ptr(),
            None if rp is None else rp.data_ptr())
    with _On(dev) as on:
        _check("moe_block_norm", lib().moe_block_norm(*args, on.stream(stream)))
    return x_out, n, rn, rp


def moe_block_norm_backward_workspace_size(T: int, H: int) -> int:
    return int(lib().moe_block_norm_backward_workspace_size(T, H))


def moe_block_norm_backward(x_out: torch.Tensor, w_next: Optional[torch.Tensor] = None,
                            rstd_next: Optional[torch.Tensor] = None, dn: Optional[torch.Tensor] = None,
                            dx_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                            w_post: Optional[torch.Tensor] = None, rstd_post: Optional[torch.Tensor] = None,
                            gate: Optional[torch.Tensor] = None, scale: float = 1.0, dx: Optional[torch.Tensor] = None,
                            dy: Optional[torch.Tensor] = None, dy_dtype=None,
                            workspace: Optional[torch.Tensor] = None, stream=None) -> dict:
    """Gradient of moe_block_norm -> dict(dx, dy, dw_next, dw_post, dgate), None for what the call had not.

    ``x_out`` is the sum that the forward call gave (without ``y``: x), ``rstd_next`` and ``rstd_post`` its reciprocal
    roots; ``dn`` and ``dx_out`` the gradients of its results, either may be missing.  dw_next, dw_post and dgate are
    fp32, dy is of ``dy_dtype`` (default: y's).  ``dx`` may be ``dx_out`` or ``dn`` itself."""
    T, H = x_out.shape
    dev, f32 = x_out.device, torch.float32
    if dx is None:
        dx = _new((T, H), x_out.dtype, dev, stream)
    if y is not None and dy is None:
        _out_dtype(y.dtype if dy_dtype is None else dy_dtype)
        dy = _new((T, H), y.dtype if dy_dtype is None else dy_dtype, dev, stream)
    dwn = _new((H,), f32, dev, stream) if w_next is not None else None
    dwp = _new((H,), f32, dev, stream) if w_post is not None else None
    dg = _new(gate.shape, f32, dev, stream) if gate is not None else None
    ws, nws, workspace = _space(workspace, int(lib().moe_block_norm_backward_workspace_size(T, H)), dev, stream)
    wdt, kind, wn, wp, g = _norm_weights(T, H, dev, w_next, w_post, gate)
    xdt, all_ = x_out.dtype, (T, H)
    yp, dyp, ydt, dydt = None, None, MOE_F32, MOE_F32
    if y is not None:
        yp, dyp, ydt, dydt = (_arg(y, "y", y.dtype, all_, dev), _arg(dy, "dy", dy.dtype, all_, dev), _out_dtype(y.dtype),
                              _out_dtype(dy.dtype))
    args = (_arg(x_out, "x_out", xdt, all_, dev), _out_dtype(xdt), yp, ydt, wn, wp, g, wdt, kind, scale,
            _arg(rstd_next, "rstd_next", f32, (T,), dev), _arg(rstd_post, "rstd_post", f32, (T,), dev),
            _arg(dx_out, "dx_out", xdt, all_, dev), _arg(dn, "dn", xdt, all_, dev), T, H, _arg(dx, "dx", xdt, all_, dev), dyp, dydt,
            None if dwn is None else dwn.data_ptr(), None if dwp is None else dwp.data_ptr(),
            None if dg is None else dg.data_ptr(), ws, nws)
    with _On(dev) as on:
        _check("moe_block_norm_backward", lib().moe_block_norm_backward(*args, on.stream(stream)))
    return {"dx": dx, "dy": dy, "dw_next": dwn, "dw_post": dwp, "dgate": dg}
