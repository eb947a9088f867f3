"""Both passes of a MoE block for training: pre-norm, router, experts, and the residual with the norm after the experts.

Host logic only, as in layer.py: which library call reads what.  The gradients are explicit results (no autograd graph),
so a step can run on any stream and be captured into a HIP graph.

    out, saved = block_forward(dev, x)
    grads = block_backward(dev, saved, d_out)

``dev`` is what layer.to_device gives (row-major bf16 or fp32 weights, of the activations' type) with the norms' weights
added: "norm_pre" [H] and optionally "norm_post" [H], "gate" ([H] or [T, 1]), "scale" and "eps".  The pieces can be
called on their own: ``experts_forward`` / ``experts_backward`` for the experts alone, on moe_permute's maps.

The gate of an assignment multiplies its intermediate row rather than the expert's output (moe_swiglu): the down
projection is linear, so the combined output is the plain sum of the rows, and the gradient of a gate is a dot product of
rows that the backward pass has at hand.  Nothing per row and hidden column is kept for the backward pass.
"""
from __future__ import annotations

from typing import Optional

import torch

from . import moe
from .layer import _on


def _rows(perm: dict) -> int:
    return perm["R_cap"] if "R_cap" in perm else perm["row_token"].shape[0]


def experts_forward(x: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor, perm: dict, stream=None):
    """SwiGLU experts [E_loc, 2I, H] and [E_loc, H, I] on the rows of ``perm`` (moe_permute), summed with the gates to
    token order -> (y [T, H] fp32, saved).  x [T, H] of the weights' type, H a multiple of 4."""
    T, k = perm["token_row"].shape
    R = _rows(perm)
    row_token, row_w = perm["row_token"][:R], perm["row_w"][:R]
    with _on(x):
        gu = moe.moe_grouped_mm(x, w_gate_up, perm["offsets"], row_index=row_token, stream=stream)
        h = moe.moe_swiglu(gu, perm["offsets"], row_w, stream=stream)
        rows = moe.moe_grouped_mm(h, w_down, perm["offsets"], dtype=torch.float32, stream=stream)
        ones = moe._new((T, k), torch.float32, x.device, stream)
        with torch.cuda.stream(moe.torch_stream(stream, x.device)):
            ones.fill_(1.0)
        y = moe.moe_combine(rows, perm["token_row"], ones, stream=stream)
    return y, {"x": x, "gu": gu, "perm": perm}


def experts_backward(saved: dict, dy: torch.Tensor, w_gate_up: torch.Tensor, w_down: torch.Tensor,
                     dw_gate_up: Optional[torch.Tensor] = None, dw_down: Optional[torch.Tensor] = None, add: bool = False,
                     dtype=torch.float32, stream=None) -> dict:
    """Gradient of experts_forward for ``dy`` [T, H] of the weights' type -> dict(dw_gate_up, dw_down, dx_rows, d_gates).

    The weights' gradients are of ``dtype``, or written to (``add``: added to) the tensors given.  ``dx_rows`` [R_cap, H]
    are the input gradients row by row, which moe_route_backward sums to tokens; ``d_gates`` [T, k] is zero for experts of
    other ranks."""
    perm, x, gu = saved["perm"], saved["x"], saved["gu"]
    off, R = perm["offsets"], _rows(perm)
    row_token, row_w, token_row = perm["row_token"][:R], perm["row_w"][:R], perm["token_row"]
    with _on(x):
        dh = moe.moe_grouped_mm(dy, w_down, off, row_index=row_token, transposed=True, stream=stream)
        dgu, h, d_row_w = moe.moe_swiglu_backward(gu, dh, off, row_w, h=dh, stream=stream)
        dw_down = moe.moe_grouped_wgrad(dy, h, off, a_index=row_token, out=dw_down, add=add, dtype=dtype, stream=stream)
        dw_gate_up = moe.moe_grouped_wgrad(dgu, x, off, b_index=row_token, out=dw_gate_up, add=add, dtype=dtype, stream=stream)
        dx_rows = moe.moe_grouped_mm(dgu, w_gate_up, off, transposed=True, stream=stream)
        with torch.cuda.stream(moe.torch_stream(stream, x.device)):
            at = token_row.clamp(min=0).long()
            d_gates = torch.where(token_row >= 0, d_row_w[at], 0.0) if R > 0 else torch.zeros_like(token_row, dtype=torch.float32)
    return {"dw_gate_up": dw_gate_up, "dw_down": dw_down, "dx_rows": dx_rows, "d_gates": d_gates}


def _check(dev: dict):
    cfg = dev["cfg"]
    if dev.get("packed") or cfg.wdt != cfg.act or cfg.act not in ("bf16", "f32"):
        raise ValueError("training takes row-major weights of the activations' type (bf16 or fp32)")
    if cfg.I_s > 0:
        raise ValueError("a block with a shared expert is not trained here")
    if cfg.E_loc != cfg.E:
        raise ValueError("a block is trained with all of its experts; a share of them: experts_forward and experts_backward, "
                         "with sums over the ranks in between")
    return cfg


def block_forward(dev: dict, x: torch.Tensor, stream=None):
    """x [T, H] (the residual stream, of the model's type) -> (out [T, H], saved):

    n = rms(x) norm_pre;  y = experts(n), routed by the router on n;  out = scale x + gate rms(y) norm_post
    (without "norm_post": scale x + gate y)."""
    cfg = _check(dev)
    scale, eps = dev.get("scale", 1.0), dev.get("eps", 1e-6)
    with _on(x):
        _, n, rstd_pre, _ = moe.moe_block_norm(x, dev["norm_pre"], eps=eps, stats=True, stream=stream)
        ids, gates = moe.moe_route(n, dev["w_router"], dev["bias"], cfg.k, stream=stream)
        perm = moe.moe_permute(ids, gates, cfg.E, 0, cfg.E, stream=stream)
        y, saved = experts_forward(n, dev["w_gate_up"], dev["w_down"], perm, stream=stream)
        out, _, _, rstd_post = moe.moe_block_norm(x, y=y, w_post=dev.get("norm_post"), gate=dev.get("gate"), scale=scale,
                                                  eps=eps, stats=True, stream=stream)
    return out, {"x": x, "rstd_pre": rstd_pre, "ids": ids, "gates": gates, "y": y, "out": out,
                 "rstd_post": rstd_post, "experts": saved}


def block_backward(dev: dict, saved: dict, d_out: torch.Tensor, grads: Optional[dict] = None, dtype=torch.float32,
                   stream=None) -> dict:
    """Gradients of block_forward for ``d_out`` [T, H] -> dict(dx, w_gate_up, w_down, w_router, bias, norm_pre, norm_post,
    gate), None for what the block has not.

    ``grads``: the dict of an earlier call.  Its w_gate_up and w_down (of ``dtype``; by far the largest) are added to in place
    and come back as the sums.  All other entries are of this call alone, with ``grads`` too: who accumulates over calls
    adds those up, before the earlier dict is let go."""
    _check(dev)
    scale, act = dev.get("scale", 1.0), saved["x"].dtype
    with _on(d_out):
        post = moe.moe_block_norm_backward(saved["out"], dx_out=d_out, y=saved["y"], w_post=dev.get("norm_post"),
                                           rstd_post=saved["rstd_post"], gate=dev.get("gate"), scale=scale, dy_dtype=act,
                                           stream=stream)
        ex = experts_backward(saved["experts"], post["dy"], dev["w_gate_up"], dev["w_down"],
                              dw_gate_up=None if grads is None else grads["w_gate_up"],
                              dw_down=None if grads is None else grads["w_down"], add=grads is not None, dtype=dtype,
                              stream=stream)
        dn, dw_router, d_bias = moe.moe_route_backward(saved["ids"], saved["gates"], ex["d_gates"], saved["experts"]["x"],
                                                       dev["w_router"], saved["experts"]["perm"], rows=ex["dx_rows"],
                                                       stream=stream)
        pre = moe.moe_block_norm_backward(saved["x"], dev["norm_pre"], saved["rstd_pre"], dn, dx_out=post["dx"],
                                          dx=post["dx"], stream=stream)
    return {"dx": pre["dx"], "w_gate_up": ex["dw_gate_up"], "w_down": ex["dw_down"], "w_router": dw_router,
            "bias": None if dev["bias"] is None else d_bias,
            "norm_pre": pre["dw_next"], "norm_post": post["dw_post"], "gate": post["dgate"]}
