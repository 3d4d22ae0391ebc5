"""Python binding of include/paro_block.h: what surrounds the products of a decoder block. The W8A8 product with
bias, activation and residual, the norms around a block with gate and residual scale, and a mixture-of-experts layer
on INT4 weights for a few tokens. Argument marshalling only, forward only, the names those of the C ABI; as in the
8-bit path a call whose operands are as they should be goes through the compiled ``_binding``, any other one through
the checks here.
"""
from __future__ import annotations

import ctypes

import torch

from . import F16, F32, GROUP, _i, _lib, _on_gpu, _ptr, _sz, _vp, _want, _want_ws
from .w8a8 import _DTYPE, _binding, _call, _channels, _f, _forward_only, _rot_p, _rows, paro_w8a8_workspace_bytes

MOE_MAX_M, MOE_MAX_E, MOE_MAX_K = 64, 512, 16
ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4, "gelu_tanh": 5}
SCORINGS = {"softmax": 0, "sigmoid": 1}


class paro_w4_experts(ctypes.Structure):
    """INT4 weights of all experts (include/paro_block.h)."""
    _fields_ = [("qweight", _vp), ("scales", _vp), ("zeros", _vp)]


_experts_p = ctypes.POINTER(paro_w4_experts)
_SIGNATURES = {
    "paro_w8a8_linear_epilogue": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _vp, _i, _vp, _sz, _vp]),
    "paro_block_norm_q8": (_i, [_i, _i, _i, _vp, _vp, _vp, _i, _vp, _f, _vp, _f, _vp, _vp, _vp, _vp]),
    "paro_block_norm": (_i, [_i, _i, _i, _vp, _vp, _vp, _i, _vp, _f, _vp, _f, _vp, _vp, _vp]),
    "paro_moe_route_workspace_bytes": (_sz, [_i, _i]),
    "paro_moe_route": (_i, [_i, _i, _i, _i, _vp, _vp, _i, _i, _i, _vp, _vp, _vp, _sz, _vp]),
    "paro_moe_workspace_bytes": (_sz, [_i, _i, _i, _i, _i]),
    "paro_moe_w4a16": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _vp, _rot_p, _rot_p, _experts_p, _experts_p, _vp, _i, _vp, _sz, _vp]),
    "paro_moe_layer_w4a16": (_i, [_i, _i, _i, _i, _i, _vp, _vp, _i, _i, _i, _rot_p, _rot_p, _experts_p, _experts_p, _vp, _i, _vp, _vp,
                                  _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args
EXPORTS_BLOCK = tuple(_SIGNATURES)
_binding.bind_block(*(ctypes.cast(getattr(_lib, _name), _vp).value for _name in EXPORTS_BLOCK))


def _one_of(table, name, what):
    if name not in table:
        raise ValueError(f"{what} must be one of {', '.join(table)}, got {name!r}")
    return table[name]


def paro_w8a8_linear_epilogue(x, x_scales, qweight, w_scales, bias=None, activation="none", residual=None, out_dtype=None, out=None,
                              ws=None):
    """y = act(x . qweight^T + bias) + residual, the product that of paro_w8a8_linear: bias [N] and residual [M][N] in
    y's type (each optional), activation one of "none", "relu", "relu2" (its square), "silu", "gelu", "gelu_tanh". The
    type of y is out_dtype, or that of out, residual or bias, or float16. ``out`` may be ``residual`` itself."""
    act = _one_of(ACTIVATIONS, activation, "activation")
    y = _binding.linear_epilogue(x, x_scales, qweight, w_scales, bias, act, residual, out_dtype, out, ws)
    if y is not None:
        return y
    for t, what in ((x, "x"), (qweight, "qweight")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{what} must be a torch.Tensor with two dimensions")
    (M, D), N = x.shape, qweight.shape[0]
    _want(x, torch.int8, (M, D), "x")
    _want(qweight, torch.int8, (N, D), "qweight")
    _want(x_scales, torch.float32, (M,), "x_scales")
    _want(w_scales, torch.float32, (N,), "w_scales")
    _channels(D)
    dtype = out_dtype or next((t.dtype for t in (out, residual, bias) if t is not None), torch.float16)
    if dtype not in _DTYPE:
        raise TypeError(f"the output must be float16, bfloat16 or float32, got {dtype}")
    for t, shape, what in ((bias, (N,), "bias"), (residual, (M, N), "residual"), (out, (M, N), "out")):
        if t is not None:
            _want(t, dtype, shape, what)
    _want_ws(ws)
    named = {"x": x, "x_scales": x_scales, "qweight": qweight, "w_scales": w_scales, "bias": bias, "residual": residual, "out": out,
             "ws": ws}
    _forward_only(named)
    dev = _on_gpu(named)
    y = torch.empty((M, N), dtype=dtype, device=dev) if out is None else out
    if ws is None and paro_w8a8_workspace_bytes(M, D, N):
        ws = torch.empty(paro_w8a8_workspace_bytes(M, D, N), dtype=torch.uint8, device=dev)
    _call(_lib.paro_w8a8_linear_epilogue, "paro_w8a8_linear_epilogue", dev, M, D, N, _ptr(x), _ptr(x_scales), _ptr(qweight),
          _ptr(w_scales), _ptr(bias), act, _ptr(residual), _ptr(y), _DTYPE[dtype], _ptr(ws), 0 if ws is None else ws.numel(),
          wrote=(out,))
    return y


def _block_norm(q8, x, residual, gamma, eps, post_gamma, gate, residual_scale, residual_out, outs):
    r = _binding.block_norm(q8, x, residual, gamma, eps, post_gamma, gate, residual_scale, residual_out, outs[0], outs[-1])
    if r is not None:
        return r
    M, D = _rows(x, "x")
    _want(residual, x.dtype, (M, D), "residual")
    _want(gamma, x.dtype, (D,), "gamma")
    if post_gamma is not None:
        _want(post_gamma, x.dtype, (D,), "post_gamma")
    gate_rows = 1
    if gate is not None:
        if not isinstance(gate, torch.Tensor) or gate.dim() not in (1, 2):
            raise ValueError("gate must be a torch.Tensor with one or two dimensions")
        gates = 1 if gate.dim() == 1 else gate.shape[0]
        _want(gate, x.dtype, (D,) if gate.dim() == 1 else (gates, D), "gate")
        if M and (gates < 1 or M % gates):
            raise ValueError(f"gate has {gates} rows, which do not divide the {M} of x")
        gate_rows = max(1, M // max(1, gates))
    if residual_out is not None:
        _want(residual_out, x.dtype, (M, D), "residual_out")
    kinds = ((torch.int8, (M, D), "q"), (torch.float32, (M,), "scales")) if q8 else ((x.dtype, (M, D), "out"),)
    for t, kind in zip(outs, kinds):
        if t is not None:
            _want(t, *kind)
    named = {"x": x, "residual": residual, "gamma": gamma, "post_gamma": post_gamma, "gate": gate, "residual_out": residual_out,
             **{k[2]: t for t, k in zip(outs, kinds)}}
    _forward_only(named)
    dev = _on_gpu(named)
    wrote = (residual_out, *outs)
    outs = [torch.empty(k[1], dtype=k[0], device=dev) if t is None else t for t, k in zip(outs, kinds)]
    if residual_out is None:
        residual_out = torch.empty_like(residual)
    name = "paro_block_norm_q8" if q8 else "paro_block_norm"
    _call(getattr(_lib, name), name, dev, M, D, _DTYPE[x.dtype], _ptr(x), _ptr(post_gamma), _ptr(gate), gate_rows, _ptr(residual),
          residual_scale, _ptr(gamma), eps, _ptr(residual_out), *map(_ptr, outs), wrote=wrote)
    return (*outs, residual_out)


def paro_block_norm_q8(x, residual, gamma, eps=1e-6, post_gamma=None, gate=None, residual_scale=1.0, out=None, residual_out=None):
    """From a block's output x and the residual stream to the next block's rows, in one kernel: p = x, or its RMS norm
    times post_gamma; h = residual_scale * residual + gate * p, rounded to x's type; then the RMS norm of h times gamma
    in 8 bits: (q int8 [M][D], scales float32 [M], h). x, residual float16 or bfloat16 [M][D]; gamma, post_gamma [D];
    gate [D], or [B][D] with B dividing M: one for each M / B rows in turn. ``out``: an optional (q, scales) pair;
    ``residual_out``: where h goes (it may be ``residual`` itself)."""
    q, scales = (None, None) if out is None else out
    return _block_norm(True, x, residual, gamma, eps, post_gamma, gate, residual_scale, residual_out, (q, scales))


def paro_block_norm(x, residual, gamma, eps=1e-6, post_gamma=None, gate=None, residual_scale=1.0, out=None, residual_out=None):
    """The same with the last norm's rows in x's type: (y [M][D], h). ``out``: an optional tensor for y."""
    return _block_norm(False, x, residual, gamma, eps, post_gamma, gate, residual_scale, residual_out, (out,))


def paro_moe_route_workspace_bytes(M: int, E: int) -> int:
    return _lib.paro_moe_route_workspace_bytes(M, E)


def paro_moe_workspace_bytes(M: int, D: int, F: int, E: int, top_k: int) -> int:
    return _lib.paro_moe_workspace_bytes(M, D, F, E, top_k)


def _tokens(x, top_k):
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError("x must be a torch.Tensor with two dimensions")
    M, D = x.shape
    _want(x, torch.float16, (M, D), "x")
    _channels(D)
    if M > MOE_MAX_M:
        raise ValueError(f"x has {M} tokens, the mixture-of-experts calls take {MOE_MAX_M} at most")
    if not 1 <= top_k <= MOE_MAX_K:
        raise ValueError(f"top_k must be 1 to {MOE_MAX_K}, got {top_k}")
    return M, D


def _router(x, router, top_k):
    """(M, D, E) of a router's operands."""
    M, D = _tokens(x, top_k)
    if not isinstance(router, torch.Tensor) or router.dim() != 2:
        raise ValueError("router must be a torch.Tensor with two dimensions")
    E = router.shape[0]
    if router.dtype not in (torch.float16, torch.float32):
        raise TypeError(f"router must be torch.float16 or torch.float32, got {router.dtype}")
    _want(router, router.dtype, (E, D), "router")
    if not top_k <= E <= MOE_MAX_E:
        raise ValueError(f"the router has {E} experts, it must have top_k = {top_k} to {MOE_MAX_E}")
    return M, D, E


def _routing(given, M, top_k):
    ids, weights = (None, None) if given is None else given
    if ids is not None:
        _want(ids, torch.int32, (M, top_k), "ids")
    if weights is not None:
        _want(weights, torch.float32, (M, top_k), "weights")
    return ids, weights


def paro_moe_route(x, router, top_k, scoring="softmax", renormalize=True, out=None, ws=None):
    """The top_k experts of each token and their weights: (ids int32 [M][top_k], weights float32 [M][top_k]), by the
    logits x . router^T, largest first, the lower index among equals. x float16 [M][D], M <= 64; router float16 or
    float32 [E][D]; scoring "softmax" (over all experts) or "sigmoid", divided by its sum over the top_k with
    ``renormalize``. ``out``: an optional (ids, weights) pair to write."""
    how = _one_of(SCORINGS, scoring, "scoring")
    r = _binding.route(x, router, top_k, how, bool(renormalize), *((None, None) if out is None else out), ws)
    if r is not None:
        return r
    M, D, E = _router(x, router, top_k)
    ids, weights = given = _routing(out, M, top_k)
    _want_ws(ws)
    named = {"x": x, "router": router, "ids": ids, "weights": weights, "ws": ws}
    _forward_only(named)
    dev = _on_gpu(named)
    ids = torch.empty((M, top_k), dtype=torch.int32, device=dev) if ids is None else ids
    weights = torch.empty((M, top_k), dtype=torch.float32, device=dev) if weights is None else weights
    if ws is None:
        ws = torch.empty(paro_moe_route_workspace_bytes(M, E), dtype=torch.uint8, device=dev)
    _call(_lib.paro_moe_route, "paro_moe_route", dev, M, D, E, top_k, _ptr(x), _ptr(router), _DTYPE[router.dtype], how,
          int(bool(renormalize)), _ptr(ids), _ptr(weights), _ptr(ws), ws.numel(), wrote=given)
    return ids, weights


def _packed(packed, what, E, N, D):
    qweight, scales, zeros = packed
    _want(qweight, torch.uint8, (E, N, D // 2), f"{what} qweight")
    _want(scales, torch.float16, (E, N, D // GROUP), f"{what} scales")
    _want(zeros, torch.float16, (E, N, D // GROUP), f"{what} zeros")
    return paro_w4_experts(qweight.data_ptr(), scales.data_ptr(), zeros.data_ptr())


def _experts(M, D, E, top_k, gate_up, down, rot_x, rot_a, out_dtype, out, ws, named):
    """Check the experts' operands; returns (F, C structs, y, y's type, ws, device). named: the call's other tensors."""
    if not isinstance(gate_up[0], torch.Tensor) or gate_up[0].dim() != 3 or gate_up[0].shape[1] % 2:
        raise ValueError("gate_up qweight must have three dimensions and as many gate rows as up rows")
    F = gate_up[0].shape[1] // 2
    _channels(F)
    E = gate_up[0].shape[0] if E is None else E
    if not 1 <= E <= MOE_MAX_E:
        raise ValueError(f"gate_up has {E} experts, it must have 1 to {MOE_MAX_E}")
    structs = _packed(gate_up, "gate_up", E, 2 * F, D), _packed(down, "down", E, D, F)
    for rot, channels, what in ((rot_x, D, "rot_x"), (rot_a, F, "rot_a")):
        if rot is not None and rot.D != channels:
            raise ValueError(f"{what} has {rot.D} channels, its rows {channels}")
    dtype = out_dtype or (out.dtype if out is not None else torch.float16)
    if dtype not in (torch.float16, torch.float32):
        raise TypeError(f"the output must be float16 or float32, got {dtype}")
    if out is not None:
        _want(out, dtype, (M, D), "out")
    _want_ws(ws)
    named = {**named, "out": out, "ws": ws, "rot_x": None if rot_x is None else rot_x.desc, "rot_a": None if rot_a is None else rot_a.desc,
             **{f"{what} {part}": t for what, packed in (("gate_up", gate_up), ("down", down))
                for part, t in zip(("qweight", "scales", "zeros"), packed)}}
    _forward_only(named)
    dev = _on_gpu(named)
    y = torch.empty((M, D), dtype=dtype, device=dev) if out is None else out
    if ws is None:
        ws = torch.empty(paro_moe_workspace_bytes(M, D, F, E, top_k), dtype=torch.uint8, device=dev)
    return E, F, structs, y, F32 if dtype == torch.float32 else F16, ws, dev


def _rot(rot):
    return None if rot is None else rot.ptr


def _compiled(x, router, top_k, how, renormalize, ids, weights, gate_up, down, rot_x, rot_a, out_dtype, out, ws):
    rots = [v for r in (rot_x, rot_a) for v in ((0, None) if r is None else (ctypes.addressof(r.handle), r.desc))]
    return _binding.moe(x, router, top_k, how, renormalize, ids, weights, gate_up, down, *rots, out_dtype, out, ws)


def paro_moe_w4a16(x, ids, weights, gate_up, down, rot_x=None, rot_a=None, out_dtype=None, out=None, ws=None):
    """The experts of up to 64 tokens on INT4 weights: y[m] = sum_j weights[m][j] * down_e(silu(gate_e x) * up_e x) with
    e = ids[m][j]; an id outside 0..E-1 takes no expert. x float16 [M][D]; ids int32, weights float32 [M][top_k];
    gate_up a (qweight uint8 [E][2F][D/2], scales, zeros float16 [E][2F][D/128]) triple, gate rows first, as
    paro_pack_weights packs the E * 2F rows; down the same [E][D][F]. rot_x, rot_a: the transforms (of D and of F
    channels) that gate_up's and down's rows were packed with. y float16 (default) or float32 [M][D]."""
    y = _compiled(x, None, None, None, None, ids, weights, gate_up, down, rot_x, rot_a, out_dtype, out, ws)
    if y is not None:
        return y
    if not isinstance(ids, torch.Tensor) or ids.dim() != 2:
        raise ValueError("ids must be a torch.Tensor with two dimensions")
    top_k = ids.shape[1]
    M, D = _tokens(x, top_k)
    if weights is None:
        raise ValueError("weights are required")
    _routing((ids, weights), M, top_k)
    E, F, (gu, dn), y, ydtype, ws, dev = _experts(M, D, None, top_k, gate_up, down, rot_x, rot_a, out_dtype, out, ws,
                                                  {"x": x, "ids": ids, "weights": weights})
    _call(_lib.paro_moe_w4a16, "paro_moe_w4a16", dev, M, D, F, E, top_k, _ptr(x), _ptr(ids), _ptr(weights), _rot(rot_x), _rot(rot_a),
          ctypes.byref(gu), ctypes.byref(dn), _ptr(y), ydtype, _ptr(ws), ws.numel(), wrote=(out,))
    return y


def paro_moe_layer_w4a16(x, router, top_k, gate_up, down, rot_x=None, rot_a=None, scoring="softmax", renormalize=True, out_dtype=None,
                         out=None, routing=None, ws=None):
    """The whole mixture-of-experts layer for up to 64 tokens: paro_moe_route, then paro_moe_w4a16 with what it chose, in
    one call: (y, ids, weights). The router sees x itself, not its transform. ``routing``: an optional (ids, weights)
    pair to write."""
    how = _one_of(SCORINGS, scoring, "scoring")
    r = _compiled(x, router, top_k, how, bool(renormalize), *((None, None) if routing is None else routing), gate_up, down, rot_x, rot_a,
                  out_dtype, out, ws)
    if r is not None:
        return r
    M, D, E = _router(x, router, top_k)
    ids, weights = given = _routing(routing, M, top_k)
    E, F, (gu, dn), y, ydtype, ws, dev = _experts(M, D, E, top_k, gate_up, down, rot_x, rot_a, out_dtype, out, ws,
                                                  {"x": x, "router": router, "ids": ids, "weights": weights})
    ids = torch.empty((M, top_k), dtype=torch.int32, device=dev) if ids is None else ids
    weights = torch.empty((M, top_k), dtype=torch.float32, device=dev) if weights is None else weights
    _call(_lib.paro_moe_layer_w4a16, "paro_moe_layer_w4a16", dev, M, D, F, E, top_k, _ptr(x), _ptr(router), _DTYPE[router.dtype], how,
          int(bool(renormalize)), _rot(rot_x), _rot(rot_a), ctypes.byref(gu), ctypes.byref(dn), _ptr(y), ydtype, _ptr(ids), _ptr(weights),
          _ptr(ws), ws.numel(), wrote=(out, *given))
    return y, ids, weights
