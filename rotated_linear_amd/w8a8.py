"""Python binding of the 8-bit path (include/paro_w8a8.h): residual RMS norm, row quantisation,
8-bit weights and the W8A8 products. Argument marshalling only, as in the package; the names mirror
the C ABI. The calls are forward only: with gradients enabled a tensor that requires one is refused
(weights to be packed aside, which become constants).

A decode-sized call takes a few microseconds on the GPU, so a call whose operands are as they should
be goes through the compiled ``_binding`` (checks, outputs and the C call in one step). Where that
declines (it returns None and has done nothing), the functions here check the operands one by one,
say what is wrong, or make the call on another GPU than the current one. Without the extension, or
with one that was built for another torch, every call goes that way: the same kernels, some 4 us more
of host time each.
"""
from __future__ import annotations

import ctypes
import re
import warnings

import torch

from . import F16, F32, GROUP, MAX_D, ParoError, _check, _i, _lib, _on_gpu, _ptr, _stream_ptr, _sz, _vp, _want, _want_ws, paro_rotation

try:
    from . import _binding
    _for = getattr(_binding, "torch_version", "another version")
    if re.match(r"\d+\.\d+\.\d+", torch.__version__)[0] != _for:  # (its headers name no pre-release)
        raise ImportError(f"it was built for torch {_for}, this is {torch.__version__}")
except ImportError as e:
    warnings.warn(f"rotated_linear_amd runs without its compiled binding ({e}): the 8-bit calls take more host time. "
                  "Build it with `python -m rotated_linear_amd._build`.", RuntimeWarning, stacklevel=2)

    class _binding:  # declines every call
        @staticmethod
        def _declines(*_):
            return None

        bind = linear = quantize = dequantize = rmsnorm = _declines

BF16 = 2
_DTYPE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}

_rot_p = ctypes.POINTER(paro_rotation)
_f = ctypes.c_float
_SIGNATURES = {
    "paro_rmsnorm_q8": (_i, [_i, _i, _i, _vp, _vp, _vp, _f, _vp, _vp, _vp, _vp]),
    "paro_rmsnorm": (_i, [_i, _i, _i, _vp, _vp, _vp, _f, _vp, _vp, _vp]),
    "paro_quantize_q8": (_i, [_rot_p, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "paro_pack_weights_q8": (_i, [_rot_p, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "paro_dequantize_q8": (_i, [_i, _i, _vp, _vp, _vp, _i, _vp]),
    "paro_w8a8_linear": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "paro_w8a8_gated_linear": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "paro_w8a8_workspace_bytes": (_sz, [_i, _i, _i]),
    "paro_w8a8_gated_workspace_bytes": (_sz, [_i, _i, _i]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args
EXPORTS_W8A8 = tuple(_SIGNATURES)
_binding.bind(*(ctypes.cast(getattr(_lib, _name), _vp).value for _name in EXPORTS_W8A8))


def _rows(t, name):
    """Refuse anything but contiguous 2-d float16 or bfloat16 rows of channels the library takes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in (torch.float16, torch.bfloat16):
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    _channels(t.shape[1])
    return t.shape


def _channels(D):
    if D % GROUP or not GROUP <= D <= MAX_D:
        raise ParoError(2, "D")


def _forward_only(named):
    """The calls have no backward pass: refuse a tensor of ``named`` (name -> tensor or None) whose gradient
    would be lost without a word."""
    if torch.is_grad_enabled():
        for name, t in named.items():
            if t is not None and t.requires_grad:
                raise RuntimeError(f"{name} requires a gradient and this call is forward only: "
                                   "detach it, or make the call under torch.no_grad()")


def _call(fn, what, dev, *args, wrote=()):
    """The C call on dev's current stream. ``wrote``: the outputs that the caller gave, whose version counters
    then tell autograd that they changed."""
    with torch.cuda.device(dev):
        _check(fn(*args, _stream_ptr(dev)), what)
    for t in wrote:
        if t is not None:
            torch.autograd.graph.increment_version(t)


def _norm(q8, x, gamma, eps, residual, residual_out, outs):
    """The checked way of a norm; outs: (q, scales) or (y,), None where they are to be made."""
    M, D = _rows(x, "x")
    _want(gamma, x.dtype, (D,), "gamma")
    if residual is not None:
        _want(residual, x.dtype, (M, D), "residual")
        if residual_out is not None:
            _want(residual_out, x.dtype, (M, D), "residual_out")
    elif residual_out is not None:
        raise ValueError("residual_out without residual")
    kinds = ((torch.int8, (M, D), "q"), (torch.float32, (M,), "scales")) if q8 else ((x.dtype, (M, D), "out"),)
    for t, kind in zip(outs, kinds):
        if t is not None:
            _want(t, *kind)
    named = {"x": x, "gamma": gamma, "residual": residual, "residual_out": residual_out, **{k[2]: t for t, k in zip(outs, kinds)}}
    _forward_only(named)
    dev = _on_gpu(named)
    wrote = (residual_out, *outs)
    outs = [torch.empty(k[1], dtype=k[0], device=dev) if t is None else t for t, k in zip(outs, kinds)]
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    name = "paro_rmsnorm_q8" if q8 else "paro_rmsnorm"
    _call(getattr(_lib, name), name, dev, M, D, _DTYPE[x.dtype], _ptr(x), _ptr(residual), _ptr(gamma), eps,
          _ptr(residual_out), *map(_ptr, outs), wrote=wrote)
    return (*outs, residual_out)


def paro_rmsnorm_q8(x, gamma, eps=1e-6, residual=None, out=None, residual_out=None):
    """h = x + residual (rounded to x's type), then the RMS norm of h times gamma in 8 bits:
    (q int8 [M][D], scales float32 [M], h). x, residual float16 or bfloat16 [M][D], gamma [D] of
    that type. ``out``: an optional (q, scales) pair to write; ``residual_out``: where h goes (it
    may be ``residual`` itself). Without ``residual``, h is None."""
    q, scales = (None, None) if out is None else out
    r = _binding.rmsnorm(True, x, gamma, eps, residual, residual_out, q, scales)
    return r if r is not None else _norm(True, x, gamma, eps, residual, residual_out, (q, scales))


def paro_rmsnorm(x, gamma, eps=1e-6, residual=None, out=None, residual_out=None):
    """The same norm with its rows in x's type, for paro_quantize_q8 behind a transform or (float16) for
    paro_rotate and the W4A16 linears: (y [M][D], h). ``out``: an optional tensor for y."""
    r = _binding.rmsnorm(False, x, gamma, eps, residual, residual_out, out, None)
    return r if r is not None else _norm(False, x, gamma, eps, residual, residual_out, (out,))


def _quantize(pack, x, rot, out):
    q, scales = (None, None) if out is None else out
    r = _binding.quantize(pack, x, 0 if rot is None else ctypes.addressof(rot.handle), None if rot is None else rot.desc, q, scales)
    if r is not None:
        return r
    name, what, qname = ("paro_pack_weights_q8", "W", "qweight") if pack else ("paro_quantize_q8", "x", "q")
    M, D = _rows(x, what)
    if rot is not None and rot.D != D:
        raise ValueError(f"{what} has {D} channels, the transform {rot.D}")
    if out is not None:
        _want(q, torch.int8, (M, D), qname)
        _want(scales, torch.float32, (M,), "scales")
    named = {what: x, qname: q, "scales": scales, "the transform": None if rot is None else rot.desc}
    _forward_only({k: t for k, t in named.items() if k != "W"})  # packed weights are constants: W may be a parameter
    dev = _on_gpu(named)
    wrote = (q, scales)
    if out is None:
        q = torch.empty((M, D), dtype=torch.int8, device=dev)
        scales = torch.empty(M, dtype=torch.float32, device=dev)
    _call(getattr(_lib, name), name, dev, None if rot is None else rot.ptr, M, D, _DTYPE[x.dtype], _ptr(x), _ptr(q), _ptr(scales),
          wrote=wrote)
    return q, scales


def paro_quantize_q8(x, rot=None, out=None):
    """Rows of x (float16 or bfloat16 [M][D]) in 8 bits: (q int8 [M][D], scales float32 [M]). With
    ``rot`` (a Rotation) the rows are transformed first, as paro_rotate does, in float32."""
    return _quantize(False, x, rot, out)


def paro_pack_weights_q8(W, rot=None, out=None):
    """Weights W (float16 or bfloat16 [N][D]) in 8 bits for the W8A8 linears: (qweight int8 [N][D],
    scales float32 [N]). With ``rot`` its transform is folded in first (build time, float64)."""
    return _quantize(True, W, rot, out)


def paro_dequantize_q8(q, scales, out_dtype=None, out=None):
    """The rows that 8-bit codes stand for: q * scales in float16 (default), bfloat16 or float32."""
    x = _binding.dequantize(q, scales, out_dtype, out)
    if x is not None:
        return x
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError("q must be a torch.Tensor with two dimensions")
    M, D = q.shape
    _want(q, torch.int8, (M, D), "q")
    _want(scales, torch.float32, (M,), "scales")
    _channels(D)
    dtype = out_dtype or (out.dtype if out is not None else torch.float16)
    if dtype not in _DTYPE:
        raise TypeError(f"the output must be float16, bfloat16 or float32, got {dtype}")
    if out is not None:
        _want(out, dtype, (M, D), "out")
    named = {"q": q, "scales": scales, "out": out}
    _forward_only(named)
    dev = _on_gpu(named)
    x = torch.empty((M, D), dtype=dtype, device=dev) if out is None else out
    _call(_lib.paro_dequantize_q8, "paro_dequantize_q8", dev, M, D, _ptr(q), _ptr(scales), _ptr(x), _DTYPE[dtype], wrote=(out,))
    return x


def paro_w8a8_workspace_bytes(M: int, D: int, N: int) -> int:
    return _lib.paro_w8a8_workspace_bytes(M, D, N)


def paro_w8a8_gated_workspace_bytes(M: int, D: int, F: int) -> int:
    return _lib.paro_w8a8_gated_workspace_bytes(M, D, F)


def _linear(gated, x, x_scales, qweight, w_scales, out_dtype, out, ws):
    y = _binding.linear(gated, x, x_scales, qweight, w_scales, out_dtype, out, ws)
    if y is not None:
        return y
    for t, what in ((x, "x"), (qweight, "qweight")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{what} must be a torch.Tensor with two dimensions")
    (M, D), rows = x.shape, qweight.shape[0]
    _want(x, torch.int8, (M, D), "x")
    _want(qweight, torch.int8, (rows, D), "qweight")
    _want(x_scales, torch.float32, (M,), "x_scales")
    _want(w_scales, torch.float32, (rows,), "w_scales")
    _channels(D)
    if gated and rows % 2:
        raise ValueError(f"qweight must hold as many gate rows as up rows, got {rows} rows")
    N = rows // 2 if gated else rows
    dtype = out_dtype or (out.dtype if out is not None else torch.float16)
    if dtype not in _DTYPE:
        raise TypeError(f"the output must be float16, bfloat16 or float32, got {dtype}")
    if out is not None:
        _want(out, dtype, (M, N), "out")
    _want_ws(ws)
    named = {"x": x, "x_scales": x_scales, "qweight": qweight, "w_scales": w_scales, "out": out, "ws": ws}
    _forward_only(named)
    dev = _on_gpu(named)
    y = torch.empty((M, N), dtype=dtype, device=dev) if out is None else out
    name, need = ("paro_w8a8_gated_linear", paro_w8a8_gated_workspace_bytes) if gated else ("paro_w8a8_linear", paro_w8a8_workspace_bytes)
    if ws is None and need(M, D, N):
        ws = torch.empty(need(M, D, N), dtype=torch.uint8, device=dev)
    _call(getattr(_lib, name), name, dev, M, D, N, _ptr(x), _ptr(x_scales), _ptr(qweight), _ptr(w_scales), _ptr(y), _DTYPE[dtype],
          _ptr(ws), 0 if ws is None else ws.numel(), wrote=(out,))
    return y


def paro_w8a8_linear(x, x_scales, qweight, w_scales, out_dtype=None, out=None, ws=None):
    """y = x . qweight^T with x_scales per row and w_scales per column: x int8 [M][D], x_scales
    float32 [M], qweight int8 [N][D], w_scales float32 [N]; y float16 (default), bfloat16 or
    float32 [M][N]. ``ws``: an optional workspace of paro_w8a8_workspace_bytes(M, D, N) bytes."""
    return _linear(False, x, x_scales, qweight, w_scales, out_dtype, out, ws)


def paro_w8a8_gated_linear(x, x_scales, qweight, w_scales, out_dtype=None, out=None, ws=None):
    """silu(gate) * up of one gated feed-forward block: qweight int8 [2F][D] holds the gate rows,
    then the up rows; y [M][F]. The rest as in paro_w8a8_linear."""
    return _linear(True, x, x_scales, qweight, w_scales, out_dtype, out, ws)
