"""Python binding of the 8-bit path (include/paro_w8a8.h): residual RMS norm, row quantisation,
8-bit weights and the W8A8 products. Argument marshalling only, as in the package; the names mirror
the C ABI. Decode-sized calls take a few microseconds on the GPU, so the checks that pass take one
comparison each and only a failing one goes through the package's checkers for its message.
"""
from __future__ import annotations

import ctypes

import torch

from . import F16, F32, GROUP, MAX_D, ParoError, _check, _i, _lib, _on_gpu, _sz, _vp, _want, _want_ws, paro_rotation

BF16 = 2
_EWORKSPACE = 5
_DTYPE = {torch.float16: F16, torch.bfloat16: BF16, torch.float32: F32}
_ROWS = (torch.float16, torch.bfloat16)

_rot_p = ctypes.POINTER(paro_rotation)
_f = ctypes.c_float
_SIGNATURES = {
    "paro_rmsnorm_q8": (_i, [_i, _i, _i, _vp, _vp, _vp, _f, _vp, _vp, _vp, _vp]),
    "paro_rmsnorm": (_i, [_i, _i, _i, _vp, _vp, _vp, _f, _vp, _vp, _vp]),
    "paro_quantize_q8": (_i, [_rot_p, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "paro_dequantize_q8": (_i, [_i, _i, _vp, _vp, _vp, _i, _vp]),
    "paro_pack_weights_q8": (_i, [_rot_p, _i, _i, _i, _vp, _vp, _vp, _vp]),
    "paro_w8a8_workspace_bytes": (_sz, [_i, _i, _i]),
    "paro_w8a8_linear": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
    "paro_w8a8_gated_workspace_bytes": (_sz, [_i, _i, _i]),
    "paro_w8a8_gated_linear": (_i, [_i, _i, _i, _vp, _vp, _vp, _vp, _vp, _i, _vp, _sz, _vp]),
}
for _name, (_res, _args) in _SIGNATURES.items():
    getattr(_lib, _name).restype = _res
    getattr(_lib, _name).argtypes = _args
EXPORTS_W8A8 = tuple(_SIGNATURES)


# The current stream's handle by device index (the lookup through a Stream object takes 2 us).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device


def _fits(t, dtype, shape, index):
    """Whether t is a contiguous tensor of this dtype and shape on GPU `index`."""
    return t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.get_device() == index >= 0


def _refuse(wants, named):
    """Raise for the first operand that is not as wanted: (tensor, dtype, shape, name) of those given,
    then where they live."""
    for t, dtype, shape, name in wants:
        if t is not None:
            _want(t, dtype, shape, name)
    _on_gpu(named)
    raise ValueError("operands do not fit together")


def _rows(t, name):
    """Refuse anything but contiguous 2-d float16 or bfloat16 rows of channels the library takes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in _ROWS:
        raise TypeError(f"{name} must be torch.float16 or torch.bfloat16, got {t.dtype}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions, got shape {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.shape[1] % GROUP or not GROUP <= t.shape[1] <= MAX_D:
        raise ParoError(2, "D")


def _call(fn, what, index, *args, ask=None):
    """fn(*args, current stream of GPU `index`), with that GPU current; raises on an error status,
    except that status `ask` is returned."""
    if _current_device() == index:
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st and st != ask:
        _check(st, what)
    return st


def _p(t):
    return 0 if t is None else t.data_ptr()


def _norm(x, gamma, residual, residual_out, outs):
    """Check a norm's operands and given outputs [(tensor, dtype, shape, name)]: (M, D, GPU)."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in _ROWS or not x.is_contiguous():
        _rows(x, "x")
    shape, dtype, index = x.shape, x.dtype, x.get_device()
    M, D = shape
    if residual is None and residual_out is not None:
        raise ValueError("residual_out without residual")
    if (index < 0 or D % GROUP or not GROUP <= D <= MAX_D
            or not isinstance(gamma, torch.Tensor) or not _fits(gamma, dtype, (D,), index)
            or (residual is not None and not (isinstance(residual, torch.Tensor) and _fits(residual, dtype, shape, index)))
            or (residual_out is not None and not (isinstance(residual_out, torch.Tensor)
                                                  and _fits(residual_out, dtype, shape, index)))
            or not all(isinstance(t, torch.Tensor) and _fits(t, dt, sh, index) for t, dt, sh, _ in outs)):
        _rows(x, "x")
        wants = [(gamma, dtype, (D,), "gamma"), (residual, dtype, shape, "residual"),
                 (residual_out, dtype, shape, "residual_out"), *outs]
        _refuse(wants, {"x": x, **{name: t for t, _, _, name in wants}})
    return M, D, index


def paro_rmsnorm_q8(x, gamma, eps=1e-6, residual=None, out=None, residual_out=None):
    """h = x + residual (rounded to x's type), then the RMS norm of h times gamma in 8 bits:
    (q int8 [M][D], scales float32 [M], h). x, residual float16 or bfloat16 [M][D], gamma [D] of
    that type. ``out``: an optional (q, scales) pair to write; ``residual_out``: where h goes (it
    may be ``residual`` itself). Without ``residual``, h is None."""
    q, sc = (None, None) if out is None else out
    M, D, index = _norm(x, gamma, residual, residual_out,
                        () if out is None else ((q, torch.int8, x.shape, "q"), (sc, torch.float32, x.shape[:1], "scales")))
    if q is None:
        q = torch.empty_like(x, dtype=torch.int8)
        sc = x.new_empty(M, dtype=torch.float32)
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    _call(_lib.paro_rmsnorm_q8, "paro_rmsnorm_q8", index, M, D, _DTYPE[x.dtype], x.data_ptr(), _p(residual),
          gamma.data_ptr(), eps, _p(residual_out), q.data_ptr(), sc.data_ptr())
    return q, sc, residual_out


def paro_rmsnorm(x, gamma, eps=1e-6, residual=None, out=None, residual_out=None):
    """The same norm with its rows in x's type, as paro_rotate and the W4A16 linears read them:
    (y [M][D], h). ``out``: an optional tensor for y."""
    M, D, index = _norm(x, gamma, residual, residual_out, () if out is None else ((out, x.dtype, x.shape, "out"),))
    y = torch.empty_like(x) if out is None else out
    if residual is not None and residual_out is None:
        residual_out = torch.empty_like(residual)
    _call(_lib.paro_rmsnorm, "paro_rmsnorm", index, M, D, _DTYPE[x.dtype], x.data_ptr(), _p(residual),
          gamma.data_ptr(), eps, _p(residual_out), y.data_ptr())
    return y, residual_out


def _quantize(fn, name, what, x, rot, out, out_names):
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype not in _ROWS or not x.is_contiguous():
        _rows(x, what)
    (M, D), index = x.shape, x.get_device()
    if rot is not None and rot.D != D:
        raise ValueError(f"{what} has {D} channels, the transform {rot.D}")
    q, sc = (None, None) if out is None else out
    if (index < 0 or D % GROUP or not GROUP <= D <= MAX_D or (rot is not None and rot.desc.get_device() != index)
            or (out is not None and not (isinstance(q, torch.Tensor) and isinstance(sc, torch.Tensor)
                                         and _fits(q, torch.int8, x.shape, index) and _fits(sc, torch.float32, (M,), index)))):
        _rows(x, what)
        for t, dtype, shape, n in () if out is None else ((q, torch.int8, (M, D), out_names[0]),
                                                          (sc, torch.float32, (M,), out_names[1])):
            _want(t, dtype, shape, n)
        _refuse((), {what: x, out_names[0]: q, out_names[1]: sc, "transform": None if rot is None else rot.desc})
    if q is None:
        q = torch.empty_like(x, dtype=torch.int8)
        sc = x.new_empty(M, dtype=torch.float32)
    _call(fn, name, index, None if rot is None else rot.ptr, M, D, _DTYPE[x.dtype], x.data_ptr(), q.data_ptr(),
          sc.data_ptr())
    return q, sc


def paro_quantize_q8(x, rot=None, out=None):
    """Rows of x (float16 or bfloat16 [M][D]) in 8 bits: (q int8 [M][D], scales float32 [M]). With
    ``rot`` (a Rotation) the rows are transformed first, as paro_rotate does, in float32."""
    return _quantize(_lib.paro_quantize_q8, "paro_quantize_q8", "x", x, rot, out, ("q", "scales"))


def paro_pack_weights_q8(W, rot=None, out=None):
    """Weights W (float16 or bfloat16 [N][D]) in 8 bits for the W8A8 linears: (qweight int8 [N][D],
    scales float32 [N]). With ``rot`` its transform is folded in first (build time, float64)."""
    return _quantize(_lib.paro_pack_weights_q8, "paro_pack_weights_q8", "W", W, rot, out, ("qweight", "scales"))


def paro_dequantize_q8(q, scales, out_dtype=torch.float16, out=None):
    """The rows that 8-bit codes stand for: q * scales in float16, bfloat16 or float32."""
    if not isinstance(q, torch.Tensor) or q.dim() != 2:
        raise ValueError("q must be a torch.Tensor with two dimensions")
    M, D = q.shape
    if out is not None:
        out_dtype = out.dtype
    if out_dtype not in _DTYPE:
        raise TypeError(f"the output must be float16, bfloat16 or float32, got {out_dtype}")
    index = q.get_device()
    if not (isinstance(scales, torch.Tensor) and _fits(q, torch.int8, (M, D), index)
            and _fits(scales, torch.float32, (M,), index) and (out is None or _fits(out, out_dtype, (M, D), index))):
        _refuse(((q, torch.int8, (M, D), "q"), (scales, torch.float32, (M,), "scales"), (out, out_dtype, (M, D), "out")),
                {"q": q, "scales": scales, "out": out})
    if D % GROUP or not GROUP <= D <= MAX_D:
        raise ParoError(2, "D")
    x = torch.empty_like(q, dtype=out_dtype) if out is None else out
    _call(_lib.paro_dequantize_q8, "paro_dequantize_q8", index, M, D, q.data_ptr(), scales.data_ptr(), x.data_ptr(),
          _DTYPE[out_dtype])
    return x


def paro_w8a8_workspace_bytes(M: int, D: int, N: int) -> int:
    return _lib.paro_w8a8_workspace_bytes(M, D, N)


def paro_w8a8_gated_workspace_bytes(M: int, D: int, F: int) -> int:
    return _lib.paro_w8a8_gated_workspace_bytes(M, D, F)


def _linear(fn, name, need_fn, gated, x, x_scales, qweight, w_scales, out_dtype, out, ws):
    for t, what in ((x, "x"), (qweight, "qweight")):
        if not isinstance(t, torch.Tensor) or t.dim() != 2:
            raise ValueError(f"{what} must be a torch.Tensor with two dimensions")
    (M, D), rows = x.shape, qweight.shape[0]
    if gated and rows % 2:
        raise ValueError(f"qweight must hold as many gate rows as up rows, got {rows} rows")
    N = rows // 2 if gated else rows
    dtype = out_dtype or (out.dtype if out is not None else torch.float16)
    index = x.get_device()
    if not (isinstance(x_scales, torch.Tensor) and isinstance(w_scales, torch.Tensor) and dtype in _DTYPE
            and x.dtype is torch.int8 is qweight.dtype and x_scales.dtype is torch.float32 is w_scales.dtype
            and qweight.shape[1] == D and x_scales.shape == (M,) and w_scales.shape == (rows,)
            and x.is_contiguous() and qweight.is_contiguous() and x_scales.is_contiguous() and w_scales.is_contiguous()
            and qweight.get_device() == x_scales.get_device() == w_scales.get_device() == index >= 0
            and (out is None or _fits(out, dtype, (M, N), index))
            and (ws is None or _fits(ws, torch.uint8, (ws.numel(),), index))):
        for a in ((x, torch.int8, (M, D), "x"), (qweight, torch.int8, (rows, D), "qweight"),
                  (x_scales, torch.float32, (M,), "x_scales"), (w_scales, torch.float32, (rows,), "w_scales")):
            _want(*a)
        if dtype not in _DTYPE:
            raise TypeError(f"the output must be float16, bfloat16 or float32, got {dtype}")
        _want_ws(ws)
        _refuse(((out, dtype, (M, N), "out"),), {"x": x, "x_scales": x_scales, "qweight": qweight, "w_scales": w_scales,
                                                "out": out, "ws": ws})
    y = x.new_empty((M, N), dtype=dtype) if out is None else out
    args = (M, D, N, x.data_ptr(), x_scales.data_ptr(), qweight.data_ptr(), w_scales.data_ptr(), y.data_ptr(), _DTYPE[dtype])
    if ws is not None:
        _call(fn, name, index, *args, ws.data_ptr(), ws.numel())
    elif _call(fn, name, index, *args, 0, 0, ask=_EWORKSPACE):  # the call wants a workspace: it has done nothing yet
        ws = x.new_empty(need_fn(M, D, N), dtype=torch.uint8)
        _call(fn, name, index, *args, ws.data_ptr(), ws.numel())
    return y


def paro_w8a8_linear(x, x_scales, qweight, w_scales, out_dtype=None, out=None, ws=None):
    """y = x . qweight^T with x_scales per row and w_scales per column: x int8 [M][D], x_scales
    float32 [M], qweight int8 [N][D], w_scales float32 [N]; y float16 (default), bfloat16 or
    float32 [M][N]. ``ws``: an optional workspace of paro_w8a8_workspace_bytes(M, D, N) bytes."""
    return _linear(_lib.paro_w8a8_linear, "paro_w8a8_linear", _lib.paro_w8a8_workspace_bytes, False, x, x_scales,
                   qweight, w_scales, out_dtype, out, ws)


def paro_w8a8_gated_linear(x, x_scales, qweight, w_scales, out_dtype=None, out=None, ws=None):
    """silu(gate) * up of one gated feed-forward block: qweight int8 [2F][D] holds the gate rows,
    then the up rows; y [M][F]. The rest as in paro_w8a8_linear."""
    return _linear(_lib.paro_w8a8_gated_linear, "paro_w8a8_gated_linear", _lib.paro_w8a8_gated_workspace_bytes, True,
                   x, x_scales, qweight, w_scales, out_dtype, out, ws)
