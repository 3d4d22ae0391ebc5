"""CPU tests of the 8-bit path's boundary (include/paro_w8a8.h) and of its oracle: exported symbols,
refusals in the library and in the binding (fake pointers and CPU tensors: every case returns before
anything is enqueued), and the oracle against hand-worked values.
"""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import q8_oracle as Q

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
rl = pytest.importorskip("rotated_linear_amd", reason="libparo.so not built")
torch = pytest.importorskip("torch")
lib = rl.lib()
A = 0x1000000  # fake 16-byte aligned addresses, far apart, never dereferenced
AT = [A * (i + 1) for i in range(12)]
F16, F32, BF16 = rl.F16, rl.F32, rl.BF16
EINVAL, ESHAPE, EWS = 1, 2, 5


def test_header_symbols_exported():
    src = open(os.path.join(ROOT, "include", "paro_w8a8.h")).read()
    names = set(re.findall(r"\b(paro_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert names == set(rl.EXPORTS_W8A8)
    out = subprocess.run(["nm", "-D", "--defined-only", rl.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\sT\s(paro_\w+)", out))


def _norm8(M=4, D=256, dt=F16, x=AT[0], r=AT[1], g=AT[2], eps=1e-6, ro=AT[3], q=AT[4], s=AT[5]):
    return lib.paro_rmsnorm_q8(M, D, dt, x, r, g, eps, ro, q, s, None)


def _norm(M=4, D=256, dt=F16, x=AT[0], r=AT[1], g=AT[2], eps=1e-6, ro=AT[3], y=AT[4]):
    return lib.paro_rmsnorm(M, D, dt, x, r, g, eps, ro, y, None)


@pytest.mark.parametrize("f", [_norm8, _norm])
def test_norm_refusals(f):
    assert f(M=0) == 0
    assert f(M=-1) == EINVAL
    for D in (0, 64, 100, 130, 16512, -128):
        assert f(D=D) == ESHAPE, D
    for dt in (F32, 3, -1):
        assert f(dt=dt) == EINVAL, dt
    for eps in (0.0, -1e-6, float("inf"), float("nan"), 1e-39):
        assert f(eps=eps) == EINVAL, eps
    for k in ("x", "g"):
        assert f(**{k: None}) == EINVAL
    assert f(r=None) == EINVAL and f(ro=None) == EINVAL  # they go together
    for k in ("x", "r", "g", "ro"):
        assert f(**{k: AT[9] + 8}) == EINVAL, k
    assert f(ro=AT[0]) == EINVAL  # residual_out over x
    assert f(ro=AT[1] + 512) == EINVAL  # the stream shifted by a row over itself
    assert f(x=AT[3]) == EINVAL
    assert f(g=AT[3] + 1024) == EINVAL


def test_norm_output_refusals():
    assert _norm(y=None) == EINVAL and _norm(y=AT[0]) == EINVAL and _norm(y=AT[3] + 16) == EINVAL
    assert _norm(y=AT[1]) == EINVAL
    assert _norm8(q=None) == EINVAL and _norm8(s=None) == EINVAL
    assert _norm8(q=AT[0] + 1024) == EINVAL and _norm8(q=AT[5] - 1008) == EINVAL and _norm8(s=AT[2]) == EINVAL
    assert _norm8(q=AT[9] + 4) == EINVAL and _norm8(s=AT[9] + 4) == EINVAL


def test_quantize_and_pack_refusals():
    rot = rl.paro_rotation(2, 256, AT[8])
    for fn, bad in ((lib.paro_quantize_q8, AT[0]), (lib.paro_pack_weights_q8, AT[0])):
        def f(M=4, D=256, dt=F16, x=AT[0], q=AT[4], s=AT[5], r=None):
            return fn(None if r is None else ctypes.byref(r), M, D, dt, x, q, s, None)
        assert f(M=0) == 0 and f(M=0, r=rot) == 0
        assert f(M=-1) == EINVAL and f(dt=F32) == EINVAL
        assert f(D=200) == ESHAPE and f(D=16512) == ESHAPE
        assert f(r=rot, D=384) == ESHAPE
        assert f(r=rl.paro_rotation(65, 256, AT[8])) == ESHAPE
        assert f(r=rl.paro_rotation(2, 256, None)) == EINVAL
        assert f(r=rl.paro_rotation(2, 256, AT[8] + 4)) == EINVAL
        for k in ("x", "q", "s"):
            assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 2}) == EINVAL
        assert f(q=bad) == EINVAL and f(s=AT[0] + 16) == EINVAL and f(q=AT[5]) == EINVAL
        assert f(r=rot, q=AT[8]) == EINVAL  # codes over the transform's descriptor


def test_dequantize_refusals():
    def f(M=4, D=256, q=AT[0], s=AT[1], x=AT[2], dt=F16):
        return lib.paro_dequantize_q8(M, D, q, s, x, dt, None)
    assert f(M=0) == 0
    assert f(M=-2) == EINVAL and f(dt=7) == EINVAL and f(D=192) == ESHAPE
    for k in ("q", "s", "x"):
        assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 1}) == EINVAL
    assert f(x=AT[0]) == EINVAL and f(x=AT[1] - 2032) == EINVAL
    assert f(x=AT[1] - 2048, dt=F32) == EINVAL  # a float32 output is twice as long


@pytest.mark.parametrize("gated", [False, True])
def test_linear_refusals(gated):
    fn = lib.paro_w8a8_gated_linear if gated else lib.paro_w8a8_linear
    need = (lib.paro_w8a8_gated_workspace_bytes if gated else lib.paro_w8a8_workspace_bytes)

    def f(M=4, D=256, N=48, x=AT[0], xs=AT[1], w=AT[2], s=AT[3], y=AT[4], dt=F16, ws=AT[5], nb=1 << 40):
        return fn(M, D, N, x, xs, w, s, y, dt, ws, nb, None)
    assert f(M=0) == 0 and f(N=0) == 0 and f(M=0, x=None, ws=None, nb=0) == 0
    assert f(M=-1) == EINVAL and f(N=-1) == EINVAL and f(dt=3) == EINVAL
    for D in (0, 64, 192, 16512):
        assert f(D=D) == ESHAPE
    if gated:
        assert f(N=1 << 29) == EINVAL and need(4, 256, 1 << 29) == 0
    for k in ("x", "xs", "w", "s", "y"):
        assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 8}) == EINVAL, k
    last = (95 if gated else 47) * 256  # the last weight row counts, up rows included
    assert f(y=AT[2] + last) == EINVAL
    assert f(y=AT[0]) == EINVAL and f(y=AT[1]) == EINVAL and f(y=AT[3]) == EINVAL
    for M, D, N in ((0, 256, 16), (4, 100, 16), (4, 256, 0), (-3, 256, 16)):
        assert need(M, D, N) == 0
    # a shape that splits its reduction, if any does, wants its whole workspace, apart from the operands
    for M, D, N in ((1, 4096, 4096), (64, 14336, 4096), (200, 8960, 257), (300, 16384, 130)):
        n = need(M, D, N)
        if n:
            assert f(M=M, D=D, N=N, ws=None, nb=0) == EWS and f(M=M, D=D, N=N, nb=n - 1) == EWS
            assert f(M=M, D=D, N=N, ws=AT[9] + 8) == EINVAL
            assert f(M=M, D=D, N=N, ws=AT[0]) == EINVAL and f(M=M, D=D, N=N, ws=AT[4]) == EINVAL


def test_binding_refusals():
    """Wrong types, shapes and strides are named before the device check; CPU tensors stop there."""
    M, D, N = 3, 256, 10
    x, g = torch.zeros(M, D, dtype=torch.float16), torch.zeros(D, dtype=torch.float16)
    q, s = torch.zeros(M, D, dtype=torch.int8), torch.zeros(M)
    w, ws = torch.zeros(N, D, dtype=torch.int8), torch.zeros(N)
    rot = rl.Rotation(2, 384, None, rl.paro_rotation(2, 384, A))

    def raises(kind, text, fn, *a, **k):
        with pytest.raises(kind, match=text):
            fn(*a, **k)

    for f in (rl.paro_rmsnorm_q8, rl.paro_rmsnorm):
        raises(TypeError, "float16 or torch.bfloat16", f, x.float(), g)
        raises(ValueError, "two dimensions", f, x[0], g)
        raises(ValueError, "x must be contiguous", f, torch.zeros(D, M, dtype=torch.float16).t(), g)
        raises(TypeError, "gamma must be", f, x, g.bfloat16())
        raises(ValueError, "gamma must have shape", f, x, g[:128])
        raises(ValueError, "residual must have shape", f, x, g, residual=x[:2])
        raises(ValueError, "residual_out without residual", f, x, g, residual_out=x)
        raises(TypeError, "residual_out must be", f, x, g, residual=x, residual_out=x.float())
        raises(rl.ParoError, "PARO_ESHAPE", f, x[:, :100].contiguous(), g[:100])
        raises(ValueError, "must live on the GPU", f, x, g, residual=x)
    raises(TypeError, "q must be", rl.paro_rmsnorm_q8, x, g, out=(q.float(), s))
    raises(ValueError, "scales must have shape", rl.paro_rmsnorm_q8, x, g, out=(q, s[:2]))
    raises(ValueError, "out must have shape", rl.paro_rmsnorm, x, g, out=x[:2])
    for f in (rl.paro_quantize_q8, rl.paro_pack_weights_q8):
        raises(TypeError, "must be torch.float16 or", f, x.double())
        raises(ValueError, "256 channels, the transform 384", f, x, rot)
        raises(rl.ParoError, "PARO_ESHAPE", f, torch.zeros(2, 16512, dtype=torch.float16))
        raises(ValueError, "must live on the GPU", f, x)
        raises(ValueError, "must live on the GPU", f, x, out=(q, s))
    raises(TypeError, "scales must be", rl.paro_quantize_q8, x, out=(q, s.double()))
    raises(TypeError, "q must be", rl.paro_dequantize_q8, x, s)
    raises(ValueError, "scales must have shape", rl.paro_dequantize_q8, q, s[:1])
    raises(TypeError, "float16, bfloat16 or float32", rl.paro_dequantize_q8, q, s, torch.float64)
    raises(ValueError, "must live on the GPU", rl.paro_dequantize_q8, q, s)
    for f, rows in ((rl.paro_w8a8_linear, N), (rl.paro_w8a8_gated_linear, N)):
        raises(TypeError, "x must be", f, x, s, w, ws)
        raises(ValueError, "qweight must have shape", f, q, s, w[:, :128].contiguous(), ws)
        raises(ValueError, "x_scales must have shape", f, q, s[:2], w, ws)
        raises(TypeError, "w_scales must be", f, q, s, w, ws.half())
        raises(ValueError, "qweight must be contiguous", f, q, s, torch.zeros(D, N, dtype=torch.int8).t(), ws)
        raises(TypeError, "float16, bfloat16 or float32", f, q, s, w, ws, torch.int32)
        raises(ValueError, "out must have shape", f, q, s, w, ws, out=torch.zeros(M, N + 1))
        raises(TypeError, "ws must be", f, q, s, w, ws, ws=torch.zeros(64))
        raises(ValueError, "must live on the GPU", f, q, s, w, ws)
    raises(ValueError, "as many gate rows as up rows", rl.paro_w8a8_gated_linear, q, s, w[:9], ws[:9])


def test_compiled_binding_declines_what_it_does_not_take():
    """It returns None, having done nothing, for CPU tensors, other objects and wrong counts; the checks
    above then speak. bind() takes nine addresses, none of them zero."""
    from rotated_linear_amd import _binding as b

    x, q, s = torch.zeros(2, 256, dtype=torch.float16), torch.zeros(2, 256, dtype=torch.int8), torch.zeros(2)
    assert b.linear(False, q, s, q, s, None, None, None) is None and b.linear(False, q, s) is None
    assert b.linear(False, None, 3, "w", s, torch.float16, None, None) is None
    assert b.quantize(False, x, 0, None, None, None) is None and b.quantize(True, 1, 0, None, None, None) is None
    assert b.dequantize(q, s, None, None) is None and b.dequantize() is None
    assert b.rmsnorm(True, x, x[0], 1e-6, None, None, None, None) is None and b.rmsnorm(None) is None
    for bad in ((), (1,) * 8, (1,) * 8 + (0,), (1,) * 8 + ("x",)):
        with pytest.raises((TypeError, ValueError)):
            b.bind(*bad)


# ---- the oracle against hand-worked values ----

def test_oracle_rounding():
    for dt, t in (("f16", torch.float16), ("bf16", torch.bfloat16), ("f32", torch.float32)):
        r = np.random.default_rng(3)
        a = np.concatenate([r.normal(0, 1, 4000) * 2.0 ** r.integers(-30, 18, 4000), [0.0, 65519.9, 65520.0, 2.0 ** -25,
                                                                                        1.5 * 2.0 ** -24, 1 + 2.0 ** -9]])
        a = a.astype(np.float32).astype(np.float64)  # torch rounds from float64 through float32
        assert np.array_equal(Q.round_to(a, dt), torch.from_numpy(a).to(t).double().numpy()), dt


def test_oracle_quantiser_hand_values():
    W = np.array([[1.0, -127.0, 63.5, 0.49, 0.5, 1.5, -0.5, 0.0], [0.0] * 8, [2.0 ** -110, 0, 0, 0, 0, 0, 0, 0]])
    q, s = Q.pack_weights(W)
    assert q[0].tolist() == [1, -127, 64, 0, 0, 2, 0, 0]  # ties to even
    assert s[0] == 1.0
    assert not q[1].any() and s[1] == np.float32(2.0 ** -100 / 127)
    assert q[2, 0] == 0  # 2^-10 of a step of 2^-100 / 127: 127 * 2^-10 = 0.124
    r, sc = Q.quantize_exact(W)
    assert r[0, 2] == 63.5 and sc[0] == 1.0


def test_oracle_norm_and_products_hand_values():
    n = Q.rmsnorm(np.array([[3.0, 4.0, 0.0, 0.0]]), [1.0, 2.0, 1.0, 1.0], 0.0)
    assert np.allclose(n, [[1.2, 3.2, 0, 0]], rtol=1e-15)
    y = Q.linear([[1, 2], [-3, 4]], [0.5, 2.0], [[10, 1], [0, -128]], [1.0, 0.25])
    assert y.tolist() == [[6.0, -32.0], [-52.0, -256.0]]
    v, g, u = Q.gated([[1, 0]], [1.0], [[2, 0], [3, 0]], [1.0, 1.0])
    assert g == 2 and u == 3 and abs(v[0, 0] - 6 / (1 + np.exp(-2.0))) < 1e-15


def test_oracle_fold_keeps_the_product():
    r = np.random.default_rng(5)
    D, K = 128, 3
    pairs = np.stack([r.permutation(D).reshape(D // 2, 2) for _ in range(K)]).astype(np.int32)
    theta = r.uniform(-3, 3, (K, D // 2)).astype(np.float32)
    s = np.exp(r.normal(0, 0.3, D)).astype(np.float32)
    x, W = r.normal(size=(5, D)), r.normal(size=(7, D))
    q, sc = Q.pack_weights(W, pairs, theta, s)
    got = Q.transform(x, pairs, theta, s) @ (q * sc[:, None].astype(np.float64)).T
    # each weight is within half a step of the folded one
    assert np.all(np.abs(got - x @ W.T) <= (0.5 + 1e-4) * np.abs(Q.transform(x, pairs, theta, s)).sum(1)[:, None] * sc + 1e-4)
