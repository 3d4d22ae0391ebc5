"""CPU tests of include/paro_block.h's boundary and of its oracle: exported symbols, refusals in the library (fake
pointers, never dereferenced: every case returns before anything is enqueued) and in the binding (CPU tensors), what
autograd would lose, and the oracle against hand-worked values.
"""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest

from oracle import block_oracle as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
rl = pytest.importorskip("rotated_linear_amd", reason="libparo.so not built")
torch = pytest.importorskip("torch")
lib = rl.lib()
A = 0x10000000
AT = [A * (i + 1) for i in range(24)]
F16, F32, BF16 = rl.F16, rl.F32, rl.BF16
EINVAL, ESHAPE, EWS = 1, 2, 5


def test_header_symbols_exported():
    src = open(os.path.join(ROOT, "include", "paro_block.h")).read()
    names = set(re.findall(r"\b(paro_[a-z0-9_]+)\s*\(", re.sub(r"/\*.*?\*/", "", src, flags=re.S)))
    assert names == set(rl.EXPORTS_BLOCK)
    out = subprocess.run(["nm", "-D", "--defined-only", rl.LIB_PATH], capture_output=True, text=True).stdout
    assert names <= set(re.findall(r"\sT\s(paro_\w+)", out))


def test_epilogue_refusals():
    def f(M=4, D=256, N=48, x=AT[0], xs=AT[1], w=AT[2], s=AT[3], b=AT[4], act=3, r=AT[5], y=AT[6], dt=F16, ws=AT[7], nb=1 << 27):
        return lib.paro_w8a8_linear_epilogue(M, D, N, x, xs, w, s, b, act, r, y, dt, ws, nb, None)
    assert f(M=0) == 0 and f(N=0) == 0 and f(M=0, x=None, b=None) == 0
    assert f(M=-1) == EINVAL and f(N=-1) == EINVAL and f(dt=3) == EINVAL and f(act=6) == EINVAL and f(act=-1) == EINVAL
    for D in (0, 64, 192, 16512):
        assert f(D=D) == ESHAPE
    for k in ("x", "xs", "w", "s", "y"):
        assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 8}) == EINVAL, k
    for k in ("b", "r"):
        assert f(**{k: AT[9] + 8}) == EINVAL, k
    for k in (0, 1, 2, 3, 4):
        assert f(y=AT[k]) == EINVAL, k
    assert f(y=AT[4] + 80) == EINVAL and f(y=AT[4] + 80, dt=F32) == EINVAL  # within the bias
    assert f(y=AT[5] + 16) == EINVAL  # the stream shifted over itself
    for M, D, N in ((200, 8960, 257), (300, 16384, 130), (64, 14336, 128)):
        n = rl.paro_w8a8_workspace_bytes(M, D, N)
        if n:
            assert f(M=M, D=D, N=N, ws=None, nb=0) == EWS and f(M=M, D=D, N=N, nb=n - 1) == EWS
            for k in (0, 2, 4, 5, 6):
                assert f(M=M, D=D, N=N, ws=AT[k]) == EINVAL, k
    assert any(rl.paro_w8a8_workspace_bytes(*s) for s in ((200, 8960, 257), (300, 16384, 130), (64, 14336, 128)))


@pytest.mark.parametrize("q8", [True, False])
def test_block_norm_refusals(q8):
    def f(M=4, D=256, dt=F16, x=AT[0], p=AT[1], t=AT[2], tr=1, r=AT[3], alpha=1.0, g=AT[4], eps=1e-6, ro=AT[5], y=AT[6], s=AT[7]):
        if q8:
            return lib.paro_block_norm_q8(M, D, dt, x, p, t, tr, r, alpha, g, eps, ro, y, s, None)
        return lib.paro_block_norm(M, D, dt, x, p, t, tr, r, alpha, g, eps, ro, y, None)
    assert f(M=0) == 0 and f(M=-1) == EINVAL
    for D in (0, 64, 100, 130, 16512, -128):
        assert f(D=D) == ESHAPE, D
    for dt in (F32, 3, -1):
        assert f(dt=dt) == EINVAL, dt
    for eps in (0.0, -1e-6, float("inf"), float("nan"), 1e-39):
        assert f(eps=eps) == EINVAL, eps
    for alpha in (float("inf"), float("-inf"), float("nan")):
        assert f(alpha=alpha) == EINVAL
    assert f(tr=0) == EINVAL and f(tr=-3) == EINVAL
    for k in ("x", "r", "g", "ro", "y"):
        assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 8}) == EINVAL, k
    for k in ("p", "t"):
        assert f(**{k: AT[9] + 8}) == EINVAL, k
    for k in range(5):
        assert f(y=AT[k]) == EINVAL, k
        assert k == 3 or f(ro=AT[k]) == EINVAL, k
    assert f(ro=AT[3] + 512) == EINVAL and f(y=AT[5]) == EINVAL
    assert f(ro=AT[2] + 1536) == EINVAL  # the last of 4 gates
    assert f(ro=AT[2] + 1024, tr=3, M=7) == EINVAL  # 3 gates for 7 rows
    if q8:
        assert f(s=None) == EINVAL and f(s=AT[9] + 4) == EINVAL and f(s=AT[0]) == EINVAL and f(s=AT[6] + 16) == EINVAL


def test_route_refusals():
    need = rl.paro_moe_route_workspace_bytes(4, 16)
    assert need >= 4 * 16 * 8
    for M, E in ((0, 16), (-1, 16), (65, 16), (4, 0), (4, 513)):
        assert rl.paro_moe_route_workspace_bytes(M, E) == 0

    def f(M=4, D=256, E=16, k=2, x=AT[0], r=AT[1], dt=F16, sc=0, ids=AT[2], w=AT[3], ws=AT[4], nb=need):
        return lib.paro_moe_route(M, D, E, k, x, r, dt, sc, 1, ids, w, ws, nb, None)
    assert f(M=0) == 0
    for bad in ({"M": -1}, {"M": 65}, {"E": 0}, {"E": 513, "nb": 1 << 30}, {"k": 0}, {"k": 17, "E": 32}, {"k": 3, "E": 2}, {"dt": BF16},
                {"dt": -1}, {"sc": 2}, {"sc": -1}):
        assert f(**bad) == EINVAL, bad
    for D in (0, 64, 192, 16512):
        assert f(D=D) == ESHAPE
    for k in ("x", "r", "ids", "w"):
        assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 8}) == EINVAL, k
    assert f(ws=None) == EWS and f(nb=need - 1) == EWS and f(ws=AT[9] + 8) == EINVAL
    for k in ("ids", "w", "ws"):
        assert f(**{k: AT[0] + 1024}) == EINVAL and f(**{k: AT[1] + 7680}) == EINVAL, k
    assert f(ids=AT[3] + 16) == EINVAL and f(ws=AT[2]) == EINVAL


def experts(q=AT[10], s=AT[11], z=AT[12]):
    return ctypes.byref(rl.block.paro_w4_experts(q, s, z))


@pytest.mark.parametrize("layer", [False, True])
def test_moe_refusals(layer):
    M0, D0, F0, E0, k0 = 4, 256, 384, 6, 2
    need = rl.paro_moe_workspace_bytes(M0, D0, F0, E0, k0)
    assert need > 0
    for s in ((0, D0, F0, E0, k0), (65, D0, F0, E0, k0), (M0, 200, F0, E0, k0), (M0, D0, 64, E0, k0), (M0, D0, F0, 0, k0),
              (M0, D0, F0, 513, k0), (M0, D0, F0, E0, 0), (M0, D0, F0, E0, 17)):
        assert rl.paro_moe_workspace_bytes(*s) == 0, s

    def f(M=M0, D=D0, F=F0, E=E0, k=k0, x=AT[0], r=AT[1], dt=F16, sc=0, ids=AT[2], w=AT[3], rx=None, ra=None, gu=experts(),
          dn=experts(AT[13], AT[14], AT[15]), y=AT[4], ydt=F16, ws=AT[5], nb=need):
        rx, ra = (None if t is None else ctypes.byref(t) for t in (rx, ra))
        if layer:
            return lib.paro_moe_layer_w4a16(M, D, F, E, k, x, r, dt, sc, 1, rx, ra, gu, dn, y, ydt, ids, w, ws, nb, None)
        return lib.paro_moe_w4a16(M, D, F, E, k, x, ids, w, rx, ra, gu, dn, y, ydt, ws, nb, None)
    assert f(M=0) == 0 and f(M=0, gu=None, dn=None) == 0
    for bad in ({"M": -1}, {"M": 65}, {"E": 0}, {"E": 513}, {"k": 0}, {"k": 17}, {"ydt": BF16}, {"ydt": 3}):
        assert f(**bad) == EINVAL, bad
    if layer:
        for bad in ({"k": 7}, {"dt": BF16}, {"sc": 2}, {"r": None}, {"r": AT[9] + 4}):
            assert f(**bad) == EINVAL, bad
        assert f(y=AT[1] + 2816) == EINVAL  # within the router
    for bad in ({"D": 192}, {"D": 16512}, {"F": 100}, {"F": 0}, {"F": 16512}):
        assert f(**bad) == ESHAPE, bad
    for k in ("x", "ids", "w", "y"):
        assert f(**{k: None}) == EINVAL and f(**{k: AT[9] + 8}) == EINVAL, k
    assert f(gu=None) == EINVAL and f(dn=None) == EINVAL
    for i in range(3):
        for bad in (None, AT[9] + 8):
            p = [AT[10], AT[11], AT[12]]
            p[i] = bad
            assert f(gu=experts(*p)) == EINVAL and f(dn=experts(*p)) == EINVAL
    assert f(ws=None) == EWS and f(nb=need - 1) == EWS and f(ws=AT[9] + 8) == EINVAL
    # y and the workspace over the inputs, their last bytes too
    for at in (AT[0] + 2032, AT[10] + E0 * 2 * F0 * D0 // 2 - 16, AT[11] + E0 * 2 * F0 * 4 - 16, AT[12], AT[13] + E0 * F0 * D0 // 2 - 16,
               AT[14] + E0 * D0 * 6 - 16, AT[15], AT[2] + 16, AT[3]):
        assert f(y=at) == EINVAL and f(ws=at) == EINVAL, hex(at)
    assert f(ws=AT[4] + 16) == EINVAL
    rx, ra = rl.paro_rotation(2, D0, AT[16]), rl.paro_rotation(2, F0, AT[17])
    for k, other in (("rx", F0), ("ra", D0)):
        assert f(**{k: rl.paro_rotation(2, other, AT[16])}) == ESHAPE
        assert f(**{k: rl.paro_rotation(65, D0 if k == "rx" else F0, AT[16])}) == ESHAPE
        assert f(**{k: rl.paro_rotation(2, D0 if k == "rx" else F0, None)}) == EINVAL
    assert f(rx=rx, y=AT[16]) == EINVAL and f(ra=ra, ws=AT[17]) == EINVAL


def tensors(device="cpu"):
    def t(*shape, dtype=torch.float16):
        return torch.ones(shape, dtype=dtype, device=device)

    M, D, N, F, E, k = 4, 256, 12, 128, 3, 2
    q8 = {"x": t(M, D, dtype=torch.int8), "x_scales": t(M, dtype=torch.float32), "qweight": t(N, D, dtype=torch.int8),
          "w_scales": t(N, dtype=torch.float32), "bias": t(N), "residual": t(M, N), "out": t(M, N)}
    norm = {"x": t(M, D), "residual": t(M, D), "gamma": t(D), "post_gamma": t(D), "gate": t(2, D), "residual_out": t(M, D)}
    route = {"x": t(M, D), "router": t(E, D), "ids": t(M, k, dtype=torch.int32), "weights": t(M, k, dtype=torch.float32)}
    packed = {f"{w} {p}": t(E, n, c // d, dtype=torch.uint8 if p == "qweight" else torch.float16)
              for w, n, c in (("gate_up", 2 * F, D), ("down", D, F)) for p, d in (("qweight", 2), ("scales", 128), ("zeros", 128))}
    return q8, norm, route, packed, t


def calls(device="cpu"):
    """(name, call by keyword, its tensors by the names that the errors use, those it writes)."""
    q8, norm, route, packed, t = tensors(device)

    def weights(kw):
        return [tuple(kw.pop(f"{w} {p}") for p in ("qweight", "scales", "zeros")) for w in ("gate_up", "down")]

    def moe(**kw):
        gu, dn = weights(kw)
        return rl.paro_moe_w4a16(gate_up=gu, down=dn, **kw)

    def layer(ids, **kw):
        gu, dn = weights(kw)
        return rl.paro_moe_layer_w4a16(top_k=2, gate_up=gu, down=dn, routing=(ids, kw.pop("weights")), **kw)

    M, D = 4, 256
    yield "epilogue", lambda **kw: rl.paro_w8a8_linear_epilogue(activation="gelu", **kw), q8, {"out"}
    yield ("block_norm_q8", lambda q, scales, **kw: rl.paro_block_norm_q8(out=(q, scales), **kw),
           {**norm, "q": t(M, D, dtype=torch.int8), "scales": t(M, dtype=torch.float32)}, {"q", "scales", "residual_out"})
    yield "block_norm", rl.paro_block_norm, {**norm, "out": t(M, D)}, {"out", "residual_out"}
    yield ("route", lambda ids, weights, **kw: rl.paro_moe_route(top_k=2, out=(ids, weights), **kw), route, {"ids", "weights"})
    yield "moe", moe, {**{k: v for k, v in route.items() if k != "router"}, **packed, "out": t(M, D)}, {"out"}
    yield "layer", layer, {**route, **packed, "out": t(M, D)}, {"out", "ids", "weights"}


def test_forward_only_and_on_the_gpu():
    """A gradient that would be lost is refused, whichever tensor asks for it; then the device is looked at."""
    for name, call, given, _ in calls():
        for which, v in given.items():
            if not v.is_floating_point():
                continue
            asked = {k: u.clone().requires_grad_(k == which) for k, u in given.items()}
            with pytest.raises(RuntimeError, match=f"{which} requires a gradient and this call is forward only"):
                call(**asked)
            with torch.no_grad(), pytest.raises(ValueError, match="must live on the GPU"):
                call(**asked)


@pytest.mark.gpu
def test_written_tensors_count_as_changed():
    for name, call, given, written in calls("cuda"):
        before = {k: v._version for k, v in given.items()}
        call(**given)
        assert {k for k, v in given.items() if v._version != before[k]} == written, name


def test_binding_refusals():
    """Wrong types, shapes, strides and choices are named before the device check."""
    every = {name: (call, given) for name, call, given, _ in calls()}

    def raises(kind, text, name, **changed):
        call, given = every[name]
        with pytest.raises(kind, match=text):
            call(**{**given, **changed})

    _, _, _, _, t = tensors()
    f32, i8 = torch.float32, torch.int8
    for name, (call, given) in every.items():
        for which, v in given.items():
            wrong = v.double()
            if name.startswith("block_norm") and which == "x":
                raises(TypeError, "x must be torch.float16 or torch.bfloat16", name, x=wrong)
            else:
                raises(TypeError, f"{'the output' if which == 'out' else which} must be|out must be", name, **{which: wrong})
            if v.dim() == 2 and which not in ("x", "qweight", "router", "ids", "gate") and "weights" not in which:
                raises(ValueError, f"{which} must have shape", name, **{which: v[:1].contiguous()})
            if v.dim() == 2:
                raises(ValueError, "must be contiguous|must have two dimensions", name, **{which: v.t().contiguous().t()})
    with pytest.raises(ValueError, match="activation must be one of none, relu, relu2"):
        rl.paro_w8a8_linear_epilogue(**{**every["epilogue"][1], "activation": "swish"})
    raises(TypeError, "bias must be torch.float32", "epilogue", out=None, residual=None, bias=t(12), out_dtype=f32)
    raises(TypeError, "float16, bfloat16 or float32", "epilogue", out=None, out_dtype=torch.int32)
    raises(rl.ParoError, "PARO_ESHAPE", "epilogue", x=t(4, 192, dtype=i8), qweight=t(12, 192, dtype=i8))
    for name in ("block_norm_q8", "block_norm"):
        raises(ValueError, "gate has 3 rows, which do not divide the 4 of x", name, gate=t(3, 256))
        raises(ValueError, "gate has 0 rows", name, gate=t(0, 256))
        raises(ValueError, "gate must have shape", name, gate=t(2, 128))
        raises(ValueError, "one or two dimensions", name, gate=t(2, 2, 256))
        raises(rl.ParoError, "PARO_ESHAPE", name, x=t(4, 200))
    for name in ("route", "layer"):
        raises(TypeError, "router must be torch.float16 or torch.float32", name, router=t(3, 256, dtype=torch.bfloat16))
        raises(ValueError, "router has 1 experts, it must have top_k = 2 to 512", name, router=t(1, 256))
        raises(ValueError, "router must have shape", name, router=t(3, 128))
    for bad, text in ((0, "top_k must be 1 to 16"), (17, "top_k must be 1 to 16")):
        with pytest.raises(ValueError, match=text):
            rl.paro_moe_route(t(4, 256), t(32, 256), bad)
    with pytest.raises(ValueError, match="scoring must be one of softmax, sigmoid"):
        rl.paro_moe_route(t(4, 256), t(32, 256), 2, "relu")
    with pytest.raises(ValueError, match="65 tokens, the mixture-of-experts calls take 64 at most"):
        rl.paro_moe_route(t(65, 256), t(32, 256), 2)
    for name in ("moe", "layer"):
        raises(ValueError, "as many gate rows as up rows", name, **{"gate_up qweight": t(3, 255, 128, dtype=torch.uint8)})
        raises(ValueError, "down qweight must have shape", name, **{"down qweight": t(3, 256, 128, dtype=torch.uint8)})
        raises(TypeError, "float16 or float32, got torch.bfloat16", name, out=None, out_dtype=torch.bfloat16)
        raises(ValueError, "rot_x has 384 channels, its rows 256", name, rot_x=rl.Rotation(2, 384, None, rl.paro_rotation(2, 384, A)))
        raises(ValueError, "rot_a has 384 channels, its rows 128", name, rot_a=rl.Rotation(2, 384, None, rl.paro_rotation(2, 384, A)))
        raises(TypeError, "ws must be", name, ws=torch.zeros(64))
    raises(ValueError, "ids must be a torch.Tensor with two dimensions", "moe", ids=t(4, dtype=torch.int32))
    raises(ValueError, "gate_up has 513 experts, it must have 1 to 512", "moe", **{"gate_up qweight": t(513, 256, 128, dtype=torch.uint8)})


def test_compiled_binding_declines_what_it_does_not_take():
    """It returns None, having done nothing, for CPU tensors, other objects and wrong counts; bind_block() takes eight
    addresses, none of them zero."""
    b = pytest.importorskip("rotated_linear_amd._binding")
    x, q, s = torch.zeros(2, 256, dtype=torch.float16), torch.zeros(2, 256, dtype=torch.int8), torch.zeros(2)
    for f, args in ((b.linear_epilogue, (q, s, q, s, None, 0, None, None, None, None)), (b.route, (x, x, 1, 0, True, None, None, None)),
                    (b.block_norm, (True, x, x, x[0], 1e-6, None, None, 1.0, None, None, None)),
                    (b.moe, (x, x, 1, 0, True, None, None, (q, s, s), (q, s, s), 0, None, 0, None, None, None, None)),
                    (b.moe, (x, None, None, None, None, q, s, (q, s, s), (q, s, s), 0, None, 0, None, None, None, None))):
        assert f(*args) is None and f(*args[1:]) is None and f() is None
        assert f(*("x" if isinstance(a, torch.Tensor) else a for a in args)) is None
    for bad in ((), (1,) * 7, (1,) * 7 + (0,), (1,) * 7 + ("x",)):
        with pytest.raises((TypeError, ValueError)):
            b.bind_block(*bad)


# ---- the oracle against hand-worked values ----

def test_oracle_activations():
    v = np.array([-2.0, -0.5, 0.0, 1.0, 3.0])
    assert B.act(v, "none").tolist() == v.tolist() and B.act(v, "relu").tolist() == [0, 0, 0, 1, 3]
    assert B.act(v, "relu2").tolist() == [0, 0, 0, 1, 9]
    e = 2.718281828459045
    assert np.allclose(B.act(v, "silu"), [-2 / (1 + e ** 2), -0.5 / (1 + e ** 0.5), 0, e / (1 + e), 3 / (1 + e ** -3)], rtol=1e-14)
    assert np.allclose(B.act(v, "gelu")[3], 0.8413447460685429, rtol=1e-14)  # the normal distribution up to 1
    z = (2 / np.pi) ** 0.5 * (v + 0.044715 * v ** 3)
    assert np.allclose(B.act(v, "gelu_tanh"), v * (1 + np.tanh(z)) / 2, rtol=1e-12)


def test_oracle_stream():
    x, res = np.array([[3.0, 4.0], [1.0, 1.0]]), np.array([[10.0, 0.0], [0.0, 10.0]])
    h, p = B.stream(x, res, 0.0, np.array([1.0, 2.0]), np.array([[1.0, 1.0], [0.0, 3.0]]), 0.5)
    r = 12.5 ** 0.5
    assert np.allclose(p, [[3 / r, 8 / r], [0, 6]]) and np.allclose(h, [[5 + 3 / r, 8 / r], [0, 11]])
    h, p = B.stream(x, res, 0.0)
    assert p.tolist() == x.tolist() and h.tolist() == (x + res).tolist()


def test_oracle_router():
    x = np.array([[1.0, 0.0], [0.0, 1.0], [np.nan, 1.0]])
    router = np.array([[0.0, np.log(2)], [np.log(4), np.log(2)], [np.log(3), 0.0], [np.log(4), -1.0]])
    ids, w = B.route(x, router, 2, renormalize=False)
    assert ids.tolist() == [[1, 3], [0, 1], [0, 1]]  # ties to the lower index, NaN in order
    assert np.allclose(w[0], [4 / 12, 4 / 12]) and np.isnan(w[2]).all()
    assert np.allclose(B.route(x, router, 3)[1][0], [4 / 11, 4 / 11, 3 / 11])
    assert np.allclose(B.route(x, router, 2, sigmoid=True, renormalize=False)[1][0], [4 / 5, 4 / 5])


def test_oracle_experts():
    x = np.zeros((3, 128))
    x[:, 0] = [1, 2, -1]
    gu, dn = np.zeros((2, 256, 128)), np.zeros((2, 128, 128))
    gu[0, 0, 0] = gu[0, 128, 0] = 1.0  # expert 0: g = u = x0 in its first channel
    gu[1, 3, 0], gu[1, 131, 0] = 2.0, 5.0
    dn[0, 7, 0], dn[1, 9, 3] = 10.0, 100.0
    ids, w = np.array([[0, 1], [1, -1], [0, 0]]), np.array([[0.5, 0.25], [1.0, 9.0], [0.25, 0.25]])
    y, bound = B.experts(x, ids, w, gu, dn)

    def silu(v):
        return v / (1 + np.exp(-v))

    want = np.zeros((3, 128))
    want[0, 7], want[0, 9] = 0.5 * 10 * silu(1.0), 0.25 * 100 * silu(2.0) * 5
    want[1, 9] = 100 * silu(4.0) * 10
    want[2, 7] = 0.5 * 10 * silu(-1.0) * -1
    assert np.allclose(y, want, rtol=1e-14) and (bound >= 0).all() and (bound[want != 0] > 2.0 ** -13 * np.abs(want[want != 0])).all()
