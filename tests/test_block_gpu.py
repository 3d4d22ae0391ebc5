"""The W8A8 product with an epilogue and the norms around a block on the GPU against their float64 oracle.

Tolerances count roundings, as in the tests of the 8-bit path: U = 2^-24 is half a float32 step, a 16-bit type adds
half of its own step.
"""
import ctypes

import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import q8_oracle as Q
from tests import gpu_common as C
from tests.test_w8a8_gpu import DT, HALF, SUB, U, guarded, on_gpu, operands, over, rows

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")
lib = rl.lib()

ACTS = ["none", "relu", "relu2", "silu", "gelu", "gelu_tanh"]


def act_bound(v, dv, kind, dt):
    """Error of act at v, where v itself is off by dv: the slope times dv, and the activation's own arithmetic. With f the
    factor that v is multiplied by (act(v) = v f(v)): float32 outputs take exp and erfc from the math library (16 units
    in the last place at most, 32 U) at arguments of two or three roundings, of size |v| (silu), v^2 / 2 (gelu) or
    1.6 |v| + 0.072 |v|^3 (gelu_tanh), and two roundings more; 16-bit outputs 2^-19 for the polynomial, 8 U for the
    instructions. The argument's error moves f by as much of its smaller part min(f, 1 - f)."""
    a = np.abs(v)
    if kind in ("none", "relu"):
        return dv
    if kind == "relu2":
        return 2 * a * dv + dv * dv + U * a * a
    arg = {"silu": a, "gelu": a * a / 2, "gelu_tanh": 1.6 * a + 0.072 * a ** 3}[kind]
    f = np.where(v == 0, 0.5, B.act(-a, kind) / np.where(v == 0, 1.0, -a))  # the smaller part
    own = a * f * ((2.0 ** -19 if kind == "gelu" and dt != "f32" else 0) + (36 if dt == "f32" else 12) * U + 6 * U * arg)
    # a factor below 2^-126 may count as 0; the product of v and the factor is one rounding
    return 1.13 * dv + own + a * 2.0 ** -126 + 2 * U * np.abs(B.act(v, kind))


def epilogue_want(xq, xs, wq, ws, bias, kind, residual, dt):
    v0 = Q.linear(xq, xs, wq, ws)
    v = v0 + (0 if bias is None else bias)
    dv = 3.1 * U * np.abs(v0) + (0 if bias is None else U * np.abs(v) * 1.01)
    y = B.act(v, kind)
    d = act_bound(v, dv, kind, dt)
    if residual is not None:
        y = y + residual
        d = d * (1 + U) + U * np.abs(y)
    return y, d + HALF[dt] * (np.abs(y) + d) + SUB[dt]


def extras(seed, M, N, dt):
    r = np.random.default_rng([seed, M, N])
    bias = torch.from_numpy(r.normal(0, 0.7, N).astype(np.float32)).to(DT[dt])
    res = torch.from_numpy(r.normal(0, 1, (M, N)).astype(np.float32)).to(DT[dt])
    return bias.cuda(), res.cuda(), bias.double().numpy(), res.double().numpy()


# a kernel for one or two rows, one for short x, the tiled one whole and split; odd and even N
SHAPES = [(1, 256, 48), (2, 384, 33), (1, 1536, 256), (7, 1152, 130), (16, 4096, 64), (40, 1024, 515), (64, 640, 1000), (65, 128, 66),
          (130, 2048, 257), (300, 384, 1030), (200, 8960, 257), (1021, 640, 77)]


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("M,D,N", SHAPES)
def test_epilogue(M, D, N, kind):
    C.log(f"epilogue M={M} D={D} N={N} {kind}")
    xq, xs, wq, ws = operands(101, M, D, N)
    ops = on_gpu(xq, xs, wq, ws)
    for dt in DT:
        bias, res, b64, r64 = extras(102, M, N, dt)
        for b, r in ((bias, None), (None, res), (bias, res), (None, None)):
            y, ok = guarded((M, N), DT[dt])
            rl.paro_w8a8_linear_epilogue(*ops, bias=b, activation=kind, residual=r, out=y)
            assert ok()
            want, bound = epilogue_want(xq, xs, wq, ws, None if b is None else b64, kind, None if r is None else r64, dt)
            assert over(y.double().cpu().numpy() - want, bound) <= 1, (dt, b is None, r is None)
            if b is None and r is None and kind == "none":
                assert torch.equal(y, rl.paro_w8a8_linear(*ops, DT[dt]))
        # the stream in place of itself, and the types that follow from the operands
        at = res.clone()
        assert rl.paro_w8a8_linear_epilogue(*ops, bias=bias, activation=kind, residual=at, out=at) is at
        got = rl.paro_w8a8_linear_epilogue(*ops, bias=bias, activation=kind, residual=res)
        assert got.dtype == DT[dt] and torch.equal(got, at)


@pytest.mark.parametrize("kind", ACTS)
@pytest.mark.parametrize("dt", list(DT))
def test_activations_over_their_range(kind, dt):
    """Products of 0 and a bias that runs through the type: every size of argument, infinities and NaN."""
    r = np.random.default_rng(7)
    v = np.concatenate([np.linspace(-20, 20, 4001), r.normal(0, 1, 400) * 2.0 ** r.integers(-40, 7, 400), [0.0, -0.0, 90.0, -90.0, 1e4, -1e4]])
    if dt != "f16":
        v = np.concatenate([v, [1e30, -1e30, 3e38, -3e38]])
    v = np.concatenate([v, [np.inf, -np.inf, np.nan, 0.5]])
    bias = torch.from_numpy(v.astype(np.float32)).to(DT[dt])
    N, v = len(v), bias.double().numpy()
    for M in (1, 3, 70):  # one kernel each
        x, xs = torch.zeros(M, 128, dtype=torch.int8, device="cuda"), torch.ones(M, device="cuda")
        w, ws = torch.zeros(N, 128, dtype=torch.int8, device="cuda"), torch.ones(N, device="cuda")
        y = rl.paro_w8a8_linear_epilogue(x, xs, w, ws, bias=bias.cuda(), activation=kind)
        y = y.double().cpu().numpy()
        assert (y[1:] == y[0]).sum() + np.isnan(y[1:]).sum() == y[1:].size
        ok = np.isfinite(v)
        want = B.act(v[ok], kind)
        top = {"f16": 65504.0, "bf16": 3.38e38, "f32": 3.4e38}[dt]
        fits = np.abs(want) < top
        bound = act_bound(v[ok], 0.0, kind, dt)
        bound = bound + HALF[dt] * (np.abs(want) + bound) + SUB[dt]
        assert over((y[0][ok] - want)[fits], bound[fits]) <= 1
        assert np.isinf(y[0][ok][~fits]).all()
        assert y[0][-4] == np.inf and np.isnan(y[0][-2])
        low = y[0][-3]
        assert (low == -np.inf) if kind == "none" else (low == 0) if kind.startswith("relu") else np.isnan(low)


@pytest.mark.parametrize("M,N", [(1, 48), (5, 48), (33, 130), (64, 258), (200, 515), (1300, 260)])
def test_rows_do_not_depend_on_their_call(M, N):
    """The same bits in a call of its own, whichever kernel that takes; a workspace full of anything."""
    D = 2048
    ops = on_gpu(*operands(103, M, D, N))
    for dt in DT:
        bias, res, _, _ = extras(104, M, N, dt)
        for kind in ("gelu", "silu", "gelu_tanh", "relu2"):
            need = rl.paro_w8a8_workspace_bytes(M, D, N)
            ws = torch.full((max(16, need),), 255, dtype=torch.uint8, device="cuda")
            y = rl.paro_w8a8_linear_epilogue(*ops, bias=bias, activation=kind, residual=res, ws=ws)
            for a, b in {(0, 1), (M // 2, M), (M - 1, M), (0, min(M, 20))}:
                got = rl.paro_w8a8_linear_epilogue(ops[0][a:b].clone(), ops[1][a:b].clone(), *ops[2:], bias=bias, activation=kind,
                                                   residual=res[a:b].clone())
                assert torch.equal(got, y[a:b]), (dt, kind, a, b)


_i, _p, _sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
lib.paro_internal_w8a8_tiled_epilogue.argtypes = [_i, _i, _i, _i, _i, _p, _p, _p, _p, _p, _i, _p, _p, _i, _p, _sz, _p]


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("tile", range(7))
def test_every_tiling(tile, splits):
    """Whole and split, more tiles than workgroups at once and fewer, rows of y at 16-byte boundaries and not."""
    for M, D, N, dt, kind in ((70, 640, 259, "f16", "gelu"), (300, 384, 520, "bf16", "silu"), (515, 512, 1030, "f32", "relu2"),
                              (2100, 384, 4104, "f16", "none"), (37, 1024, 4, "bf16", "relu"), (33, 384, 1, "f32", "gelu_tanh")):
        C.log(f"tiling {tile} splits {splits} M={M} D={D} N={N} {dt}")
        ops = on_gpu(*operands(105, M, D, N))
        bias, res, _, _ = extras(106, M, N, dt)
        y, ok = guarded((M, N), DT[dt])
        y.copy_(res)  # in place
        need = lib.paro_internal_w8a8_tiled_workspace_bytes(M, N, 0, splits)
        ws = torch.full((max(need, 16),), 85, dtype=torch.uint8, device="cuda")
        st = lib.paro_internal_w8a8_tiled_epilogue(tile, splits, M, D, N, *(t.data_ptr() for t in ops), bias.data_ptr(), ACTS.index(kind),
                                                   y.data_ptr(), y.data_ptr(), {"f16": rl.F16, "bf16": rl.BF16, "f32": rl.F32}[dt],
                                                   ws.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and ok()
        assert torch.equal(y, rl.paro_w8a8_linear_epilogue(*ops, bias=bias, activation=kind, residual=res))


NORMS = [(1, 128), (1, 4096), (1, 16384), (2, 256), (3, 1152), (6, 1536), (33, 4480), (64, 14336), (130, 384), (600, 1024), (2050, 256),
         (300, 5120), (521, 16384)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,D", NORMS)
def test_block_norm(M, D, dt):
    C.log(f"block norm M={M} D={D} {dt}")
    x, x64 = rows(111, M, D, dt)
    res, r64 = rows(112, M, D, dt, 10.0)
    r = np.random.default_rng(D)

    def vector(n, mean, spread):
        t = torch.from_numpy(r.normal(mean, spread, (n, D)).astype(np.float32)).to(DT[dt])
        return t.cuda(), t.double().numpy()

    gamma, g64 = vector(1, 1, 0.3)
    post, p64 = vector(1, 0.6, 0.2)
    eps = 1e-5
    every = next(g for g in (3, 2, 1) if M % g == 0)
    for with_post, gates, alpha in ((True, 0, 1.0), (True, every, 0.3), (False, 1, 1.0), (False, M, -0.7), (False, 0, 1.0)):
        gate, t64 = vector(gates, 0, 0.5) if gates else (None, None)
        kw = {"post_gamma": post[0] if with_post else None, "gate": gate if gates != 1 else gate[0], "residual_scale": alpha}
        h64, p = B.stream(x64, r64, eps, p64[0] if with_post else None, t64, np.float64(np.float32(alpha)))
        (q, qok), (sc, scok), (y, yok), (ho, hok) = (guarded(s, t) for s, t in (((M, D), torch.int8), ((M,), torch.float32),
                                                                                ((M, D), DT[dt]), ((M, D), DT[dt])))
        _, _, h = rl.paro_block_norm_q8(x, res, gamma[0], eps, out=(q, sc), residual_out=ho, **kw)
        assert h is ho and qok() and scok() and hok()
        got = h.double().cpu().numpy()
        # 1 / sqrt, three products, the fused sum; then the type's rounding
        d = 4.1 * U * np.abs(p) + U * np.abs(h64)
        assert over(got - h64, d + HALF[dt] * (np.abs(h64) + d) + SUB[dt]) <= 1
        _, h = rl.paro_block_norm(x, res, gamma[0], eps, out=y, residual_out=ho.zero_(), **kw)
        assert yok() and hok() and np.array_equal(h.double().cpu().numpy(), got)
        # the second norm is that of the rounded stream, the quantiser that of the rows: as in the test of paro_rmsnorm_q8
        n = Q.rmsnorm(got, g64, eps)
        assert over(y.double().cpu().numpy() - n, np.abs(n) * (4 * U + HALF[dt]) + SUB[dt]) <= 1
        real, want = Q.quantize_exact(n)
        assert over(sc.double().cpu().numpy() - want, want * 5 * U) <= 1
        code = q.cpu().numpy().astype(np.float64)
        assert np.abs(code - real).max() <= 0.5 + 127 * 6 * U
        # bit for bit what the norm of the stream gives
        q2, s2, _ = rl.paro_rmsnorm_q8(h.contiguous(), gamma[0], eps)
        assert torch.equal(q2, q) and torch.equal(s2, sc)
        if not with_post and not gates and alpha == 1.0:
            y2, h2 = rl.paro_rmsnorm(x, gamma[0], eps, residual=res)
            assert torch.equal(y2, y) and torch.equal(h2, h)
        # in place of the stream, each row by itself
        at = res.clone()
        rl.paro_block_norm(x, at, gamma[0], eps, residual_out=at, **kw)
        assert torch.equal(at, h)
        m = M - 1
        one = {**kw, "gate": None if not gates else gate[m // (M // gates)]}
        y1, h1 = rl.paro_block_norm(x[m:].clone(), res[m:].clone(), gamma[0], eps, **one)
        assert torch.equal(y1[0], y[m]) and torch.equal(h1[0], h[m])


def test_block_norm_odd_rows():
    """Zero rows, infinities and NaN stay in their rows; bfloat16 rows whose squares, or whose 1 / sqrt, pass float32."""
    D = 1536
    for dt in ("bf16", "f16"):
        x, _ = rows(121, 8, D, dt)
        res, _ = rows(122, 8, D, dt)
        x[1] = 0
        res[1] = 0
        x[2, 700] = float("inf")
        x[3, 1] = float("nan")
        res[4, 5] = float("-inf")
        if dt == "bf16":
            x[5] *= 2.0 ** 100  # their squares pass float32
            x[6] *= 2.0 ** -100
            x[7] = 2.0 ** 127  # 1 / sqrt lies under 2^-126
            res[7] = 0
        g = torch.full((D,), 0.5, dtype=DT[dt], device="cuda")
        gate = torch.full((8, D), 2.0, dtype=DT[dt], device="cuda")
        q, s, h = rl.paro_block_norm_q8(x, res, g, 1e-6, post_gamma=g, gate=gate)
        assert not q[1].any() and float(s[1]) > 0 and not h[1].any()
        for r in (2, 3, 4):
            assert not q[r].any() and bool(s[r].isnan()), r
        ok = [0, 5, 6, 7]
        h64, p = B.stream(x[ok].double().cpu().numpy(), res[ok].double().cpu().numpy(), 1e-6, np.full(D, 0.5), np.full((4, D), 2.0))
        d = 4.1 * U * np.abs(p) + U * np.abs(h64)
        assert over(h[ok].double().cpu().numpy() - h64, d + HALF[dt] * (np.abs(h64) + d) + SUB[dt]) <= 1
        n = Q.rmsnorm(h[ok].double().cpu().numpy(), np.full(D, 0.5), 1e-6)
        real, sc = Q.quantize_exact(n)
        assert over(s[ok].double().cpu().numpy() - sc, sc * 5 * U) <= 1
        assert np.abs(q[ok].cpu().numpy() - real).max() <= 0.5 + 127 * 6 * U
    # an x of infinities behind a gate of 0 is a NaN, as the formula says; a residual scale of 0 takes nothing but those
    x, res = torch.ones(2, 128).half().cuda(), torch.ones(2, 128).half().cuda()
    y, h = rl.paro_block_norm(x, res, torch.ones(128).half().cuda(), 1e-6, gate=torch.zeros(128).half().cuda(), residual_scale=0.0)
    assert not y.any() and not h.any()
