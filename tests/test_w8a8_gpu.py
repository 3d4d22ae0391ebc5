"""The 8-bit path on the GPU against its float64 oracle: residual RMS norm, row quantiser (plain and
behind the transform), read-back, weight packing, the W8A8 products, and a run of them together.

Tolerances count roundings: u = 2^-24 is half a float32 step, a 16-bit type adds half of its own
step (2^-11 for float16, 2^-8 for bfloat16). Real-valued codes are compared before rounding: a code
is right if it is within 1/2 plus the arithmetic's error of the exact quotient.
"""
import numpy as np
import pytest

from oracle import q8_oracle as Q
from tests import gpu_common as C
import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": U}
# half the spacing of the type's subnormal numbers
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}


def rows(seed, M, D, dt, mult=30.0):
    """Activation-like rows on the GPU and their exact float64 values."""
    r = np.random.default_rng([seed, M, D])
    x = r.normal(0, 1, (M, D))
    x[:, r.choice(D, max(1, D // 200), replace=False)] *= mult
    t = torch.from_numpy(x.astype(np.float32)).to(DT[dt])
    return t.cuda(), t.double().numpy()


def guarded(shape, dtype, fill=7):
    """A contiguous tensor followed by 4 KiB of `fill` bytes: (tensor, the tail's check)."""
    n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
    buf = torch.full((n + 4096,), fill, dtype=torch.uint8, device="cuda")
    t = buf[:n].view(dtype).view(shape)
    return t, lambda: bool((buf[n:] == fill).all())


def over(err, bound):
    return C.over_bound(np.asarray(err), np.asarray(bound))


SHAPES = [(1, 128), (1, 4096), (1, 16384), (2, 256), (3, 1152), (5, 1536), (17, 2048), (33, 4480), (64, 14336), (7, 8960),
          (130, 384), (600, 1024), (2050, 256), (300, 5120)]


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,D", SHAPES)
def test_rmsnorm(M, D, dt):
    C.log(f"rmsnorm M={M} D={D} {dt}")
    x, x64 = rows(1, M, D, dt)
    res, r64 = rows(2, M, D, dt, 10.0)
    r = np.random.default_rng(D)
    g = torch.from_numpy(r.normal(1, 0.3, D).astype(np.float32)).to(DT[dt])
    g64 = g.double().numpy()
    g = g.cuda()
    eps = 1e-5
    for residual in (res, None):
        h64 = Q.round_to(Q.round_to(x64 + r64, "f32"), dt) if residual is not None else x64
        n = Q.rmsnorm(h64, g64, eps)
        q, qok = guarded((M, D), torch.int8)
        sc, scok = guarded((M,), torch.float32)
        y, yok = guarded((M, D), DT[dt])
        ho, hok = guarded((M, D), DT[dt])
        kw = {} if residual is None else {"residual": residual, "residual_out": ho}
        _, _, h = rl.paro_rmsnorm_q8(x, g, eps, out=(q, sc), **kw)
        assert qok() and scok() and hok()
        if residual is not None:
            assert np.array_equal(h.double().cpu().numpy(), h64)
            ho.zero_()
        else:
            assert h is None
        _, h = rl.paro_rmsnorm(x, g, eps, out=y, **kw)
        assert yok() and hok()
        if residual is not None:
            assert np.array_equal(h.double().cpu().numpy(), h64)
        # n: h * gamma, 1 / sqrt and their product, one float32 rounding each, then the type's own
        got = y.double().cpu().numpy()
        assert over(got - n, np.abs(n) * (4 * U + HALF[dt]) + SUB[dt]) <= 1
        # scale: those three and the division by 127. Codes: h * gamma, the step and the product.
        real, want = Q.quantize_exact(n)
        s = sc.double().cpu().numpy()
        assert over(s - want, want * 5 * U) <= 1
        code = q.cpu().numpy().astype(np.float64)
        assert np.abs(code - real).max() <= 0.5 + 127 * 6 * U
        assert np.abs(code).max() == 127


def test_rmsnorm_in_place_stream_and_odd_rows():
    """residual_out = residual; a zero row; a row with an infinity; a row with a NaN; bfloat16 rows
    whose squares pass float32; very small rows (eps decides)."""
    D = 1536
    x, _ = rows(3, 6, D, "bf16")
    res, _ = rows(4, 6, D, "bf16")
    x[1] = 0
    res[1] = 0
    x[2, 700] = float("inf")
    x[3, 1] = float("nan")
    x[4] *= 1e25
    res[4] = 0
    x[5] *= 1e-30
    res[5] = 0
    g = torch.full((D,), 0.5, dtype=torch.bfloat16, device="cuda")
    stream = res.clone()
    q, s, h = rl.paro_rmsnorm_q8(x, g, 1e-6, residual=stream, residual_out=stream)
    assert h.data_ptr() == stream.data_ptr()
    want = (x.float() + res.float()).bfloat16()
    assert torch.equal(h.nan_to_num(nan=3e38), want.nan_to_num(nan=3e38))
    n = Q.rmsnorm(want[[0, 4, 5]].double().cpu().numpy(), np.full(D, 0.5), 1e-6)
    real, sc = Q.quantize_exact(n)
    assert over(s[[0, 4, 5]].double().cpu().numpy() - sc, sc * 5 * U) <= 1
    assert np.abs(q[[0, 4, 5]].cpu().numpy() - real).max() <= 0.5 + 127 * 6 * U
    assert not q[1].any() and float(s[1]) > 0
    assert not q[2].any() and not q[3].any() and bool(s[2:4].isnan().all())
    y, _ = rl.paro_rmsnorm(x, g, 1e-6, residual=res)
    assert not y[1].any() and bool(y[2].isnan().any()) and bool(y[3].isnan().all())
    assert bool(y[[0, 1, 4, 5]].isfinite().all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,D", SHAPES)
def test_quantize_plain_and_read_back(M, D, dt):
    C.log(f"quantize M={M} D={D} {dt}")
    x, x64 = rows(5, M, D, dt)
    q, qok = guarded((M, D), torch.int8)
    sc, scok = guarded((M,), torch.float32)
    rl.paro_quantize_q8(x, out=(q, sc))
    assert qok() and scok()
    real, want = Q.quantize_exact(x64)
    s = sc.double().cpu().numpy()
    assert np.array_equal(s, Q.round_to(want, "f32"))  # the maximum is exact: one rounding
    code = q.cpu().numpy().astype(np.float64)
    assert np.abs(code - real).max() <= 0.5 + 127 * 2 * U  # the step's rounding and the product's
    for o in ("f16", "bf16", "f32"):
        back, ok = guarded((M, D), DT[o])
        rl.paro_dequantize_q8(q, sc, out=back)
        assert ok()
        # the product rounds to float32 once, then to the type
        assert np.array_equal(back.double().cpu().numpy(), Q.round_to(Q.round_to(code * s[:, None], "f32"), o))


def test_quantize_odd_rows():
    """Zero rows, rows of the smallest and largest numbers, infinities and NaN, ties to even."""
    D = 256
    x = torch.zeros(8, D, dtype=torch.bfloat16)
    x[1] = float("inf")
    x[2, 255] = float("nan")
    x[3, 7] = -float("inf")
    x[4, 3] = 3.3e38
    x[5, 9] = 2.0 ** -110
    x[6] = torch.arange(D).bfloat16() / 2
    x[6, 0] = -127.0
    x[6, 128:] = 0
    q, s = rl.paro_quantize_q8(x.cuda())
    q, s = q.cpu(), s.cpu()
    tiny = np.float32(2.0 ** -100 / 127)
    assert not q[0].any() and s[0] == tiny and not q[7].any()
    for r in (1, 2, 3):
        assert not q[r].any() and s[r].isnan()
    assert int(q[4, 3]) == 127 and int(q[4].abs().sum()) == 127
    assert s[5] == tiny and not q[5].any()
    want = np.rint(np.arange(128) / 2)
    want[0] = -127
    assert float(s[6]) == 1.0 and np.array_equal(q[6, :128].numpy(), want.astype(np.int8))
    back = rl.paro_dequantize_q8(q.cuda(), s.cuda(), torch.float32)
    assert bool(back[1:4].isnan().all()) and bool(back[[0, 4, 5, 6, 7]].isfinite().all())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_values_half_way_between_codes_go_to_the_even_one(dt):
    """Rows whose maximum is 127 m 2^e hold values m (2 k + 1) 2^(e-1), exactly half way between two
    codes, also where 127 / maximum has no exact float32: k rounds to even there. The same through the
    norm with a gamma of one number."""
    ms = [1, 3, 5, 7, 9, 11, 13, 15] if dt == "f16" else [1]  # 127 m in the type's digits
    D = 256
    k = np.arange(D) - 128
    x = np.stack([np.where(np.abs(k) == 128, 127.0, np.clip(k + 0.5, -127, 127)) * m * 2.0 ** e for m in ms for e in (-9, 0, 4)])
    ok = Q.round_to(x, dt) == x  # the halves that the type holds
    x = np.where(ok, x, 0.0)
    x[:, 0] = np.abs(x).max(axis=1)
    want = np.rint(Q.quantize_exact(x)[0])
    t = torch.from_numpy(x).to(DT[dt]).cuda()
    assert np.array_equal(t.double().cpu().numpy(), x)
    assert (np.abs(Q.quantize_exact(x)[0] % 1 - 0.5) < 1e-9).sum() > 20 * len(ms)
    q, _ = rl.paro_quantize_q8(t)
    assert np.array_equal(q.cpu().numpy(), want)
    q, _ = rl.paro_pack_weights_q8(t)
    assert np.array_equal(q.cpu().numpy(), want) and np.array_equal(Q.pack_weights(x)[0], want)
    q, _, _ = rl.paro_rmsnorm_q8(t, torch.full((D,), 0.75, dtype=DT[dt], device="cuda"), 1e-6)
    assert np.array_equal(q.cpu().numpy(), want)


ROT = [(1, 128, 1, "f16"), (1, 1536, 8, "f16"), (16, 1536, 8, "bf16"), (3, 256, 2, "f16"), (65, 4096, 8, "f16"), (257, 1152, 8, "bf16"),
       (520, 2048, 8, "f16"), (2, 14336, 8, "f16"), (300, 8960, 8, "f16"), (5, 16384, 8, "bf16"), (1100, 512, 12, "f16"),
       (9, 640, 0, "f16"), (2, 4096, 64, "f16"), (513, 9216, 2, "f16"), (600, 12288, 2, "bf16"), (260, 16384, 1, "f16"),
       (1030, 4224, 3, "f16")]


def rotated_bounds(x64, scale, K, real, sc):
    """Error of the float32 transform (as in rotate_bound: a few float32 roundings of the row's norm
    per stage), in codes: the element's own, and the maximum's through the step."""
    delta = (K + 2) * 4 * U * np.linalg.norm(x64, axis=1, keepdims=True) / scale[None, :].astype(np.float64)
    dtop = delta.max(axis=1, keepdims=True)
    return dtop[:, 0], (delta + np.abs(real) / 127 * dtop) / sc[:, None] * 1.01


@pytest.mark.parametrize("M,D,K,dt", ROT)
def test_quantize_behind_the_transform(M, D, K, dt):
    C.log(f"rotate+quantize M={M} D={D} K={K} {dt}")
    L = W.custom_linear(31, 1, D, 16, K)
    rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
    x, x64 = rows(6, M, D, dt)
    q, qok = guarded((M, D), torch.int8)
    sc, scok = guarded((M,), torch.float32)
    rl.paro_quantize_q8(x, rot, out=(q, sc))
    assert qok() and scok()
    pick = C.sample_rows(M, 48, 1)
    a = Q.transform(x64[pick], L.pairs, L.theta, L.scale)
    real, want = Q.quantize_exact(a)
    dtop, dcode = rotated_bounds(x64[pick], L.scale, K, real, want)
    s = sc.double().cpu().numpy()[pick]
    assert over(s - want, dtop / 127 + want * 2 * U) <= 1
    code = q.cpu().numpy()[pick].astype(np.float64)
    assert over(code - real, 0.5 + 127 * 2 * U + dcode) <= 1
    # rows are independent: each one alone gives the same bits
    for m in {0, M // 2, M - 1}:
        q1, s1 = rl.paro_quantize_q8(x[m:m + 1].clone(), rot)
        assert torch.equal(q1[0], q[m]) and torch.equal(s1[0], sc[m]), m


@pytest.mark.parametrize("D", [128, 256, 512, 640, 768, 896, 1024, 1280, 1536, 1664, 2048, 2304, 2944, 4096, 4224, 5120, 6144, 6272,
                               7168, 7296, 8192, 8320, 8960, 9088, 9216, 9344, 10240, 10368, 12288, 12416, 14336, 14464, 16384])
def test_quantize_behind_the_transform_at_every_width(D):
    """One, two and four rows a workgroup, with pairs that divide over its threads and that do not."""
    K, M = 3, 520
    L = W.custom_linear(31, 5, D, 16, K)
    rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
    x, x64 = rows(9, M, D, "f16")
    (q, qok), (sc, scok) = guarded((M, D), torch.int8), guarded((M,), torch.float32)
    rl.paro_quantize_q8(x, rot, out=(q, sc))
    assert qok() and scok()
    pick = C.sample_rows(M, 12, 1)
    real, want = Q.quantize_exact(Q.transform(x64[pick], L.pairs, L.theta, L.scale))
    dtop, dcode = rotated_bounds(x64[pick], L.scale, K, real, want)
    assert over(sc.double().cpu().numpy()[pick] - want, dtop / 127 + want * 2 * U) <= 1
    assert over(q.cpu().numpy()[pick].astype(np.float64) - real, 0.5 + 127 * 2 * U + dcode) <= 1
    for a, b in ((0, 300), (M - 7, M)):  # the same rows in calls of two rows and of one row a workgroup
        (qb, qbok), (sb, sbok) = guarded((b - a, D), torch.int8), guarded((b - a,), torch.float32)
        rl.paro_quantize_q8(x[a:b].clone(), rot, out=(qb, sb))
        assert qbok() and sbok() and torch.equal(qb, q[a:b]) and torch.equal(sb, sc[a:b])


def test_quantize_behind_the_transform_odd_rows():
    D = 512
    L = W.custom_linear(33, 1, D, 16, 8)
    rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
    x, _ = rows(8, 7, D, "f16")
    clean = x.clone()
    x[1, 5] = float("nan")
    x[3, 500] = float("inf")
    x[5] = 0
    q, s = rl.paro_quantize_q8(x, rot)
    qc, sc = rl.paro_quantize_q8(clean, rot)
    for r in (1, 3):
        assert not q[r].any() and bool(s[r].isnan())
    assert not q[5].any() and float(s[5]) > 0
    for r in (0, 2, 4, 6):
        assert torch.equal(q[r], qc[r]) and torch.equal(s[r], sc[r])


@pytest.mark.parametrize("N,D,K,dt", [(1, 128, 2, "f16"), (5, 256, None, "f16"), (33, 1536, 8, "bf16"), (64, 4096, 8, "f16"),
                                      (3, 16384, 2, "f16"), (7, 8960, None, "bf16"), (40, 384, 0, "f16"), (9, 640, 64, "f16")])
def test_pack_weights_bit_exact(N, D, K, dt):
    C.log(f"pack N={N} D={D} K={K} {dt}")
    L = W.custom_linear(41, 1, D, 16, K or 0)
    w, w64 = rows(9, N, D, dt, 10.0)
    q, qok = guarded((N, D), torch.int8)
    sc, scok = guarded((N,), torch.float32)
    if K is None:
        rl.paro_pack_weights_q8(w, out=(q, sc))
        oq, osc = Q.pack_weights(w64)
    else:
        rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
        rl.paro_pack_weights_q8(w, rot, out=(q, sc))
        oq, osc = Q.pack_weights(w64, L.pairs, L.theta, L.scale)
    assert qok() and scok()
    assert np.array_equal(q.cpu().numpy(), oq)
    assert np.array_equal(sc.cpu().numpy(), osc)


def test_pack_weights_odd_rows():
    w, _ = rows(10, 5, 256, "f16")
    w[1] = 0
    w[2, 3] = float("nan")
    w[4, 255] = float("-inf")
    q, s = rl.paro_pack_weights_q8(w)
    assert not q[1].any() and float(s[1]) > 0
    for r in (2, 4):
        assert not q[r].any() and bool(s[r].isnan())
    assert bool(s[[0, 1, 3]].isfinite().all()) and int(q[0].abs().max()) == 127


def operands(seed, M, D, N, full=False):
    r = np.random.default_rng([seed, M, D, N])
    if full:  # the whole int8 range, -128 included
        xq, wq = r.integers(-128, 128, (M, D)), r.integers(-128, 128, (N, D))
    else:
        xq, wq = (np.clip(np.rint(r.normal(0, 32, (n, D))), -127, 127) for n in (M, N))
    xs = r.uniform(0.02, 0.06, M).astype(np.float32)
    ws = (r.uniform(0.5, 1.5, N) / (32 * np.sqrt(D))).astype(np.float32)
    return xq.astype(np.int8), xs, wq.astype(np.int8), ws


def on_gpu(*a):
    return [torch.from_numpy(v).cuda() for v in a]


def linear_bound(ref, dt):
    """int -> float32, times xs, times ws (one rounding each), then the output's rounding."""
    return np.abs(ref) * (3.1 * U + (0 if dt == "f32" else HALF[dt])) + SUB[dt]


def gated_bound(v, g, u, dt):
    """In units of U: g and u are three roundings each; exp(-g) takes g's error and the argument's
    two more roundings into |g| times as much (5 |g|), and the exponential's own (2); 1 + e (1), its
    reciprocal (2), two products (2). Far below -87 exp(-g) or the reciprocal leaves float32."""
    rel = (5 * np.abs(g) + 16) * U + (0 if dt == "f32" else HALF[dt])
    return np.abs(v) * rel + np.abs(g * u) * 2.0 ** -120 + SUB[dt]


LIN = [(1, 128, 1), (1, 4096, 4096), (1, 16384, 130), (2, 1536, 257), (3, 384, 15), (4, 1152, 64), (5, 256, 17), (8, 2048, 300),
       (9, 4480, 65), (15, 640, 63), (16, 8960, 129), (17, 128, 16), (31, 1536, 1000), (32, 14336, 48), (33, 1024, 255),
       (48, 4096, 512), (49, 512, 33), (63, 3968, 80), (64, 14336, 256), (65, 1536, 256), (77, 1152, 1003), (100, 128, 31),
       (128, 4096, 384), (129, 640, 257), (200, 8960, 257), (255, 2176, 511), (256, 1024, 1024), (257, 384, 129), (300, 16384, 130),
       (513, 1536, 640), (1021, 1280, 1537), (1500, 256, 2000), (2, 256, 70001), (4100, 128, 3)]


@pytest.mark.parametrize("M,D,N", LIN)
def test_linear(M, D, N):
    C.log(f"w8a8 linear M={M} D={D} N={N}")
    xq, xs, wq, ws = operands(51, M, D, N, full=(M + N) % 2 == 1)
    ref = Q.linear(xq, xs, wq, ws)
    d = on_gpu(xq, xs, wq, ws)
    for dt in ("f16", "bf16", "f32"):
        y, ok = guarded((M, N), DT[dt])
        need = rl.paro_w8a8_workspace_bytes(M, D, N)
        work = torch.full((max(need, 16),), 0xA5, dtype=torch.uint8, device="cuda")  # nothing in it needs to start at zero
        rl.paro_w8a8_linear(*d, out=y, ws=work)
        assert ok()
        assert over(y.double().cpu().numpy() - ref, linear_bound(ref, dt)) <= 1, dt
    y2 = rl.paro_w8a8_linear(*d, torch.float32)
    assert torch.equal(y, y2)  # the same bits every time


@pytest.mark.parametrize("M,D,F", [(1, 128, 1), (1, 4096, 700), (2, 1536, 129), (5, 1536, 8960), (8, 256, 33), (16, 4480, 64), (17, 128, 15),
                                   (33, 1152, 130), (64, 4096, 257), (65, 384, 100), (100, 2048, 129), (128, 640, 512),
                                   (200, 8960, 65), (257, 1024, 385), (300, 16384, 70), (1000, 512, 1111), (2, 256, 33001)])
def test_gated_linear(M, D, F):
    C.log(f"w8a8 gated M={M} D={D} F={F}")
    xq, xs, wq, ws = operands(52, M, D, 2 * F)
    ws = ws * np.float32(20)  # gates of a few units to a hundred
    v, g, u = Q.gated(xq, xs, wq, ws)
    d = on_gpu(xq, xs, wq, ws)
    for dt in ("f16", "bf16", "f32"):
        y, ok = guarded((M, F), DT[dt])
        need = rl.paro_w8a8_gated_workspace_bytes(M, D, F)
        work = torch.full((max(need, 16),), 0xA5, dtype=torch.uint8, device="cuda")
        rl.paro_w8a8_gated_linear(*d, out=y, ws=work)
        assert ok()
        got = y.double().cpu().numpy()
        big = np.abs(v) > 65000 if dt == "f16" else np.zeros_like(v, bool)  # past float16: an infinity is right there
        assert over((got - v)[~big], gated_bound(v, g, u, dt)[~big]) <= 1, dt
    assert torch.equal(y, rl.paro_w8a8_gated_linear(*d, torch.float32))


# Shapes that the plan spreads over the tilings of the tiled kernel, whole and split, with ragged ends and rows
# of y at 16-byte boundaries. (test_w8a8_tilings.py runs each tiling by name.)
TILED = [(654, 384, 11023, False), (1606, 256, 15152, False), (138, 11904, 5769, False), (258, 384, 11466, True), (1158, 256, 9798, True),
         (134, 12032, 2840, True), (129, 128, 12350, False), (514, 128, 13270, False), (514, 128, 13272, False), (68, 128, 8478, True),
         (260, 128, 10981, True), (260, 128, 10984, True), (71, 9472, 8197, True), (129, 512, 13533, False), (2075, 13824, 65, False),
         (2881, 9728, 70, False), (66, 640, 8975, True), (2713, 8064, 37, True), (2778, 9728, 34, True), (4409, 128, 391, False),
         (3739, 256, 1032, False), (2831, 2688, 23, False), (4163, 128, 193, True), (2973, 256, 665, True), (2841, 6912, 17, True),
         (69, 128, 11270, False), (270, 128, 11200, False), (33, 4224, 1481, False), (702, 5504, 134, False), (33, 128, 9174, True),
         (130, 128, 8624, True), (33, 4224, 803, True), (1060, 4736, 33, True), (413, 128, 4667, False), (1160, 768, 3330, False),
         (1067, 7808, 265, False), (278, 15488, 544, False), (820, 128, 1219, True), (1185, 768, 1666, True), (1303, 11008, 65, True),
         (129, 384, 10994, False), (1034, 3200, 17, False), (65, 384, 9115, True), (34, 2688, 713, True),
         # one row of tiles (each starts its walk over the channels elsewhere), whole and split
         (64, 2048, 9000, False), (40, 1536, 7000, True), (64, 14336, 264, False), (50, 8960, 120, True),
         (715, 128, 13689, False), (3335, 128, 7016, False), (329, 128, 14149, True), (1095, 128, 9883, True), (140, 6656, 8597, True),
         (579, 128, 9795, False), (1417, 128, 10819, False), (135, 13184, 8885, False), (193, 128, 12305, True), (3196, 128, 2479, True),
         (145, 11520, 4205, True), (199, 128, 12575, False), (520, 128, 12901, False), (4134, 16000, 69, False), (67, 128, 12863, True),
         (322, 128, 9902, True), (4418, 15232, 34, True), (66, 256, 11509, False), (716, 512, 5400, False), (4138, 5120, 19, False),
         (2991, 6272, 18, False), (66, 256, 5591, True), (2483, 512, 769, True), (1368, 9088, 34, True), (1380, 9728, 35, True),
         (161, 128, 11014, False), (1370, 4864, 18, False), (66, 128, 11288, True), (325, 11648, 33, True), (35, 15872, 1600, True),
         (263, 128, 13751, False), (584, 128, 13224, False), (129, 128, 11001, True), (324, 128, 10946, True),
         (8, 8320, 18, False), (1427, 4224, 16, False), (8, 5504, 17, True), (8, 15488, 1455, True),
         # three stages of 256 x 128 tiles, whole, aligned and ragged
         (268, 1536, 13633, False), (322, 1536, 11376, False), (136, 1536, 11013, True), (146, 1536, 11176, True),
         (193, 2048, 8193, True), (579, 2048, 6584, False)]


@pytest.mark.parametrize("M,D,N,gated", TILED)
def test_tiled_kernel(M, D, N, gated):
    C.log(f"w8a8 tiled M={M} D={D} N={N} gated={gated}")
    xq, xs, wq, ws = operands(54, M, D, N * (2 if gated else 1))
    if gated:
        ws = ws * np.float32(20)
        ref, g, u = Q.gated(xq, xs, wq, ws)
    else:
        ref = Q.linear(xq, xs, wq, ws)
    fn = rl.paro_w8a8_gated_linear if gated else rl.paro_w8a8_linear
    need = (rl.paro_w8a8_gated_workspace_bytes if gated else rl.paro_w8a8_workspace_bytes)(M, D, N)
    d = on_gpu(xq, xs, wq, ws)
    work = torch.full((max(need, 16),), 0xA5, dtype=torch.uint8, device="cuda")
    for dt in ("bf16", "f32"):
        y, ok = guarded((M, N), DT[dt])
        fn(*d, out=y, ws=work)
        assert ok()
        bound = gated_bound(ref, g, u, dt) if gated else linear_bound(ref, dt)
        assert over(y.double().cpu().numpy() - ref, bound) <= 1, dt


# 16 columns a workgroup: one to four fragments of rows, fewer steps than waves, few and many
# workgroups, ragged rows and columns, and streamed rows with tails of every kind.
COLUMN = [(3, 128, 15), (16, 384, 200), (9, 1152, 4100), (17, 128, 33), (32, 2048, 48), (24, 640, 4500), (33, 1152, 200), (64, 384, 4111),
          (50, 2048, 900), (64, 128, 17), (48, 1536, 4099), (31, 896, 4112), (8, 4096, 4096), (1, 128, 4), (2, 384, 1030), (1, 640, 9000),
          (2, 4352, 33), (1, 16128, 12)]


@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("M,D,N", COLUMN)
def test_short_x_kernels(M, D, N, gated):
    C.log(f"w8a8 short x M={M} D={D} N={N} gated={gated}")
    xq, xs, wq, ws = operands(57, M, D, N * (2 if gated else 1), full=not gated)
    if gated:
        ws = ws * np.float32(20)
        ref, g, u = Q.gated(xq, xs, wq, ws)
    else:
        ref = Q.linear(xq, xs, wq, ws)
    fn = rl.paro_w8a8_gated_linear if gated else rl.paro_w8a8_linear
    d = on_gpu(xq, xs, wq, ws)
    for dt in ("bf16", "f32"):
        y, ok = guarded((M, N), DT[dt])
        fn(*d, out=y)
        assert ok()
        bound = gated_bound(ref, g, u, dt) if gated else linear_bound(ref, dt)
        assert over(y.double().cpu().numpy() - ref, bound) <= 1, dt


@pytest.mark.parametrize("D,N", [(256, 70), (1536, 256), (4096, 640), (8960, 136)])
def test_rows_do_not_depend_on_the_other_rows(D, N):
    """A row alone (streamed weights), in a short batch and in a long one (every kernel and split):
    the same bits, for the linears, the gated ones and the row kernels."""
    M = 600
    xq, xs, wq, ws = on_gpu(*operands(55, M, D, N))
    x, _ = rows(56, M, D, "f16")
    g = torch.ones(D, dtype=torch.float16, device="cuda")
    for dt in (torch.float16, torch.float32):
        full = rl.paro_w8a8_linear(xq, xs, wq, ws, dt)
        full_g = rl.paro_w8a8_gated_linear(xq, xs, wq, ws, dt)
        for m in (1, 2, 3, 7, 12, 16, 17, 33, 40, 64, 65, 130, 300):
            assert torch.equal(rl.paro_w8a8_linear(xq[:m], xs[:m], wq, ws, dt), full[:m]), (m, dt)
            assert torch.equal(rl.paro_w8a8_gated_linear(xq[:m], xs[:m], wq, ws, dt), full_g[:m]), (m, dt)
    q, s, h = rl.paro_rmsnorm_q8(x, g, residual=x)
    p, t = rl.paro_quantize_q8(x)
    for m in (1, 5, 100):
        q1, s1, h1 = rl.paro_rmsnorm_q8(x[:m], g, residual=x[:m])
        assert torch.equal(q1, q[:m]) and torch.equal(s1, s[:m]) and torch.equal(h1, h[:m])
        p1, t1 = rl.paro_quantize_q8(x[:m])
        assert torch.equal(p1, p[:m]) and torch.equal(t1, t[:m])


@pytest.mark.parametrize("M", [1, 40, 300])
def test_linear_extreme_sums(M):
    """All codes -128 or 127 at D = 16384: sums of +-2^28 are exact in float32."""
    D, N = 16384, 20
    xq = np.full((M, D), -128, np.int8)
    wq = np.full((N, D), -128, np.int8)
    wq[1::2] = 127
    y = rl.paro_w8a8_linear(*on_gpu(xq, np.ones(M, np.float32), wq, np.ones(N, np.float32)), torch.float32)
    want = np.where(np.arange(N) % 2, -128.0 * 127 * D, 2.0 ** 28)
    assert np.array_equal(y.double().cpu().numpy(), np.broadcast_to(want, (M, N)))


@pytest.mark.parametrize("M,D,N", [(3, 256, 40), (40, 4096, 100), (130, 8960, 96)])
def test_linear_scales_that_are_not_finite_stay_in_their_row_and_column(M, D, N):
    xq, xs, wq, ws = operands(53, M, D, N)
    clean = rl.paro_w8a8_linear(*on_gpu(xq, xs, wq, ws), torch.float32)
    gated_clean = rl.paro_w8a8_gated_linear(*on_gpu(xq, xs, wq, ws), torch.float32)
    xs[1] = np.nan
    ws[7] = np.nan
    xs[2] = 0
    y = rl.paro_w8a8_linear(*on_gpu(xq, xs, wq, ws), torch.float32)
    keep = torch.ones(M, N, dtype=torch.bool, device="cuda")
    keep[1:3] = False
    keep[:, 7] = False
    assert torch.equal(y[keep], clean[keep])
    assert bool(y[1].isnan().all()) and bool(y[:, 7].isnan().all())
    assert not y[2, :7].any() and not y[2, 8:].any()
    y = rl.paro_w8a8_gated_linear(*on_gpu(xq, xs, wq, ws), torch.float32)
    assert torch.equal(y[keep[:, :N // 2]], gated_clean[keep[:, :N // 2]])
    assert bool(y[1].isnan().all()) and bool(y[:, 7].isnan().all())


def test_empty_calls():
    e = torch.empty
    for M, N in ((0, 32), (4, 0), (0, 0)):
        x, w = e(M, 256, dtype=torch.int8, device="cuda"), e(N, 256, dtype=torch.int8, device="cuda")
        assert rl.paro_w8a8_linear(x, e(M, device="cuda"), w, e(N, device="cuda")).shape == (M, N)
        assert rl.paro_w8a8_gated_linear(x, e(M, device="cuda"), w, e(N, device="cuda")).shape == (M, N // 2)
    x = e(0, 256, dtype=torch.float16, device="cuda")
    g = torch.ones(256, dtype=torch.float16, device="cuda")
    q, s, h = rl.paro_rmsnorm_q8(x, g, residual=x)
    assert q.shape == (0, 256) and s.shape == (0,) and h.shape == (0, 256)
    assert rl.paro_rmsnorm(x, g)[0].shape == (0, 256)
    assert rl.paro_quantize_q8(x)[0].shape == (0, 256) and rl.paro_pack_weights_q8(x)[0].shape == (0, 256)
    assert rl.paro_dequantize_q8(q, s).shape == (0, 256)
    torch.cuda.synchronize()


class Unusual(torch.Tensor):
    pass


def test_both_ways_of_the_binding_agree():
    """Calls that fit go through the compiled binding; a tensor subclass goes the checked way to the
    same library call, with and without given outputs."""
    from rotated_linear_amd import _binding as b

    M, D, N = 70, 1024, 200
    x, _ = rows(95, M, D, "f16")
    g = torch.ones(D, dtype=torch.float16, device="cuda")
    L = W.custom_linear(96, 1, D, 16, 4)
    rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
    wq, ws = rl.paro_pack_weights_q8(rows(97, N, D, "f16")[0])
    q, s = rl.paro_quantize_q8(x, rot)
    assert b.linear(False, q, s, wq, ws, None, None, None) is not None
    assert b.quantize(False, x, 0, None, None, None) is not None
    assert b.dequantize(q, s, torch.float32, None) is not None
    assert b.rmsnorm(True, x, g, 1e-6, x, None, None, None) is not None
    u = x.as_subclass(Unusual)
    uq = q.as_subclass(Unusual)
    assert b.quantize(False, u, 0, None, None, None) is None and b.linear(False, uq, s, wq, ws, None, None, None) is None
    plain = torch.Tensor
    for f, a, ua in ((rl.paro_quantize_q8, (x, rot), (u, rot)), (rl.paro_pack_weights_q8, (x, rot), (u, rot)),
                     (rl.paro_rmsnorm_q8, (x, g, 1e-6, x), (u, g, 1e-6, u)), (rl.paro_rmsnorm, (x, g, 1e-6, x), (u, g, 1e-6, u)),
                     (rl.paro_dequantize_q8, (q, s), (uq, s)),
                     (rl.paro_w8a8_linear, (q, s, wq, ws), (uq, s, wq, ws)),
                     (rl.paro_w8a8_gated_linear, (q, s, wq, ws), (uq, s, wq, ws))):
        got, want = f(*ua), f(*a)
        for t, v in zip(*((o if isinstance(o, tuple) else (o,)) for o in (got, want))):
            assert torch.equal(t.as_subclass(plain), v), f
    eq, es = torch.empty_like(q), torch.empty_like(s)
    r = rl.paro_quantize_q8(x, rot, out=(eq, es))
    assert r[0].data_ptr() == eq.data_ptr() and torch.equal(eq, q) and torch.equal(es, s)
    y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
    assert rl.paro_w8a8_linear(q, s, wq, ws, out=y).data_ptr() == y.data_ptr()
    with pytest.raises(rl.ParoError, match="EINVAL"):  # an odd address is refused by the library
        rl.paro_dequantize_q8(q, torch.zeros(M + 1, device="cuda")[1:])
    with pytest.raises(rl.ParoError, match="EWORKSPACE"):
        big = torch.zeros(200, 8960, dtype=torch.int8, device="cuda")
        rl.paro_w8a8_linear(big, torch.ones(200, device="cuda"), big, torch.ones(200, device="cuda"),
                            ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(rl.ParoError, match="EINVAL"):  # h over x
        rl.paro_rmsnorm_q8(x, g, 1e-6, residual=x.clone(), residual_out=x)
    torch.cuda.synchronize()


# ---- a decoder layer's MLP: norm, gate and up, quantiser behind the transform, down ----

class Mlp:
    def __init__(self, seed, D, F, K=8):
        r = np.random.default_rng(seed)
        self.D, self.F = D, F
        self.gamma = torch.from_numpy(r.normal(1, 0.2, D).astype(np.float16)).cuda()
        t = W.custom_linear(seed, 1, F, 16, K)
        self.t = t
        self.rot = rl.paro_rotation_prepare(t.pairs, t.theta, t.scale)
        self.w_gu = torch.from_numpy((r.normal(0, 1, (2 * F, D)) / np.sqrt(D)).astype(np.float16)).cuda()
        self.w_d = torch.from_numpy((r.normal(0, 1, (D, F)) / np.sqrt(F)).astype(np.float16)).cuda()
        self.gu = rl.paro_pack_weights_q8(self.w_gu)
        self.d = rl.paro_pack_weights_q8(self.w_d, self.rot)

    def run(self, x, stream):
        xq, xs, _ = rl.paro_rmsnorm_q8(x, self.gamma, 1e-5, residual=stream, residual_out=stream)
        a = rl.paro_w8a8_gated_linear(xq, xs, *self.gu)
        aq, as_ = rl.paro_quantize_q8(a, self.rot)
        return xq, xs, a, aq, as_, rl.paro_w8a8_linear(aq, as_, *self.d)

    def check(self, x, stream0, out):
        xq, xs, a, aq, as_, y = [t.double().cpu().numpy() for t in out]
        h = Q.round_to(x.double().cpu().numpy() + stream0.double().cpu().numpy(), "f16")
        # each step against the oracle on what it was given
        real, sc = Q.quantize_exact(Q.rmsnorm(h, self.gamma.double().cpu().numpy(), 1e-5))
        assert np.abs(xq - real).max() <= 0.5 + 127 * 6 * U and over(xs - sc, 5 * U * sc) <= 1
        v, g, u = Q.gated(xq, xs, *[t.double().cpu().numpy() for t in self.gu])
        assert over(a - v, gated_bound(v, g, u, "f16")) <= 1
        real, sc = Q.quantize_exact(Q.transform(a, self.t.pairs, self.t.theta, self.t.scale))
        dtop, dcode = rotated_bounds(a, self.t.scale, 8, real, sc)
        assert over(aq - real, 0.5 + 127 * 2 * U + dcode) <= 1 and over(as_ - sc, dtop / 127 + 2 * U * sc) <= 1
        ref = Q.linear(aq, as_, *[t.double().cpu().numpy() for t in self.d])
        assert over(y - ref, linear_bound(ref, "f16")) <= 1
        # and the block against itself without any quantisation: 8 bits keep two digits
        n = Q.rmsnorm(h, self.gamma.double().cpu().numpy(), 1e-5)
        gu = n @ self.w_gu.double().cpu().numpy().T
        g, u = gu[:, :self.F], gu[:, self.F:]
        full = (g / (1 + np.exp(-g)) * u) @ self.w_d.double().cpu().numpy().T
        return np.linalg.norm(y - full) / np.linalg.norm(full)


@pytest.mark.parametrize("M", [1, 5, 40, 200])
def test_mlp_block(M):
    C.log(f"mlp M={M}")
    mlp = Mlp(61, 512, 1152)
    x, _ = rows(62, M, 512, "f16", 5.0)
    stream, _ = rows(63, M, 512, "f16", 5.0)
    kept = stream.clone()
    out = mlp.run(x, stream)
    # three 8-bit roundings of tensors whose steps are about 4 sigma / 127: each about 1 % of its tensor
    assert mlp.check(x, kept, out) < 0.05
    assert torch.equal(stream, (x.float() + kept.float()).half())


@pytest.mark.parametrize("M", [3, 40, 150])
def test_mlp_block_captured_and_replayed(M):
    """Captured once, replayed with new inputs and eager work of another instance in between; the
    library allocates nothing, so a graph owns what its calls were given."""
    C.log(f"mlp graph M={M}")
    mlp = Mlp(64, 384, 1024)
    xin, _ = rows(65, M, 384, "f16", 5.0)
    stream, _ = rows(66, M, 384, "f16", 5.0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        mlp.run(xin, stream.clone())
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = mlp.run(xin, stream)
    for rep in range(4):
        x, _ = rows(70 + rep, M, 384, "f16", 5.0)
        st, _ = rows(80 + rep, M, 384, "f16", 5.0)
        want = mlp.run(x, st.clone())
        torch.cuda.synchronize()
        xin.copy_(x)
        stream.copy_(st)
        for t in out:
            t.zero_()
        g.replay()
        mlp.run(x, st.clone())  # the program's own work beside the replay
        torch.cuda.synchronize()
        for k, (a, b) in enumerate(zip(out, want)):
            assert torch.equal(a, b), (rep, k)
    del g


def test_two_streams_at_once():
    """Calls on two streams, each with its own outputs and workspace."""
    a = on_gpu(*operands(91, 200, 8960, 257))
    b = on_gpu(*operands(92, 33, 4096, 700))
    want = [rl.paro_w8a8_linear(*t, torch.float32) for t in (a, b)]
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(5):
        with torch.cuda.stream(s1):
            y1 = rl.paro_w8a8_linear(*a, torch.float32)
        with torch.cuda.stream(s2):
            y2 = rl.paro_w8a8_linear(*b, torch.float32)
        got.append((y1, y2))
    torch.cuda.synchronize()
    for y1, y2 in got:
        assert torch.equal(y1, want[0]) and torch.equal(y2, want[1])


def test_outputs_are_ordinary_tensors():
    """Outputs the calls make: torch's own kind, memory that torch counts and takes back, also in
    inference mode and for inputs whose memory torch has not allocated."""
    x = torch.randn(3, 256, device="cuda").half()
    like = torch.empty(3, 256, dtype=torch.int8, device="cuda")
    q, s = rl.paro_quantize_q8(x)
    assert q.device == like.device and q.stride() == like.stride() and not q.requires_grad
    assert torch._C._dispatch_keys(q) == torch._C._dispatch_keys(like)
    other = torch.from_dlpack(x)
    q2, s2 = rl.paro_quantize_q8(other)
    assert torch.equal(q, q2) and torch.equal(s, s2)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    kept = [rl.paro_quantize_q8(x) for _ in range(4)]
    assert torch.cuda.memory_allocated() == before + 4 * (1024 + 512)
    del kept
    assert torch.cuda.memory_allocated() == before
    with torch.inference_mode():
        qi, _ = rl.paro_quantize_q8(x)
        y = rl.paro_w8a8_linear(qi, s, like.zero_(), torch.ones(3, device="cuda"))
        assert qi.is_inference() and y.is_inference() and torch.equal(y, torch.zeros_like(y))
    assert torch.equal((q + 1) - 1, q)
