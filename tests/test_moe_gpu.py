"""The mixture-of-experts calls on the GPU against their float64 oracle: the router with its ties and odd rows, the
experts over token counts, ids and sizes, the layer as a whole, and a decoder block's run of all of it.
"""
import ctypes

import numpy as np
import pytest

import oracle as O
import workloads as W
from oracle import block_oracle as B
from tests import gpu_common as C
from tests.test_w8a8_gpu import U, guarded, over

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")


def pack(r, E, N, D):
    """Random packed experts: the library's operands and the dequantized weights [E][N][D]."""
    q = np.clip(np.rint(r.normal(7.5, 2.7, (E * N, D))), 0, 15).astype(np.uint8)
    sc = (r.uniform(0.7, 1.3, (E * N, D // 128)) / (2.7 * np.sqrt(D))).astype(np.float16)
    z = r.integers(5, 11, (E * N, D // 128)).astype(np.float16)
    w = (q.reshape(E * N, D // 128, 128) - z[..., None].astype(np.float64)) * sc[..., None].astype(np.float64)
    qw = W.qweight_to_blocked(q[:, 0::2] | (q[:, 1::2] << 4))
    ops = tuple(torch.from_numpy(np.ascontiguousarray(t)).cuda().view(E, N, -1) for t in (qw, sc, z))
    return ops, w.reshape(E, N, D)


def tokens(r, M, D):
    x = r.normal(0, 1, (M, D)).astype(np.float16)
    return torch.from_numpy(x).cuda(), x.astype(np.float64)


def choose(r, M, E, k, holes=0.0):
    ids = np.argsort(r.random((M, E)), axis=1)[:, :k].astype(np.int32)
    ids[r.random((M, k)) < holes] = -1
    w = r.uniform(0, 1, (M, k)).astype(np.float32)
    return ids, w


def check(y, want, bound, half):
    got = y.double().cpu().numpy()
    assert over(got - want, bound + half * (np.abs(want) + bound) + (2.0 ** -25 if half > U else 0)) <= 1
    if np.linalg.norm(want) > 0:
        assert np.linalg.norm(got - want) <= C.REL_L2 * np.linalg.norm(want)


SIZES = [  # M, D, F, E, top_k
    (1, 128, 128, 1, 1), (1, 2048, 1024, 64, 8), (2, 256, 384, 4, 2), (3, 1152, 128, 7, 3), (5, 128, 2176, 5, 5), (13, 640, 256, 60, 4),
    (16, 512, 512, 3, 2), (17, 256, 128, 2, 1), (33, 384, 640, 4, 3), (48, 256, 256, 512, 16), (64, 256, 384, 16, 8), (64, 128, 128, 1, 1),
    (64, 1024, 128, 2, 2), (7, 4096, 1408, 9, 2), (4, 256, 14336, 3, 2), (4, 16384, 256, 3, 2), (31, 768, 896, 40, 6),
    (3, 2560, 256, 5, 2), (9, 5120, 256, 3, 2), (5, 8192, 128, 3, 1), (40, 10368, 128, 3, 2), (64, 768, 1408, 24, 6), (50, 2048, 640, 30, 4)]


def down_plan(*size):
    """(16-column tiles of a workgroup, workgroups that share them) of the down product."""
    out = [ctypes.c_int() for _ in range(2)]
    rl.lib().paro_internal_moe_down_plan(*size, *map(ctypes.byref, out))
    return tuple(v.value for v in out)


def test_the_sizes_reach_every_kernel():
    plans = {down_plan(*s) for s in SIZES}
    assert {t for t, s in plans if s == 1} >= {1, 4} and {t for t, s in plans if s > 1} == {1, 2, 4}
    # the gate and up product: four, eight or sixteen waves by the groups of channels, one to four of them to a wave, or any number
    assert {min(65, D // 128) for _, D, _, _, _ in SIZES} >= {1, 2, 4, 5, 6, 8, 9, 16, 20, 32, 40, 64, 65}


@pytest.mark.parametrize("M,D,F,E,k", SIZES)
def test_experts(M, D, F, E, k):
    C.log(f"experts M={M} D={D} F={F} E={E} k={k}")
    r = np.random.default_rng([M, D, F, E, k])
    gu, gw = pack(r, E, 2 * F, D)
    dn, dw = pack(r, E, D, F)
    x, x64 = tokens(r, M, D)
    for holes in (0.0, 0.5):
        ids, w = choose(r, M, E, k, holes)
        want, bound = B.experts(x64, ids, w.astype(np.float64), gw, dw)
        di, dwt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
        ws = torch.full((rl.paro_moe_workspace_bytes(M, D, F, E, k),), 255, dtype=torch.uint8, device="cuda")
        outs = []
        for t, half in ((torch.float32, U), (torch.float16, 2.0 ** -11)):
            y, ok = guarded((M, D), t)
            rl.paro_moe_w4a16(x, di, dwt, gu, dn, out=y, ws=ws)
            assert ok()
            check(y, want, bound, half)
            outs.append(y)
        assert torch.equal(outs[0].half(), outs[1])
        # a token in a call of its own: the sums may be taken in another order, the bound is the same
        for m in {0, M // 2, M - 1}:
            one = rl.paro_moe_w4a16(x[m:m + 1].clone(), di[m:m + 1].clone(), dwt[m:m + 1].clone(), gu, dn, out_dtype=torch.float32)
            check(one, want[m:m + 1], bound[m:m + 1], U)
        assert not outs[0][torch.from_numpy((ids < 0).all(1)).cuda()].any()


def test_ids_of_every_kind():
    """All tokens at one expert, ids out of range, the same expert twice, more ids than experts, no expert at all."""
    r = np.random.default_rng(5)
    M, D, F, E = 64, 256, 256, 5
    gu, gw = pack(r, E, 2 * F, D)
    dn, dw = pack(r, E, D, F)
    x, x64 = tokens(r, M, D)
    for k, make in ((1, lambda: np.full((M, 1), 3)), (3, lambda: r.integers(-2, E + 3, (M, 3))), (2, lambda: np.full((M, 2), 4)),
                    (16, lambda: r.integers(0, E, (M, 16))), (4, lambda: np.full((M, 4), -1)),
                    (2, lambda: np.full((M, 2), [2 ** 31 - 1, -2 ** 31]))):
        ids = make().astype(np.int32)
        w = r.uniform(0, 1, (M, k)).astype(np.float32)
        w[(ids < 0) | (ids >= E)] = np.nan  # not read into the sum
        want, bound = B.experts(x64, ids, w.astype(np.float64), gw, dw)
        bound = bound + 16 * U * np.abs(want)  # the weights of an expert named twice are added first
        y = rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, out_dtype=torch.float32)
        check(y, want, bound, U)
        assert k != 4 or not y.any()


def test_odd_rows_stay_in_their_rows():
    """NaN, infinities and a NaN weight reach their own token only; an expert that no token names is not read."""
    r = np.random.default_rng(6)
    M, D, F, E, k = 20, 384, 256, 6, 2
    gu, _ = pack(r, E, 2 * F, D)
    dn, _ = pack(r, E, D, F)
    x, _ = tokens(r, M, D)
    ids, w = choose(r, M, E - 1, k)
    di, dwt = torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda()
    clean = rl.paro_moe_w4a16(x, di, dwt, gu, dn)
    for t in (gu, dn):
        t[1][E - 1] = float("nan")
        t[2][E - 1] = float("inf")
    x[3, 5] = float("nan")
    x[11, 383] = float("inf")
    dwt[17, 1] = float("nan")
    y = rl.paro_moe_w4a16(x, di, dwt, gu, dn)
    rest = [m for m in range(M) if m not in (3, 11, 17)]
    assert torch.equal(y[rest], clean[rest])
    assert bool(y[[3, 17]].isnan().all()) and not bool(y[11].isfinite().any())


@pytest.mark.parametrize("M,D,F,E,k,K", [(1, 256, 128, 4, 2, 2), (13, 1536, 1408, 6, 2, 8), (64, 384, 256, 5, 3, 8), (6, 4224, 128, 3, 1, 3),
                                         (64, 256, 640, 6, 5, 2), (60, 256, 1408, 6, 5, 2), (64, 128, 2176, 6, 5, 1)])
def test_rotated_experts(M, D, F, E, k, K):
    """Experts packed with a transform for x and one for the rows between the products, against the unquantized layer's
    own packing: the oracle's transforms in float64, a rounded to float16 behind its own."""
    C.log(f"rotated experts M={M} D={D} F={F} E={E} k={k} K={K}")
    r = np.random.default_rng([M, D, F, E, k, K])
    Lx, La = W.custom_linear(51, 1, D, 16, K), W.custom_linear(52, 1, F, 16, K)
    rot_x, rot_a = (rl.paro_rotation_prepare(L.pairs, L.theta, L.scale) for L in (Lx, La))

    def packed(rot, N, C_):
        w = torch.from_numpy((r.normal(0, 1, (E * N, C_)) / np.sqrt(C_)).astype(np.float16)).cuda()
        q, s, z = rl.paro_pack_weights(rot, w)
        host = C.host_weights((q, s, z))
        return (q.view(E, N, -1), s.view(E, N, -1), z.view(E, N, -1)), O.dequantize(*host).reshape(E, N, C_)

    gu, gw = packed(rot_x, 2 * F, D)
    dn, dw = packed(rot_a, D, F)
    x, x64 = tokens(r, M, D)
    ids, w = choose(r, M, E, k, 0.2)
    xt = O.transform_activations(x64.astype(np.float16), Lx.pairs, Lx.theta, Lx.scale)

    def between(a):
        return C.f16_of(O.transform_activations(a, La.pairs, La.theta, La.scale))

    want, _ = B.experts(xt, ids, w.astype(np.float64), gw, dw, between)
    y, ok = guarded((M, D), torch.float32)
    rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, rot_x, rot_a, out=y)
    assert ok()
    got = y.double().cpu().numpy()
    # the library's bar for rotated products
    assert np.abs(got - want).max() <= C.MAX_ABS and np.linalg.norm(got - want) <= C.REL_L2 * np.linalg.norm(want)
    # x' keeps float32's digits, and the oracle rounds a as the library does: a row's float32 error, (K + 2) 4 U of its
    # norm, some 40 times an element at these widths, is under a quarter of a float16 step, so at most a quarter of a is
    # a step off, sqrt(1/4) 2^-11 of it (rows of paro_rotate would leave more: every element of x' half a step at most).
    # Where an expert has up to 8 tokens the library keeps what a's rounding takes away, and the oracle's rounding is the
    # difference: a step of 2^-10 over a mantissa m between 1 and 2, 1 / sqrt(12) of it in the mean of squares, and 1 / m^2
    # is 3 / (8 ln 2) in the mean: 0.212 * 2^-10, under 2^-12
    assert np.linalg.norm(got - want) <= 2.0 ** -12 * np.linalg.norm(want)


LARGE = [  # M, D, F, E, top_k, K
    (64, 4096, 1408, 64, 8, 0), (8, 512, 16384, 8, 4, 0), (8, 1024, 8192, 8, 4, 0), (8, 1536, 8192, 8, 4, 0), (8, 2048, 4096, 8, 4, 0),
    (8, 2560, 2048, 16, 4, 0), (8, 5120, 2048, 8, 4, 0), (8, 8192, 1024, 8, 4, 0), (2, 16384, 1024, 4, 2, 0), (8, 512, 16384, 8, 4, 2),
    (8, 1024, 8192, 8, 4, 2), (8, 1536, 8192, 8, 4, 2), (8, 4096, 2048, 8, 4, 2), (2, 16384, 1024, 4, 2, 2)]


@pytest.mark.parametrize("M,D,F,E,k,K", LARGE)
def test_large_experts(M, D, F, E, k, K):
    """Experts of tens of megabytes, whose weights go past the caches, against the formulas in float64 on the GPU."""
    C.log(f"large experts M={M} D={D} F={F} E={E} k={k} K={K}")
    r = np.random.default_rng([M, D, F, E, k, K])
    torch.manual_seed(M + D + F)

    def packed(N, n):
        q = torch.randint(0, 256, (E, N, n // 2), dtype=torch.uint8, device="cuda")
        sc = ((torch.rand(E, N, n // 128, device="cuda") * 0.6 + 0.7) / (4.6 * n ** 0.5)).half()
        return q, sc, torch.randint(5, 11, (E, N, n // 128), device="cuda").half()

    def expert(p, e):
        q, sc, z = (t[e] for t in p)
        N, half = q.shape
        q = q.view(N // 16, half // 64, 16, 64).transpose(1, 2).reshape(N, half)
        q = torch.stack([q & 15, q >> 4], -1).view(N, half // 64, 128).double()
        return ((q - z.double()[..., None]) * sc.double()[..., None]).view(N, 2 * half)

    gu, dn = packed(2 * F, D), packed(D, F)
    x, x64 = tokens(r, M, D)
    ids, w = choose(r, M, E, k)
    rots = None, None
    if K:
        Lx, La = W.custom_linear(51, 1, D, 16, K), W.custom_linear(52, 1, F, 16, K)
        rots = [rl.paro_rotation_prepare(L.pairs, L.theta, L.scale) for L in (Lx, La)]
        x64 = O.transform_activations(x64.astype(np.float16), Lx.pairs, Lx.theta, Lx.scale)
    xd = torch.from_numpy(np.asarray(x64, np.float64)).cuda()
    want, bound = (torch.zeros(M, D, dtype=torch.float64, device="cuda") for _ in range(2))
    for e in range(E):
        at = np.nonzero((ids == e).any(axis=1))[0]
        if not len(at):
            continue
        we = torch.from_numpy(np.where(ids[at] == e, w[at], 0).sum(axis=1).astype(np.float64)).cuda()[:, None]
        g, d, xe = expert(gu, e), expert(dn, e), xd[at]
        p, off = xe @ g.T, (140 + D // 128) * U * (xe.abs() @ g.abs().T)
        a = p[:, :F] * torch.sigmoid(p[:, :F]) * p[:, F:]
        # block_oracle.experts derives the bound
        gate, up, og, ou = p[:, :F].abs(), p[:, F:].abs(), off[:, :F], off[:, F:]
        da = 1.1 * up * og + gate * ou + 1.1 * og * ou + (4 + gate) * U * a.abs()
        da = da + (2.0 ** -11 * (a.abs() + da)).clamp(min=2.0 ** -25)
        if K:
            a = torch.from_numpy(np.asarray(O.transform_activations(a.cpu().numpy(), La.pairs, La.theta, La.scale), np.float64)).cuda()
        want[at] += we * (a @ d.T)
        bound[at] += we * (da @ d.abs().T + (160 + k + F // 128) * U * ((a.abs() + da) @ d.abs().T))
    y, ok = guarded((M, D), torch.float32)
    rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, *rots, out=y)
    assert ok()
    if K:
        # a is off by half a float16 step of each value, 2^-11 of it at most and 2^-11 / sqrt(3) in the mean of squares; the
        # sums turn that into as much of y, with float32's errors far below
        assert float((y.double() - want).norm()) <= 2.0 ** -11 * float(want.norm())
    else:
        check(y, want.cpu().numpy(), bound.cpu().numpy(), U)


ROUTES = [(1, 128, 1, 1), (1, 2048, 64, 8), (3, 256, 5, 5), (64, 4096, 128, 8), (17, 384, 60, 4), (64, 128, 512, 16), (33, 16384, 3, 2),
          (2, 1536, 257, 16)]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("M,D,E,k", ROUTES)
def test_route(M, D, E, k, scoring):
    C.log(f"route M={M} D={D} E={E} k={k} {scoring}")
    r = np.random.default_rng([M, D, E, k])
    x, x64 = tokens(r, M, D)
    router = (r.normal(0, 1.5, (E, D)) / np.sqrt(D)).astype(np.float32)
    for dt in (np.float32, np.float16):
        rt = router.astype(dt)
        for renorm in (True, False):
            want, w64 = B.route(x64, rt.astype(np.float64), k, scoring == "sigmoid", renorm)
            (ids, iok), (w, wok) = guarded((M, k), torch.int32), guarded((M, k), torch.float32)
            ws = torch.full((rl.paro_moe_route_workspace_bytes(M, E),), 255, dtype=torch.uint8, device="cuda")
            rl.paro_moe_route(x, torch.from_numpy(rt).cuda(), k, scoring, renorm, out=(ids, w), ws=ws)
            assert iok() and wok()
            assert np.array_equal(ids.cpu().numpy(), want)
            # float64 throughout, one rounding to float32
            assert over(w.double().cpu().numpy() - w64, w64 * U * 1.0001) <= 1


def test_route_ties_and_odd_rows():
    """Equal logits go by index; a NaN ranks last; an infinite logit has all the softmax, two make it NaN."""
    D, E, k = 256, 40, 6
    r = np.random.default_rng(9)
    x, x64 = tokens(r, 6, D)
    base = (r.normal(0, 1, (8, D)) / 16).astype(np.float16)
    router = base[r.integers(0, 8, E)]  # many equal rows
    ids, w = rl.paro_moe_route(x, torch.from_numpy(router).cuda(), k)
    want, w64 = B.route(x64, router.astype(np.float64), k)
    assert np.array_equal(ids.cpu().numpy(), want) and over(w.double().cpu().numpy() - w64, w64 * U * 1.0001) <= 1
    x[1] = 0  # all logits equal
    x[2, 3] = float("nan")
    x[4, 7] = float("inf")
    ids, w = rl.paro_moe_route(x, torch.from_numpy(router).cuda(), k)
    assert ids[1].tolist() == list(range(k)) and w[1].tolist() == [float(np.float32(1 / 6))] * k
    assert ids[2].tolist() == list(range(k)) and bool(w[2].isnan().all())
    ids = ids.cpu().numpy()
    assert np.array_equal(ids[[0, 3, 5]], want[[0, 3, 5]])
    assert len(set(ids[4])) == k and (0 <= ids[4]).all() and (ids[4] < E).all()
    # one expert's row is NaN: it is never taken while others are left, and takes the softmax with it
    bad = torch.from_numpy(router).cuda()
    bad[11] = float("nan")
    for scoring in ("softmax", "sigmoid"):
        ids, w = rl.paro_moe_route(x[:1], bad, E if E <= 16 else 16, scoring)
        assert 11 not in ids[0].tolist() and bool(w.isnan().all()) == (scoring == "softmax")
    small = torch.from_numpy(router[:3].copy()).cuda()
    small[0] = float("nan")
    ids, w = rl.paro_moe_route(x[:1], small, 3, "sigmoid", False)
    assert ids[0].tolist()[2] == 0 and bool(w[0, 2].isnan()) and bool(w[0, :2].isfinite().all())


@pytest.mark.parametrize("M,E,k", [(1, 2, 2), (3, 61, 16), (25, 40, 7), (64, 15, 15), (64, 300, 9)])
def test_route_close_logits(M, E, k):
    """Logits a float32's last digit apart, of either sign, some of them equal."""
    D = 128
    r = np.random.default_rng([M, E, k])
    x = np.zeros((M, D), np.float16)
    x[:, 0] = r.choice([1, -1, 0.5, -0.25], M)
    router = np.zeros((E, D), np.float32)
    router[:, 0] = 1 + r.integers(0, 2 * E, E) * 2.0 ** -23
    want, w64 = B.route(x.astype(np.float64), router.astype(np.float64), k)
    ids, w = rl.paro_moe_route(torch.from_numpy(x).cuda(), torch.from_numpy(router).cuda(), k)
    assert np.array_equal(ids.cpu().numpy(), want) and over(w.double().cpu().numpy() - w64, w64 * U * 1.0001) <= 1


@pytest.mark.parametrize("M,E,k,rotated", [(1, 64, 8, False), (4, 8, 2, True), (64, 24, 3, False), (23, 7, 7, True)])
def test_layer_is_its_parts(M, E, k, rotated):
    D, F = 512, 384
    r = np.random.default_rng([M, E, k])
    gu, _ = pack(r, E, 2 * F, D)
    dn, _ = pack(r, E, D, F)
    x, _ = tokens(r, M, D)
    router = torch.from_numpy((r.normal(0, 1, (E, D)) / 16).astype(np.float16)).cuda()
    rots = {}
    if rotated:
        for name, n in (("rot_x", D), ("rot_a", F)):
            L = W.custom_linear(61, 1, n, 16, 4)
            rots[name] = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
    (y, yok), (ids, iok), (w, wok) = guarded((M, D), torch.float16), guarded((M, k), torch.int32), guarded((M, k), torch.float32)
    rl.paro_moe_layer_w4a16(x, router, k, gu, dn, out=y, routing=(ids, w), **rots)
    assert yok() and iok() and wok()
    i2, w2 = rl.paro_moe_route(x, router, k)
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    assert torch.equal(y, rl.paro_moe_w4a16(x, i2, w2, gu, dn, **rots))


def test_without_the_compiled_binding(monkeypatch):
    """The calls' own checks and ctypes, as where the binding declines."""
    r = np.random.default_rng(5)
    M, D, F, E, k = 6, 256, 128, 5, 2
    gu, _ = pack(r, E, 2 * F, D)
    dn, _ = pack(r, E, D, F)
    x, _ = tokens(r, M, D)
    h, _ = tokens(r, M, D)
    router = torch.from_numpy((r.normal(0, 1, (E, D)) / 16).astype(np.float16)).cuda()
    g, bias = (torch.from_numpy(r.normal(1, 0.1, n).astype(np.float16)).cuda() for n in (D, 2 * F))
    wq, ws = rl.paro_pack_weights_q8(torch.from_numpy(r.normal(0, 1, (2 * F, D)).astype(np.float16)).cuda())

    def run():
        q, s, n8 = rl.paro_block_norm_q8(x, h, g, post_gamma=g, gate=g, residual_scale=0.5)
        res = torch.full((M, 2 * F), 0.25, dtype=torch.float16, device="cuda")
        rl.paro_w8a8_linear_epilogue(q, s, wq, ws, bias=bias, activation="gelu", residual=res, out=res)
        layer = rl.paro_moe_layer_w4a16(x, router, k, gu, dn)
        ids, w = rl.paro_moe_route(x, router, k, "sigmoid")
        return (q, s, n8, res, *layer, ids, w, *rl.paro_block_norm(x, h, g), rl.paro_moe_w4a16(x, ids, w, gu, dn, out_dtype=torch.float32))

    want = run()

    class Declines:
        linear_epilogue = block_norm = route = moe = staticmethod(lambda *a: None)

    monkeypatch.setattr(rl.block, "_binding", Declines)
    assert all(torch.equal(a, b) for a, b in zip(run(), want, strict=True))


class Block:
    """One decoder block's products, served: norms on both sides, a projection with bias, one that ends in the stream,
    and a mixture of experts; attention, which is not the library's, is left out."""

    def __init__(self, D=512, F=384, E=12, k=3):
        r = np.random.default_rng(71)
        self.D, self.k = D, k

        def half(*s, mean=0.0, spread=1.0):
            return torch.from_numpy(r.normal(mean, spread, s).astype(np.float16)).cuda()

        self.v = rl.paro_pack_weights_q8(half(D, D, spread=D ** -0.5))
        self.o = rl.paro_pack_weights_q8(half(D, D, spread=D ** -0.5))
        self.bias, self.router = half(D, spread=0.2), half(E, D, spread=D ** -0.5)
        self.g1, self.g2, self.g3, self.post = (half(D, mean=1, spread=0.1) for _ in range(4))
        self.gate = half(D, mean=0.8, spread=0.1)
        L = W.custom_linear(72, 1, D, 16, 4)
        self.rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
        one = rl.paro_rotation_prepare(np.zeros((0, F // 2, 2), np.int32), np.zeros((0, F // 2), np.float32), np.ones(F, np.float32))
        q = rl.paro_pack_weights(self.rot, half(E * 2 * F, D, spread=D ** -0.5))
        self.gu = tuple(t.view(E, 2 * F, -1) for t in q)
        q = rl.paro_pack_weights(one, half(E * D, F, spread=F ** -0.5))
        self.dn = tuple(t.view(E, D, -1) for t in q)

    def run(self, x, stream):
        xq, xs, h = rl.paro_rmsnorm_q8(x, self.g1, 1e-6, residual=stream)
        v = rl.paro_w8a8_linear_epilogue(xq, xs, *self.v, bias=self.bias, activation="gelu", out_dtype=torch.float16)
        vq, vs = rl.paro_quantize_q8(v)
        h = rl.paro_w8a8_linear_epilogue(vq, vs, *self.o, residual=h, out=h)
        n, _ = rl.paro_rmsnorm(h, self.g2, 1e-6)
        y, ids, w = rl.paro_moe_layer_w4a16(n, self.router, self.k, self.gu, self.dn, rot_x=self.rot)
        q, s, h2 = rl.paro_block_norm_q8(y, h, self.g3, 1e-6, post_gamma=self.post, gate=self.gate)
        return v, h, y, ids, w, q, s, h2


@pytest.mark.parametrize("M", [1, 9, 64])
def test_a_block_captured_and_replayed(M):
    """The run as a graph, with other inputs each time, beside the program's own eager runs."""
    b = Block()
    g = torch.Generator(device="cuda").manual_seed(M)

    def new():
        return torch.randn(M, b.D, generator=g, device="cuda").half()

    x, stream = new(), new()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.run(x, stream)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = b.run(x, stream)
    for rep in range(4):
        nx, ns = new(), new()
        want = b.run(nx, ns)
        torch.cuda.synchronize()
        x.copy_(nx)
        stream.copy_(ns)
        for t in out:
            t.zero_()
        graph.replay()
        b.run(new(), new())
        torch.cuda.synchronize()
        for i, (a, c) in enumerate(zip(out, want)):
            assert torch.equal(a, c), (rep, i)
            assert not a.is_floating_point() or bool(a.isfinite().all())
    del graph


def test_two_streams_at_once():
    b = Block()
    g = torch.Generator(device="cuda").manual_seed(1)
    ins = [(torch.randn(M, b.D, generator=g, device="cuda").half(), torch.randn(M, b.D, generator=g, device="cuda").half()) for M in (3, 40)]
    want = [b.run(*i) for i in ins]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ins]
    got = []
    for _ in range(4):
        for i, s in zip(ins, streams):
            with torch.cuda.stream(s):
                got.append(b.run(*i))
    torch.cuda.synchronize()
    for n, out in enumerate(got):
        for a, c in zip(out, want[n % 2]):
            assert torch.equal(a, c), n
