"""Numbers of the 8-bit path where they can go wrong, on the GPU: half-way values behind a transform.

Tolerances count roundings: U = 2^-24 is half a float32 step.
"""
import numpy as np
import pytest

from oracle import q8_oracle as Q
from tests import gpu_common as C

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")

U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def still(D, K):
    """A transform that moves nothing: K stages of angle 0 (c = 1, s = 0) and channel scales of 1."""
    r = np.random.default_rng([D, K])
    pairs = np.stack([r.permutation(D).reshape(D // 2, 2) for _ in range(K)]) if K else np.zeros((0, D // 2, 2))
    return rl.paro_rotation_prepare(pairs.astype(np.int32), np.zeros((K, D // 2), np.float32), np.ones(D, np.float32))


def half_way_rows(M, D, dt):
    """Rows with maximum 127 m 2^e and values m (2 k + 1) 2^(e - 1), half way between two codes."""
    ms = [1, 3, 5, 7, 9, 11, 13, 15] if dt == "f16" else [1]  # 127 m in the type's digits
    k = np.arange(D) % 256 - 128
    base = np.where(k == -128, 127.0, np.clip(k + 0.5, -126.5, 126.5))
    x = np.stack([base * ms[i % len(ms)] * 2.0 ** (i % 7 - 3) for i in range(M)])
    x = np.where(Q.round_to(x, dt) == x, x, 0.0)  # the halves that the type holds
    assert np.all(np.abs(x).max(axis=1) == 127.0 * np.array([ms[i % len(ms)] * 2.0 ** (i % 7 - 3) for i in range(M)]))
    return x


# one, two and four rows a workgroup; the widest four-row blocks, whose channel scales are read twice
@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("M,D,K", [(9, 256, 0), (40, 256, 2), (300, 384, 3), (530, 512, 0), (520, 4096, 1), (513, 8704, 0), (514, 9216, 2)])
def test_half_way_values_behind_a_transform_go_to_the_even_code(M, D, K, dt):
    """The codes of a row are the same whether it comes through a transform that moves nothing or not:
    rint of the exact quotient, ties to even."""
    C.log(f"half way behind a transform M={M} D={D} K={K} {dt}")
    x = half_way_rows(M, D, dt)
    real, scale = Q.quantize_exact(x)
    want = np.rint(real)
    t = torch.from_numpy(x).to(DT[dt]).cuda()
    q, s = rl.paro_quantize_q8(t, still(D, K))
    assert np.array_equal(q.cpu().numpy(), want)
    assert np.array_equal(s.double().cpu().numpy(), Q.round_to(scale, "f32"))
    p, ps = rl.paro_quantize_q8(t)
    assert torch.equal(p, q) and torch.equal(ps, s)


@pytest.mark.parametrize("with_residual", [True, False])
@pytest.mark.parametrize("M,D", [(7, 128), (6, 1536), (530, 4096), (1100, 6144), (700, 16384)])
def test_norm_of_bfloat16_rows_at_the_ends_of_the_range(M, D, with_residual):
    """n is an ordinary number where h * gamma is not: rows of large numbers under a large gamma, rows of
    small ones under a small gamma (eps decides their norm), rows whose 1 / sqrt is under 2^-126, and
    ordinary rows among them. A workgroup walks several rows in the larger calls."""
    C.log(f"norm range M={M} D={D} residual={with_residual}")
    r = np.random.default_rng([M, D])
    eps = 2.0 ** -126
    for power, g_power in ((124, 6), (-118, -24), (126, -10)):
        x = r.normal(0, 1, (M, D))
        if power == 126:
            x = np.sign(x) * r.uniform(0.8, 1.9, (M, D))  # rms above 2^126
        x[1::2] = np.ldexp(x[1::2], power)
        res = np.zeros((M, D)) if power == 126 else x[::-1][: M] * 0.25 if M % 2 else np.roll(x, 2, axis=0) * 0.25
        g = np.ldexp(r.normal(1, 0.3, D), g_power)
        x, res, g = (torch.from_numpy(v.astype(np.float32)).bfloat16() for v in (x, res, g))
        h64 = x.double().numpy()
        if with_residual:
            h64 = Q.round_to(Q.round_to(h64 + res.double().numpy(), "f32"), "bf16")
        assert np.isfinite(h64).all()
        n = Q.rmsnorm(h64, g.double().numpy(), eps)
        kw = {"residual": res.cuda()} if with_residual else {}
        y, h = rl.paro_rmsnorm(x.cuda(), g.cuda(), eps, **kw)
        q, s, h8 = rl.paro_rmsnorm_q8(x.cuda(), g.cuda(), eps, **kw)
        if with_residual:
            assert np.array_equal(h.double().cpu().numpy(), h64) and torch.equal(h, h8)
            stream = res.cuda()  # and the stream updated in place
            y2, h2 = rl.paro_rmsnorm(x.cuda(), g.cuda(), eps, residual=stream, residual_out=stream)
            assert torch.equal(y2, y) and torch.equal(h2, h)
        # the bounds of the ordinary rows: three float32 roundings and the type's own, the scale's division,
        # the codes' step and product
        assert C.over_bound(y.double().cpu().numpy() - n, np.abs(n) * (4 * U + 2.0 ** -8) + 2.0 ** -134) <= 1, power
        real, want = Q.quantize_exact(n)
        assert C.over_bound(s.double().cpu().numpy() - want, want * 5 * U) <= 1, power
        assert np.abs(q.cpu().numpy() - real).max() <= 0.5 + 127 * 6 * U, power


def exact_gates(seed, M, D, F):
    """Codes and scales (powers of two) whose gates and ups are exact in float32: sums under 2^24 over a
    power of two, gates from a fraction to about +-100, so that nothing but the activation rounds."""
    r = np.random.default_rng([seed, M, D, F])
    xq = r.integers(-127, 128, (M, D)).astype(np.int8)
    wq = r.integers(-127, 128, (2 * F, D)).astype(np.int8)
    xs = np.ldexp(1.0, r.integers(-3, 3, M)).astype(np.float32)
    spread = int(np.rint(np.log2(73.0 * 73.0 * np.sqrt(D))))  # a sum's standard deviation, about
    ws = np.ldexp(1.0, r.integers(1, 6, 2 * F) - spread).astype(np.float32)
    return xq, xs, wq, ws


# streamed, by columns, tiled, and tiled with a split reduction
@pytest.mark.parametrize("M,D,F", [(1, 128, 600), (2, 256, 129), (8, 256, 300), (40, 1152, 200), (64, 128, 33), (130, 640, 515), (200, 8960, 65),
                                   (700, 512, 1030)])
def test_silu_in_float32(M, D, F):
    """A float32 output of the gated linear carries the activation to float32, whatever the gate. With exact
    g and u, in units of U: exp(-|g|) 2 (one float32 step), for a negative gate its product with g 1; 1 + exp
    1 and at most 1 of exp's own; the quotient 1; the product with u 1: 7, 2 % more for their products.
    Under 2^-126 exp(-|g|) is off by the last digit there, 2^-149, and the products and the quotient by half
    of one each."""
    C.log(f"silu f32 M={M} D={D} F={F}")
    xq, xs, wq, ws = exact_gates(71, M, D, F)
    v, g, u = Q.gated(xq, xs, wq, ws)
    assert np.array_equal(g, g.astype(np.float32)) and np.array_equal(u, u.astype(np.float32))
    if M * F > 20000:
        assert g.min() < -95 and g.max() > 95 and np.abs(g).min() < 0.01
    y = rl.paro_w8a8_gated_linear(*(torch.from_numpy(a).cuda() for a in (xq, xs, wq, ws)), torch.float32).double().cpu().numpy()
    assert C.over_bound(y - v, 7.15 * U * np.abs(v) + 2.0 ** -149 * (np.abs(g * u) + np.abs(u) + 1)) <= 1
