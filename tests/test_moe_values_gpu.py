"""What the experts hold between their products, seen in a float32 y against float64 oracles that round nothing."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from oracle import block_oracle as B
from tests import gpu_common as C
from tests.test_moe_gpu import choose, pack, test_large_experts as large_experts, tokens

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")

# Rows in two float16 parts are off by 2^-22 of a value, an element of a float32 sum of n <= 384 products by some
# sqrt(n / 2) U < 2^-20 of the sum's own spread, in each of the three products that y goes through: some 2^-19 together.
# One float16 part is off by 2^-11 / sqrt(12) / (a mantissa's mean square) of a, and so of y: 2^-12.2, and 2^-13 where
# only half the units lose theirs.
EXACT = 2.0 ** -16


def relative(y, want):
    return np.linalg.norm(y.double().cpu().numpy() - want) / np.linalg.norm(want)


@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (8, 1, 1), (8, 6, 2), (9, 1, 1), (9, 6, 2), (16, 1, 1), (17, 2, 1), (29, 4, 2), (64, 1, 1), (64, 12, 3),
                                   (64, 60, 4)])
@pytest.mark.parametrize("K", [0, 2])
def test_digits_of_the_rows_between_the_products(M, E, k, K):
    """Whatever the number of tokens that share an expert."""
    D, F = 256, 384
    C.log(f"digits M={M} E={E} k={k} K={K}")
    r = np.random.default_rng([M, E, k, K])
    gu, gw = pack(r, E, 2 * F, D)
    dn, dw = pack(r, E, D, F)
    x, x64 = tokens(r, M, D)
    ids, w = choose(r, M, E, k)
    rots, between = (None, None), None
    if K:
        Lx, La = W.custom_linear(51, 1, D, 16, K), W.custom_linear(52, 1, F, 16, K)
        rots = [rl.paro_rotation_prepare(L.pairs, L.theta, L.scale) for L in (Lx, La)]
        x64 = O.transform_activations(x64.astype(np.float16), Lx.pairs, Lx.theta, Lx.scale)

        def between(a):
            return O.transform_activations(a, La.pairs, La.theta, La.scale)

    want, _ = B.experts(np.asarray(x64, np.float64), ids, w.astype(np.float64), gw, dw, between)
    y = rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, *rots, out_dtype=torch.float32)
    assert relative(y, want) <= EXACT


@pytest.mark.parametrize("M,E,k", [(1, 2, 2), (8, 3, 2), (40, 3, 2)])
@pytest.mark.parametrize("K", [0, 2])
def test_rows_of_every_scale(M, E, k, K):
    """Rows from 2^-14 to 2^13 side by side, so that the rows between the products run from 2^-30 to 2^27: each
    keeps its digits."""
    D, F = 256, 384
    C.log(f"scales M={M} E={E} k={k} K={K}")
    r = np.random.default_rng([M, E, k, K, 1])
    gu, gw = pack(r, E, 2 * F, D)
    dn, dw = pack(r, E, D, F)
    rots, between = (None, None), None
    if K:
        Lx, La = W.custom_linear(51, 1, D, 16, K), W.custom_linear(52, 1, F, 16, K)
        rots = [rl.paro_rotation_prepare(L.pairs, L.theta, L.scale) for L in (Lx, La)]

        def between(a):
            return O.transform_activations(a, La.pairs, La.theta, La.scale)

    ids, w = choose(r, M, E, k)
    for powers in ([-14], [-8], [8], [13], [-14, -3, 13, 6]):
        x64 = r.normal(0, 1, (M, D)).clip(-3.9, 3.9) * np.exp2(np.resize(powers, M))[:, None]
        x64[0, 7] = 3.9 * 2.0 ** powers[0]
        x = torch.from_numpy(x64.astype(np.float16)).cuda()
        x64 = x.cpu().numpy().astype(np.float64)
        assert np.isfinite(x64).all()
        if K:
            x64 = np.asarray(O.transform_activations(x64.astype(np.float16), Lx.pairs, Lx.theta, Lx.scale), np.float64)
        want, _ = B.experts(x64, ids, w.astype(np.float64), gw, dw, between)
        y = rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, *rots, out_dtype=torch.float32)
        for m in range(M):
            assert relative(y[m], want[m]) <= EXACT, (powers, m)


def test_transformed_rows_past_the_range_of_float16():
    D, F, E = 256, 384, 2
    r = np.random.default_rng(12)
    gu, gw = pack(r, E, 2 * F, D)
    dn, dw = pack(r, E, D, F)
    L = W.custom_linear(51, 1, D, 16, 2)
    rot = rl.paro_rotation_prepare(L.pairs, L.theta, L.scale)
    v = r.normal(0, 1, (3, D))
    v[1, np.argmin(L.scale)] = 2.0 ** 17
    x = O.untransform_activations(v, L.pairs, L.theta, L.scale).astype(np.float16)
    x64 = np.asarray(O.transform_activations(x, L.pairs, L.theta, L.scale), np.float64)
    assert np.isfinite(x).all() and np.abs(x64).max() > 65504
    ids, w = choose(r, 3, E, 2)
    want, _ = B.experts(x64, ids, w.astype(np.float64), gw, dw)
    y = rl.paro_moe_w4a16(torch.from_numpy(x).cuda(), torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, rot, out_dtype=torch.float32)
    for m in range(3):
        assert relative(y[m], want[m]) <= EXACT


def test_rows_of_zeros():
    r = np.random.default_rng(8)
    M, D, F, E = 12, 256, 384, 2
    gu, _ = pack(r, E, 2 * F, D)
    dn, _ = pack(r, E, D, F)
    x, _ = tokens(r, M, D)
    ids, w = choose(r, M, E, 1)
    x[5] = 0
    y = rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn)
    assert not y[5].any() and bool((y[[m for m in range(M) if m != 5]] != 0).any(1).all())


MORE = [(7, 4096, 256, 9, 2), (8, 4096, 8192, 8, 8)]  # M, D, F, E, top_k: kernels that no other test's sizes reach


@pytest.mark.parametrize("M,D,F,E,k", MORE)
def test_more_sizes(M, D, F, E, k):
    large_experts(M, D, F, E, k, 0)


# A transform's kernel is one of nine by the row's width, each for widths that its threads divide and for others.
WIDTHS = [640, 1024, 1152, 2048, 2176, 3200, 4096, 4224, 6144, 6272, 10240, 10368, 12288, 12416, 14336, 14464, 16384]


def transformed(seed, width, K):
    """(the library's transform, the oracle's function)"""
    r = np.random.default_rng([seed, width, K])
    pairs = np.stack([r.permutation(width).reshape(-1, 2) for _ in range(K)]).astype(np.int32) if K else np.zeros((0, width // 2, 2), np.int32)
    theta = r.uniform(-np.pi, np.pi, (K, width // 2)).astype(np.float32)
    scale = np.exp(r.normal(0, 0.3, width)).astype(np.float32)
    return rl.paro_rotation_prepare(pairs, theta, scale), lambda v: np.asarray(O.transform_activations(v, pairs, theta, scale), np.float64)


def experts_against_the_oracle(seed, M, D, F, E, k, K_x, K_a):
    """K_x, K_a: stages of the transforms, None for no transform."""
    r = np.random.default_rng([seed, M, D, F, E, k])
    gu, gw = pack(r, E, 2 * F, D)
    dn, dw = pack(r, E, D, F)
    x, x64 = tokens(r, M, D)
    rot_x, turn_x = (None, lambda v: v) if K_x is None else transformed(1, D, K_x)
    rot_a, turn_a = (None, None) if K_a is None else transformed(2, F, K_a)
    ids, w = choose(r, M, E, k)
    want, _ = B.experts(turn_x(x64), ids, w.astype(np.float64), gw, dw, turn_a)
    y = rl.paro_moe_w4a16(x, torch.from_numpy(ids).cuda(), torch.from_numpy(w).cuda(), gu, dn, rot_x, rot_a, out_dtype=torch.float32)
    # (sums of more products are sums of sums: of 128 in a group, of the groups of a wave, of up to 16 waves; a stage of a
    # transform costs some U of an element. EXACT leaves room for both)
    assert relative(y, want) <= EXACT


@pytest.mark.parametrize("K", [0, 1, 3])
@pytest.mark.parametrize("width", WIDTHS)
def test_transforms_of_every_width(width, K):
    C.log(f"transforms of {width}, K={K}")
    experts_against_the_oracle(21, 3, width, 128, 2, 1, K, None)
    experts_against_the_oracle(22, 3, 128, width, 2, 1, None, K)


@pytest.mark.parametrize("width", [640, 1024, 1152, 2048, 2176, 4096])
def test_transforms_of_many_rows(width):
    """More rows between the products than the GPU has CUs: two rows to a workgroup."""
    C.log(f"transforms of many rows of {width}")
    experts_against_the_oracle(23, 64, 128, width, 5, 5, 2, 2)
