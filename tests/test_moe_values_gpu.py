"""What the experts hold between their products, seen in a float32 y against float64 oracles that round nothing."""
import numpy as np
import pytest

import oracle as O
import workloads as W
from oracle import block_oracle as B
from tests import gpu_common as C
from tests.test_moe_gpu import choose, pack, tokens

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
