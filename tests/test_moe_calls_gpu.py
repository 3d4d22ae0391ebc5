"""The mixture-of-experts calls on the GPU: the arguments that they refuse, with operands that are right otherwise."""
import numpy as np
import pytest

from tests.test_moe_gpu import pack, tokens

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")


def test_a_layer_without_a_router_is_refused():
    """Even where a routing to write is given, which the experts alone would read."""
    r = np.random.default_rng(3)
    M, D, F, E, k = 4, 256, 128, 3, 2
    gu, _ = pack(r, E, 2 * F, D)
    dn, _ = pack(r, E, D, F)
    x, _ = tokens(r, M, D)
    routing = torch.zeros(M, k, dtype=torch.int32, device="cuda"), torch.ones(M, k, device="cuda")
    for given in (None, routing):
        with pytest.raises(ValueError, match="router"):
            rl.paro_moe_layer_w4a16(x, None, k, gu, dn, routing=given)
