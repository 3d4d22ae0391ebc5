"""A decoder layer's MLP whose every product sees rotated rows: residual RMS norm, quantiser behind the gate and
up projections' transform, gated linear, quantiser behind the down projection's, down."""
import numpy as np
import pytest

from oracle import q8_oracle as Q
from tests import gpu_common as C
from tests.test_w8a8_gpu import Mlp, U, gated_bound, linear_bound, over, rotated_bounds, rows
import workloads as W

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd")


class RotatedMlp(Mlp):
    def __init__(self, seed, D, F, K=8):
        super().__init__(seed, D, F, K)
        self.tx = W.custom_linear(seed, 2, D, 16, K)
        self.rot_x = rl.paro_rotation_prepare(self.tx.pairs, self.tx.theta, self.tx.scale)
        self.gu = rl.paro_pack_weights_q8(self.w_gu, self.rot_x)

    def run(self, x, stream):
        n, _ = rl.paro_rmsnorm(x, self.gamma, 1e-5, residual=stream, residual_out=stream)
        xq, xs = rl.paro_quantize_q8(n, self.rot_x)
        a = rl.paro_w8a8_gated_linear(xq, xs, *self.gu)
        aq, as_ = rl.paro_quantize_q8(a, self.rot)
        return n, xq, xs, a, aq, as_, rl.paro_w8a8_linear(aq, as_, *self.d)

    def check(self, x, stream0, out):
        """Each step against the oracle on what it was given; then the block against itself in 64 bits without
        any quantisation: the relative error."""
        n, xq, xs, a, aq, as_, y = [t.double().cpu().numpy() for t in out]
        h = Q.round_to(x.double().cpu().numpy() + stream0.double().cpu().numpy(), "f16")
        n64 = Q.rmsnorm(h, self.gamma.double().cpu().numpy(), 1e-5)
        assert over(n - n64, np.abs(n64) * (4 * U + 2.0 ** -11) + 2.0 ** -25) <= 1
        for row, q, s, t in ((n, xq, xs, self.tx), (a, aq, as_, self.t)):
            real, sc = Q.quantize_exact(Q.transform(row, t.pairs, t.theta, t.scale))
            dtop, dcode = rotated_bounds(row, t.scale, 8, real, sc)
            assert over(q - real, 0.5 + 127 * 2 * U + dcode) <= 1 and over(s - sc, dtop / 127 + 2 * U * sc) <= 1
        v, g, u = Q.gated(xq, xs, *[t.double().cpu().numpy() for t in self.gu])
        assert over(a - v, gated_bound(v, g, u, "f16")) <= 1
        ref = Q.linear(aq, as_, *[t.double().cpu().numpy() for t in self.d])
        assert over(y - ref, linear_bound(ref, "f16")) <= 1
        gu = n64 @ self.w_gu.double().cpu().numpy().T
        g, u = gu[:, :self.F], gu[:, self.F:]
        full = (g / (1 + np.exp(-g)) * u) @ self.w_d.double().cpu().numpy().T
        return np.linalg.norm(y - full) / np.linalg.norm(full)


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_rotated_mlp_block(M):
    C.log(f"rotated mlp M={M}")
    mlp = RotatedMlp(61, 512, 1152)
    x, _ = rows(62, M, 512, "f16", 5.0)
    stream, _ = rows(63, M, 512, "f16", 5.0)
    kept = stream.clone()
    out = mlp.run(x, stream)
    # the oracle's own block (its quantisers and products, in 64 bits) is 3.3 % off the block without quantisation
    assert mlp.check(x, kept, out) < 0.05
    assert torch.equal(stream, (x.float() + kept.float()).half())


@pytest.mark.parametrize("M", [3, 150])
def test_rotated_mlp_block_captured_and_replayed(M):
    C.log(f"rotated mlp graph M={M}")
    mlp = RotatedMlp(64, 384, 1024)
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
