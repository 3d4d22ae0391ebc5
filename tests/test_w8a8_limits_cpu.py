"""Sizes at the ends of the 8-bit products' range (fake pointers: every case returns before anything is
enqueued)."""
import pytest

rl = pytest.importorskip("rotated_linear_amd", reason="libparo.so not built")
lib = rl.lib()
AT = [1 << (42 + i) for i in range(6)]  # never dereferenced, farther apart than any operand is long
MOST = 2 ** 31 - 512


@pytest.mark.parametrize("gated", [False, True])
def test_rows_that_no_tile_count_holds_are_refused(gated):
    """M or N within a tile of 2^31: their tiles are counted in ints."""
    fn = lib.paro_w8a8_gated_linear if gated else lib.paro_w8a8_linear
    need = lib.paro_w8a8_gated_workspace_bytes if gated else lib.paro_w8a8_workspace_bytes
    x, xs, w, s, y, ws = AT
    for over in (MOST + 1, MOST + 300, 2 ** 31 - 1):
        for M, N in ((over, 3), (3, over), (over, 0), (0, over)):
            assert fn(M, 128, N, x, xs, w, s, y, 0, ws, 1 << 40, None) == 1, (M, N)
            assert need(M, 128, N) == 0
    assert fn(MOST, 128, 0, x, xs, w, s, y, 0, ws, 1 << 40, None) == 0  # the largest, nothing to do
    assert fn(0, 128, 2 ** 29 - 1 if gated else MOST, x, xs, w, s, y, 0, ws, 1 << 40, None) == 0
