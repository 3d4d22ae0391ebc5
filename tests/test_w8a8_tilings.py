"""Every tiling of the tiled 8-bit product by name, whatever the plan would choose: plain and gated, whole and
in parts, fewer tiles than the GPU holds workgroups and more (so that loads and scales pass from one tile of a
workgroup to its next), rows of y at 16-byte boundaries and not, in every output type. And what the plan
chooses: each tiling somewhere, and the largest one for the prompts that it is there for.

The library's entries for this are in no header of its own (csrc/q8_internal.h).
"""
import ctypes

import numpy as np
import pytest

torch = pytest.importorskip("torch")
rl = pytest.importorskip("rotated_linear_amd", reason="libparo.so not built")

lib = rl.lib()
_i, _p, _sz = ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
_ip = ctypes.POINTER(_i)
lib.paro_internal_w8a8_plan.argtypes = [_i, _i, _i, _i, _ip, _ip, _ip]
lib.paro_internal_w8a8_plan.restype = None
lib.paro_internal_w8a8_tiling.argtypes = [_i, _ip, _ip, _ip]
lib.paro_internal_w8a8_tiled_workspace_bytes.argtypes = [_i, _i, _i, _i]
lib.paro_internal_w8a8_tiled_workspace_bytes.restype = _sz
lib.paro_internal_w8a8_tiled.argtypes = [_i, _i, _i, _i, _i, _i, _p, _p, _p, _p, _p, _i, _p, _sz, _p]

STREAM, COLUMN, TILED = 0, 1, 2
TILINGS = range(7)
U = 2.0 ** -24
DT = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
CODE = {"f16": rl.F16, "bf16": rl.BF16, "f32": rl.F32}
HALF = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": U}
SUB = {"f16": 2.0 ** -25, "bf16": 2.0 ** -134, "f32": 2.0 ** -150}


def plan(M, D, N, gated):
    """(kernel, tiling or -1, parts) of a product."""
    out = [_i() for _ in range(3)]
    lib.paro_internal_w8a8_plan(M, D, N, int(gated), *map(ctypes.byref, out))
    return tuple(v.value for v in out)


def tiling(tile):
    """(rows of x, rows of w, workgroups that the GPU holds) of a tiling."""
    out = [_i() for _ in range(3)]
    assert lib.paro_internal_w8a8_tiling(tile, *map(ctypes.byref, out)) == 1
    return tuple(v.value for v in out)


def test_there_are_these_tilings():
    assert [tiling(t)[:2] for t in TILINGS] == [(256, 256), (256, 128), (128, 128), (128, 128), (128, 64), (64, 64), (32, 64)]
    assert lib.paro_internal_w8a8_tiling(7, _i(), _i(), _i()) == 0 and lib.paro_internal_w8a8_tiling(-1, _i(), _i(), _i()) == 0


def test_the_plan_reaches_every_kernel_and_tiling():
    """Nothing is built that no size takes: over sizes spread by their logarithms, each kernel, and each tiling
    whole and in parts."""
    r = np.random.default_rng(1)

    def log(lo, hi, n):
        return np.rint(np.exp(r.uniform(np.log(lo), np.log(hi), n))).astype(int).tolist()

    n = 60000
    seen = set()
    for M, d, N, g in zip(log(1, 8192, n), log(1, 128, n), log(16, 32768, n), r.integers(0, 2, n).tolist()):
        kernel, tile, parts = plan(M, 128 * d, N, g)
        assert kernel == TILED or (tile, parts) == (-1, 1)
        need = (lib.paro_w8a8_gated_workspace_bytes if g else lib.paro_w8a8_workspace_bytes)(M, 128 * d, N)
        assert need == (lib.paro_internal_w8a8_tiled_workspace_bytes(M, N, g, parts) if kernel == TILED else 0)
        seen.add((kernel, tile, parts > 1))
    assert seen == {(STREAM, -1, False), (COLUMN, -1, False)} | {(TILED, t, p) for t in TILINGS for p in (False, True)}


@pytest.mark.parametrize("M,D,N,gated", [(4096, 4096, 14336, True), (4096, 4096, 14336, False), (512, 4096, 14336, True),
                                         (4096, 4096, 4096, False), (8192, 8192, 8192, False)])
def test_large_prompts_take_the_largest_tiles_whole(M, D, N, gated):
    assert plan(M, D, N, gated) == (TILED, 0, 1)


def test_tiled_entry_refusals():
    a = [1 << (42 + i) for i in range(6)]  # never dereferenced

    def f(tile=0, splits=1, M=300, D=512, N=300, dt=0, nb=1 << 40, ws=a[5]):
        return lib.paro_internal_w8a8_tiled(tile, splits, 0, M, D, N, *a[:5], dt, ws, nb, None)

    assert f(tile=-1) == 1 and f(tile=7) == 1 and f(splits=0) == 1 and f(splits=5) == 1 and f(dt=3) == 1
    assert f(D=200) == 2 and f(M=-1) == 1
    assert f(splits=4, nb=lib.paro_internal_w8a8_tiled_workspace_bytes(300, 300, 0, 4) - 1) == 5 and f(splits=2, ws=None) == 5
    assert f(M=0) == 0


def sizes(tile, gated, splits, several, aligned):
    """Sizes with ragged rows and columns, and a tile count on the wanted side of the GPU's workgroups."""
    bm, bn, workgroups = tiling(tile)
    yn = bn // 2 if gated else bn
    steps = {(1, False): 5, (1, True): 5 if aligned else 2, (3, False): 7, (3, True): 5}[splits, several]
    per = -(-steps // splits)
    parts = -(-steps // per)
    if several:
        tiles_m = 5  # a whole group of four rows of tiles and one more
        tiles_n = -(-int(1.2 * workgroups) // (parts * tiles_m)) + 1
    else:
        tiles_m, tiles_n = (1, 4) if aligned else (2, 3)
    units = tiles_m * tiles_n * parts
    assert units > 1.1 * workgroups if several else units < workgroups
    return tiles_m * bm - 5, 128 * steps, tiles_n * yn - (8 if aligned else 3)


def guarded(M, N, dtype):
    """[M][N] followed by 4 KiB of sevens: (tensor, the tail's check)."""
    n = M * N * dtype.itemsize
    buf = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
    return buf[:n].view(dtype).view(M, N), lambda: bool((buf[n:] == 7).all())


@pytest.mark.gpu
@pytest.mark.parametrize("aligned", [True, False], ids=["aligned", "ragged"])
@pytest.mark.parametrize("several", [False, True], ids=["one tile", "several"])
@pytest.mark.parametrize("splits", [1, 3], ids=["whole", "parts"])
@pytest.mark.parametrize("gated", [False, True], ids=["plain", "gated"])
@pytest.mark.parametrize("tile", TILINGS)
def test_tiling(tile, gated, splits, several, aligned):
    """Bounds, in units of U = 2^-24: a product is three roundings (the sum's, xs, ws). The gated output takes
    those of g into 1 + |g| times as much and those of u; the activation adds 7.15 in a float32 output and, with
    its exponential's argument rounded, 1.25 |g| + 12 in a 16-bit one, whose own rounding follows; where
    1 / (1 + exp(-g)) leaves float32 it counts as 0."""
    M, D, N = sizes(tile, gated, splits, several, aligned)
    print(f"[case] tiling {tile} gated={gated} parts={splits} M={M} D={D} N={N}", flush=True)
    assert (N % 8 == 0) == aligned
    g = torch.Generator(device="cuda").manual_seed(1000 * tile + M + N)
    rows = 2 * N if gated else N

    def codes(n):  # the whole range, -128 included
        return torch.randint(-128, 128, (n, D), generator=g, device="cuda", dtype=torch.int8)

    x, w = codes(M), codes(rows)
    xs = 0.02 + 0.04 * torch.rand(M, generator=g, device="cuda")
    ws = (0.5 + torch.rand(rows, generator=g, device="cuda")) / (5.0 if gated else 74.0) / D ** 0.5
    ref = (x.double() @ w.double().t()) * xs.double()[:, None] * ws.double()
    if gated:
        gate, up = ref[:, :N], ref[:, N:]
        ref = gate / (1 + torch.exp(-gate)) * up
    need = lib.paro_internal_w8a8_tiled_workspace_bytes(M, N, int(gated), splits)
    assert (need > 0) == (splits > 1)
    work = torch.full((max(need, 256),), 0xA5, dtype=torch.uint8, device="cuda")
    public = rl.paro_w8a8_gated_linear if gated else rl.paro_w8a8_linear
    for dt in ("f16", "bf16", "f32"):
        y, tail = guarded(M, N, DT[dt])
        st = lib.paro_internal_w8a8_tiled(tile, splits, int(gated), M, D, N, x.data_ptr(), xs.data_ptr(), w.data_ptr(), ws.data_ptr(),
                                          y.data_ptr(), CODE[dt], work.data_ptr(), need, torch.cuda.current_stream().cuda_stream)
        assert st == 0 and tail()
        if gated:
            own = 7.15 * U if dt == "f32" else (1.25 * gate.abs() + 12) * U + HALF[dt]
            bound = ref.abs() * ((3.1 * (1 + gate.abs()) + 3.1) * U + own) + (gate * up).abs() * 2.0 ** -120 + SUB[dt]
        else:
            bound = ref.abs() * (3.1 * U + (0 if dt == "f32" else HALF[dt])) + SUB[dt]
        off = (y.double() - ref).abs()
        if dt == "f16":
            off = torch.where(ref.abs() > 65000, 0, off)  # past float16: an infinity is right there
        assert bool((off <= bound).all()), (dt, float((off / bound).max()))
        # whichever kernel the plan takes gives the same bits
        assert torch.equal(public(x, xs, w, ws, DT[dt]), y)
