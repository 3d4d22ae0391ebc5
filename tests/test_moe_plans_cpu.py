"""How the experts' products are cut, by the sizes of a call."""
import ctypes

import pytest

from tests.test_moe_gpu import LARGE, SIZES, down_plan, test_rotated_experts as _rotated
from tests.test_moe_values_gpu import MORE, WIDTHS

rl = pytest.importorskip("rotated_linear_amd")
ROTATED = next(m.args[1] for m in _rotated.pytestmark if m.name == "parametrize")


def gate_up_plan(*size, parts=1):
    """(waves of a workgroup, groups of a wave, whether weights go past the caches)"""
    out = [ctypes.c_int() for _ in range(3)]
    rl.lib().paro_internal_moe_gate_up_plan(*size, parts, *map(ctypes.byref, out))
    return tuple(v.value for v in out)


@pytest.mark.parametrize("D,F", [(4096, 14336), (1024, 4096), (4096, 4096), (128, 16384), (16384, 256)])
def test_units_of_an_expert_count(D, F):
    """Every token at every expert: one expert of 64 tokens is as much work as four of 16, and three of 33 as nine of 11."""
    assert down_plan(64, D, F, 1, 1) == down_plan(16, D, F, 4, 4)
    assert down_plan(33, D, F, 3, 3) == down_plan(11, D, F, 9, 9)


def test_weights_that_are_read_again_stay_in_the_caches():
    size = 4096, 14336
    assert gate_up_plan(4, *size, 8, 2)[2] and gate_up_plan(24, *size, 2, 1)[2]
    assert not gate_up_plan(64, *size, 4, 2)[2] and not gate_up_plan(64, *size, 1, 1)[2] and not gate_up_plan(17, *size, 1, 1)[2]
    assert not gate_up_plan(1, 2048, 1024, 64, 8)[2]  # few bytes


@pytest.mark.parametrize("parts", [1, 2])
def test_a_row_fits_its_waves(parts):
    for groups in range(1, 129):
        waves, each, _ = gate_up_plan(4, 128 * groups, 256, 8, 2, parts=parts)
        assert waves in (4, 8, 16) and (each == 0 or (waves * each >= groups and parts * each <= 4))
        assert each or groups > 64 // parts


def down_kernel(*size):
    """(16-column tiles of a workgroup, whether no expert can have more than 8 tokens, whether weights go past the caches)"""
    out = [ctypes.c_int() for _ in range(3)]
    rl.lib().paro_internal_moe_down_kernel(*size, *map(ctypes.byref, out))
    return tuple(v.value for v in out)


def test_the_gpu_tests_reach_every_kernel():
    calls = [(*s, 1) for s in SIZES + MORE] + [(*s[:5], 2 if s[5] else 1) for s in LARGE]
    calls += [(*s[:5], 2) for s in ROTATED] + [(3, w, 128, 2, 1, 2) for w in WIDTHS] + [(3, 128, w, 2, 1, 1) for w in WIDTHS]
    gate_up = {(parts, *gate_up_plan(*size, parts=parts)) for *size, parts in calls}
    plain = (4, 1), (4, 2), (4, 3), (4, 4), (8, 3), (8, 4), (16, 3), (16, 4), (16, 0)
    behind = (4, 1), (8, 1), (8, 2), (16, 2), (16, 0)
    assert gate_up == {(parts, *plan, once) for parts, plans in ((1, plain), (2, behind)) for plan in plans for once in (0, 1)}
    down = {(*down_kernel(*size), down_plan(*size)[1] > 1) for *size, _ in calls}
    assert down >= {(tiles, few, 0, shared) for tiles in (1, 2, 4) for few in (0, 1) for shared in (False, True)}
    assert {d[:3] for d in down if d[2]} == {(4, 0, 1), (4, 1, 1)}
