"""How the experts' products are cut, by the sizes of a call."""
import ctypes

import pytest

from tests.test_moe_gpu import down_plan

rl = pytest.importorskip("rotated_linear_amd")


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
