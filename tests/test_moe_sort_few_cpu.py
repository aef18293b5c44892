"""moe_sort of more slots a token than experts (a device's share of them): not refused, without a GPU."""
import pytest

import tiled_dense_gemm_bias_amd as gba
from tests.test_abi_cpu import _gpu_present
from tests.test_moe_cpu import DEVICE, SCRATCH, SHAPE, at, grad, route, sort


def test_more_slots_than_experts():
    lib = gba.moe.moe_lib()
    assert sort(lib, E=2, k=33) == SHAPE and sort(lib, E=0, k=8) == SHAPE
    assert sort(lib, E=2, k=8, T=1 << 20, ws=at(8), nb=4) == SCRATCH
    assert gba.moe_sort_workspace(16384, 2, 8) == 256 * 4 * 4 and gba.moe_sort_workspace(8, 2, 8) == 0
    assert route(lib, E=2, k=8) == SHAPE and grad(lib, E=2, k=8) == SHAPE     # a choice of 8 of 2 is none
    if _gpu_present():
        pytest.skip("a GPU is present; the rest checks the GPU-less path")
    assert sort(lib, E=2, k=8) == sort(lib, E=1, k=32) == DEVICE
