"""What the header and the docstrings say of cases that the code cannot settle, or settles in a way that a caller has to know."""
import re

import pytest

import tiled_dense_gemm_bias_amd as gba


@pytest.fixture(scope="module")
def header():
    """The header's comments as running text."""
    return re.sub(r"\s*\n \*\s*", " ", open(gba.moe.MOE_HEADER).read())


def test_rows_of_two_slots(header):
    """Several waves write a row, in no order."""
    assert "holds one of the two" not in header
    assert "No row belongs to two slots" in header and "(but for rows that two slots name, see below)" in header
    assert "mixture of both" in gba.moe.__doc__


def test_gradients_of_rows_without_a_slot(header):
    assert "NaN where moe_route's weights are NaN for its logits" in header
    assert "NaN where moe_route's weights are NaN" in " ".join(gba.moe_route_grad.__doc__.split())


def test_slots_without_a_row_in_combine(header):
    """An infinity or a NaN among their weights makes the token's sums NaN."""
    doc = " ".join(gba.moe_combine.__doc__.split())
    assert "left out" not in doc and "A slot of -1 adds its weight times 0" in doc
    assert "A slot of -1 adds weight times 0" in header


def test_range_of_the_scales_product(header):
    assert "a scales' product below 2^-126 has fewer bits, one of 2^128 or more is an infinity" in header


def test_accuracy_of_routing_weights(header):
    """What tests/moe_oracle.py's route_tol holds them to."""
    assert "off by up to (2 D + 40) 2^-24 of themselves" in header
    import torch
    from tests import moe_oracle as orc
    w, depth = torch.tensor([[0.5]], dtype=torch.float64), torch.tensor([3.0], dtype=torch.float64)
    assert abs(orc.route_tol(w, depth).item() - 46 * 2.0 ** -25) < 2.0 ** -100
