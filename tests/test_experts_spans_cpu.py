"""Overlap checks of the grouped and 4-bit products where an array ends near the end of the address space."""
from tests.test_experts_cpu import ALIAS, NULL, P, at, dense4, fwd, grad, lib, mx4, wgrad  # noqa: F401

TOP = (1 << 64) - (1 << 20)


def test_a_workspace_over_everything_is_an_overlap(lib):  # noqa: F811
    """Its end lies past the last address, so that a sum of address and size wraps round."""
    for call in (fwd, grad, wgrad, mx4, dense4):
        for nb in ((1 << 64) - 1, (1 << 64) - P, (1 << 64) - 1 - at(3)):
            assert call(lib, ws=P, nb=nb) == ALIAS, (call.__name__, nb)


def test_arrays_at_the_top_of_the_address_space(lib):  # noqa: F811
    assert fwd(lib, C=TOP, ws=TOP - (1 << 20), nb=(1 << 20) + 16) == ALIAS
    assert fwd(lib, C=TOP, ws=TOP + 16, nb=1 << 40) == ALIAS
    assert fwd(lib, C=None, ws=TOP, nb=1 << 40) == NULL
