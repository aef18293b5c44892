"""Sizes that reach the persistent kernel of the 8-bit products, as moe_cases.PRODUCTS."""
from tests.moe_cases import _case

# The persistent kernel where tiles have few slices (two to five, whole and cut short), several tiles a CU, more than 64 experts; with
# columns in whole 128-byte lines (N a multiple of 64) whole tiles are stored without masks, beside the ragged ends of groups.
_LARGE = ("persistent", 256, 256, False)
LARGE = [
    _case(_LARGE, 3500, 1, 4096, 144, 0),
    _case(_LARGE, 7000, 2, 4160, 256, 0, 3, 0),
    _case(_LARGE, 3000, 5, 4160, 272, 0, 1, 2),
    _case(_LARGE, 3000, 8, 4096, 384, 0),
    _case(_LARGE, 1500, 3, 8256, 400, 0, 0, 5),
    _case(_LARGE, 10000, 5, 4160, 272, 0),
    _case(_LARGE, 11000, 3, 4096, 144, 0, 0, 1),
    _case(_LARGE, 12000, 66, 4096, 272, 0, 2, 3),
    _case(_LARGE, 15000, 70, 2048, 528, 0),
    _case(_LARGE, 15000, 66, 8200, 272, 0),
]
