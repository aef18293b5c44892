"""The choice of kernel by depth, without a GPU: what is chosen goes by the number of slices of 128, not by whether rows are a
multiple of 2 KiB; and few rows on weights that HBM has to deliver are streamed."""
import pytest

from tiled_dense_gemm_bias_amd import moe


@pytest.mark.parametrize("T,E", [(9, 1), (96, 1), (400, 1), (2000, 1), (200, 4), (1000, 4), (1000, 16), (2000, 16)])
def test_whole_2_kib_take_the_tile_of_their_slices(T, E):
    for N in (512, 520, 1024, 2048, 2816, 4096, 8192, 14336):
        for K in (2048, 4096, 6144, 8192, 14336):
            for ws in (0, 8 << 20):
                assert moe.plan(T, E, N, K, ws) == moe.plan(T, E, N, K - 16, ws), (N, K, ws)


def test_few_rows():
    for T, E, N, K in ((16, 32, 2816, 2048), (1, 1, 4096, 4096), (8, 8, 4096, 4096), (4, 4, 2816, 8192), (1, 1, 11008, 14336)):
        assert moe.plan(T, E, N, K)["kind"] == "stream", (T, E, N, K)
    for T, E, N, K in ((8, 1, 14336, 4096), (96, 16, 28672, 2048)):
        assert moe.plan(T, E, N, K)["kind"] == "ring", (T, E, N, K)
