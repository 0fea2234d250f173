"""Sizes of the grouped projections at their largest row counts, on the CPU."""
import pytest

MOST = (1 << 31) - 513      # rows


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__ as g

    g.build()
    from mixture_experts_layer_mok_gb300 import _lib

    return _lib.load()


@pytest.mark.parametrize("N", [8, 256, 264, 2048, 256 * 1216, 256 * 1216 + 8, 1 << 20])
@pytest.mark.parametrize("M", [1, 1 << 20, (1 << 31) - 4096, (1 << 31) - 1216, (1 << 31) - 1215, MOST])
def test_the_bias_sums_take_few_chunks_of_any_row_count(lib, M, N):
    """Chunks of rows are made so that there are 8 blocks or so for each of 152
    SMs: at most ceil(1216 / column blocks) of them, and one more part for each
    expert."""
    E, size = 3, lib.mok_grouped_linear_bwd_workspace_bytes
    parts = size(M, E, N, 0, 0, 1) - size(M, E, N, 0, 0, 0)
    cols = -(-N // 256)
    assert (E + 1) * N * 4 <= parts <= (-(-1216 // cols) + E) * N * 4 + 255
    assert size(MOST + 1, E, N, 0, 0, 1) == 0
