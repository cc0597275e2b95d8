"""Sizes of the prompt weights' workspace: host arithmetic, no GPU."""
import pytest

BF16, F32 = 1, 0


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_116_gb300 import build

    build.build()
    from paged_kv_cache_116_gb300 import _binding

    return _binding.lib()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("heads", [(32, 8), (64, 8), (12, 2)])
@pytest.mark.parametrize("seqs", [1, 4])
def test_a_window_needs_space_for_the_rows_it_counts(lib, dtype, heads, seqs):
    """The statistics are of the counted rows: with a window of 32 a prompt of 131,072 tokens needs no more than one of
    1,024 over the same context."""
    def size(new, window):
        return lib.pa_prompt_weights_workspace_size(seqs, seqs * new, new, *heads, 128, 16, 131072, window, dtype)

    assert size(131072, 32) == size(1024, 32)
    # in pieces of the keys at most 64 times (maximum, sum) per row, and once a 4-byte statistic in tiles of up to
    # twice the rows
    rows = seqs * 32 * heads[0]
    assert size(131072, 32) <= 64 * rows * 8 + 2 * (rows + (seqs + 2) * 128 * heads[1]) * 4 + 4096
    assert size(131072, 0) > size(131072, 32)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_window_beyond_the_prompt_changes_nothing(lib, dtype):
    for window in (300, 4096, 2 ** 31 - 1):
        a = lib.pa_prompt_weights_workspace_size(3, 600, 300, 8, 2, 128, 16, 400, window, dtype)
        assert a == lib.pa_prompt_weights_workspace_size(3, 600, 300, 8, 2, 128, 16, 400, 0, dtype)
