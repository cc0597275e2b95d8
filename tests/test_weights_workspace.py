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


GIB = 1 << 30


@pytest.mark.parametrize("fp8", [False, True])
def test_dense_keys_of_many_long_requests_are_laid_out_in_parts(lib, fp8):
    """Blocks that no box fits, and codes: a copy of the keys of as many requests at a time as some GiB hold."""
    def size(seqs, context, bs=12):
        fn = lib.pa_prompt_weights_fp8_workspace_size if fp8 else lib.pa_prompt_weights_workspace_size
        return fn(seqs, seqs, 1, 32, 8, 128, bs, context, 0, BF16)

    one = 131072 * 8 * 128 * 2
    assert one < size(1, 131072) < 1.1 * one
    assert size(64, 131072) <= 4.5 * GIB
    assert size(100000, 131072) <= 4.5 * GIB
    # one request is never cut: what it needs is asked for
    assert size(2, 1 << 23) >= (1 << 23) * 8 * 128 * 2


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_of_many_long_sequences_are_kept_in_parts(lib, fp8):
    def size(seqs, context):
        fn = lib.pa_decode_weights_fp8_workspace_size if fp8 else lib.pa_decode_weights_workspace_size
        return fn(seqs, 32, 8, 128, 16, context, BF16)

    assert size(1, 131072) >= 131072 * 32 * 4
    assert size(4096, 131072) <= 4.5 * GIB
    assert size(2, 1 << 29) >= (1 << 29) * 32 * 4


@pytest.mark.parametrize("seqs", [129, 200, 256, 300, 4096])
def test_parts_are_of_one_size(lib, seqs):
    """129 sequences of 33 MB are two parts of 65 and 64, not 128 and a single one."""
    per = 262144 * 32 * 4
    parts = -(-seqs // ((4 * GIB) // per))
    space = lib.pa_decode_weights_workspace_size(seqs, 32, 8, 128, 16, 262144, BF16)
    assert 0 <= space - -(-seqs // parts) * per < 64 << 20  # (and the split records)
