"""Waits that run out are reported, by whatever role of a kernel they are made."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_an_item_that_never_comes_is_not_the_end_of_the_items():
    """Warps that take handed-out work give up on a ring that nobody fills, or nobody empties, with an answer of its
    own -- not with the end of the list, after which a kernel would return as if all its work were done."""
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    pa.pa_device_status(clear=True)
    for polls in (1, 500):
        pa.pa_selftest_wait_timeout(polls)
        with pytest.raises(pa.PAError, match="PA_ERR_TIMEOUT"):
            pa.pa_device_status(clear=True)
        pa.pa_device_status(clear=True)
    assert float(torch.ones(4, device="cuda:0").sum()) == 4.0  # the context is usable
