"""Check mode of the latent-cache and shared-prefix entry points: index arrays
that do not fit are refused on the host, before anything runs."""
import pytest
import torch

from latent_ops import LatentBatch, SharedBatch, rand

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    pa.pa_set_check_mode(True)
    yield pa
    pa.pa_set_check_mode(False)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _refused(pa, f, what):
    with pytest.raises(pa.PAError, match=what):
        f()


def test_latent_write(pa):
    n, row = 5, 576
    kv = rand((n, row), "bf16", 1).to(DEV)
    inv, pos = torch.ones(32, dtype=torch.float64, device=DEV), torch.arange(n, device=DEV)
    cache = torch.zeros((2, 16, row), dtype=torch.bfloat16, device=DEV)
    for slots, what in (([0, 1, 2, 3, 32], "outside the pool"), ([0, 1, 2, 3, 1], "written twice")):
        _refused(pa, lambda: pa.pa_latent_write(kv, pos, inv, torch.tensor(slots, device=DEV), cache), what)
    assert (cache == 0).all()
    pa.pa_latent_write(kv, pos, inv, torch.tensor([0, 1, -1, -1, 31], device=DEV), cache)


def test_latent_attention(pa):
    b = LatentBatch([40, 20], 512, 64, 16, "bf16", 1).to(DEV)
    q = rand((2, 16, 576), "bf16", 2).to(DEV)
    out = torch.zeros((2, 16, 512), dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(pa.pa_latent_varlen_workspace_size(2, 2, 1, 16, 512, 64, 16, 40, q.dtype), dtype=torch.uint8,
                     device=DEV)

    def decode(lens, tables=b.dtables, ctx=40):
        return pa.pa_latent_decode(out, q, b.dcache, tables, _i32(lens), ctx, 0.1, workspace=ws)

    decode([40, 20])
    _refused(pa, lambda: decode([41, 20]), "outside")
    _refused(pa, lambda: decode([-1, 20]), "outside")
    _refused(pa, lambda: decode([40, 20], tables=b.dtables[:, :2].contiguous()), "needs 3 blocks")
    bad = b.dtables.clone()
    bad[1, 0] = b.num_blocks
    _refused(pa, lambda: decode([40, 20], tables=bad), "maps to")
    for lens, cu, max_q in (([40, 20], [0, 1, 1], 1), ([40, 20], [0, 2, 2], 1), ([1, 20], [0, 2, 2], 2), ([40, 20], [0, 2, 1], 2)):
        with pytest.raises(pa.PAError):
            pa.pa_latent_varlen(out, q, b.dcache, b.dtables, _i32(lens), _i32(cu), max_q, 40, 0.1, workspace=ws)


def test_shared(pa):
    b = SharedBatch([(32, [5, 9]), (48, [1, 2])], 2, 64, 16, "bf16", 1, [7]).to(DEV)
    q = rand((5, 8, 64), "bf16", 2).to(DEV)
    pa.pa_set_option(1, 2)
    try:
        ws = torch.empty(pa.pa_decode_shared_workspace_size(5, 2, 8, 2, 64, 16, b.max_context, q.dtype), dtype=torch.uint8,
                         device=DEV)

        def run(starts=(0, 2, 4), prefix=(32, 48), tables=b.dtables):
            return pa.pa_decode_shared(torch.zeros_like(q), q, b.dk, b.dv, tables, b.dlens, _i32(starts), _i32(prefix),
                                       b.max_context, 0.1, workspace=ws)

        run()
        run(starts=(1, 1, 3), prefix=(32, 0))
        for starts, what in (((-1, 2, 4), "group_starts"), ((0, 2, 6), "group_starts"), ((0, 3, 2), "non-decreasing"),
                             ((0, 99, 4), "non-decreasing")):
            _refused(pa, lambda: run(starts=starts), what)
        for prefix, what in (((33, 48), "multiple"), ((-16, 48), "multiple"), ((48, 48), "longer than"), ((32, 64), "longer than")):
            _refused(pa, lambda: run(prefix=prefix), what)
        bad = b.dtables.clone()
        bad[1, 1] = b.dtables[3, 0]
        _refused(pa, lambda: run(tables=bad), "does not share")
        _refused(pa, lambda: run(starts=(0, 3, 4)), "longer than|does not share")
    finally:
        pa.pa_set_option(1, 0)
