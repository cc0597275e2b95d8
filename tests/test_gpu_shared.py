"""pa_decode_shared against attention in 64 bits (bounds in
latent_ops.attention) and against pa_decode's contract."""
import pytest
import torch

from latent_ops import SharedBatch, close, rand, shared_exact

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    yield pa
    pa.pa_set_option(1, 0)


@pytest.fixture(autouse=True)
def _apart(pa):
    """Small batches are worked as pa_decode unless the tensor cores are pinned; the pin is off where they do not
    apply (shared, below)."""
    yield
    pa.pa_set_option(1, 0)


def shared(pa, b, q, scale, out=None, fill=0xFF, starts=None, prefix=None, kernel=2):
    S, hq, hd = q.shape
    pa.pa_set_option(1, kernel if _tensor_cores(b, hq) else 0)
    starts = b.dstarts if starts is None else starts
    prefix = b.dprefix if prefix is None else prefix
    if out is None:
        out = torch.full_like(q, float("nan"))
    size = pa.pa_decode_shared_workspace_size(S, prefix.numel(), hq, b.hkv, hd, b.bs, b.max_context, q.dtype)
    ws = torch.full((max(16, size),), fill, dtype=torch.uint8, device=DEV)
    pa.pa_decode_shared(out, q, b.dk, b.dv, b.dtables, b.dlens, starts, prefix, b.max_context, scale, workspace=ws)
    return out


CASES = [
    # groups (prefix, tails), loners, hq, hkv, hd, bs, dtype
    ([(64, [5, 0, 30])], [], 32, 8, 128, 16, "bf16"),
    ([(288, [13, 40, 200, 256])] * 5, [1, 0, 77], 12, 2, 128, 16, "bf16"),
    ([(1024, list(range(0, 64)))], [], 8, 8, 64, 16, "f16"),          # the tail's tiles: empty, partial, several
    ([(16, [1]), (32, [2, 3]), (0, [50, 60]), (48, [])], [9], 16, 1, 128, 16, "bf16"),
    ([(2048, [7] * 13)], [], 28, 4, 128, 32, "f16"),
    ([(120, [1, 9, 64]), (8, [3] * 20)], [], 32, 8, 128, 8, "bf16"),   # 8-token blocks: the tail starts inside a tile
    ([(3000 // 48 * 48, [100] * 40)], [], 32, 8, 128, 48, "bf16"),
    ([(512, [10] * 200)], [500], 32, 8, 128, 16, "bf16"),              # more rows than a tile
    ([(256, [10, 20, 0])], [5], 16, 2, 256, 16, "bf16"),
    ([(256, [0, 0, 0])], [], 40, 40, 128, 16, "f16"),                  # nothing but the prefix
    ([(64, [3, 50])] * 60, [], 12, 2, 128, 16, "bf16"),
    ([(4096, [33] * 3)], [], 16, 16, 128, 64, "f16"),
    ([(60, [1, 2, 3])], [4], 8, 2, 128, 12, "bf16"),                   # no box: as pa_decode
    ([(64, [5, 30])], [8], 8, 2, 64, 16, "f32"),
    ([(64, [5, 30])], [8], 34, 2, 128, 16, "bf16"),                    # 17 heads per KV head: CUDA cores
    ([(64, [5, 30])], [8], 8, 2, 96, 16, "bf16"),
]


def _tensor_cores(b, hq):
    return b.dtype != "f32" and b.hd in (64, 128, 256) and hq // b.hkv <= 16


@pytest.mark.parametrize("groups,loners,hq,hkv,hd,bs,dtype", CASES)
def test_against_64_bits(pa, groups, loners, hq, hkv, hd, bs, dtype):
    b = SharedBatch(groups, hkv, hd, bs, dtype, 3, loners).to(DEV)
    q = rand((len(b.lens), hq, hd), dtype, 4)
    scale = hd ** -0.5
    exact, bound = shared_exact(b, q, scale, _tensor_cores(b, hq))
    for kernel in (2, 0):  # apart, and as the sizes say
        out = shared(pa, b, q.to(DEV), scale, kernel=kernel)
        close(out, exact, bound)
        for s, L in enumerate(b.lens):
            if L == 0:
                assert (out[s] == 0).all()
    assert pa.lib().pa_device_status(1) == 0


def test_without_groups_it_is_the_plain_decode(pa):
    b = SharedBatch([], 8, 128, 16, "bf16", 3, [100, 0, 900, 16]).to(DEV)
    q = rand((4, 32, 128), "bf16", 4).to(DEV)
    out = shared(pa, b, q, 0.1, prefix=torch.zeros(0, dtype=torch.int32, device=DEV),
                 starts=torch.zeros(1, dtype=torch.int32, device=DEV))
    ws = torch.zeros(max(16, pa.pa_decode_workspace_size(4, 32, 8, 128, 16, b.max_context, q.dtype)), dtype=torch.uint8,
                     device=DEV)
    plain = torch.zeros_like(q)
    pa.pa_decode(plain, q, b.dk, b.dv, b.dtables, b.dlens, b.max_context, 0.1, workspace=ws)
    assert torch.equal(out, plain)


def test_large_batches_are_worked_apart(pa):
    """Without a pinned kernel: 64 requests behind 2,048 tokens, and the workspace that takes."""
    b = SharedBatch([(2048, [5 + 3 * i for i in range(64)])], 8, 128, 16, "bf16", 6).to(DEV)
    q = rand((64, 32, 128), "bf16", 7)
    size, plain = (f(64, *g, 32, 8, 128, 16, b.max_context, q.dtype) for f, g in
                   ((pa.pa_decode_shared_workspace_size, (1,)), (pa.pa_decode_workspace_size, ())))
    assert size > plain
    close(shared(pa, b, q.to(DEV), 0.09, kernel=0), *shared_exact(b, q, 0.09, True))


def test_groups_may_lie_anywhere(pa):
    """Sequences before the first group and behind the last are worked on their own."""
    b = SharedBatch([(0, [40, 50]), (160, [8, 1, 30])], 2, 128, 16, "bf16", 6, [200]).to(DEV)
    q = rand((6, 12, 128), "bf16", 7)
    starts = torch.tensor([2, 5], dtype=torch.int32, device=DEV)
    out = shared(pa, b, q.to(DEV), 0.09, starts=starts, prefix=torch.tensor([160], dtype=torch.int32, device=DEV))
    close(out, *shared_exact(b, q, 0.09, True))


def test_scores_that_grow_and_values_that_differ(pa):
    """The prefix's and the tail's maxima far apart, either way round."""
    for up in (True, False):
        b = SharedBatch([(256, [64, 100, 1])], 2, 128, 16, "bf16", 6)
        lead = b.tables[0, :16].long()
        b.k[lead] *= 0.05 if up else 4.0
        b.to(DEV)
        q = rand((3, 12, 128), "bf16", 7, 3.0)
        close(shared(pa, b, q.to(DEV), 0.3), *shared_exact(b, q, 0.3, True))


def test_relabelled_blocks_give_the_same_bits(pa):
    b = SharedBatch([(512, [10, 300, 0])], 8, 128, 16, "bf16", 6, [70]).to(DEV)
    q = rand((4, 32, 128), "bf16", 7).to(DEV)
    first = shared(pa, b, q, 0.09)
    perm = torch.randperm(b.num_blocks, generator=torch.Generator().manual_seed(9))
    for name in ("k", "v"):
        pool = torch.empty_like(getattr(b, name))
        pool[perm] = getattr(b, name)
        setattr(b, "d" + name, pool.to(DEV))
    b.dtables = torch.where(b.tables >= 0, perm[b.tables.long().clamp(min=0)].int(), b.tables).to(DEV)
    assert torch.equal(first, shared(pa, b, q, 0.09, fill=0))


def test_graph_replays_follow_lengths_and_groups(pa):
    b = SharedBatch([(256, [64, 100, 1]), (128, [5, 300])], 2, 128, 16, "bf16", 6).to(DEV)
    q = rand((5, 12, 128), "bf16", 7).to(DEV)
    out = torch.zeros_like(q)
    pa.pa_set_option(1, 2)
    ws = torch.zeros(pa.pa_decode_shared_workspace_size(5, 2, 12, 2, 128, 16, b.max_context, q.dtype),
                     dtype=torch.uint8, device=DEV)
    run = lambda: pa.pa_decode_shared(out, q, b.dk, b.dv, b.dtables, b.dlens, b.dstarts, b.dprefix,  # noqa: E731
                                      b.max_context, 0.09, workspace=ws)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens, prefix in (([320, 356, 257, 133, 428], [256, 128]), ([300, 256, 250, 0, 128], [240, 0]),
                         ([17, 20, 30, 16, 200], [16, 16])):
        q.copy_(rand((5, 12, 128), "bf16", sum(lens)))
        b.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        b.dprefix.copy_(torch.tensor(prefix, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        run()
        assert torch.equal(got, out)
        b.lens = lens
        close(out, *shared_exact(b, q.cpu(), 0.09, True))


@pytest.mark.parametrize("ctas", [1, 7, 152, 3000])
def test_any_split_of_the_rests(pa, ctas):
    """PA_OPT_DECODE_CTAS from one CTA (units worked whole) to more warps than tiles (one tile or none each)."""
    b = SharedBatch([(96, [0, 1, 40, 300]), (16, [5, 5])], 2, 128, 16, "bf16", 8, [33]).to(DEV)
    q = rand((7, 12, 128), "bf16", 9)
    exact = shared_exact(b, q, 0.09, True)
    pa.pa_set_option(2, ctas)
    try:
        close(shared(pa, b, q.to(DEV), 0.09), *exact)
    finally:
        pa.pa_set_option(2, 0)


def test_no_group_shares_anything(pa):
    """Groups without a prefix, of one member, or of none: the work of the prefixes is empty."""
    b = SharedBatch([(0, [40, 50]), (64, [8]), (32, [])], 2, 128, 16, "f16", 6, [200]).to(DEV)
    q = rand((4, 12, 128), "f16", 7)
    close(shared(pa, b, q.to(DEV), 0.09), *shared_exact(b, q, 0.09, True))


def test_streams_side_by_side(pa):
    parts = []
    for i in range(3):
        b = SharedBatch([(256 + 64 * i, [64, 100, 1, 7])], 2, 128, 16, "bf16", i, [90]).to(DEV)
        parts.append((b, rand((5, 12, 128), "bf16", 50 + i).to(DEV)))
    alone = [shared(pa, b, q, 0.09) for b, q in parts]
    torch.cuda.synchronize()
    outs = []
    for b, q in parts:
        with torch.cuda.stream(torch.cuda.Stream()):
            outs.append([shared(pa, b, q, 0.09) for _ in range(5)])
    torch.cuda.synchronize()
    for a, os_ in zip(alone, outs):
        for o in os_:
            assert torch.equal(a, o)


def test_back_to_back_calls_share_a_workspace(pa):
    """Calls of different sizes on one stream, one scratch for all: none sees what another leaves."""
    parts = []
    for i, (pre, tails) in enumerate(((512, [5] * 20), (16, [300, 2]), (0, [40, 50]), (2048, [0, 9]))):
        b = SharedBatch([(pre, tails)], 4, 128, 16, "bf16", i, [17]).to(DEV)
        parts.append((b, rand((len(b.lens), 16, 128), "bf16", 70 + i).to(DEV)))
    pa.pa_set_option(1, 2)
    size = max(pa.pa_decode_shared_workspace_size(len(b.lens), 1, 16, 4, 128, 16, b.max_context, q.dtype) for b, q in parts)
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(6):
        for b, q in parts:
            out = torch.empty_like(q)
            pa.pa_decode_shared(out, q, b.dk, b.dv, b.dtables, b.dlens, b.dstarts, b.dprefix, b.max_context, 0.09,
                                workspace=ws)
            outs.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        b, q = parts[i % len(parts)]
        assert torch.equal(out, outs[i % len(parts)])
    for (b, q), out in zip(parts, outs):
        close(out, *shared_exact(b, q.cpu(), 0.09, True))
