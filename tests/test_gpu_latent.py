"""pa_latent_decode and pa_latent_varlen against attention in 64 bits; bounds in
latent_ops.attention."""
import pytest
import torch

from cache_ops import DTYPES
from latent_ops import LatentBatch, close, latent_exact, rand

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
OPT = {"decode": 1, "varlen": 3}


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    yield pa
    for o in OPT.values():
        pa.pa_set_option(o, 0)


def _tensor_cores(b):
    return b.dtype != "f32" and (b.lat, b.rot) == (512, 64)


def decode(pa, b, q, scale, out=None, ws_fill=0xFF, stream=None):
    S, H, _ = q.shape
    if out is None:
        out = torch.full((S, H, b.lat), float("nan"), dtype=q.dtype, device=DEV)
    size = pa.pa_latent_decode_workspace_size(S, H, b.lat, b.rot, b.bs, b.max_context, q.dtype)
    ws = torch.full((max(16, size),), ws_fill, dtype=torch.uint8, device=DEV)
    pa.pa_latent_decode(out, q, b.dcache, b.dtables, b.dlens, b.max_context, scale, workspace=ws, stream=stream)
    return out


def varlen(pa, b, q, cu, scale, causal, out=None):
    T, H, _ = q.shape
    if out is None:
        out = torch.full((T, H, b.lat), float("nan"), dtype=q.dtype, device=DEV)
    max_q = max(cu[i + 1] - cu[i] for i in range(len(cu) - 1))
    size = pa.pa_latent_varlen_workspace_size(len(b.lens), T, max_q, H, b.lat, b.rot, b.bs, b.max_context, q.dtype)
    ws = torch.full((max(16, size),), 0xFF, dtype=torch.uint8, device=DEV)
    pa.pa_latent_varlen(out, q, b.dcache, b.dtables, b.dlens, torch.tensor(cu, dtype=torch.int32, device=DEV), max_q,
                        b.max_context, scale, causal=causal, workspace=ws)
    return out


DECODE = [
    # lens, heads, lat, rot, bs, dtype
    ([1], 16, 512, 64, 16, "bf16"),
    ([1, 0, 64, 65, 127, 128, 129, 300], 16, 512, 64, 16, "bf16"),
    ([5, 1999, 40], 128, 512, 64, 16, "bf16"),
    ([700, 3, 0, 256], 20, 512, 64, 8, "f16"),
    ([13, 250], 1, 512, 64, 32, "bf16"),
    ([1000, 90], 200, 512, 64, 64, "f16"),          # more heads than a tile has rows
    ([333, 128, 17], 64, 512, 64, 48, "bf16"),
    ([2100], 40, 512, 64, 128, "f16"),
    ([400, 31], 8, 512, 64, 256, "bf16"),
    ([100] * 97 + [777], 16, 512, 64, 16, "bf16"),   # more units than SM pairs
    ([4000, 4100], 32, 512, 64, 16, "f16"),          # a unit in many pieces
    ([130, 7, 300], 16, 512, 64, 12, "bf16"),        # boxes of four rows
    ([257, 66], 40, 512, 64, 4, "f16"),
    ([140, 501], 24, 512, 64, 24, "bf16"),
    ([130, 7], 16, 512, 64, 6, "bf16"),              # boxes of two rows
    ([129, 500, 0, 64], 128, 512, 64, 10, "f16"),
    ([90, 0, 5], 7, 512, 64, 1, "f16"),              # boxes of one row
    ([128, 1, 1100, 33, 95], 130, 512, 64, 1, "bf16"),
    ([63, 400], 16, 512, 64, 7, "bf16"),
    ([100] * 90 + [515], 16, 512, 64, 2, "bf16"),
    ([150, 64], 16, 512, 64, 16, "f32"),
    ([70, 33], 9, 96, 32, 16, "bf16"),
    ([70, 33], 3, 50, 0, 4, "f32"),
    ([20], 5, 256, 32, 16, "f16"),
    ([3000], 4, 512, 64, 16, "f32"),                 # CUDA cores, a row's keys in pieces
    ([900, 0, 1, 70], 6, 96, 32, 4, "f16"),
    ([600, 0, 33], 37, 512, 64, 16, "f32"),          # several CTAs of heads, the last one short
    ([77, 8, 1], 12, 300, 13, 16, "bf16"),           # rows that are no vectors
    ([40, 515], 8, 129, 0, 3, "f32"),
    ([200, 9], 1, 512, 64, 16, "f32"),
]


@pytest.mark.parametrize("lens,heads,lat,rot,bs,dtype", DECODE)
def test_decode(pa, lens, heads, lat, rot, bs, dtype):
    b = LatentBatch(lens, lat, rot, bs, dtype, 7).to(DEV)
    q = rand((len(lens), heads, lat + rot), dtype, 8)
    scale = (128 + rot) ** -0.5
    out = decode(pa, b, q.to(DEV), scale)
    close(out, *latent_exact(b, q, None, scale, True, _tensor_cores(b)))
    for s, L in enumerate(lens):
        if L == 0:
            assert (out[s] == 0).all()
    assert pa.lib().pa_device_status(1) == 0


VARLEN = [
    # (new, context) per request, heads, bs, dtype, causal
    ([(1, 1), (5, 5), (0, 20), (64, 300), (129, 129)], 16, 16, "bf16", True),
    ([(3, 130), (1, 500), (0, 0), (40, 128)], 20, 8, "f16", True),
    ([(17, 140), (1, 128), (9, 9)], 128, 64, "bf16", True),
    ([(17, 140), (1, 128), (9, 9)], 24, 16, "bf16", False),
    ([(300, 700)], 8, 32, "f16", True),
    ([(2, 1000), (700, 700)], 1, 16, "bf16", True),
    ([(5, 77)], 200, 48, "bf16", True),
    ([(4, 20), (6, 6), (70, 200)], 6, 4, "bf16", True),
    ([(4, 20), (6, 6)], 6, 3, "bf16", True),          # boxes of one row
    ([(300, 333), (1, 258)], 16, 1, "bf16", True),
    ([(70, 201), (129, 129)], 24, 14, "f16", True),   # boxes of two rows
    ([(30, 100), (1, 3)], 5, 16, "f32", True),
    ([(30, 100), (1, 3)], 5, 16, "f32", False),
]


@pytest.mark.parametrize("reqs,heads,bs,dtype,causal", VARLEN)
def test_varlen(pa, reqs, heads, bs, dtype, causal):
    lens, cu = [L for _, L in reqs], [0]
    for n, _ in reqs:
        cu.append(cu[-1] + n)
    b = LatentBatch(lens, 512, 64, bs, dtype, 17).to(DEV)
    q = rand((cu[-1], heads, 576), dtype, 18)
    scale = 192 ** -0.5
    out = varlen(pa, b, q.to(DEV), cu, scale, causal)
    close(out, *latent_exact(b, q, cu, scale, causal, _tensor_cores(b)))
    assert pa.lib().pa_device_status(1) == 0


def test_rows_behind_the_last_request_stay(pa):
    for dtype in ("bf16", "f32"):
        b = LatentBatch([20, 500], 512, 64, 16, dtype, 3).to(DEV)
        q = rand((40, 16, 576), dtype, 4)
        out = torch.full((40, 16, 512), 3.0, dtype=q.dtype, device=DEV)
        varlen(pa, b, q.to(DEV), [0, 7, 30], 0.07, True, out=out)
        assert (out[30:] == 3).all()
        exact, bound = latent_exact(b, q[:30], [0, 7, 30], 0.07, True, _tensor_cores(b))
        close(out[:30], exact, bound)


def test_relabelled_blocks_give_the_same_bits(pa):
    b = LatentBatch([500, 129, 64], 512, 64, 16, "bf16", 5).to(DEV)
    q = rand((3, 32, 576), "bf16", 6).to(DEV)
    first = decode(pa, b, q, 0.07)
    perm = torch.randperm(b.num_blocks, generator=torch.Generator().manual_seed(9))
    cache = torch.empty_like(b.cache)
    cache[perm] = b.cache
    tables = torch.where(b.tables >= 0, perm[b.tables.long().clamp(min=0)].int(), b.tables)
    b.dcache, b.dtables = cache.to(DEV), tables.to(DEV)
    assert torch.equal(first, decode(pa, b, q, 0.07, ws_fill=0))


def test_large_scores_and_growing_maxima(pa):
    """Scores of hundreds, the largest ones last: the running maximum moves by much more than its slack, tile by tile."""
    for dtype in ("bf16", "f16"):
        b = LatentBatch([700, 1500], 512, 64, 16, dtype, 5)
        for s, L in enumerate(b.lens):
            for t in range(L):
                b.cache[b.tables[s, t // 16].long(), t % 16] *= 0.2 + 1.5 * t / L
        b.k = b.cache[:, :, None]
        b.to(DEV)
        q = rand((2, 16, 576), dtype, 6, 2.0)
        out = decode(pa, b, q.to(DEV), 0.3)
        close(out, *latent_exact(b, q, None, 0.3, True, True))
        out = decode(pa, b, q.to(DEV), -0.3)
        close(out, *latent_exact(b, q, None, -0.3, True, True))


def test_graph_replays_follow_new_queries_and_lengths(pa):
    b = LatentBatch([300, 1000, 64], 512, 64, 16, "bf16", 5).to(DEV)
    q = rand((3, 16, 576), "bf16", 6).to(DEV)
    out = torch.zeros((3, 16, 512), dtype=torch.bfloat16, device=DEV)
    ws = torch.zeros(pa.pa_latent_decode_workspace_size(3, 16, 512, 64, 16, b.max_context, q.dtype), dtype=torch.uint8,
                     device=DEV)
    run = lambda: pa.pa_latent_decode(out, q, b.dcache, b.dtables, b.dlens, b.max_context, 0.07, workspace=ws)  # noqa: E731
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for lens in ([300, 1000, 64], [1, 999, 0], [17, 3, 60]):
        q.copy_(rand((3, 16, 576), "bf16", sum(lens)))
        b.dlens.copy_(torch.tensor(lens, dtype=torch.int32))
        out.fill_(9)
        graph.replay()
        got = out.clone()
        run()
        assert torch.equal(got, out)
        b.lens = lens
        close(out, *latent_exact(b, q.cpu(), None, 0.07, True, True))


def test_streams_side_by_side(pa):
    parts = []
    for i in range(3):
        b = LatentBatch([400 + 100 * i, 77], 512, 64, 16, "bf16", i).to(DEV)
        parts.append((b, rand((2, 16, 576), "bf16", 50 + i)))
    alone = [decode(pa, b, q.to(DEV), 0.07) for b, q in parts]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in parts]
    qs = [q.to(DEV) for _, q in parts]
    torch.cuda.synchronize()
    outs = []
    for (b, _), q, st in zip(parts, qs, streams):
        with torch.cuda.stream(st):
            outs.append([decode(pa, b, q, 0.07) for _ in range(5)])
    torch.cuda.synchronize()
    for a, os_ in zip(alone, outs):
        for o in os_:
            assert torch.equal(a, o)


@pytest.mark.parametrize("op", ["decode", "varlen"])
def test_both_kernels_agree(pa, op):
    b = LatentBatch([129, 300], 512, 64, 16, "bf16", 2).to(DEV)
    cu = [0, 1, 2] if op == "decode" else [0, 40, 41]
    q = rand((cu[-1], 16, 576), "bf16", 3)
    for kernel in (1, 2):
        pa.pa_set_option(OPT[op], kernel)
        try:
            out = decode(pa, b, q.to(DEV), 0.07) if op == "decode" else varlen(pa, b, q.to(DEV), cu, 0.07, True)
        finally:
            pa.pa_set_option(OPT[op], 0)
        close(out, *latent_exact(b, q, cu, 0.07, True, kernel == 2))


def test_more_sequences_than_a_launch_lists(pa):
    S = 2600
    lens = [1 + (i * 7) % 40 for i in range(S)]
    b = LatentBatch(lens, 512, 64, 16, "bf16", 2).to(DEV)
    q = rand((S, 2, 576), "bf16", 3)
    close(decode(pa, b, q.to(DEV), 0.07), *latent_exact(b, q, None, 0.07, True, True))
    cu = list(range(S + 1))
    close(varlen(pa, b, q.to(DEV), cu, 0.07, True), *latent_exact(b, q, cu, 0.07, True, True))


def test_back_to_back_calls_share_a_workspace(pa):
    """Prompts and single tokens of different sizes on one stream with one scratch: none sees what another leaves."""
    parts, size = [], 0
    for i, (new, lens) in enumerate((([1] * 4, [900, 5, 64, 333]), ([70, 3], [70, 500]), ([1], [1]), ([300], [300]))):
        b = LatentBatch(lens, 512, 64, 16, "bf16", i).to(DEV)
        cu = [0]
        for n in new:
            cu.append(cu[-1] + n)
        parts.append((b, cu, rand((cu[-1], 24, 576), "bf16", 70 + i).to(DEV)))
        size = max(size, pa.pa_latent_varlen_workspace_size(len(lens), cu[-1], max(new), 24, 512, 64, 16, b.max_context,
                                                            torch.bfloat16))
    ws = torch.empty(size, dtype=torch.uint8, device=DEV)
    outs = []
    for _ in range(6):
        for b, cu, q in parts:
            out = torch.empty((q.shape[0], 24, 512), dtype=q.dtype, device=DEV)
            if cu == list(range(len(cu))):
                pa.pa_latent_decode(out, q, b.dcache, b.dtables, b.dlens, b.max_context, 0.07, workspace=ws)
            else:
                pa.pa_latent_varlen(out, q, b.dcache, b.dtables, b.dlens, torch.tensor(cu, dtype=torch.int32, device=DEV),
                                    max(b_ - a for a, b_ in zip(cu, cu[1:])), b.max_context, 0.07, workspace=ws)
            outs.append(out)
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        assert torch.equal(out, outs[i % len(parts)])
    for (b, cu, q), out in zip(parts, outs):
        close(out, *latent_exact(b, q.cpu(), cu, 0.07, True, True))


def test_infinite_and_nan_tokens_reach_only_who_sees_them(pa):
    """A NaN row of one sequence, and one of a token that comes after the query: the other sequences, and earlier rows
    whose tiles do not hold it, are what they are without it."""
    b = LatentBatch([300, 300], 512, 64, 16, "bf16", 2)
    q = rand((2, 16, 576), "bf16", 3)
    clean = decode(pa, b.to(DEV), q.to(DEV), 0.07)
    b.dcache[b.tables[0, 3].long(), 5] = float("nan")
    out = decode(pa, b, q.to(DEV), 0.07)
    assert torch.isnan(out[0].float()).all() and torch.equal(out[1], clean[1])
