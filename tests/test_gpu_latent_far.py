"""The latent-cache and shared-prefix operators where sizes are far out: pools
whose offsets pass 32 bits, a million tokens of context, bounds on lengths far
above the lengths, scales of nothing."""
import pytest
import torch

from latent_ops import LatentBatch, SharedBatch, attention, close, latent_exact, rand, shared_exact

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
DECODE, VARLEN = 1, 3  # the options that pin a kernel


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    yield pa
    torch.cuda.empty_cache()


@pytest.fixture(autouse=True)
def _unpinned(pa):
    yield
    pa.pa_set_option(DECODE, 0)
    pa.pa_set_option(VARLEN, 0)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _decode(pa, q, cache, tables, lens, ctx, scale):
    out = torch.full((*q.shape[:2], 512), float("nan"), dtype=q.dtype, device=DEV)
    size = pa.pa_latent_decode_workspace_size(q.shape[0], q.shape[1], 512, 64, cache.shape[1], ctx, q.dtype)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    pa.pa_latent_decode(out, q, cache, tables, lens, ctx, scale, workspace=ws)
    return out


def _varlen(pa, q, cache, tables, lens, cu, ctx, scale, causal):
    out = torch.full((*q.shape[:2], 512), float("nan"), dtype=q.dtype, device=DEV)
    max_q = max(b - a for a, b in zip(cu, cu[1:]))
    size = pa.pa_latent_varlen_workspace_size(len(cu) - 1, q.shape[0], max_q, q.shape[1], 512, 64, cache.shape[1], ctx,
                                              q.dtype)
    ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    pa.pa_latent_varlen(out, q, cache, tables, lens, _i32(cu), max_q, ctx, scale, causal=causal, workspace=ws)
    return out


@pytest.mark.parametrize("bs,dtype", [(16, "bf16"), (6, "f16"), (1, "bf16"), (16, "f32")])
def test_latent_pools_beyond_32_bits(pa, bs, dtype):
    """The same blocks at the two ends of a pool of 2.2 G elements give the same bits."""
    b = LatentBatch([300, 77], 512, 64, bs, dtype, 3).to(DEV)
    n, far = b.num_blocks, 2_200_000_000 // (576 * bs)
    assert (far - n) * bs * 576 > 2 ** 31
    q = rand((2, 16, 576), dtype, 4).to(DEV)
    new = rand((20, 16, 576), dtype, 5).to(DEV)
    pool = torch.empty((far, bs, 576), dtype=q.dtype, device=DEV)
    pool[far - n:] = b.dcache
    moved = torch.where(b.dtables >= 0, b.dtables + (far - n), b.dtables)
    cu = [0, 13, 20]
    for kernel in (1, 2) if dtype != "f32" else (0,):
        pa.pa_set_option(DECODE, kernel)
        pa.pa_set_option(VARLEN, kernel)
        near = _decode(pa, q, b.dcache, b.dtables, b.dlens, b.max_context, 0.07)
        assert torch.isfinite(near).all()
        assert torch.equal(near, _decode(pa, q, pool, moved, b.dlens, b.max_context, 0.07))
        near = _varlen(pa, new, b.dcache, b.dtables, b.dlens, cu, b.max_context, 0.07, True)
        assert torch.isfinite(near).all()
        assert torch.equal(near, _varlen(pa, new, pool, moved, b.dlens, cu, b.max_context, 0.07, True))
    # and rows written there
    kv, pos = rand((20, 576), dtype, 6).to(DEV), torch.arange(20, device=DEV)
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).to(DEV)
    small = torch.zeros((32, 1, 576), dtype=q.dtype, device=DEV)
    pa.pa_latent_write(kv, pos, inv, pos, small)
    pa.pa_latent_write(kv, pos, inv, far * bs - 20 + pos, pool)
    assert torch.equal(small[:20, 0], pool.view(-1, 576)[-20:])


def test_shared_pools_beyond_32_bits(pa):
    b = SharedBatch([(256, [5, 0, 40]), (64, [9, 200])], 8, 128, 16, "bf16", 3, loners=[70]).to(DEV)
    S, n, far = len(b.lens), b.num_blocks, 2_200_000_000 // (16 * 8 * 128)
    q = rand((S, 32, 128), "bf16", 4).to(DEV)
    pools = [torch.empty((far, 16, 8, 128), dtype=q.dtype, device=DEV) for _ in range(2)]
    for pool, small in zip(pools, (b.dk, b.dv)):
        pool[far - n:] = small
    moved = torch.where(b.dtables >= 0, b.dtables + (far - n), b.dtables)
    pa.pa_set_option(DECODE, 2)
    size = pa.pa_decode_shared_workspace_size(S, 2, 32, 8, 128, 16, b.max_context, q.dtype)
    ws, outs = torch.empty(size, dtype=torch.uint8, device=DEV), []
    for k, v, t in ((b.dk, b.dv, b.dtables), (*pools, moved)):
        outs.append(torch.full_like(q, float("nan")))
        pa.pa_decode_shared(outs[-1], q, k, v, t, b.dlens, b.dstarts, b.dprefix, b.max_context, 0.07, workspace=ws)
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)


@pytest.mark.parametrize("op", ["decode", "varlen", "shared"])
def test_a_million_tokens(pa, op):
    """One block over and over: attention over its 16 tokens.  A piece of the work is at most the tiles of one of 70 SM
    pairs or more (7,813 / 70 + 1 of 128 tokens; shared: of one SM), each added in 8 products of 16 tokens, and 152
    pieces are joined at most: no sum is deeper than 8 * 113 + 17 + 152."""
    L = 1_000_000
    deep = 2 * (8 * 113 + 17 + 152) * 2.0 ** -23
    seen = torch.ones((1, 16), dtype=torch.bool)
    if op == "shared":
        k, v = rand((1, 16, 1, 128), "bf16", 1), rand((1, 16, 1, 128), "bf16", 2)
        q = rand((4, 8, 128), "bf16", 3)
        rest = 16 * 40
        tables = torch.zeros((4, (L + rest) // 16), dtype=torch.int32, device=DEV)
        lens = [L + rest] * 4
        out = torch.full_like(q, float("nan"), device=DEV)
        pa.pa_set_option(DECODE, 2)
        size = pa.pa_decode_shared_workspace_size(4, 1, 8, 1, 128, 16, L + rest, q.dtype)
        ws = torch.empty(size, dtype=torch.uint8, device=DEV)
        pa.pa_decode_shared(out, q.to(DEV), k.to(DEV), v.to(DEV), tables, _i32(lens), _i32([0, 4]), _i32([L]), L + rest,
                            0.09, workspace=ws)
        rows, keys, values = q.view(-1, 128), k.view(16, 128), v.view(16, 128)
        exact, bound = attention(rows, keys, values, 0.09, seen, "bf16", True)
    else:
        cache = rand((1, 16, 576), "bf16", 1)
        q = rand((1 if op == "decode" else 3, 16, 576), "bf16", 2)
        tables = torch.zeros((1, L // 16), dtype=torch.int32, device=DEV)
        if op == "decode":
            out = _decode(pa, q.to(DEV), cache.to(DEV), tables, _i32([L]), L, 0.07)
        else:
            out = _varlen(pa, q.to(DEV), cache.to(DEV), tables, _i32([L]), [0, 3], L, 0.07, False)
        rows, keys, values = q.view(-1, 576), cache[0], cache[0, :, :512]
        exact, bound = attention(rows, keys, values, 0.07, seen, "bf16", True)
    x = torch.softmax(rows.double() @ keys.double().t() * (0.09 if op == "shared" else 0.07), -1)
    close(out.view(exact.shape), exact, bound + deep * (x @ values.double().abs()))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_a_bound_far_above_the_lengths(pa, dtype):
    b = LatentBatch([300, 0, 7], 512, 64, 16, dtype, 3).to(DEV)
    q = rand((3, 4, 576), dtype, 4)
    out = _decode(pa, q.to(DEV), b.dcache, b.dtables, b.dlens, 2 ** 31 - 1, 0.07)
    close(out, *latent_exact(b, q, None, 0.07, True, dtype != "f32"))
    q = rand((8, 4, 576), dtype, 5)
    out = _varlen(pa, q.to(DEV), b.dcache, b.dtables, b.dlens, [0, 5, 5, 8], 2 ** 31 - 1, 0.07, True)
    close(out, *latent_exact(b, q, [0, 5, 5, 8], 0.07, True, dtype != "f32"))


@pytest.mark.parametrize("scale", [0.0, 1e-30, -0.05])
def test_scales_of_nothing_and_below(pa, scale):
    b = LatentBatch([300, 17, 129], 512, 64, 16, "bf16", 3).to(DEV)
    q = rand((3, 16, 576), "bf16", 4)
    for kernel in (1, 2):
        pa.pa_set_option(DECODE, kernel)
        out = _decode(pa, q.to(DEV), b.dcache, b.dtables, b.dlens, b.max_context, scale)
        close(out, *latent_exact(b, q, None, scale, True, kernel == 2))
    s = SharedBatch([(256, [5, 0, 40])], 2, 128, 16, "bf16", 3).to(DEV)
    q = rand((3, 8, 128), "bf16", 4)
    size = pa.pa_decode_shared_workspace_size(3, 1, 8, 2, 128, 16, s.max_context, q.dtype)
    ws, out = torch.empty(size, dtype=torch.uint8, device=DEV), torch.full_like(q, float("nan"), device=DEV)
    pa.pa_decode_shared(out, q.to(DEV), s.dk, s.dv, s.dtables, s.dlens, s.dstarts, s.dprefix, s.max_context, scale,
                        workspace=ws)
    close(out, *shared_exact(s, q, scale, True))
