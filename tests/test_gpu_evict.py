"""pa_evict against a plain ranking: kept tokens, their places, positions and
rows are decisions and moves, so everything is compared bit for bit."""
import numpy as np
import pytest
import torch

from cache_ops import Batch, evict_exact

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


def _bits(t):
    return t.contiguous().view({4: torch.int32, 2: torch.int16, 1: torch.uint8}[t.element_size()])


def _weights(S, hkv, stride, kind, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.exp(2 * torch.randn((S, hkv, stride), generator=g))
    if kind == "ties":
        w = torch.randint(0, 3, (S, hkv, stride), generator=g).float()
    elif kind == "equal":
        w = torch.full_like(w, 0.25)
    elif kind == "signs":
        w = torch.randn((S, hkv, stride), generator=g).mul(2).round() / 2
        w[w == 0] *= torch.where(torch.rand(w[w == 0].shape, generator=g) < 0.5, -1.0, 1.0)
    elif kind == "special":
        for i, x in enumerate((float("nan"), float("inf"), -float("inf"), 0.0, -0.0, 1e-42, -1e-42)):
            w[torch.rand(w.shape, generator=g) < 0.04] = x
    return w


def _run(pa, b, w, keep, sink, recent, new_tables=None, pos=None, rec=None, seen=None, in_place=False, mc=None):
    """(new_lens, weights_out, positions_out) after the call on b's device pools."""
    S, hkv, stride = w.shape
    i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    dw = w.to(DEV)
    wo = dw if in_place else torch.full_like(dw, -7.0)
    dp = None if pos is None else pos.to(DEV)
    po = dp if in_place and dp is not None else torch.full((S, hkv, stride), -9, dtype=torch.int32, device=DEV)
    new_lens = torch.full((S,), -1, dtype=torch.int32, device=DEV)
    nt = b.dtables if new_tables is None else new_tables.to(DEV)
    mc = b.max_context if mc is None else mc
    ws = torch.full((max(16, pa.pa_evict_workspace_size(S, hkv, mc, keep)),), 0xFF, dtype=torch.uint8, device=DEV)
    sc = dict(k_scales=b.dscales[0], v_scales=b.dscales[1]) if b.fp8 else {}
    pa.pa_evict(new_lens, wo, po, dw, b.dk, b.dv, b.dtables, nt, b.dlens, mc, keep, sink, recent, positions=dp,
                recorded_lens=i32(rec), seen_lens=i32(seen), workspace=ws, **sc)
    torch.cuda.synchronize()
    return new_lens.cpu(), wo.cpu(), po.cpu()


def _check(b, w, got, keep, sink, recent, new_tables=None, pos=None, rec=None, seen=None, in_place=False):
    new_lens, wo, po = got
    nt = b.tables if new_tables is None else new_tables
    k, v = b.k.clone(), b.v.clone()
    sc = [x.clone() for x in b.scales] if b.fp8 else []
    wn, pn = w.numpy(), None if pos is None else pos.numpy()
    before_w = w if in_place else torch.full_like(w, -7.0)
    before_p = pos if in_place and pos is not None else torch.full(w.shape, -9, dtype=torch.int32)
    for s, L in enumerate(b.lens):
        n = L if seen is None else seen[s]
        c = 0 if rec is None else rec[s]
        assert int(new_lens[s]) == min(L, keep)
        for h in range(b.hkv):
            src, p = evict_exact(wn[s, h], None if pn is None else pn[s, h], L, n, c, keep, sink, recent)
            m = len(src)
            assert np.array_equal(_bits(wo)[s, h, :m].numpy(), _bits(w)[s, h].numpy()[src]), (s, h)
            assert np.array_equal(po[s, h, :m].numpy(), p), (s, h)
            assert torch.equal(_bits(wo)[s, h, m:], _bits(before_w)[s, h, m:])
            assert torch.equal(po[s, h, m:], before_p[s, h, m:])
            i = np.arange(m)
            fb, tb = b.tables[s].numpy()[src // b.bs], nt[s].numpy()[i // b.bs]
            for pool, old in ((k, b.k), (v, b.v)):
                pool[tb, i % b.bs, h] = old[fb, src % b.bs, h]
            for pool, old in zip(sc, b.scales or []):
                pool[tb, h, i % b.bs] = old[fb, h, src % b.bs]
    assert torch.equal(_bits(b.dk.cpu()), _bits(k)) and torch.equal(_bits(b.dv.cpu()), _bits(v))
    for d, want in zip(b.dscales or [], sc):
        assert torch.equal(_bits(d.cpu()), _bits(want))


CASES = [
    # lens, hkv, hd, bs, dtype, fp8, keep, sink, recent, weights
    ([100, 7, 0, 64, 65, 300], 2, 128, 16, "bf16", False, 64, 4, 16, "spread"),
    ([40, 33, 20], 3, 32, 4, "f32", False, 20, 0, 0, "ties"),
    ([50, 51], 2, 64, 12, "f16", False, 13, 2, 11, "equal"),       # sink + recent == keep
    ([90, 2, 1], 1, 128, 16, "bf16", False, 1, 0, 0, "special"),
    ([200, 150], 4, 128, 16, "bf16", False, 149, 3, 20, "special"),
    ([2500, 1025, 1024], 2, 128, 16, "bf16", False, 1024, 4, 512, "spread"),
    ([5000], 8, 64, 64, "f16", False, 700, 1, 0, "ties"),
    ([37, 80], 2, 7, 1, "f32", False, 30, 0, 1, "signs"),          # 28-byte rows
    ([33, 40], 2, 5, 16, "bf16", False, 17, 0, 5, "spread"),       # 10-byte rows
    ([600, 90, 91], 8, 128, 16, "bf16", True, 90, 2, 30, "ties"),
    ([64, 65], 3, 33, 8, "bf16", True, 40, 0, 0, "spread"),        # 33-byte rows of codes
    ([20000, 9000], 1, 8, 32, "bf16", False, 3000, 4, 200, "ties"),
    ([60000, 100], 1, 8, 64, "f16", False, 5000, 4, 200, "ties"),   # past the keys that shared memory holds
    ([60000], 1, 8, 64, "f16", False, 50000, 0, 1000, "special"),
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("how", ["in_place", "fresh", "mixed"])
def test_evict(pa, case, how):
    lens, hkv, hd, bs, dtype, fp8, keep, sink, recent, kind = case
    width = -(-min(max(lens), keep) // bs)
    b = Batch(lens, hkv, hd, bs, dtype, 11, fp8, extra_blocks=width * len(lens)).to(DEV)
    nt = b.tables[:, :width].clone()
    first = b.num_blocks - width * len(lens)
    for s in range(len(lens)):
        for j in range(width):
            if how == "fresh" or (how == "mixed" and (s + j) % 2):
                nt[s, j] = first + s * width + j
    w = _weights(len(lens), hkv, max(lens) + 3, kind, 5)
    got = _run(pa, b, w, keep, sink, recent, nt, in_place=how == "in_place")
    _check(b, w, got, keep, sink, recent, nt, in_place=how == "in_place")


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("keep", [40, 25])
def test_evict_again(pa, keep, in_place):
    """A second eviction: recorded positions in any order, tokens appended since, a smaller budget."""
    lens, rec, seen = [60, 41, 40, 30], [40, 40, 40, 10], [200, 141, 40, 30]
    b = Batch(lens, 2, 128, 16, "bf16", 13).to(DEV)
    g = torch.Generator().manual_seed(3)
    w = _weights(4, 2, 64, "ties", 6)
    pos = torch.full((4, 2, 64), 12345, dtype=torch.int32)
    for s in range(4):
        for h in range(2):
            pos[s, h, : rec[s]] = torch.randperm(seen[s] - (lens[s] - rec[s]), generator=g)[: rec[s]].to(torch.int32)
    got = _run(pa, b, w, keep, 3, 20, pos=pos, rec=rec, seen=seen, in_place=in_place)
    _check(b, w, got, keep, 3, 20, pos=pos, rec=rec, seen=seen, in_place=in_place)


def test_evict_shared_blocks(pa):
    """Two sequences over one prompt's blocks, evicted into blocks of their own."""
    b = Batch([80, 80], 2, 128, 16, "bf16", 13, extra_blocks=6)
    b.tables[1] = b.tables[0]
    b.to(DEV)
    nt = torch.arange(b.num_blocks - 6, b.num_blocks, dtype=torch.int32).view(2, 3)
    w = _weights(2, 2, 80, "spread", 6)
    got = _run(pa, b, w, 40, 2, 8, nt)
    _check(b, w, got, 40, 2, 8, nt)


def test_evict_wide_max_context_and_no_positions(pa):
    """max_context far above the lengths; positions_out left out; nothing to drop at all."""
    b = Batch([30, 12], 2, 64, 16, "bf16", 13).to(DEV)
    w = _weights(2, 2, 5000, "spread", 6)
    got = _run(pa, b, w, 20, 0, 4, mc=5000)
    _check(b, w, got, 20, 0, 4)
    b = Batch([30, 12], 2, 64, 16, "bf16", 13).to(DEV)
    new_lens = torch.zeros(2, dtype=torch.int32, device=DEV)
    dw = w.to(DEV)
    pa.pa_evict(new_lens, dw, None, dw, b.dk, b.dv, b.dtables, b.dtables, b.dlens, 30, 30, 0, 0)
    assert new_lens.tolist() == [30, 12] and torch.equal(dw.cpu(), w)
    assert torch.equal(_bits(b.dk.cpu()), _bits(b.k))


def test_evict_graph(pa):
    """Captured once, replayed with other weights: the same as an eager call."""
    b = Batch([700, 90, 513], 2, 128, 16, "bf16", 13, extra_blocks=3 * 32).to(DEV)
    nt = torch.arange(b.num_blocks - 96, b.num_blocks, dtype=torch.int32).view(3, 32).to(DEV)
    S, stride = 3, 700
    dw = torch.empty((S, 2, stride), device=DEV)
    outs = []
    ws = torch.empty(pa.pa_evict_workspace_size(S, 2, 700, 512), dtype=torch.uint8, device=DEV)
    for _ in range(2):
        outs.append((torch.zeros(S, dtype=torch.int32, device=DEV), torch.zeros_like(dw),
                     torch.zeros(dw.shape, dtype=torch.int32, device=DEV)))

    def call(o):
        pa.pa_evict(*o, dw, b.dk, b.dv, b.dtables, nt, b.dlens, 700, 512, 4, 100, workspace=ws)

    dw.copy_(_weights(S, 2, stride, "spread", 1))
    call(outs[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        call(outs[0])
    for seed in (2, 3):
        dw.copy_(_weights(S, 2, stride, "spread", seed))
        g.replay()
        torch.cuda.synchronize()
        pools = b.dk.clone(), b.dv.clone()
        call(outs[1])
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(*outs))
        assert torch.equal(_bits(pools[0]), _bits(b.dk)) and torch.equal(_bits(pools[1]), _bits(b.dv))


def test_evict_check_mode(pa):
    """A block written for one sequence and read by another, a block given twice, lengths that do not fit."""
    b = Batch([80, 80], 2, 64, 16, "bf16", 13, extra_blocks=6).to(DEV)
    w = _weights(2, 2, 80, "spread", 6)
    fresh = torch.arange(b.num_blocks - 6, b.num_blocks, dtype=torch.int32).view(2, 3)
    pa.pa_set_check_mode(True)
    try:
        for bad in ("read", "twice", "range"):
            nt = fresh.clone()
            if bad == "read":
                nt[0, 0] = b.tables[1, 0]
            elif bad == "twice":
                nt[0, 0] = nt[1, 1]
            else:
                nt[1, 2] = b.num_blocks
            with pytest.raises(pa.PAError) as e:
                _run(pa, b, w, 40, 2, 8, nt)
            assert e.value.status == 3
        pos = torch.zeros((2, 2, 80), dtype=torch.int32)
        for rec, seen in (([81, 0], [90, 90]), ([10, 10], [79, 90])):
            with pytest.raises(pa.PAError) as e:
                _run(pa, b, w, 40, 2, 8, fresh, pos=pos, rec=rec, seen=seen)
            assert e.value.status == 3
        got = _run(pa, b, w, 40, 2, 8, fresh)
    finally:
        pa.pa_set_check_mode(False)
    _check(b, w, got, 40, 2, 8, fresh)
