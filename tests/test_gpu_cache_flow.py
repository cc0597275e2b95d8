"""The cache-side operators together, as a long-context server uses them: a
prompt is rotated into the cache, attended, weighed and pruned; then tokens are
generated one by one, each rotated in, attended with the weights kept, and the
cache brought back to its budget every few steps.

The oracle keeps, per (sequence, KV head), the list of held tokens with their
positions, stored rows and weights, and works in 64 bits.  It follows the
device's evictions only through the weights, which it checks first: a token
is expected to go where the device's own fp32 weights (read back) say, since a
64-bit weight may order two nearly equal tokens the other way."""
import numpy as np
import pytest
import torch

from cache_ops import DTYPES, EPS, evict_exact, rope, softmax_rows, weight_rtol
from helpers import ATOL, RTOL

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


@pytest.mark.parametrize("dtype, hq, hkv, hd, bs, fp8", [("bf16", 8, 2, 128, 16, False), ("f32", 4, 2, 32, 4, False),
                                                         ("f16", 6, 2, 128, 16, True)])
def test_prompt_prune_generate_evict(pa, dtype, hq, hkv, hd, bs, fp8):
    S, keep, sink, recent, every, steps = 3, 48, 2, 20, 5, 12
    prompt = [150, 97, 30]
    td, G, scale = DTYPES[dtype], hq // hkv, hd ** -0.5
    mc = max(prompt)
    g = torch.Generator().manual_seed(5)
    width = -(-mc // bs)
    nb = S * width
    tables = torch.randperm(nb, generator=g).to(torch.int32).view(S, width)
    half = hd // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    dinv, dtab = inv.to(DEV), tables.to(DEV)
    pool = torch.uint8 if fp8 else td
    kc, vc = (torch.zeros((nb, bs, hkv, hd), dtype=pool, device=DEV) for _ in range(2))
    sc = [torch.zeros((nb, hkv, bs), device=DEV) for _ in range(2)] if fp8 else []
    scales = dict(k_scales=sc[0], v_scales=sc[1]) if fp8 else {}
    w = torch.zeros((S, hkv, mc), device=DEV)
    pos = torch.zeros((S, hkv, mc), dtype=torch.int32, device=DEV)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731

    def rows(which, s, h, n):
        """The first n rows of head h of sequence s as the device holds them, in 64 bits."""
        t = tables[s, : -(-n // bs)].long()
        x = (kc, vc)[which].cpu()[t, :, h]
        if fp8:
            x = x.view(torch.float8_e4m3fn).double() * sc[which].cpu()[t, h].double()[..., None]
        return x.double().reshape(-1, hd)[:n]

    def write(q, k, v, positions, seqs, idx):
        """Rotated q; k (rotated) and v of token i go to index idx[i] of sequence seqs[i]."""
        slots = torch.tensor([int(tables[s, j // bs]) * bs + j % bs for s, j in zip(seqs, idx)], device=DEV)
        out = torch.empty_like(q)
        args = (out, q, k, v, torch.tensor([positions], device=DEV), dinv, slots)
        if fp8:
            pa.pa_rope_write_kv_fp8(*args, kc, vc, *sc)
        else:
            pa.pa_rope_write_kv(*args, kc, vc)
        want = rope(q.cpu(), torch.tensor([positions]), inv, None, False)
        assert float((out.cpu().double() - want).abs().max()) <= 2 * EPS[dtype] * float(want.abs().max()) + 2e-6
        return out

    def evict(lens, recorded, seen):
        before = [(rows(0, s, h, lens[s]), rows(1, s, h, lens[s])) for s in range(S) for h in range(hkv)]
        wb, pb = w.cpu().numpy(), pos.cpu().numpy()
        new = torch.empty(S, dtype=torch.int32, device=DEV)
        ws = torch.empty(max(16, pa.pa_evict_workspace_size(S, hkv, mc, keep)), dtype=torch.uint8, device=DEV)
        pa.pa_evict(new, w, pos, w, kc, vc, dtab, dtab, i32(lens), mc, keep, sink, recent, positions=pos,
                    recorded_lens=i32(recorded), seen_lens=i32(seen), workspace=ws, **scales)
        got = new.tolist()
        for s in range(S):
            assert got[s] == min(lens[s], keep)
            for h in range(hkv):
                src, p = evict_exact(wb[s, h], pb[s, h], lens[s], seen[s], recorded[s], keep, sink, recent)
                assert np.array_equal(pos[s, h, : got[s]].cpu().numpy(), p)
                k0, v0 = before[s * hkv + h]
                assert torch.equal(rows(0, s, h, got[s]), k0[src]) and torch.equal(rows(1, s, h, got[s]), v0[src])
                assert np.array_equal(w[s, h, : got[s]].cpu().numpy(), wb[s, h][src])
        return got

    # the prompts
    T = sum(prompt)
    q, k, v = (torch.randn((T, n, hd), generator=g).to(td).to(DEV) for n in (hq, hkv, hkv))
    seqs = [s for s in range(S) for _ in range(prompt[s])]
    idx = [j for s in range(S) for j in range(prompt[s])]
    rq = write(q, k, v, idx, seqs, idx)
    cu = [0] + list(np.cumsum(prompt))
    size = pa.pa_prompt_weights_fp8_workspace_size if fp8 else pa.pa_prompt_weights_workspace_size
    ws = torch.empty(size(S, T, mc, hq, hkv, hd, bs, mc, 0, td), dtype=torch.uint8, device=DEV)
    if fp8:
        pa.pa_prompt_weights_fp8(w, rq, kc, sc[0], dtab, i32(prompt), i32(cu), mc, mc, 0, scale, workspace=ws)
    else:
        pa.pa_prompt_weights(w, rq, kc, dtab, i32(prompt), i32(cu), mc, mc, 0, scale, workspace=ws)
    for s in range(S):
        L = prompt[s]
        seen_mask = torch.arange(L)[:, None] >= torch.arange(L)
        for h in range(hkv):
            want, rt = torch.zeros(L, dtype=torch.float64), 0.0
            for j in range(G):
                p, mag = softmax_rows(rq[cu[s]:cu[s + 1], h * G + j].cpu(), rows(0, s, h, L), scale, seen_mask)
                want += p.sum(0)
                rt = max(rt, weight_rtol(hd, mag, L, L * G))
            assert bool(((w[s, h, :L].cpu().double() - want).abs() <= rt * want).all())
    lens = evict(prompt, [0] * S, prompt)
    recorded, seen = list(lens), list(prompt)

    # generation
    size = pa.pa_decode_weights_fp8_workspace_size if fp8 else pa.pa_decode_weights_workspace_size
    ws = torch.empty(size(S, hq, hkv, hd, bs, mc, td), dtype=torch.uint8, device=DEV)
    for step in range(steps):
        q, k, v = (torch.randn((S, n, hd), generator=g).to(td).to(DEV) for n in (hq, hkv, hkv))
        rq = write(q, k, v, seen, list(range(S)), lens)
        lens = [x + 1 for x in lens]
        seen = [x + 1 for x in seen]
        out = torch.empty_like(q)
        old = w.cpu().double()
        if fp8:
            pa.pa_decode_weights_fp8(out, w, rq, kc, vc, *sc, dtab, i32(lens), mc, scale, workspace=ws)
        else:
            pa.pa_decode_weights(out, w, rq, kc, vc, dtab, i32(lens), mc, scale, workspace=ws)
        got, ow = w.cpu().double(), out.cpu().double()
        for s in range(S):
            L = lens[s]
            for h in range(hkv):
                p, mag = softmax_rows(rq[s, h * G:(h + 1) * G].cpu(), rows(0, s, h, L), scale,
                                      torch.ones((G, L), dtype=torch.bool))
                o = p @ rows(1, s, h, L)
                err = (ow[s, h * G:(h + 1) * G] - o).abs()
                assert bool((err <= ATOL[dtype] + RTOL[dtype] * o.abs()).all())
                want = p.sum(0)
                want[: L - 1] += old[s, h, : L - 1]
                rt = weight_rtol(hd, mag, L, G) + 2.0 ** -23
                assert bool(((got[s, h, :L] - want).abs() <= rt * want).all())
        if (step + 1) % every == 0:
            lens = evict(lens, recorded, seen)
            recorded = list(lens)
    assert max(lens) > keep  # some tokens came after the last eviction
