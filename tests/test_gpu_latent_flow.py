"""The latent-cache operators as a server runs them -- prompts written and
attended in chunks, forks of a prompt, generated tokens -- against attention in
64 bits over the rows that the cache then holds; and shared prefixes made by
forking a prompt (copy-on-write tails, appended tokens)."""
import pytest
import torch

from cache_ops import EPS, DTYPES
from latent_ops import attention, close, latent_write, rand

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LAT, ROT = 512, 64
INV = 10000.0 ** (-torch.arange(ROT // 2, dtype=torch.float64) / (ROT // 2))


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    yield pa
    pa.pa_set_option(1, 0)


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype,bs,heads", [("bf16", 16, 16), ("f16", 64, 128), ("f32", 16, 4)])
def test_prompts_in_chunks_then_tokens(pa, dtype, bs, heads):
    dt = DTYPES[dtype]
    prompts, steps, S = [70, 129, 1], 4, 3
    blocks = [-(-(n + steps) // bs) for n in prompts]
    perm = torch.randperm(sum(blocks) + 1, generator=torch.Generator().manual_seed(1)).tolist()
    tables = torch.full((S, max(blocks)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(blocks):
        tables[s, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
        at += n
    cache = torch.full((len(perm), bs, LAT + ROT), float("nan"), dtype=dt, device=DEV)
    norm = (1 + 0.1 * rand((LAT,), "f32", 2)).to(dt)
    dtables, inv = tables.to(DEV), INV.to(DEV)
    ctx, scale = max(prompts) + steps, 192 ** -0.5
    held = [torch.zeros((0, LAT + ROT), dtype=torch.float64) for _ in range(S)]  # what the cache has, read back
    lens = [0] * S

    def step(new, seed, single):
        """New tokens per sequence: rows and queries into place, then attention; checks both."""
        T = sum(new)
        kv = rand((T, LAT + ROT), dtype, seed, 0.7)
        q = rand((T, heads, LAT + ROT), dtype, seed + 1)
        seq = torch.cat([torch.full((n,), s, dtype=torch.int32) for s, n in enumerate(new)])
        pos = torch.cat([torch.arange(lens[s], lens[s] + n) for s, n in enumerate(new)])
        slots = pa.pa_slot_mapping(dtables, seq.to(DEV), pos.to(DEV), bs)
        dq = q.to(DEV)
        pa.pa_latent_write(kv.to(DEV), pos.to(DEV), inv, slots, cache, norm_weight=norm.to(DEV), q=dq[..., LAT:],
                           q_out=dq[..., LAT:], interleaved=True)
        q = dq.cpu()
        rows, bound = latent_write(kv, pos, INV, norm, 1e-6, True, LAT)
        flat = cache.view(-1, LAT + ROT).cpu()
        got = flat[slots.cpu()].double()
        assert ((got - rows).abs() <= (bound + EPS[dtype] * rows.abs()) * 1.001 + 2.0 ** -24).all()
        cu = [0]
        for s, n in enumerate(new):
            held[s] = torch.cat((held[s], got[cu[-1]:cu[-1] + n]))
            lens[s] += n
            cu.append(cu[-1] + n)
        out = torch.full((T, heads, LAT), float("nan"), dtype=dt, device=DEV)
        dlens = _i32(lens)
        if single:
            size = pa.pa_latent_decode_workspace_size(S, heads, LAT, ROT, bs, ctx, dt)
            ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
            pa.pa_latent_decode(out, dq, cache, dtables, dlens, ctx, scale, workspace=ws)
        else:
            size = pa.pa_latent_varlen_workspace_size(S, T, max(new), heads, LAT, ROT, bs, ctx, dt)
            ws = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
            pa.pa_latent_varlen(out, dq, cache, dtables, dlens, _i32(cu), max(new), ctx, scale, workspace=ws)
        for s, n in enumerate(new):
            if n == 0:
                continue
            seen = (torch.arange(lens[s] - n, lens[s])[:, None] >= torch.arange(lens[s])).repeat_interleave(heads, 0)
            o, e = attention(q[cu[s]:cu[s + 1]].reshape(-1, LAT + ROT), held[s], held[s][:, :LAT], scale, seen, dtype,
                             dtype != "f32")
            close(out[cu[s]:cu[s + 1]].reshape(-1, LAT), o, e)

    step([40, 100, 0], 10, False)          # first chunks; the third prompt waits
    step([30, 29, 1], 20, False)           # the rest of the prompts
    for i in range(steps):
        step([1, 1, 1], 30 + 2 * i, True)  # generated tokens
    assert lens == [n + steps for n in prompts]


def test_forks_of_a_prompt_share_it(pa):
    """A prompt of 100 tokens forked four times: the partial last block is copied, each fork appends its own tokens, and
    the shared decode gives what the plain decode gives, up to rounding, at every step."""
    hq, hkv, hd, bs, n, forks, steps = 16, 4, 128, 16, 100, 4, 20
    g = torch.Generator().manual_seed(3)
    own = -(-(n + steps) // bs) - n // bs  # blocks of each fork behind the shared ones
    lead = n // bs
    total = lead + forks * own
    perm = torch.randperm(total, generator=g).to(torch.int32)
    tables = torch.cat((perm[:lead].repeat(forks, 1), perm[lead:].view(forks, own)), 1).to(DEV)
    kc, vc = (torch.full((total, bs, hkv, hd), float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    k, v = (torch.randn((n, hkv, hd), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
    pos = torch.arange(n, device=DEV)
    slots = pa.pa_slot_mapping(tables, torch.zeros(n, dtype=torch.int32, device=DEV), pos, bs)
    pa.pa_write_kv(k, v, slots, kc, vc)
    pairs = torch.stack([torch.stack((tables[0, lead], tables[f, lead])) for f in range(1, forks)]).long().contiguous()
    pa.pa_copy_blocks(kc, vc, pairs)
    starts, prefix = _i32([0, forks]), _i32([lead * bs])
    pa.pa_set_option(1, 2)
    ctx = n + steps
    ws = torch.empty(pa.pa_decode_shared_workspace_size(forks, 1, hq, hkv, hd, bs, ctx, torch.bfloat16),
                     dtype=torch.uint8, device=DEV)
    for i in range(steps):
        q = torch.randn((forks, hq, hd), generator=g).to(torch.bfloat16).to(DEV)
        nk, nv = (torch.randn((forks, hkv, hd), generator=g).to(torch.bfloat16).to(DEV) for _ in range(2))
        lens = _i32([n + i + 1] * forks)
        plain, out = torch.empty_like(q), torch.empty_like(q)
        pa.pa_decode_append(plain, q, nk, nv, kc, vc, tables, lens, ctx, hd ** -0.5, workspace=ws)
        pa.pa_decode_shared(out, q, kc, vc, tables, lens, starts, prefix, ctx, hd ** -0.5, workspace=ws)
        L = n + i + 1
        keys, vals = (c[tables.long()].reshape(forks, -1, hkv, hd)[:, :L].cpu() for c in (kc, vc))
        for f in range(forks):
            for h in range(hkv):
                s = slice(h * 4, h * 4 + 4)
                o, e = attention(q[f, s].cpu(), keys[f, :, h], vals[f, :, h], hd ** -0.5,
                                 torch.ones((4, L), dtype=torch.bool), "bf16", True)
                close(out[f, s], o, e)
                close(plain[f, s], o, e)
