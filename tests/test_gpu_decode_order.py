"""What follows a decode on its stream may write what the decode read: the library's calls, launched as dependents of one
another, run in order also where no sequence's result has to be joined from pieces."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


@pytest.mark.parametrize("form", ["decode", "decode_fp8", "weights"])
def test_a_write_after_the_decode_of_whole_sequences(pa, form):
    """As many equal (sequence, KV head) units as the decode has warps: each is worked whole by one of them."""
    S, hkv, hq, hd, bs, L = 152, 8, 16, 128, 16, 2048
    fp8 = form == "decode_fp8"
    S = S * 3 // 2 if fp8 else S  # (three CTAs of four warps per SM over codes, one of eight otherwise)
    nb = S * L // bs
    gen = torch.Generator(device=DEV).manual_seed(1)
    q = torch.randn((S, hq, hd), generator=gen, device=DEV).to(torch.bfloat16)
    tables = torch.randperm(nb, generator=gen, device=DEV).to(torch.int32).view(S, L // bs)
    lens = torch.full((S,), L, dtype=torch.int32, device=DEV)
    if fp8:
        pools = [torch.randint(0, 0x70, (nb, bs, hkv, hd), generator=gen, device=DEV, dtype=torch.uint8)
                 for _ in range(2)]
        scales = [torch.rand((nb, hkv, bs), generator=gen, device=DEV) * 0.01 for _ in range(2)]
    else:
        pools = [torch.randn((nb, bs, hkv, hd), generator=gen, device=DEV).to(torch.bfloat16) for _ in range(2)]
        scales = []
    size = {"decode": pa.pa_decode_workspace_size, "decode_fp8": pa.pa_decode_fp8_workspace_size,
            "weights": pa.pa_decode_weights_workspace_size}[form]
    ws = torch.empty(size(S, hq, hkv, hd, bs, L, torch.bfloat16), dtype=torch.uint8, device=DEV)
    rows = torch.zeros((S, hkv, L), device=DEV)

    def decode(out):
        if form == "weights":
            pa.pa_decode_weights(out, rows, q, *pools, tables, lens, L, 0.09, ws)
        elif fp8:
            pa.pa_decode_fp8(out, q, *pools, *scales, tables, lens, L, 0.09, workspace=ws)
        else:
            pa.pa_decode(out, q, *pools, tables, lens, L, 0.09, workspace=ws)

    # (the tokens read last: a warp's latest tiles)
    pos = torch.arange(L - 64, L, device=DEV)
    slots = (tables[:, pos // bs].long() * bs + pos % bs).reshape(-1)
    new = torch.full((slots.numel(), hkv, hd), 3.0, dtype=torch.bfloat16, device=DEV)
    want, got = torch.empty_like(q), torch.empty_like(q)
    decode(want)
    torch.cuda.synchronize()
    for _ in range(4):
        got.fill_(7.0)
        keep = [p.clone() for p in pools + scales]
        torch.cuda.synchronize()
        decode(got)
        if fp8:
            pa.pa_write_kv_fp8(new, new, slots, *pools, *scales)
        else:
            pa.pa_write_kv(new, new, slots, *pools)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        for p, k in zip(pools + scales, keep):
            assert not torch.equal(p, k)
            p.copy_(k)
