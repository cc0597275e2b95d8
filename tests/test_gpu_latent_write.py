"""pa_latent_write against its definition in 64 bits: bounds of the fp32 steps
in latent_ops.latent_write, then one rounding to the element type."""
import pytest
import torch

from cache_ops import DTYPES, EPS, rope, rope_bound
from latent_ops import LOW, latent_write, rand

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


def _slots(n, blocks, bs, seed):
    slots = torch.randperm(blocks * bs, generator=torch.Generator().manual_seed(seed))[:n].contiguous()
    if n > 3:
        slots[2] = -1
    return slots


CASES = [
    # n, heads, lat, rot, bs, dtype, norm, interleaved, elements before each head's rotated part, kv padding
    (1, 16, 512, 64, 16, "bf16", True, True, 128, 0),
    (64, 16, 512, 64, 16, "bf16", True, False, 128, 8),
    (33, 128, 512, 64, 64, "f16", True, True, 128, 0),
    (7, 20, 512, 64, 8, "f32", True, False, 0, 4),
    (5, 3, 500, 62, 4, "bf16", True, True, 1, 3),     # element by element
    (6, 2, 100, 2, 1, "f32", False, True, 0, 0),
    (9, 1, 96, 32, 16, "f16", False, False, 0, 0),
    (3, 5, 1600, 128, 16, "bf16", True, True, 16, 0),  # more vectors than a lane keeps
    (4, 2, 4096, 256, 2, "f32", True, False, 0, 0),
    (700, 8, 512, 64, 16, "bf16", False, True, 0, 0),  # several tokens per CTA
    (2500, 4, 256, 32, 32, "f16", True, False, 64, 0),
]


@pytest.mark.parametrize("n,heads,lat,rot,bs,dtype,norm,interleaved,lead,pad", CASES)
def test_rows_and_queries(pa, n, heads, lat, rot, bs, dtype, norm, interleaved, lead, pad):
    kv = rand((n, lat + rot + pad), dtype, 1, 0.7)
    q = rand((n, heads, lead + rot), dtype, 2)
    w = rand((lat,), dtype, 3) if norm else None
    pos = torch.randint(-(1 << 20), 1 << 20, (n,), generator=torch.Generator().manual_seed(4))
    inv = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / (rot // 2))
    blocks = -(-n // bs) + 2
    slots = _slots(n, blocks, bs, 5)
    nan = float("nan")
    cache = torch.full((blocks, bs, lat + rot), nan, dtype=DTYPES[dtype], device=DEV)
    wide = torch.full((n, heads, lat + rot), nan, dtype=DTYPES[dtype], device=DEV)
    pa.pa_latent_write(kv.to(DEV)[:, : lat + rot], pos.to(DEV), inv.to(DEV), slots.to(DEV), cache,
                       norm_weight=None if w is None else w.to(DEV), eps=1e-6, q=q.to(DEV)[..., lead:],
                       q_out=wide[..., lat:], interleaved=interleaved)
    rows, bound = latent_write(kv[:, : lat + rot], pos, inv, w, 1e-6, interleaved, lat)
    # the test's own angles lose |angle| 2^-53
    bound[:, lat:] += rope_bound(kv[:, None, lat: lat + rot], rot // 2, interleaved)[:, 0] * 2.0 ** -30
    got = cache.cpu().view(blocks * bs, lat + rot)
    fine = slots >= 0
    err = (got[slots[fine]].double() - rows[fine]).abs()
    assert (err <= bound[fine] + EPS[dtype] * (rows[fine].abs() + bound[fine]) + LOW[dtype]).all()
    if not norm:  # moved, not computed
        assert torch.equal(got[slots[fine]][:, :lat], kv[fine][:, :lat])
    rest = torch.ones(blocks * bs, dtype=torch.bool)
    rest[slots[fine]] = False
    assert torch.isnan(got[rest].float()).all()
    want = rope(q[..., lead:], pos[None], inv, None, interleaved)
    qb = rope_bound(q[..., lead:], rot // 2, interleaved) * (6 * 2.0 ** -24 + 2.0 ** -30)
    out = wide.cpu()
    assert ((out[..., lat:].double() - want).abs() <= qb + EPS[dtype] * (want.abs() + qb) + LOW[dtype]).all()
    assert torch.isnan(out[..., :lat].float()).all()


def test_far_positions_turn_by_whole_turns(pa):
    """A position whose angle is a multiple of a turn rotates by nothing: integer arithmetic drops whole turns."""
    inv = torch.tensor([2 * 3.141592653589793 / 4096], dtype=torch.float64, device=DEV)
    kv = rand((4, 66), "f32", 1).to(DEV)
    pos = torch.tensor([0, 4096 << 20, -(4096 << 25), 4096 << 28], device=DEV)
    cache = torch.zeros((4, 1, 66), device=DEV)
    pa.pa_latent_write(kv, pos, inv, torch.arange(4, device=DEV), cache)
    assert torch.allclose(cache[:, 0], kv, rtol=0, atol=2e-6)


def test_in_place_queries_and_rows_only(pa):
    n, heads, rot, lat = 37, 6, 64, 512
    kv, q = rand((n, lat + rot), "bf16", 1).to(DEV), rand((n, heads, rot), "bf16", 2).to(DEV)
    pos, inv = torch.arange(n, device=DEV), (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).to(DEV)
    slots = torch.arange(n, device=DEV)
    caches = [torch.zeros((3, 16, lat + rot), dtype=torch.bfloat16, device=DEV) for _ in range(3)]
    out = torch.zeros_like(q)
    pa.pa_latent_write(kv, pos, inv, slots, caches[0], q=q, q_out=out)
    same = q.clone()
    pa.pa_latent_write(kv, pos, inv, slots, caches[1], q=same, q_out=same)
    assert torch.equal(out, same) and torch.equal(caches[0], caches[1])
    pa.pa_latent_write(kv, pos, inv, slots, caches[2])
    assert torch.equal(caches[0], caches[2])
    # heads outermost
    turned = torch.zeros((heads, n, rot), dtype=torch.bfloat16, device=DEV)
    pa.pa_latent_write(kv, pos, inv, slots, caches[2], q=q.transpose(0, 1).contiguous().transpose(0, 1),
                       q_out=turned.transpose(0, 1))
    assert torch.equal(turned.transpose(0, 1), out)


def test_zero_rows_and_no_tokens(pa):
    lat, rot = 512, 64
    inv = torch.ones(32, dtype=torch.float64, device=DEV)
    cache = torch.full((1, 16, lat + rot), 7.0, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(lat, dtype=torch.bfloat16, device=DEV)
    none = torch.zeros(0, dtype=torch.int64, device=DEV)
    pa.pa_latent_write(torch.zeros((0, lat + rot), dtype=torch.bfloat16, device=DEV), none, inv, none, cache, norm_weight=w)
    assert (cache == 7).all()
    one = torch.zeros(1, dtype=torch.int64, device=DEV)
    pa.pa_latent_write(torch.zeros((1, lat + rot), dtype=torch.bfloat16, device=DEV), one, inv, one, cache, norm_weight=w)
    assert (cache[0, 0] == 0).all() and (cache[0, 1:] == 7).all()
