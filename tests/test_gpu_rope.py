"""pa_rope_write_kv and its quantizing form against the 64-bit rotation.

Tolerance: the half turn x in [-1, 1) is rounded once to fp32 (2^-25, times pi
for the angle: below 1.6 2^-24), sincospif is good to one unit (2^-24), the two
products and their sum round once each (2 2^-24 of |x1| + |x2|): below
6 2^-24 (|x1| + |x2|) in all.  Then one rounding to the element type: half a
step relative, and for f16 below its normal range (2^-14) half of the fixed
step 2^-24 there, 2^-25, which is more than 2^-11 of such a value."""
import pytest
import torch

from cache_ops import DTYPES, EPS, rope, rope_bound

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
LOW = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


def _inputs(n, hq, hkv, hd, bs, dtype, axes, rot, far, seed, fused=True, pad=0):
    g = torch.Generator().manual_seed(seed)
    width = (hq + 2 * hkv) * hd
    qkv = torch.randn((n, width + pad), generator=g).to(DTYPES[dtype])
    dq = qkv.to(DEV)
    cut = (0, hq * hd, (hq + hkv) * hd, width)
    cpu = [qkv[:, cut[i]:cut[i + 1]].reshape(n, -1, hd) for i in range(3)]
    dev = [dq[:, cut[i]:cut[i + 1]].unflatten(1, (-1, hd)) for i in range(3)]
    if not fused:
        dev = [x.contiguous() for x in dev]
    pos = torch.randint(0, far, (axes, n), generator=g)
    half = rot // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    axis = (torch.arange(half) % axes).to(torch.int32) if axes > 1 else None
    blocks = -(-n // bs) + 2
    slots = torch.randperm(blocks * bs, generator=g)[:n].contiguous()
    if n > 3:
        slots[2] = -1
    return cpu, dev, pos, inv, axis, slots, blocks


def _dev(x):
    return None if x is None else x.to(DEV)


CASES = [
    # n, hq, hkv, hd, bs, dtype, axes, rot, interleaved, far, fused, pad
    (1, 32, 8, 128, 16, "bf16", 3, 128, False, 4096, True, 0),
    (64, 32, 8, 128, 16, "bf16", 3, 128, True, 1 << 20, True, 0),
    (5, 4, 2, 32, 4, "f32", 1, 32, False, 1000, False, 0),
    (17, 12, 2, 128, 16, "f16", 2, 64, True, 1 << 17, True, 8),
    (33, 6, 3, 40, 12, "bf16", 2, 24, False, 50000, True, 0),     # no 16-byte vectors over the pairs
    (9, 2, 1, 7, 1, "f32", 1, 6, True, 300, True, 3),             # odd head_dim and stride
    (700, 8, 8, 256, 32, "f16", 3, 256, False, 1 << 20, True, 0),
    (5000, 4, 1, 64, 16, "bf16", 1, 64, False, 200000, True, 0),  # several tokens per CTA
    (40, 0, 4, 128, 16, "bf16", 1, 128, False, 9000, True, 0),    # keys and values only
]


@pytest.mark.parametrize("case", CASES)
@pytest.mark.parametrize("fp8", [False, True])
def test_matches_the_rotation(pa, case, fp8):
    n, hq, hkv, hd, bs, dtype, axes, rot, inter, far, fused, pad = case
    (q, k, v), (dq, dk, dv), pos, inv, axis, slots, blocks = _inputs(n, hq, hkv, hd, bs, dtype, axes, rot, far, 3,
                                                                     fused, pad)
    kw = dict(pair_axis=_dev(axis), interleaved=inter)
    q_out = torch.full((n, hq, hd), float("nan"), dtype=DTYPES[dtype], device=DEV) if hq else None
    half, u = rot // 2, 2.0 ** -24
    args = (q_out, dq if hq else None, dk, dv, pos.to(DEV), inv.to(DEV), slots.to(DEV))
    fine = slots >= 0
    to = slots[fine]
    kx = rope(k, pos, inv, axis, inter)
    if fp8:
        kc, vc = (torch.full((blocks, bs, hkv, hd), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks, vs = (torch.full((blocks, hkv, bs), -3.0, device=DEV) for _ in range(2))
        pa.pa_rope_write_kv_fp8(*args, kc, vc, ks, vs, **kw)
        # v rows: bit for bit what the quantizing write stores
        kc2, vc2, ks2, vs2 = kc.clone().fill_(0x55), vc.clone().fill_(0x55), ks.clone().fill_(-3.0), vs.clone().fill_(-3.0)
        pa.pa_write_kv_fp8(dk.contiguous(), dv.contiguous(), slots.to(DEV), kc2, vc2, ks2, vs2)
        assert torch.equal(vc, vc2) and torch.equal(vs, vs2)
        codes, scales = kc.cpu().view(-1, hkv, hd), ks.cpu().transpose(1, 2).reshape(-1, hkv)
        untouched = torch.ones(blocks * bs, dtype=torch.bool)
        untouched[to] = False
        assert bool((codes[untouched] == 0x55).all()) and bool((scales[untouched] == -3.0).all())
        top = kx[fine].abs().amax(-1)
        sc = scales[to].double()
        # |x1| + |x2| <= 2 max|row|: the maximum is off by 12 2^-24, the division by one more
        assert bool(((sc - top / 448).abs() <= 13 * u * top / 448).all())
        got = codes[to].view(torch.float8_e4m3fn).double() * sc[..., None]
        # half a step of E4M3 (2^-4 relative, 2^-10 below the normal range), and the fp32 errors above
        tol = kx[fine].abs() * (2.0 ** -4 + 40 * u) + sc[..., None] * 2.0 ** -10 + 40 * u * top[..., None]
        assert bool(((got - kx[fine]).abs() <= tol).all())
    else:
        kc, vc = (torch.full((blocks, bs, hkv, hd), float("nan"), dtype=DTYPES[dtype], device=DEV) for _ in range(2))
        pa.pa_rope_write_kv(*args, kc, vc, **kw)
        rows = kc.cpu().view(-1, hkv, hd)
        want = torch.full(rows.shape, float("nan"), dtype=torch.float64)
        want[to] = kx[fine]
        tol = 6 * u * rope_bound(k, half, inter)
        tol = tol + EPS[dtype] * (kx.abs() + tol) + LOW[dtype]
        assert torch.equal(rows.isnan(), want.isnan())
        assert bool(((rows[to].double() - kx[fine]).abs() <= tol[fine]).all())
        vrows = torch.full(rows.shape, float("nan"), dtype=DTYPES[dtype])
        vrows[to] = v[fine]
        it = torch.int32 if dtype == "f32" else torch.int16
        assert torch.equal(vc.cpu().view(-1, hkv, hd).contiguous().view(it), vrows.view(it))
    if hq:
        want = rope(q, pos, inv, axis, inter)
        tol = 6 * u * rope_bound(q, half, inter)
        tol = tol + EPS[dtype] * (want.abs() + tol) + LOW[dtype]
        assert bool(((q_out.cpu().double() - want).abs() <= tol).all())


def test_far_and_negative_positions(pa):
    """Positions up to 2^31 and below zero: against angles reduced in integers (frequencies that are whole fractions
    of a turn have exact angles)."""
    n, hd = 12, 16
    pos = torch.tensor([[0, 1, -1, 2 ** 20 + 3, -(2 ** 20) - 3, 2 ** 31 - 1, 2 ** 40 + 5, -(2 ** 40) - 5, 7, -7, 4, -4]])
    turns = torch.tensor([8, 5, 12, 1000, 7, 3, 64, 999])  # positions per turn
    import math

    inv = 2 * math.pi / turns.double()
    x = torch.randn((n, 1, hd), generator=torch.Generator().manual_seed(1))
    frac = (pos[0][:, None] % turns).double() / turns
    c, s = torch.cos(2 * math.pi * frac)[:, None], torch.sin(2 * math.pi * frac)[:, None]
    a, b = x[..., :8].double(), x[..., 8:].double()
    want = torch.cat((a * c - b * s, b * c + a * s), -1)
    q_out = torch.empty((n, 1, hd), device=DEV)
    kc, vc = (torch.zeros((2, 8, 1, hd), device=DEV) for _ in range(2))
    dx = x.to(DEV)
    pa.pa_rope_write_kv(q_out, dx, dx, dx, pos.to(DEV), inv.to(DEV), torch.arange(n, device=DEV), kc, vc)
    # the frequency itself is rounded to 2^-53 relative: |position| 2^-53 radians more
    tol = (6 * 2.0 ** -24 + pos[0].abs().double()[:, None, None] * 2.0 ** -51) * rope_bound(x, 8, False)
    assert bool(((q_out.cpu().double() - want).abs() <= tol + 2.0 ** -24 * want.abs()).all())


def test_in_place_q_stream_and_graph(pa):
    (q, k, v), (dq, dk, dv), pos, inv, axis, slots, blocks = _inputs(200, 8, 2, 128, 16, "bf16", 3, 128, 70000, 9,
                                                                     fused=False)
    kc, vc = (torch.zeros((blocks, 16, 2, 128), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    args = (dk, dv, pos.to(DEV), inv.to(DEV), slots.to(DEV), kc, vc)
    ref = torch.empty_like(dq)
    pa.pa_rope_write_kv(ref, dq, *args, pair_axis=_dev(axis))
    kref = kc.clone()
    kc.zero_()
    own = dq.clone()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        pa.pa_rope_write_kv(own, own, *args, pair_axis=_dev(axis))
    st.synchronize()
    assert torch.equal(own, ref) and torch.equal(kc, kref)
    out = torch.empty_like(dq)
    ax = _dev(axis)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        pa.pa_rope_write_kv(out, dq, *args, pair_axis=ax)
    dq.copy_(dq.flip(0))
    kc.zero_()
    g.replay()
    pa.pa_rope_write_kv(ref, dq, *args, pair_axis=ax)
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(kc, kref)


def test_check_mode(pa):
    (q, k, v), (dq, dk, dv), pos, inv, axis, slots, blocks = _inputs(8, 4, 2, 64, 16, "bf16", 2, 64, 100, 9)
    kc, vc = (torch.zeros((blocks, 16, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.zeros((8, 4, 64), dtype=torch.bfloat16, device=DEV)
    twice, far, ax = slots.clone(), slots.clone(), axis.clone()
    twice[4], far[4], ax[3] = twice[5], blocks * 16, 2
    pa.pa_set_check_mode(True)
    try:
        for sl, a in ((twice, axis), (far, axis), (slots, ax)):
            with pytest.raises(pa.PAError) as e:
                pa.pa_rope_write_kv(out, dq, dk, dv, pos.to(DEV), inv.to(DEV), sl.to(DEV), kc, vc, pair_axis=a.to(DEV))
            assert e.value.status == 3
        assert not bool(out.any()) and not bool(kc.any())
        pa.pa_rope_write_kv(out, dq, dk, dv, pos.to(DEV), inv.to(DEV), slots.to(DEV), kc, vc, pair_axis=axis.to(DEV))
    finally:
        pa.pa_set_check_mode(False)
    assert bool(kc.any())


def test_binding_refuses(pa):
    (q, k, v), (dq, dk, dv), pos, inv, axis, slots, blocks = _inputs(8, 4, 2, 64, 16, "bf16", 1, 64, 100, 9)
    kc, vc = (torch.zeros((blocks, 16, 2, 64), dtype=torch.bfloat16, device=DEV) for _ in range(2))
    out = torch.zeros((8, 4, 64), dtype=torch.bfloat16, device=DEV)
    good = [out, dq, dk, dv, pos.to(DEV), inv.to(DEV), slots.to(DEV), kc, vc]
    for i, bad in ((0, out[:, :2]), (1, dq.float()), (2, dk[:4]), (3, dv.transpose(1, 2)), (4, pos.to(DEV).int()),
                   (5, inv.to(DEV).float()), (6, slots.to(DEV)[:4]), (2, k)):
        args = list(good)
        args[i] = bad
        with pytest.raises((ValueError, TypeError)):
            pa.pa_rope_write_kv(*args)
