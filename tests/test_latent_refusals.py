"""Refusals of the latent-cache and shared-prefix entry points, on the CPU: the
C checks answer before anything is enqueued, and the binding's before the call."""
import ctypes

import pytest
import torch

vp = ctypes.c_void_p
ONE = vp(1024)
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_116_gb300 import build

    build.build()
    from paged_kv_cache_116_gb300 import _binding

    return _binding.lib()


def _write(lib, **kw):
    a = dict(q_out=ONE, qos=640, qoh=64, q=ONE, qs=640, qh=64, kv=ONE, kvs=576, norm=ONE, eps=1e-6, pos=ONE, inv=ONE,
             rot=64, inter=0, slots=ONE, n=4, cache=ONE, nb=4, bs=16, heads=10, lat=512, dtype=1, stream=None)
    a.update(kw)
    return lib.pa_latent_write(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(rot=0), INVALID), (dict(rot=63), INVALID), (dict(rot=258), INVALID), (dict(lat=0), INVALID),
    (dict(lat=4097), UNSUPPORTED), (dict(heads=-1), INVALID), (dict(dtype=3), INVALID), (dict(n=-1), INVALID),
    (dict(n=1 << 31), UNSUPPORTED), (dict(kv=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID),
    (dict(pos=None), INVALID), (dict(inv=None), INVALID), (dict(slots=None), INVALID), (dict(cache=None), INVALID),
    (dict(cache=vp(1032)), INVALID), (dict(kv=vp(1025)), INVALID), (dict(norm=vp(1025)), INVALID),
    (dict(kvs=575), INVALID), (dict(qoh=63), INVALID), (dict(qos=639), INVALID), (dict(qs=-1), INVALID),
    (dict(qos=64, qoh=64 * 4 - 1), INVALID), (dict(nb=0), INVALID), (dict(nb=1 << 28), UNSUPPORTED)])
def test_write_refuses(lib, kw, status):
    assert _write(lib, **kw) == status


def test_write_of_nothing_is_fine(lib):
    assert _write(lib, n=0, kv=None) == 0


def _decode(lib, **kw):
    a = dict(out=ONE, q=ONE, cache=ONE, tables=ONE, max_blocks=8, lens=ONE, S=2, heads=16, lat=512, rot=64, nb=16,
             bs=16, ctx=100, scale=0.1, dtype=1, ws=ONE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.pa_latent_decode(*a.values())


def _varlen(lib, **kw):
    a = dict(out=ONE, q=ONE, cache=ONE, tables=ONE, max_blocks=8, lens=ONE, cu=ONE, S=2, T=10, max_q=9, heads=16,
             lat=512, rot=64, nb=16, bs=16, ctx=100, scale=0.1, causal=1, dtype=1, ws=ONE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.pa_latent_varlen(*a.values())


REFUSED = [
    (dict(lat=0), INVALID), (dict(rot=-1), INVALID), (dict(lat=513), UNSUPPORTED), (dict(heads=0), INVALID),
    (dict(dtype=3), INVALID), (dict(S=-1), INVALID), (dict(max_blocks=-1), INVALID), (dict(ctx=-1), INVALID),
    (dict(out=None), INVALID), (dict(q=None), INVALID), (dict(cache=None), INVALID), (dict(tables=None), INVALID),
    (dict(lens=None), INVALID), (dict(out=vp(1032)), INVALID), (dict(q=vp(1032)), INVALID),
    (dict(cache=vp(1032)), INVALID), (dict(nb=0), INVALID), (dict(nb=1 << 28), UNSUPPORTED),
    (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(ws=vp(1032)), INVALID)]


@pytest.mark.parametrize("kw,status", REFUSED)
def test_attention_refuses(lib, kw, status):
    assert _decode(lib, **kw) == status
    assert _varlen(lib, **kw) == status


def test_attention_of_nothing_is_fine(lib):
    assert _decode(lib, S=0, q=None) == 0
    assert _varlen(lib, T=0, q=None) == 0
    assert _varlen(lib, cu=None) == INVALID and _varlen(lib, T=-1) == INVALID and _varlen(lib, max_q=-1) == INVALID
    assert _varlen(lib, T=1 << 28, heads=128, ctx=1 << 20) == UNSUPPORTED


def test_pinned_tensor_cores_refuse_what_they_do_not_take(lib):
    for opt, call in ((1, _decode), (3, _varlen)):
        assert lib.pa_set_option(opt, 2) == 0
        try:
            for kw in (dict(dtype=0), dict(lat=256), dict(rot=32)):
                assert call(lib, **kw) == UNSUPPORTED
        finally:
            lib.pa_set_option(opt, 0)


def test_workspace_sizes(lib):
    size = lib.pa_latent_decode_workspace_size
    assert size(0, 16, 512, 64, 16, 100, 1) == 0
    assert size(4, 16, 512, 64, 16, 64, 0) == 0          # CUDA cores: pieces of 64 keys at least
    assert 0 < size(4, 16, 512, 64, 6, 1000, 0) < size(4, 16, 512, 64, 6, 4000, 0)
    assert size(4000, 16, 512, 64, 6, 4000, 0) == 0     # rows enough
    small, full = size(64, 16, 512, 64, 16, 4000, 1), size(1, 128, 512, 64, 16, 100, 1)  # a tile has 128 rows
    assert 0 < small < full
    assert lib.pa_latent_varlen_workspace_size(4, 1000, 500, 128, 512, 64, 16, 4000, 1) == full
    assert lib.pa_latent_varlen_workspace_size(0, 0, 0, 128, 512, 64, 16, 4000, 1) == 0


def _shared(lib, **kw):
    a = dict(out=ONE, q=ONE, k=ONE, v=ONE, tables=ONE, max_blocks=8, lens=ONE, starts=ONE, prefix=ONE, groups=1, S=4,
             hq=32, hkv=8, hd=128, nb=16, bs=16, ctx=100, scale=0.1, dtype=1, ws=ONE, wsb=1 << 40, stream=None)
    a.update(kw)
    return lib.pa_decode_shared(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(groups=-1), INVALID), (dict(starts=None), INVALID), (dict(prefix=None), INVALID), (dict(hq=33), INVALID),
    (dict(dtype=3), INVALID), (dict(hd=257), UNSUPPORTED), (dict(out=None), INVALID), (dict(q=None), INVALID),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(tables=None), INVALID), (dict(lens=None), INVALID),
    (dict(q=vp(1032)), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=16), WORKSPACE), (dict(ws=vp(1032)), INVALID)])
def test_shared_refuses(lib, kw, status):
    assert _shared(lib, **kw) == status
    assert _shared(lib, **{**kw, "S": 0}) in (0, status)


def test_binding_refuses(monkeypatch):
    """CPU tensors, and parts that do not fit each other (their devices aside)."""
    from paged_kv_cache_116_gb300 import _binding as pa

    f = torch.zeros
    with pytest.raises(ValueError):
        pa.pa_latent_decode(f(1, 2, 512), f(1, 2, 576), f(2, 16, 576), f(1, 4, dtype=torch.int32),
                            f(1, dtype=torch.int32), 10, 0.1)
    monkeypatch.setattr(pa, "_dev", lambda *ts: None)
    i32 = dict(dtype=torch.int32)
    good = dict(out=f(2, 4, 512), q=f(2, 4, 576), latent_cache=f(2, 16, 576), block_tables=f(2, 4, **i32),
                context_lens=f(2, **i32))
    for key, bad in (("out", f(2, 4, 577)), ("out", f(2, 3, 512)), ("q", f(2, 4, 575)), ("q", f(2, 576)),
                     ("latent_cache", f(2, 16, 1, 576)), ("latent_cache", f(2, 16, 576).half()),
                     ("out", f(2, 4, 512).half()), ("block_tables", f(3, 4, **i32)), ("context_lens", f(3, **i32))):
        with pytest.raises(ValueError):
            pa.pa_latent_decode(**{**good, key: bad}, max_context=10, scale=0.1)
    for key, bad in (("block_tables", f(2, 4)), ("context_lens", f(2))):
        with pytest.raises(TypeError):
            pa.pa_latent_decode(**{**good, key: bad}, max_context=10, scale=0.1)
    good["seq_lens"] = good.pop("context_lens")
    with pytest.raises(ValueError):
        pa.pa_latent_varlen(**good, cu_seqlens_q=f(2, **i32), max_q=1, max_context=10, scale=0.1)
    with pytest.raises(TypeError):
        pa.pa_latent_varlen(**good, cu_seqlens_q=f(3), max_q=1, max_context=10, scale=0.1)
    good = dict(out=f(2, 4, 64), q=f(2, 4, 64), k_cache=f(4, 16, 2, 64), v_cache=f(4, 16, 2, 64),
                block_tables=f(2, 4, **i32), context_lens=f(2, **i32), group_starts=f(2, **i32), prefix_lens=f(1, **i32))
    for key, bad in (("out", f(2, 4, 32)), ("k_cache", f(4, 16, 2, 32)), ("v_cache", f(4, 16, 2, 64).half()),
                     ("block_tables", f(3, 4, **i32)), ("context_lens", f(3, **i32)), ("group_starts", f(3, **i32))):
        with pytest.raises(ValueError):
            pa.pa_decode_shared(**{**good, key: bad}, max_context=10, scale=0.1)
    for key, bad in (("group_starts", f(2)), ("prefix_lens", f(1)), ("block_tables", f(2, 4))):
        with pytest.raises(TypeError):
            pa.pa_decode_shared(**{**good, key: bad}, max_context=10, scale=0.1)
    i64, f64 = dict(dtype=torch.int64), dict(dtype=torch.float64)
    good = dict(kv=f(3, 96), positions=f(3, **i64), inv_freq=f(16, **f64), slot_mapping=f(3, **i64),
                latent_cache=f(2, 4, 96))
    for key, bad in (("positions", f(3, **i32)), ("inv_freq", f(16)), ("slot_mapping", f(3, **i32))):
        with pytest.raises(TypeError):
            pa.pa_latent_write(**{**good, key: bad})
    for extra in (dict(), dict(latent_cache=f(2, 4, 95)), dict(positions=f(1, 3, **i64))):  # (CPU tensors to begin with)
        with pytest.raises(ValueError):
            pa.pa_latent_write(**{**good, **extra})
