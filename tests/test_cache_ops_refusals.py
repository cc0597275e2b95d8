"""Argument refusals of the cache-side operators: answered on the host, no GPU."""
import ctypes

import pytest

INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 4
BF16, F32, FP8 = 1, 0, 3


@pytest.fixture(scope="module")
def lib():
    from paged_kv_cache_116_gb300 import build

    build.build()
    from paged_kv_cache_116_gb300 import _binding

    return _binding.lib()


P = ctypes.c_void_p
ONE = P(16)


def _rope(lib, fp8=False, **kw):
    a = dict(q_out=P(32), q=ONE, k=ONE, v=ONE, qs=1024, ks=256, vs=256, pos=ONE, axes=1, inv=ONE, axis=None, rot=128,
             inter=0, slots=ONE, n=4, kc=ONE, vc=ONE, scl=ONE, nb=10, bs=16, hq=8, hkv=2, hd=128, dt=BF16)
    a.update(kw)
    s = (a["scl"], a["scl"]) if fp8 else ()
    fn = lib.pa_rope_write_kv_fp8 if fp8 else lib.pa_rope_write_kv
    return fn(a["q_out"], a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["pos"], a["axes"], a["inv"], a["axis"],
              a["rot"], a["inter"], a["slots"], a["n"], a["kc"], a["vc"], *s, a["nb"], a["bs"], a["hq"], a["hkv"],
              a["hd"], a["dt"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw, status", [
    (dict(rot=127), INVALID), (dict(rot=0), INVALID), (dict(rot=130), INVALID), (dict(axes=0), INVALID),
    (dict(n=-1), INVALID), (dict(hd=258, rot=2), UNSUPPORTED), (dict(hq=7), INVALID), (dict(hq=-1), INVALID),
    (dict(qs=1023), INVALID), (dict(ks=255), INVALID), (dict(vs=100), INVALID), (dict(pos=None), INVALID),
    (dict(inv=None), INVALID), (dict(slots=None), INVALID), (dict(kc=P(24)), INVALID), (dict(dt=3), INVALID),
    (dict(q_out=None), INVALID), (dict(q_out=ONE, qs=2048), INVALID), (dict(bs=0), INVALID),
    (dict(n=1 << 31), UNSUPPORTED)])
def test_rope_refuses(lib, kw, status, fp8):
    assert _rope(lib, fp8, **kw) == status, lib.pa_last_error()


def test_rope_nothing_to_do(lib):
    assert _rope(lib, n=0, q=None, k=None, v=None) == 0
    assert _rope(lib, fp8=True, scl=None) == INVALID


def _decode(lib, fp8=False, **kw):
    a = dict(out=ONE, w=ONE, stride=64, q=ONE, kc=ONE, vc=ONE, scl=ONE, bt=ONE, mb=4, lens=ONE, S=2, hq=8, hkv=2,
             hd=128, nb=10, bs=16, mc=64, dt=BF16, ws=ONE, wsb=1 << 40)
    a.update(kw)
    s = (a["scl"], a["scl"]) if fp8 else ()
    fn = lib.pa_decode_weights_fp8 if fp8 else lib.pa_decode_weights
    return fn(a["out"], a["w"], a["stride"], a["q"], a["kc"], a["vc"], *s, a["bt"], a["mb"], a["lens"], a["S"],
              a["hq"], a["hkv"], a["hd"], a["nb"], a["bs"], a["mc"], 1.0, a["dt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw, status", [
    (dict(stride=63), INVALID), (dict(w=None), INVALID), (dict(hq=9), INVALID), (dict(S=-1), INVALID),
    (dict(mc=-1), INVALID), (dict(wsb=8), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(hd=300), UNSUPPORTED),
    (dict(out=P(24)), INVALID), (dict(q=None), INVALID), (dict(dt=3), INVALID), (dict(ws=P(24)), INVALID)])
def test_decode_weights_refuses(lib, kw, status, fp8):
    assert _decode(lib, fp8, **kw) == status, lib.pa_last_error()


def test_decode_weights_nothing_to_do(lib):
    assert _decode(lib, S=0, w=None, q=None) == 0
    assert _decode(lib, fp8=True, scl=None) == INVALID


def _prompt(lib, fp8=False, **kw):
    a = dict(w=ONE, stride=64, q=ONE, kc=ONE, scl=ONE, bt=ONE, mb=4, lens=ONE, cu=ONE, S=2, T=8, mq=6, hq=8, hkv=2,
             hd=128, nb=10, bs=16, mc=64, win=0, dt=BF16, ws=ONE, wsb=1 << 40)
    a.update(kw)
    s = (a["scl"],) if fp8 else ()
    fn = lib.pa_prompt_weights_fp8 if fp8 else lib.pa_prompt_weights
    return fn(a["w"], a["stride"], a["q"], a["kc"], *s, a["bt"], a["mb"], a["lens"], a["cu"], a["S"], a["T"], a["mq"],
              a["hq"], a["hkv"], a["hd"], a["nb"], a["bs"], a["mc"], a["win"], 1.0, 1, a["dt"], a["ws"], a["wsb"],
              None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw, status", [
    (dict(stride=10), INVALID), (dict(w=None), INVALID), (dict(cu=None), INVALID), (dict(win=-1), INVALID),
    (dict(hq=9), INVALID), (dict(T=-1), INVALID), (dict(wsb=8), WORKSPACE), (dict(ws=None), WORKSPACE),
    (dict(ws=P(24)), INVALID), (dict(hd=300), UNSUPPORTED), (dict(kc=P(24)), INVALID), (dict(dt=4), INVALID)])
def test_prompt_weights_refuses(lib, kw, status, fp8):
    assert _prompt(lib, fp8, **kw) == status, lib.pa_last_error()


def test_prompt_weights_nothing_to_do(lib):
    assert _prompt(lib, S=0, q=None) == 0 and _prompt(lib, T=0, q=None) == 0
    assert _prompt(lib, fp8=True, scl=None) == INVALID


def _evict(lib, **kw):
    a = dict(wo=ONE, po=ONE, nl=P(32), w=ONE, pos=None, rec=None, seen=None, stride=64, kc=ONE, vc=ONE, ks=None,
             vs=None, bt=ONE, mb=4, nt=ONE, nmb=4, lens=ONE, S=2, hkv=2, hd=128, nb=10, bs=16, mc=64, keep=32, sink=2,
             rcnt=8, dt=BF16, ws=ONE, wsb=1 << 40)
    a.update(kw)
    return lib.pa_evict(a["wo"], a["po"], a["nl"], a["w"], a["pos"], a["rec"], a["seen"], a["stride"], a["kc"],
                        a["vc"], a["ks"], a["vs"], a["bt"], a["mb"], a["nt"], a["nmb"], a["lens"], a["S"], a["hkv"],
                        a["hd"], a["nb"], a["bs"], a["mc"], a["keep"], a["sink"], a["rcnt"], a["dt"], a["ws"],
                        a["wsb"], None)


@pytest.mark.parametrize("kw, status", [
    (dict(keep=0), INVALID), (dict(sink=-1), INVALID), (dict(rcnt=-1), INVALID), (dict(sink=25), INVALID),
    (dict(sink=2 ** 31 - 1, rcnt=2 ** 31 - 1), INVALID), (dict(stride=63), INVALID), (dict(wo=None), INVALID),
    (dict(nl=None), INVALID), (dict(nl=ONE), INVALID), (dict(rec=P(48)), INVALID), (dict(pos=P(48)), INVALID),
    (dict(pos=P(48), rec=P(32)), INVALID), (dict(seen=P(32)), INVALID), (dict(ks=ONE, vs=ONE), INVALID),
    (dict(dt=FP8), INVALID), (dict(dt=FP8, ks=ONE), INVALID), (dict(dt=9), INVALID), (dict(kc=P(24)), INVALID),
    (dict(wsb=8), WORKSPACE), (dict(ws=None), WORKSPACE), (dict(ws=P(24)), INVALID), (dict(hkv=0), INVALID),
    (dict(mc=-1), INVALID), (dict(S=1 << 24), UNSUPPORTED), (dict(mc=(1 << 19) + 1, stride=1 << 20), UNSUPPORTED)])
def test_evict_refuses(lib, kw, status):
    assert _evict(lib, **kw) == status, lib.pa_last_error()


def test_evict_nothing_to_do(lib):
    assert _evict(lib, S=0, w=None) == 0
    assert lib.pa_evict_workspace_size(4, 2, 100, 100) == 0  # nothing can exceed the budget
    assert lib.pa_evict_workspace_size(0, 2, 100, 50) == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_empty_contexts_and_huge_sizes(lib, fp8):
    """max_context 0: no request holds a token.  Sizes beyond int32 are refused before any launch."""
    assert _prompt(lib, fp8, mc=0, stride=0) == 0
    assert _prompt(lib, fp8, mq=0) == 0
    assert _prompt(lib, fp8, mc=1 << 30, stride=1 << 30, bs=12, wsb=1 << 62) == UNSUPPORTED
    assert _rope(lib, fp8, hkv=1 << 22, hq=1 << 23, ks=1 << 40, vs=1 << 40, qs=1 << 40, nb=1, bs=1) == UNSUPPORTED


@pytest.mark.parametrize("name, count", [
    ("pa_decode_weights_workspace_size", 7), ("pa_decode_weights_fp8_workspace_size", 7),
    ("pa_prompt_weights_workspace_size", 10), ("pa_prompt_weights_fp8_workspace_size", 10),
    ("pa_evict_workspace_size", 4)])
def test_workspace_sizes_answer_any_numbers(lib, name, count):
    """Zeros, negatives and the largest integers: a number comes back, nothing divides by zero."""
    gen = __import__("random").Random(1)
    for _ in range(4000):
        getattr(lib, name)(*[gen.choice((-2 ** 31, -1, 0, 1, 7, 16, 64, 128, 1000, 2 ** 31 - 1)) for _ in range(count)])
