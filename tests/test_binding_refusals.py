"""What the bindings of the cache-side operators refuse before the library sees it.  No GPU: host tensors that pass
for CUDA tensors, and a library that notes whether it was reached."""
import types

import pytest
import torch

from paged_kv_cache_116_gb300 import _binding as B


class _Cuda(torch.Tensor):
    is_cuda = property(lambda self: True)

    def get_device(self):
        return getattr(self, "_on", 0)


def _t(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype).as_subclass(_Cuda)


class _Lib:
    reached = 0

    def __getattr__(self, name):
        def call(*args):
            self.reached += 1
            return 0

        return call


@pytest.fixture
def lib(monkeypatch):
    fake = _Lib()
    monkeypatch.setattr(B, "lib", lambda: fake)
    monkeypatch.setattr(B, "_current_device", lambda: 0)
    monkeypatch.setattr(B, "_device_count", 2)
    return fake


STREAM = types.SimpleNamespace(cuda_stream=0, device_index=0)
I32, F32, U8, F8 = torch.int32, torch.float32, torch.uint8, torch.float8_e4m3fn
NB, BS, HKV, HQ, HD, S, N, MC = 6, 16, 2, 8, 64, 3, 5, 40


def _pool(dtype=torch.bfloat16, nb=NB):
    return _t(nb, BS, HKV, HD, dtype=dtype)


def _scales(nb=NB):
    return _t(nb, HKV, BS, dtype=F32)


def _decode(**kw):
    a = dict(out=_t(S, HQ, HD), weights=_t(S, HKV, MC, dtype=F32), q=_t(S, HQ, HD), k=_pool(), v=_pool(), sc=None,
             tables=_t(S, 3, dtype=I32), lens=_t(S, dtype=I32))
    a.update(kw)
    rest = (a["tables"], a["lens"], MC, 0.1, _t(64, dtype=U8), STREAM)
    if a["sc"] is None:
        B.pa_decode_weights(a["out"], a["weights"], a["q"], a["k"], a["v"], *rest)
    else:
        B.pa_decode_weights_fp8(a["out"], a["weights"], a["q"], a["k"], a["v"], *a["sc"], *rest)


def _prompt(**kw):
    a = dict(weights=_t(S, HKV, MC, dtype=F32), q=_t(N, HQ, HD), k=_pool(), sc=None, tables=_t(S, 3, dtype=I32),
             lens=_t(S, dtype=I32), cu=_t(S + 1, dtype=I32))
    a.update(kw)
    rest = (a["tables"], a["lens"], a["cu"], 3, MC, 0, 0.1, True, _t(64, dtype=U8), STREAM)
    if a["sc"] is None:
        B.pa_prompt_weights(a["weights"], a["q"], a["k"], *rest)
    else:
        B.pa_prompt_weights_fp8(a["weights"], a["q"], a["k"], a["sc"], *rest)


def _rope(**kw):
    a = dict(q_out=_t(N, HQ, HD), q=_t(N, HQ, HD), k=_t(N, HKV, HD), v=_t(N, HKV, HD),
             pos=_t(1, N, dtype=torch.int64), inv=_t(HD // 2, dtype=torch.float64), slots=_t(N, dtype=torch.int64),
             kc=_pool(), vc=_pool(), sc=None, axis=None)
    a.update(kw)
    args = (a["q_out"], a["q"], a["k"], a["v"], a["pos"], a["inv"], a["slots"], a["kc"], a["vc"])
    if a["sc"] is None:
        B.pa_rope_write_kv(*args, pair_axis=a["axis"], stream=STREAM)
    else:
        B.pa_rope_write_kv_fp8(*args, *a["sc"], pair_axis=a["axis"], stream=STREAM)


def _codes(dtype=U8, nb=NB):
    return dict(k=_pool(dtype, nb), v=_pool(dtype, nb), sc=(_scales(nb), _scales(nb)))


def _rope_codes(dtype=U8, nb=NB):
    return dict(kc=_pool(dtype, nb), vc=_pool(dtype, nb), sc=(_scales(nb), _scales(nb)))


def _prompt_codes(dtype=U8):
    return dict(k=_pool(dtype), sc=_scales())


@pytest.mark.parametrize("call, kw", [
    (_decode, {}), (_decode, _codes()), (_decode, _codes(F8)), (_prompt, {}), (_prompt, _prompt_codes()),
    (_prompt, _prompt_codes(F8)), (_rope, {}), (_rope, _rope_codes()), (_rope, _rope_codes(F8)),
    (_rope, dict(q=None, q_out=None)), (_rope, dict(q=None)), (_rope, dict(pos=_t(N, dtype=torch.int64)))])
def test_parts_that_fit_reach_the_library(lib, call, kw):
    call(**kw)
    assert lib.reached == 1


@pytest.mark.parametrize("call, kw", [
    # codes read as 16-bit rows would be read twice as far as they reach, and 16-bit rows are no codes
    (_decode, dict(k=_pool(U8), v=_pool(U8))), (_decode, _codes(torch.bfloat16)), (_decode, _codes(torch.int8)),
    (_prompt, dict(k=_pool(U8))), (_prompt, _prompt_codes(torch.bfloat16)),
    # results of another type, pools that differ from each other
    (_decode, dict(out=_t(S, HQ, HD, dtype=F32))), (_decode, {**_codes(), "out": _t(S, HQ, HD, dtype=torch.float16)}),
    (_decode, dict(v=_pool(torch.float16))), (_decode, dict(v=_pool(F32))), (_decode, {**_codes(), "v": _pool(F8, 3)}),
    (_rope, dict(vc=_pool(nb=3))), (_rope, dict(vc=_pool(torch.float16))),
    (_rope, dict(vc=_t(NB, BS, HKV, HD // 2))), (_rope, _rope_codes(torch.bfloat16)),
    (_rope, {**_rope_codes(), "vc": _pool(U8, 3)}), (_rope, {**_rope_codes(), "vc": _pool()}),
    (_rope, {**_rope_codes(), "kc": _pool(torch.int16)}),
    # a query without a place for its rotation; positions and slots of more dimensions than they have
    (_rope, dict(q_out=None)), (_rope, dict(pos=_t(1, N, 2, dtype=torch.int64))),
    (_rope, dict(slots=_t(N, 2, dtype=torch.int64)))])
def test_parts_that_do_not_fit_are_refused(lib, call, kw):
    with pytest.raises(ValueError):
        call(**kw)
    assert lib.reached == 0


def _evict(**kw):
    a = dict(new_lens=_t(S, dtype=I32), weights_out=_t(S, HKV, MC, dtype=F32), positions_out=None,
             weights=_t(S, HKV, MC, dtype=F32), k_cache=_pool(), v_cache=_pool(), block_tables=_t(S, 3, dtype=I32),
             new_block_tables=_t(S, 3, dtype=I32), context_lens=_t(S, dtype=I32), max_context=MC, keep=8, num_sink=0,
             num_recent=0, workspace=_t(64, dtype=U8), stream=STREAM)
    a.update(kw)
    B.pa_evict(**a)


_RECORDED = dict(positions=_t(S, HKV, MC, dtype=I32), recorded_lens=_t(S, dtype=I32), seen_lens=_t(S, dtype=I32))
_CODE_POOLS = dict(k_cache=_pool(U8), v_cache=_pool(U8), k_scales=_scales(), v_scales=_scales())


@pytest.mark.parametrize("kw", [{}, _RECORDED, _CODE_POOLS])
def test_evict_reaches_the_library(lib, kw):
    _evict(**kw)
    assert lib.reached == 1


@pytest.mark.parametrize("kw", [
    {**_RECORDED, "recorded_lens": _t(S - 1, dtype=I32)}, {**_RECORDED, "seen_lens": _t(1, dtype=I32)},
    {**_RECORDED, "seen_lens": _t(S, 2, dtype=I32)}, dict(new_lens=_t(S, 2, dtype=I32)),
    {**_CODE_POOLS, "v_scales": None}, {**_CODE_POOLS, "k_scales": None},
    {**_CODE_POOLS, "v_scales": _scales(2)}])
def test_evict_refuses_lengths_and_scales_that_do_not_fit(lib, kw):
    """A length per sequence: a shorter array would be read past its end."""
    with pytest.raises(ValueError):
        _evict(**kw)
    assert lib.reached == 0


def _on(device, t):
    t._on = device
    return t


@pytest.mark.parametrize("call, kw", [
    (_decode, dict(v=_on(1, _pool()))), (_decode, dict(tables=_on(1, _t(S, 3, dtype=I32)))),
    (_prompt, dict(q=_on(1, _t(N, HQ, HD)))), (_rope, dict(k=_on(1, _t(N, HKV, HD)))),
    (_rope, dict(pos=_on(1, _t(1, N, dtype=torch.int64)))), (_rope, dict(vc=_on(1, _pool()))),
    (_evict, dict(k_cache=_on(1, _pool()))), (_evict, dict(weights=_on(1, _t(S, HKV, MC, dtype=F32))))])
def test_tensors_of_another_device_are_refused(lib, call, kw):
    with pytest.raises(ValueError, match="device"):
        call(**kw)
    assert lib.reached == 0


@pytest.mark.parametrize("call", [_decode, _prompt, _rope, _evict])
def test_a_current_device_other_than_the_tensors_is_refused(lib, monkeypatch, call):
    """The library launches on the current device."""
    monkeypatch.setattr(B, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="device"):
        call()
    assert lib.reached == 0


@pytest.mark.parametrize("call", [_decode, _prompt, _rope])
def test_a_stream_of_another_device_is_refused(lib, monkeypatch, call):
    monkeypatch.setattr(STREAM, "device_index", 1)
    with pytest.raises(ValueError, match="device"):
        call()
    assert lib.reached == 0
