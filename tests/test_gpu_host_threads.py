"""Host threads call the same entry point at once, each on a stream and with
buffers of its own, two of each of two sizes: every call is answered, and as a
single thread's is.  (The sizes differ in the shared memory their launches ask
for, a limit that belongs to the kernel and so to both threads.)"""
import threading

import pytest
import torch

from cache_ops import Batch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


def _evict(pa, big):
    """One short sequence; max_context decides the launch."""
    mc = 40000 if big else 10000
    b = Batch([300], 1, 64, 16, "bf16", 5, extra_blocks=8).to(DEV)
    w = torch.rand((1, 1, mc), generator=torch.Generator().manual_seed(3)).to(DEV)
    to = torch.arange(b.num_blocks - 8, b.num_blocks, dtype=torch.int32, device=DEV).view(1, 8)
    n, wo = torch.zeros(1, dtype=torch.int32, device=DEV), torch.zeros_like(w)
    ws = torch.empty(pa.pa_evict_workspace_size(1, 1, mc, 128), dtype=torch.uint8, device=DEV)

    def call(stream=None):
        pa.pa_evict(n, wo, None, w, b.dk, b.dv, b.dtables, to, b.dlens, mc, 128, 4, 16, workspace=ws, stream=stream)
        return wo

    return call


def _batch(big, per=1, L=9):
    """Sequences of one block each: many, or three."""
    S = 4000 if big else 3
    b = Batch([L] * S, 1, 64, 16, "bf16", 5).to(DEV)
    q = torch.randn((S * per, 2, 64), generator=torch.Generator().manual_seed(4)).to(torch.bfloat16).to(DEV)
    return S, b, q


def _prompt(pa, big):
    S, b, q = _batch(big, 2, 2)
    w = torch.zeros((S, 1, 9), device=DEV)
    cu = torch.arange(0, 2 * S + 1, 2, dtype=torch.int32, device=DEV)
    ws = torch.empty(pa.pa_prompt_weights_workspace_size(S, 2 * S, 2, 2, 1, 64, 16, 9, 1, torch.bfloat16),
                     dtype=torch.uint8, device=DEV)

    def call(stream=None):
        # (every token is new: its weight is set, not added to)
        pa.pa_prompt_weights(w, q, b.dk, b.dtables, b.dlens, cu, 2, 9, 1, 0.1, workspace=ws, stream=stream)
        return w

    return call


def _decode_weights(pa, big):
    S, b, q = _batch(big)
    w, out = torch.zeros((S, 1, 9), device=DEV), torch.zeros_like(q)
    ws = torch.empty(pa.pa_decode_weights_workspace_size(S, 2, 1, 64, 16, 9, torch.bfloat16), dtype=torch.uint8,
                     device=DEV)

    def call(stream=None):
        pa.pa_decode_weights(out, w, q, b.dk, b.dv, b.dtables, b.dlens, 9, 0.1, ws, stream=stream)
        return out

    return call


def _decode(pa, big):
    S, b, q = _batch(big)
    out = torch.zeros_like(q)
    ws = torch.empty(pa.pa_decode_workspace_size(S, 2, 1, 64, 16, 9, torch.bfloat16), dtype=torch.uint8, device=DEV)

    def call(stream=None):
        pa.pa_decode(out, q, b.dk, b.dv, b.dtables, b.dlens, 9, 0.1, workspace=ws, stream=stream)
        return out

    return call


def _varlen(pa, big):
    S, b, q = _batch(big, 2)
    out = torch.zeros_like(q)
    cu = torch.arange(0, 2 * S + 1, 2, dtype=torch.int32, device=DEV)

    def call(stream=None):  # (without the workspace, whose plan would take the batch out of shared memory)
        pa.pa_varlen(out, q, b.dk, b.dv, b.dtables, b.dlens, cu, 2, 9, 0.1, stream=stream)
        return out

    return call


class _Recorder:
    """The library; keeps what its last entry point was called with."""

    def __init__(self, lib):
        self.lib = lib

    def __getattr__(self, name):
        fn = getattr(self.lib, name)

        def call(*args):
            self.last = fn, args
            return fn(*args)

        return call


@pytest.mark.parametrize("make", [_evict, _prompt, _decode_weights, _decode, _varlen])
def test_threads_with_launches_of_different_size(pa, make, monkeypatch):
    from paged_kv_cache_116_gb300 import _binding

    rec = _Recorder(pa.lib())
    calls = [make(pa, big) for big in (False, True, False, True)]
    want = [c().clone() for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    raw = []  # the entry points themselves: a thread spends its time in the library, not in Python
    with monkeypatch.context() as m:
        m.setattr(_binding, "lib", lambda: rec)
        for c, st in zip(calls, streams):
            c(st)
            raw.append(rec.last)
    torch.cuda.synchronize()
    failed, start = [], threading.Barrier(len(calls))

    def work(i):
        torch.cuda.set_device(DEV)
        fn, args = raw[i]
        start.wait()
        for k in range(3000):
            if fn(*args) != 0:
                failed.append(pa.lib().pa_last_error())
                return
            if k % 100 == 99:
                streams[i].synchronize()  # (a full launch queue would have the threads wait in turn)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not failed, failed[0]
    for c, st, ref in zip(calls, streams, want):
        got = c(st)
        st.synchronize()
        assert torch.equal(got, ref)


@pytest.mark.parametrize("make", [_evict, _prompt, _decode_weights, _decode, _varlen])
@pytest.mark.parametrize("ctas", [0, 3])
def test_first_call_of_a_thread(pa, make, ctas):
    """A thread that has made no CUDA call yet: its first is the library's (with a pinned decode grid nothing is asked
    of the device on the way)."""
    pa.pa_set_option(pa.PA_OPT_DECODE_CTAS, ctas)
    try:
        _first_call(make(pa, False))
    finally:
        pa.pa_set_option(pa.PA_OPT_DECODE_CTAS, 0)


def _first_call(call):
    want = call().clone()
    torch.cuda.synchronize()
    stream, got = torch.cuda.current_stream(), []

    def work():
        try:
            got.append(call(stream))
        except Exception as e:  # noqa: BLE001 (reported by the test's thread)
            got.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert torch.is_tensor(got[0]), got[0]
    assert torch.equal(got[0], want)
