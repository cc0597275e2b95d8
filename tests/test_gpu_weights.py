"""pa_decode_weights and pa_prompt_weights (16-bit, fp32 and quantized caches)
against 64-bit softmax weights; tolerances from cache_ops.weight_rtol."""
import numpy as np
import pytest
import torch

from cache_ops import Batch, DTYPES, decode_exact, prompt_exact, weight_rtol
from helpers import within_tol

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module")
def pa():
    import __graft_entry__

    __graft_entry__.build()
    import paged_kv_cache_116_gb300 as pa

    return pa


def _start_weights(S, hkv, stride, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.rand((S, hkv, stride), generator=g) * 0.1


def _check_weights(got, want, before, b, rtol):
    """Entries inside each sequence within rtol (of the added part and the stored sum), the others untouched."""
    for s, L in enumerate(b.lens):
        assert torch.equal(got[s, :, L:], before[s, :, L:]), s
        x, y = got[s, :, :L].double(), want[s, :, :L]
        bad = (x - y).abs() > (rtol + 2.0 ** -23) * y.abs()
        assert not bool(bad.any()), (s, float(((x - y).abs() / y.abs()).max()), rtol)


def _decode(pa, b, dq, w, scale, ws=None, max_context=None):
    S, hq, hd = dq.shape
    mc = b.max_context if max_context is None else max_context
    size = pa.pa_decode_weights_fp8_workspace_size if b.fp8 else pa.pa_decode_weights_workspace_size
    if ws is None:
        ws = torch.full((max(16, size(S, hq, b.hkv, hd, b.bs, mc, dq.dtype)),), 0xFF, dtype=torch.uint8, device=DEV)
    out = torch.full_like(dq, float("nan"))
    if b.fp8:
        pa.pa_decode_weights_fp8(out, w, dq, b.dk, b.dv, *b.dscales, b.dtables, b.dlens, mc, scale, workspace=ws)
    else:
        pa.pa_decode_weights(out, w, dq, b.dk, b.dv, b.dtables, b.dlens, mc, scale, workspace=ws)
    return out


DECODE = [
    # lens, hq, hkv, hd, bs, dtype, fp8
    ([6, 13, 1, 20], 4, 2, 32, 4, "f32", False),
    ([1, 17, 300, 0, 64, 1000], 32, 8, 128, 16, "bf16", False),
    ([5, 1, 2, 16, 33], 12, 2, 128, 16, "f16", False),
    ([700, 31], 40, 40, 64, 16, "f16", False),
    ([129, 64, 2000], 16, 1, 128, 8, "bf16", False),
    ([257, 90], 6, 2, 256, 64, "bf16", False),
    ([77, 200], 8, 2, 128, 12, "bf16", False),      # a block size that is gathered row by row
    ([40, 0, 3], 34, 2, 128, 16, "bf16", False),    # more query heads than the tensor-core kernel takes
    ([50, 120], 4, 4, 100, 16, "f16", False),       # a head_dim it does not take
    ([5000], 32, 8, 128, 16, "bf16", False),        # one long sequence, split
    ([16000, 3], 12, 2, 64, 8, "bf16", False),      # few units in hundreds of pieces
    ([9000, 70], 4, 1, 256, 16, "f16", False),
    ([12000], 8, 1, 128, 16, "bf16", True),
    ([3500, 12, 1, 800], 32, 8, 128, 16, "bf16", True),
    ([100, 37], 12, 2, 256, 16, "f16", True),
    ([60, 19], 8, 8, 128, 8, "f16", True),
    ([21, 48], 4, 2, 64, 16, "f32", True),
]


@pytest.mark.parametrize("case", DECODE)
def test_decode_weights(pa, case):
    lens, hq, hkv, hd, bs, dtype, fp8 = case
    b = Batch(lens, hkv, hd, bs, dtype, 7, fp8).to(DEV)
    q = torch.randn((len(lens), hq, hd), generator=torch.Generator().manual_seed(2)).to(DTYPES[dtype])
    stride = b.max_context + 5
    before = _start_weights(len(lens), hkv, stride, 4)
    w = before.to(DEV)
    scale = hd ** -0.5
    out = _decode(pa, b, q.to(DEV), w, scale)
    eo, ew, rtol = decode_exact(b, q, scale, before)
    ok, err = within_tol(out.double().cpu().numpy(), eo.numpy(), dtype)
    assert ok, err
    _check_weights(w.cpu(), ew, before, b, rtol)


def test_decode_weights_accumulate_and_repeat(pa):
    """Three steps add up; two runs from the same start give the same bits; a larger max_context changes nothing
    beyond the tolerance."""
    b = Batch([900, 33, 256], 8, 128, 16, "bf16", 5).to(DEV)
    q = torch.randn((3, 3, 32, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    before = _start_weights(3, 8, 1000, 4)
    runs = []
    for mc in (None, None, 1000):
        w = before.to(DEV)
        for i in range(3):
            _decode(pa, b, q[i].to(DEV), w, 0.088, max_context=mc)
        runs.append(w.cpu())
    want, rtol = before, 0.0
    for i in range(3):
        _, want, r = decode_exact(b, q[i], 0.088, want)
        rtol = max(rtol, r)
    for got in runs:
        _check_weights(got, want, before, b, rtol + 3 * 2.0 ** -24)
    assert torch.equal(runs[0], runs[1])


def test_decode_weights_shared_blocks(pa):
    """Two sequences over the same blocks keep separate weights."""
    b = Batch([200, 200], 2, 128, 16, "bf16", 6)
    b.tables[1] = b.tables[0]
    b.to(DEV)
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    before = _start_weights(2, 2, 200, 4)
    w = before.to(DEV)
    _decode(pa, b, q.to(DEV), w, 0.1)
    _, want, rtol = decode_exact(b, q, 0.1, before)
    _check_weights(w.cpu(), want, before, b, rtol)


def test_decode_weights_large_scores(pa):
    """Scores of several hundred: the weights stay within the tolerance their magnitude gives."""
    b = Batch([300, 64], 2, 128, 16, "bf16", 6, spread=6.0).to(DEV)
    q = (torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(2)) * 6).to(torch.bfloat16)
    before = torch.zeros((2, 2, 300))
    w = before.to(DEV)
    _decode(pa, b, q.to(DEV), w, 0.2)
    _, want, rtol = decode_exact(b, q, 0.2, before)
    got = w.cpu()
    for s, L in enumerate(b.lens):
        err = (got[s, :, :L].double() - want[s, :, :L]).abs()
        assert bool((err <= rtol * want[s, :, :L] + 1e-30).all())


def test_decode_weights_nan_stays_in_its_sequence(pa):
    b = Batch([100, 80], 2, 128, 16, "bf16", 6)
    b.k[b.tables[0, 1].long(), 3, 0] = float("nan")  # a key of sequence 0, head 0
    b.to(DEV)
    q = torch.randn((2, 8, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    w = torch.zeros((2, 2, 100), device=DEV)
    out = _decode(pa, b, q.to(DEV), w, 0.1).cpu()
    got = w.cpu()
    assert bool(got[0, 0].isnan().all()) and bool(out[0, :4].isnan().all())
    assert bool(got[0, 1].isfinite().all()) and bool(got[1].isfinite().all()) and bool(out[1].isfinite().all())


def test_decode_weights_graph_and_stream(pa):
    b = Batch([1500, 1, 333, 64], 8, 128, 16, "bf16", 8).to(DEV)
    gen = torch.Generator().manual_seed(1)
    dq = torch.randn((4, 32, 128), generator=gen).to(torch.bfloat16).to(DEV)
    n = pa.pa_decode_weights_workspace_size(4, 32, 8, 128, 16, 1500, torch.bfloat16)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    w = torch.zeros((4, 8, 1500), device=DEV)
    out = torch.empty_like(dq)

    def step(out, w, ws):
        pa.pa_decode_weights(out, w, dq, b.dk, b.dv, b.dtables, b.dlens, 1500, 0.088, workspace=ws)

    step(out, w, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="thread_local"):
        step(out, w, ws)
    ref_w, ref = torch.zeros_like(w), torch.empty_like(out)
    w.zero_()
    st = torch.cuda.Stream()
    ws2 = torch.empty_like(ws)
    st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        dq.copy_(torch.randn(dq.shape, generator=gen).to(torch.bfloat16))
        g.replay()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step(ref, ref_w, ws2)
        torch.cuda.current_stream().wait_stream(st)
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(w, ref_w)


def _prompt(pa, b, dq, cu, window, scale, w, causal=True):
    T, hq, hd = dq.shape
    S = len(b.lens)
    mq = max(cu[i + 1] - cu[i] for i in range(S))
    size = pa.pa_prompt_weights_fp8_workspace_size if b.fp8 else pa.pa_prompt_weights_workspace_size
    n = size(S, T, mq, hq, b.hkv, hd, b.bs, b.max_context, window, dq.dtype)
    ws = torch.full((max(16, n),), 0xFF, dtype=torch.uint8, device=DEV)
    dcu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    if b.fp8:
        pa.pa_prompt_weights_fp8(w, dq, b.dk, b.dscales[0], b.dtables, b.dlens, dcu, mq, b.max_context, window, scale,
                                 causal=causal, workspace=ws)
    else:
        pa.pa_prompt_weights(w, dq, b.dk, b.dtables, b.dlens, dcu, mq, b.max_context, window, scale, causal=causal,
                             workspace=ws)


PROMPT = [
    # new, lens, hq, hkv, hd, bs, dtype, window, causal, fp8
    ([5, 3, 1], [6, 13, 1], 4, 2, 32, 4, "f32", 0, True, False),
    ([300, 64, 1, 0, 17], [300, 200, 40, 25, 17], 12, 2, 128, 16, "bf16", 0, True, False),
    ([300, 64, 1, 0, 17], [300, 200, 40, 25, 17], 12, 2, 128, 16, "bf16", 32, True, False),
    ([129, 700], [129, 1500], 8, 2, 64, 16, "f16", 0, True, False),
    ([40, 33], [2000, 129], 32, 8, 128, 32, "bf16", 16, True, False),
    ([200, 90], [260, 128], 4, 4, 128, 8, "f16", 0, False, False),
    ([64, 10], [200, 500], 40, 2, 128, 16, "bf16", 8, True, False),
    ([3], [5000], 16, 1, 128, 16, "bf16", 0, True, False),
    ([90, 31], [150, 260], 6, 2, 256, 16, "bf16", 0, True, False),
    ([50, 60], [77, 80], 4, 2, 128, 12, "f16", 0, True, False),
    ([130, 20], [300, 600], 8, 2, 128, 16, "bf16", 0, True, True),
    ([64, 20], [64, 900], 12, 2, 128, 16, "f16", 24, True, True),
    ([20, 9], [50, 9], 4, 2, 64, 16, "f32", 0, True, True),
    ([1200, 300], [1300, 4000], 8, 2, 128, 16, "f16", 0, True, False),
    ([600, 2], [900, 3], 14, 2, 64, 64, "bf16", 0, True, False),
    ([70, 5], [90, 700], 128, 1, 64, 16, "bf16", 0, True, False),
    ([40, 129], [40, 260], 4, 2, 256, 8, "f16", 0, True, False),
    ([33, 1], [9000, 2500], 32, 8, 128, 256, "bf16", 32, True, False),
    ([900, 40], [1300, 2000], 8, 2, 128, 16, "bf16", 0, True, True),
    ([40, 33], [6000, 300], 32, 8, 128, 16, "f16", 32, True, True),
    ([200, 31], [260, 500], 6, 2, 64, 24, "bf16", 0, True, True),
    ([50, 130], [500, 140], 4, 2, 256, 16, "f16", 0, False, True),
    ([300, 20], [400, 900], 12, 2, 128, 1, "bf16", 0, True, False),
]


@pytest.mark.parametrize("case", PROMPT)
def test_prompt_weights(pa, case):
    new, lens, hq, hkv, hd, bs, dtype, window, causal, fp8 = case
    b = Batch(lens, hkv, hd, bs, dtype, 17, fp8).to(DEV)
    cu = [0] + list(np.cumsum(new))
    q = torch.randn((cu[-1], hq, hd), generator=torch.Generator().manual_seed(12)).to(DTYPES[dtype])
    before = _start_weights(len(lens), hkv, b.max_context + 3, 4)
    w = before.to(DEV)
    scale = hd ** -0.5
    _prompt(pa, b, q.to(DEV), cu, window, scale, w, causal)
    want, rtol = prompt_exact(b, q, cu, window, scale, causal, before)
    got = w.cpu()
    _check_weights(got, want, before, b, rtol)
    again = before.to(DEV)
    _prompt(pa, b, q.to(DEV), cu, window, scale, again, causal)
    assert torch.equal(again.cpu(), got)


def test_prompt_weights_of_single_tokens_match_decode(pa):
    """One new token per request: the prompt form and the decode form add the same weights."""
    b = Batch([300, 5, 64, 1], 2, 128, 16, "bf16", 21).to(DEV)
    q = torch.randn((4, 8, 128), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    before = _start_weights(4, 2, 300, 9)
    w1, w2 = before.to(DEV), before.to(DEV)
    _decode(pa, b, q.to(DEV), w1, 0.09)
    _prompt(pa, b, q.to(DEV), [0, 1, 2, 3, 4], 0, 0.09, w2)
    _, want, rtol = decode_exact(b, q, 0.09, before)
    _check_weights(w1.cpu(), want, before, b, rtol)
    _check_weights(w2.cpu(), want, before, b, rtol)


def test_prompt_weights_many_requests(pa):
    """More requests than one launch lists (their prefix lives in shared memory)."""
    S = 4100
    b = Batch([2] * S, 1, 64, 16, "bf16", 3).to(DEV)
    q = torch.randn((S, 2, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    before = torch.zeros((S, 1, 2))
    for form in ("prompt", "decode"):
        w = before.to(DEV)
        if form == "prompt":
            _prompt(pa, b, q.to(DEV), list(range(S + 1)), 0, 0.125, w)
        else:
            _decode(pa, b, q.to(DEV), w, 0.125)
        k = torch.stack([b.k[b.tables[s, 0].long(), :2, 0] for s in range(S)]).double()
        want = torch.softmax(torch.einsum("sgd,std->sgt", q.double(), k) * 0.125, -1).sum(1)
        assert bool(((w.cpu()[:, 0].double() - want).abs() <= 1e-4 * want).all()), form


def test_prompt_weights_infinite_key(pa):
    """A key every query gives a score of -infinity weighs 0, whatever the group size pads a query tile with."""
    b = Batch([200], 1, 128, 16, "f16", 3)
    b.k.clamp_(min=0.01)
    b.k[b.tables[0, 2].long(), 5, 0, 7] = -float("inf")  # token 37
    b.to(DEV)
    q = torch.rand((150, 6, 128), generator=torch.Generator().manual_seed(3)).clamp(min=0.01).to(torch.float16)
    before = torch.zeros((1, 1, 200))
    w = before.to(DEV)
    _prompt(pa, b, q.to(DEV), [0, 150], 0, 0.05, w)
    b.k[b.tables[0, 2].long(), 5, 0, 7] = -60000.0  # finite for the reference: the weight underflows to 0 as well
    want, rtol = prompt_exact(b, q, [0, 150], 0, 0.05, True, before)
    got = w.cpu()
    assert float(got[0, 0, 37]) == 0.0
    want[0, 0, 37] = 0.0
    b.k[b.tables[0, 2].long(), 5, 0, 7] = 0.01
    _, rtol = prompt_exact(b, q, [0, 150], 0, 0.05, True, before)
    assert bool(((got.double() - want).abs() <= rtol * want).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_pinned_kernels_and_grids_agree(pa, fp8):
    """The CUDA-core and the tensor-core forms, and decode grids of other sizes, within the tolerance."""
    b = Batch([700, 33, 90], 2, 128, 16, "bf16", 23, fp8).to(DEV)
    new, cu = [64, 1, 90], [0, 64, 65, 155]
    gen = torch.Generator().manual_seed(4)
    q1 = torch.randn((3, 8, 128), generator=gen).to(torch.bfloat16)
    qp = torch.randn((cu[-1], 8, 128), generator=gen).to(torch.bfloat16)
    before = _start_weights(3, 2, 700, 4)
    _, want1, r1 = decode_exact(b, q1, 0.09, before)
    wantp, rp = prompt_exact(b, qp, cu, 40, 0.09, True, before)
    try:
        for kernel, ctas in ((1, 0), (2, 0), (2, 3), (2, 400)):
            pa.pa_set_option(pa.PA_OPT_DECODE_KERNEL, kernel)
            pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, kernel)
            pa.pa_set_option(pa.PA_OPT_DECODE_CTAS, ctas)
            w = before.to(DEV)
            _decode(pa, b, q1.to(DEV), w, 0.09)
            _check_weights(w.cpu(), want1, before, b, r1)
            w = before.to(DEV)
            _prompt(pa, b, qp.to(DEV), cu, 40, 0.09, w)
            _check_weights(w.cpu(), wantp, before, b, rp)
    finally:
        for o in (pa.PA_OPT_DECODE_KERNEL, pa.PA_OPT_VARLEN_KERNEL, pa.PA_OPT_DECODE_CTAS):
            pa.pa_set_option(o, 0)


def test_check_mode_refuses_bad_batches(pa):
    """Check mode: indexes are validated on the host, nothing is launched, the weights stay as they are."""
    b = Batch([50, 20], 2, 128, 16, "bf16", 23).to(DEV)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device=DEV)
    w = torch.full((2, 2, 50), 3.0, device=DEV)
    pa.pa_set_check_mode(True)
    try:
        for bad in ("length", "block"):
            lens, tables = b.dlens.clone(), b.dtables.clone()
            if bad == "length":
                lens[1] = 51
            else:
                tables[0, 1] = b.num_blocks
            keep = b.dlens, b.dtables
            b.dlens, b.dtables = lens, tables
            with pytest.raises(pa.PAError) as e:
                _decode(pa, b, q, w, 0.1)
            assert e.value.status == 3
            with pytest.raises(pa.PAError) as e:
                _prompt(pa, b, q, [0, 1, 2], 0, 0.1, w)
            assert e.value.status == 3
            b.dlens, b.dtables = keep
        with pytest.raises(pa.PAError) as e:
            _prompt(pa, b, torch.zeros((71, 8, 128), dtype=torch.bfloat16, device=DEV), [0, 50, 71], 0, 0.1, w)
        assert e.value.status == 3  # more new tokens than context
        _decode(pa, b, q, w, 0.1)
    finally:
        pa.pa_set_check_mode(False)
    assert float(w[0, 0, 49]) != 3.0 and float(w[1, 0, 20]) == 3.0


def test_prompt_weights_more_requests_than_a_launch(pa):
    """Over 4,096 requests with long ones on both sides of the cut; the CUDA-core form answers for all of them."""
    S, hkv, hd = 4105, 2, 64
    new = [1] * S
    lens = [2 + s % 5 for s in range(S)]
    for s, n in ((0, 200), (4095, 150), (4096, 180), (4104, 300)):
        new[s], lens[s] = n, n + s % 3
    cu = np.concatenate(([0], np.cumsum(new))).tolist()
    b = Batch(lens, hkv, hd, 16, "bf16", 31).to(DEV)
    q = torch.randn((cu[-1], 4, hd), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    before = _start_weights(S, hkv, 301, 2)
    got, ref = before.to(DEV), before.to(DEV)
    _prompt(pa, b, q, cu, 0, 0.1, got)
    try:
        pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, 1)
        _prompt(pa, b, q, cu, 0, 0.1, ref)
    finally:
        pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, 0)
    mag = float(q.float().norm(dim=-1).max() * b.k.float().nan_to_num().norm(dim=-1).max()) * 0.1 * 1.45
    rtol = 2 * weight_rtol(hd, mag, 301, 600)  # both are off
    for s in range(S):
        lens_s = lens[s]
        assert torch.equal(got[s, :, lens_s:], ref[s, :, lens_s:])
    assert bool(((got - ref).abs() <= rtol * ref.abs()).all()), float(((got - ref).abs() / ref.abs()).max())


def test_prompt_weights_graphs_share_a_workspace_and_streams_do_not(pa):
    """Two captured calls on one workspace, replayed in turn; then the same two and an attention step at once on three
    streams with memory of their own.  Every run gives the eager call's bits."""
    b = Batch([700, 90, 1500], 4, 64, 16, "bf16", 41).to(DEV)
    cu, mq, mc = [0, 600, 640, 1000], 600, 1500
    gen = torch.Generator().manual_seed(3)
    q = [torch.randn((1000, 8, 64), generator=gen).to(torch.bfloat16).to(DEV) for _ in range(2)]
    dcu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    size = [pa.pa_prompt_weights_workspace_size(3, 1000, mq, 8, 4, 64, 16, mc, win, torch.bfloat16) for win in (0, 16)]

    def call(i, w, ws):
        pa.pa_prompt_weights(w, q[i], b.dk, b.dtables, b.dlens, dcu, mq, mc, (0, 16)[i], 0.125, workspace=ws)

    want = [torch.zeros((3, 4, mc), device=DEV) for _ in range(2)]
    got = [torch.zeros((3, 4, mc), device=DEV) for _ in range(2)]
    shared = torch.empty(max(size), dtype=torch.uint8, device=DEV)
    for i in range(2):
        call(i, want[i], shared)
        want[i].zero_()
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, capture_error_mode="thread_local"):
            call(i, got[i], shared)
        graphs.append(g)
    for _ in range(3):
        for i in range(2):
            graphs[i].replay()
    own = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in size]
    for _ in range(3):
        for i in range(2):
            call(i, want[i], own[i])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

    def attend(out, ws):
        pa.pa_varlen(out, q[0], b.dk, b.dv, b.dtables, b.dlens, dcu, mq, mc, 0.125, workspace=ws)

    n = pa.pa_varlen_workspace_size(3, 1000, mq, 8, 4, 64, 16, mc, torch.bfloat16)
    vws = torch.empty(max(n, 16), dtype=torch.uint8, device=DEV)
    ref, out = torch.empty_like(q[0]), torch.empty_like(q[0])
    attend(ref, vws)
    for t in got + want:
        t.zero_()
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                call(i, got[i], own[i])
        with torch.cuda.stream(streams[2]):
            attend(out, vws)
    torch.cuda.synchronize()
    for _ in range(8):
        for i in range(2):
            call(i, want[i], shared)
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(out, ref)


@pytest.mark.parametrize("scale", [-0.09, 0.0, 3.0])
@pytest.mark.parametrize("fp8", [False, True])
def test_weights_at_any_scale(pa, scale, fp8):
    """A negative scale turns the order of the scores round, zero makes them equal, a large one leaves one key each."""
    b = Batch([900, 40, 333], 2, 128, 16, "f16", 51, fp8).to(DEV)
    new, cu = [700, 5, 40], [0, 700, 705, 745]
    gen = torch.Generator().manual_seed(6)
    q1 = torch.randn((3, 8, 128), generator=gen).to(torch.float16)
    qp = torch.randn((cu[-1], 8, 128), generator=gen).to(torch.float16)
    before = _start_weights(3, 2, 900, 5)
    _, want, rtol = decode_exact(b, q1, scale, before)
    w = before.to(DEV)
    _decode(pa, b, q1.to(DEV), w, scale)
    _close(w.cpu(), want, rtol)
    for window in (0, 16):
        want, rtol = prompt_exact(b, qp, cu, window, scale, True, before)
        w = before.to(DEV)
        _prompt(pa, b, qp.to(DEV), cu, window, scale, w)
        _close(w.cpu(), want, rtol)


def _close(got, want, rtol):
    """As _check_weights, and of up to 4,096 terms each may be lost below the smallest normal number."""
    assert bool(((got.double() - want).abs() <= (rtol + 2.0 ** -23) * want.abs() + 4096 * 2.0 ** -126).all())


def test_bindings_refuse_parts_that_do_not_fit(pa):
    b = Batch([50, 20], 2, 128, 16, "bf16", 23).to(DEV)
    q = torch.zeros((2, 8, 128), dtype=torch.bfloat16, device=DEV)
    w, cu = torch.zeros((2, 2, 50), device=DEV), torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    ws, out = torch.empty(1 << 24, dtype=torch.uint8, device=DEV), torch.empty_like(q)
    good = dict(out=out, weights=w, q=q, k_cache=b.dk, v_cache=b.dv, block_tables=b.dtables, context_lens=b.dlens,
                max_context=50, scale=0.1, workspace=ws)
    for bad in (dict(q=q.float(), out=out.float()), dict(q=q[..., :64].contiguous()), dict(out=out[:1]),
                dict(block_tables=b.dtables[:1]), dict(context_lens=b.dlens[:1]), dict(v_cache=b.dv[:2]),
                dict(weights=w[:1]), dict(weights=w.double())):
        with pytest.raises(ValueError):
            pa.pa_decode_weights(**{**good, **bad})
    good = dict(weights=w, q=q, k_cache=b.dk, block_tables=b.dtables, seq_lens=b.dlens, cu_seqlens_q=cu, max_q=1,
                max_context=50, window=0, scale=0.1, workspace=ws)
    for bad in (dict(q=q.half()), dict(cu_seqlens_q=cu[:2]), dict(block_tables=b.dtables[:1]),
                dict(weights=w[:, :1].contiguous())):
        with pytest.raises(ValueError):
            pa.pa_prompt_weights(**{**good, **bad})
    good = dict(new_lens=torch.zeros(2, dtype=torch.int32, device=DEV), weights_out=w.clone(), positions_out=None,
                weights=w, k_cache=b.dk, v_cache=b.dv, block_tables=b.dtables, new_block_tables=b.dtables,
                context_lens=b.dlens, max_context=50, keep=10, num_sink=0, num_recent=1, workspace=ws)
    for bad in (dict(new_block_tables=b.dtables[:1]), dict(v_cache=b.dv.half()),
                dict(weights_out=w[..., :40].contiguous())):
        with pytest.raises(ValueError):
            pa.pa_evict(**{**good, **bad})
    assert not bool(w.any())
