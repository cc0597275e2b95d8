"""Batches whose scratch space (scores of a decode, dense keys of a prompt) is
beyond what one launch keeps: worked in parts, with max_context far above the
lengths."""
import pytest
import torch

from cache_ops import Batch, decode_exact, prompt_exact
from helpers import within_tol
from test_gpu_weights import DEV, _check_weights, _decode, pa  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs, fp8, window", [(12, False, 0), (16, True, 0), (16, True, 8), (12, False, 5)])
def test_dense_keys_in_parts(pa, bs, fp8, window):  # noqa: F811
    mc, S = 1 << 20, 7  # 4 heads of 128: 1.07 GB of 16-bit keys each, three requests at a time
    lens = [40, 300, 1, 0, 700, 33, 90]
    new = [30, 300, 1, 0, 20, 33, 1]
    b = Batch(lens, 4, 128, bs, "bf16", 7, fp8)
    b.max_context = mc
    b.to(DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], 8, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    before = torch.rand((S, 4, 700), generator=torch.Generator().manual_seed(4))
    w = torch.zeros((S, 4, mc), device=DEV)
    w[:, :, :700] = before.to(DEV)
    size = pa.pa_prompt_weights_fp8_workspace_size if fp8 else pa.pa_prompt_weights_workspace_size
    n = size(S, cu[-1], 300, 8, 4, 128, bs, mc, window, torch.bfloat16)
    assert n < 5 << 30
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV)
    dcu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    args = (b.dtables, b.dlens, dcu, 300, mc, window, 0.09)
    if fp8:
        pa.pa_prompt_weights_fp8(w, q.to(DEV), b.dk, b.dscales[0], *args, workspace=ws)
    else:
        pa.pa_prompt_weights(w, q.to(DEV), b.dk, *args, workspace=ws)
    want, rtol = prompt_exact(b, q, cu, window, 0.09, True, before)
    _check_weights(w[:, :, :700].cpu(), want, before, b, rtol)
    assert not bool(w[:, :, 700:].any())


@pytest.mark.parametrize("fp8", [False, True])
def test_scores_in_parts(pa, fp8):  # noqa: F811
    mc, S = 1 << 21, 45  # 16 heads: 134 MB of scores a sequence, 32 sequences at a time
    lens = [1 + (37 * s) % 400 for s in range(S)]
    lens[5] = lens[40] = 0
    b = Batch(lens, 4, 128, 16, "bf16", 7, fp8).to(DEV)
    q = torch.randn((S, 16, 128), generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    before = torch.rand((S, 4, 400), generator=torch.Generator().manual_seed(4))
    w = torch.zeros((S, 4, mc), device=DEV)
    w[:, :, :400] = before.to(DEV)
    out = _decode(pa, b, q.to(DEV), w, 0.09, max_context=mc)
    eo, ew, rtol = decode_exact(b, q, 0.09, before)
    ok, err = within_tol(out.double().cpu().numpy(), eo.numpy(), "bf16")
    assert ok, err
    _check_weights(w[:, :, :400].cpu(), ew, before, b, rtol)
    assert not bool(w[:, :, 400:].any())
