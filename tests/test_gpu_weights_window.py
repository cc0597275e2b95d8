"""pa_prompt_weights with a window much shorter than the prompt: the statistics
are then laid out by counted row, request by request."""
import pytest
import torch

from cache_ops import Batch, DTYPES, prompt_exact, weight_rtol
from test_gpu_weights import DEV, _check_weights, _prompt, _start_weights, pa  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("new, lens, hq, hkv, hd, bs, dtype, window, causal, fp8", [
    ([3000, 1, 700, 0, 40], [3000, 900, 5000, 30, 41], 12, 2, 128, 16, "bf16", 40, True, False),
    ([6000], [6000], 32, 8, 128, 16, "f16", 32, True, False),
    ([900, 2100, 33], [900, 2100, 33], 8, 2, 64, 16, "bf16", 500, True, False),
    ([2500, 7, 600], [3000, 7, 600], 4, 2, 256, 16, "bf16", 16, False, False),
    ([2000, 40], [2000, 3000], 8, 2, 128, 16, "bf16", 24, True, True),
    ([700, 60, 1], [700, 500, 9], 6, 2, 40, 12, "f32", 17, True, False)])
def test_short_window_over_long_prompts(pa, new, lens, hq, hkv, hd, bs, dtype, window, causal, fp8):  # noqa: F811
    b = Batch(lens, hkv, hd, bs, dtype, 19, fp8).to(DEV)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn((cu[-1], hq, hd), generator=torch.Generator().manual_seed(13)).to(DTYPES[dtype])
    before = _start_weights(len(lens), hkv, b.max_context, 4)
    w = before.to(DEV)
    _prompt(pa, b, q.to(DEV), cu, window, hd ** -0.5, w, causal)
    want, rtol = prompt_exact(b, q, cu, window, hd ** -0.5, causal, before)
    _check_weights(w.cpu(), want, before, b, rtol)


@pytest.mark.parametrize("kernel", [0, 1])
def test_more_requests_than_a_launch_takes(pa, kernel):  # noqa: F811
    """Each launch's requests use the same rows of the workspace again."""
    S, window = 4105, 2
    b = Batch([5] * S, 1, 64, 16, "bf16", 3).to(DEV)
    q = torch.randn((4 * S, 2, 64), generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
    w = torch.full((S, 1, 5), 2.0, device=DEV)
    pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, kernel)
    try:
        _prompt(pa, b, q.to(DEV), list(range(0, 4 * S + 1, 4)), window, 0.125, w)
    finally:
        pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, 0)
    k = torch.stack([b.k[b.tables[s, 0].long(), :5, 0] for s in range(S)]).double()
    x = torch.einsum("srgd,std->sgrt", q.view(S, 4, 2, 64)[:, 2:].double(), k) * 0.125
    x[:, :, 0, 4] = -float("inf")
    want = torch.softmax(x, -1).sum((1, 2))
    want[:, 0] += 2.0  # the one token that was there before
    mag = float(torch.einsum("srgd,std->sgrt", q.view(S, 4, 2, 64).double().abs(), k.abs()).max()) * 0.125
    assert bool(((w.cpu()[:, 0].double() - want).abs() <= (weight_rtol(64, mag, 5, 4) + 2.0 ** -23) * want).all())
