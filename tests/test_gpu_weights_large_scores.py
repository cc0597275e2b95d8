"""Equal keys under scores of thousands: every row's weights are equal whatever the
scores' size is, so a statistic that loses bits to it shows."""
import pytest
import torch

from cache_ops import Batch, DTYPES
from test_gpu_weights import DEV, _decode, _prompt, pa  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu


def _equal_keys(lens, hkv, hd, bs, dtype, fp8):
    b = Batch(lens, hkv, hd, bs, dtype, 7, fp8)
    if fp8:
        b.k.fill_(0x50)  # 8 in E4M3
        b.scales[0].fill_(1.0)
    else:
        b.k.fill_(8.0)
    return b.to(DEV)


@pytest.mark.parametrize("kernel", [0, 1])
@pytest.mark.parametrize("new, lens, hq, hkv, hd, bs, dtype, window, fp8", [
    ([61, 1], [61, 37], 8, 2, 128, 16, "bf16", 0, False), ([61, 23], [75, 23], 12, 2, 64, 16, "f16", 0, False),
    ([61, 50], [61, 70], 8, 2, 128, 16, "bf16", 7, False), ([300], [301], 4, 2, 256, 16, "bf16", 0, False),
    ([61, 1], [61, 37], 8, 2, 128, 16, "bf16", 0, True), ([700], [701], 8, 2, 128, 16, "f16", 0, False)])
def test_rows_of_equal_scores_weigh_their_keys_alike(pa, kernel, new, lens, hq, hkv, hd, bs, dtype, window,  # noqa: F811
                                                     fp8):
    b = _equal_keys(lens, hkv, hd, bs, dtype, fp8)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.full((cu[-1], hq, hd), 7.5, dtype=DTYPES[dtype], device=DEV)
    w = torch.zeros((len(lens), hkv, max(lens)), device=DEV)
    pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, kernel)
    try:
        _prompt(pa, b, q, cu, window, 0.37, w)
    finally:
        pa.pa_set_option(pa.PA_OPT_VARLEN_KERNEL, 0)
    for s, L in enumerate(lens):
        rows = new[s] if window == 0 else min(new[s], window)
        want = torch.zeros(L, dtype=torch.float64)
        for p in range(L - rows, L):
            want[:p + 1] += (hq // hkv) / (p + 1)
        # equal terms: their sums' roundings, as many as there are keys and rows, and the division's
        tol = (L + rows * (hq // hkv) + 8) * 2.0 ** -24
        got = w[s, :, :L].cpu().double()
        assert bool(((got - want).abs() <= tol * want).all()), (s, float(((got - want).abs() / want).max()), tol)


@pytest.mark.parametrize("fp8", [False, True])
def test_a_decode_of_equal_scores(pa, fp8):  # noqa: F811
    b = _equal_keys([61, 700], 2, 128, 16, "bf16", fp8)
    q = torch.full((2, 8, 128), 7.5, dtype=torch.bfloat16, device=DEV)
    w = torch.zeros((2, 2, 700), device=DEV)
    _decode(pa, b, q, w, 0.37)
    for s, L in enumerate(b.lens):
        assert bool(((w[s, :, :L].cpu().double() * L / 4 - 1).abs() <= (L + 12) * 2.0 ** -24).all())
