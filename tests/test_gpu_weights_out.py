"""pa_decode_weights' out beside pa_decode's: the same up to the roundings each makes."""
import pytest
import torch

from cache_ops import Batch, DTYPES, EPS, softmax_rows
from test_gpu_weights import DEV, _decode, pa  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens, hq, hkv, hd, bs, dtype, fp8", [
    ([1, 17, 300, 0, 1000], 32, 8, 128, 16, "bf16", False), ([700, 31], 12, 2, 64, 16, "f16", False),
    ([5000], 32, 8, 128, 16, "bf16", False), ([9000, 70], 4, 1, 256, 16, "f16", False),
    ([77, 200], 8, 2, 128, 12, "bf16", False), ([60, 5], 4, 2, 40, 16, "f32", False),
    ([3500, 12, 1, 800], 32, 8, 128, 16, "bf16", True), ([100, 37], 12, 2, 256, 16, "f16", True)])
def test_out_is_the_decodes(pa, lens, hq, hkv, hd, bs, dtype, fp8):  # noqa: F811
    b = Batch(lens, hkv, hd, bs, dtype, 7, fp8).to(DEV)
    S, G = len(lens), hq // hkv
    q = torch.randn((S, hq, hd), generator=torch.Generator().manual_seed(2)).to(DTYPES[dtype])
    dq, scale, mc = q.to(DEV), hd ** -0.5, b.max_context
    out = _decode(pa, b, dq, torch.zeros((S, hkv, mc), device=DEV), scale).double().cpu()
    size = pa.pa_decode_fp8_workspace_size if fp8 else pa.pa_decode_workspace_size
    ws = torch.empty(max(16, size(S, hq, hkv, hd, bs, mc, dq.dtype)), dtype=torch.uint8, device=DEV)
    plain = torch.full_like(dq, float("nan"))
    if fp8:
        pa.pa_decode_fp8(plain, dq, b.dk, b.dv, *b.dscales, b.dtables, b.dlens, mc, scale, workspace=ws)
    else:
        pa.pa_decode(plain, dq, b.dk, b.dv, b.dtables, b.dlens, mc, scale, workspace=ws)
    plain = plain.double().cpu()
    for s, L in enumerate(lens):
        if L == 0:
            assert not bool(out[s].any()) and not bool(plain[s].any())
            continue
        for h in range(hkv):
            rows = slice(h * G, (h + 1) * G)
            p, mag = softmax_rows(q[s, rows], b.rows(0, s, h), scale, torch.ones((G, L), dtype=torch.bool))
            pv = p @ b.rows(1, s, h).abs()
            # each side rounds its probabilities (half a step of the type, f16 over codes) and its result once; the
            # scores' and sums' fp32 roundings as in weight_rtol; over codes the plain side rounds the scaled query to
            # f16, which enters the exponential and the row's sum
            eps = EPS["f16"] if fp8 else EPS[dtype]
            rel = 2 * eps + 4 * (hd + 4) * 2.0 ** -23 * max(mag, 1.0) + 2 * L * 2.0 ** -24
            if fp8:
                rel += 2 * 2.0 ** -11 * mag
            tol = rel * pv + 2 * EPS[dtype] * torch.maximum(out[s, rows].abs(), plain[s, rows].abs())
            assert bool(((out[s, rows] - plain[s, rows]).abs() <= tol).all()), (s, h)
