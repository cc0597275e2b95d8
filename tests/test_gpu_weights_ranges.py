"""pa_decode_weights_fp8 with queries of any size: a code cache's scores are
products in f16, which the query's own range must not be cut to."""
import pytest
import torch

from cache_ops import Batch, decode_exact
from helpers import within_tol
from test_gpu_weights import DEV, _check_weights, _decode, _start_weights, pa  # noqa: F401 (pa: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq, hkv, hd", [(8, 2, 128), (24, 2, 128), (4, 1, 256), (20, 2, 256)])
@pytest.mark.parametrize("size", ["large", "small", "mixed", "zero"])
def test_queries_beyond_the_f16_range(pa, hq, hkv, hd, size):  # noqa: F811
    b = Batch([300, 17, 64], hkv, hd, 16, "bf16", 3, True).to(DEV)
    q = torch.randn((3, hq, hd), generator=torch.Generator().manual_seed(8))
    at = torch.full((1, hq, 1), {"large": 2.0 ** 20, "small": 2.0 ** -24, "mixed": 1.0, "zero": 0.0}[size])
    if size == "mixed":  # heads of one KV head far apart
        at[0, ::2, 0], at[0, 1::2, 0] = 2.0 ** 18, 2.0 ** 9
    q = (q * at).to(torch.bfloat16)
    scale = hd ** -0.5 / (float(at.max()) or 1.0)
    before = _start_weights(3, hkv, 310, 4)
    w = before.to(DEV)
    out = _decode(pa, b, q.to(DEV), w, scale)
    eo, ew, rtol = decode_exact(b, q, scale, before)
    ok, err = within_tol(out.double().cpu().numpy(), eo.numpy(), "bf16")
    assert ok, err
    _check_weights(w.cpu(), ew, before, b, rtol)


def test_an_infinite_query_stays_in_its_head(pa):  # noqa: F811
    """Its softmax is NaN, the other heads' are not; a NaN element neither raises nor lowers the others."""
    b = Batch([100], 2, 128, 16, "bf16", 3, True).to(DEV)
    q = torch.randn((1, 4, 128), generator=torch.Generator().manual_seed(8)).to(torch.bfloat16)
    q[0, 0, 5] = float("inf")
    w = torch.zeros((1, 2, 100), device=DEV)
    out = _decode(pa, b, q.to(DEV), w, 0.1).cpu()
    assert not bool(out[0, 0].isfinite().any()) and bool(out[0, 1:].isfinite().all())
    assert bool(w[0, 0].isnan().all()) and bool(w[0, 1].isfinite().all())
    q[0, 0, 5] = float("nan")
    w.zero_()
    out = _decode(pa, b, q.to(DEV), w, 0.1).cpu()
    assert bool(out[0, 0].isnan().all()) and bool(out[0, 1:].isfinite().all())
