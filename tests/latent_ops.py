"""Plain 64-bit forms of the latent-cache and shared-prefix operators and the
inputs their tests share.  Written from the definitions in include/pa.h, on CPU
tensors; the product never imports this."""
import torch

from cache_ops import DTYPES, EPS, Batch, rope, rope_bound

LOW = {"f32": 0.0, "bf16": 0.0, "f16": 2.0 ** -25}  # half of the fixed step below the normal range


def latent_write(kv, positions, inv_freq, norm, eps, interleaved, lat):
    """(rows, bound of their error before the rounding to the type), in 64 bits."""
    x = kv.double()
    c = x[:, :lat]
    if norm is not None:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps) * norm.double()
    r = x[:, None, lat:]
    turned = rope(r, positions[None], inv_freq, None, interleaved)[:, 0]
    # the latent part: the sum of lat squares (lat 2^-24), division, eps, root, reciprocal (below 2 2^-24 on the root's
    # argument, so half of that on the result, and 2 roundings), two products
    bound = torch.cat((c.abs() * ((lat / 2 + 8) * 2.0 ** -24 if norm is not None else 0.0),
                       6 * 2.0 ** -24 * rope_bound(r, inv_freq.numel(), interleaved)[:, 0]), 1)
    return torch.cat((c, turned), 1), bound


class LatentBatch(Batch):
    """A paged latent cache with NaN in every unused slot."""

    def __init__(self, lens, lat, rot, bs, dtype, seed):
        super().__init__(lens, 1, lat + rot, bs, dtype, seed)
        self.lat, self.rot = lat, rot
        self.cache = self.k[:, :, 0].contiguous()

    def to(self, dev):
        self.dcache, self.dtables = self.cache.to(dev), self.tables.to(dev)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        return self


def attention(q, k, v, scale, seen, dtype, umma):
    """(out, bound) of rows q [rows, d] over keys k [L, d] and values v [L, e], in 64 bits.

    A score is d exact products summed in fp32 (the tensor cores cut where fp32 addition rounds: 2^-23 each), scaled by
    two more roundings; it enters the weight and the sum of the weights, so twice.  exp2 is good to 2^-21.  The weights
    are rounded to the type (tensor cores only; below f16's normal range by up to 2^-25, of a sum of at least one), n
    products are summed in fp32, joining pieces costs a few more, and the result is rounded to the type."""
    if k.shape[0] == 0:
        return torch.zeros((q.shape[0], v.shape[1]), dtype=torch.float64), torch.zeros((q.shape[0], 1), dtype=torch.float64)
    x = q.double() @ k.double().t() * scale
    p = torch.softmax(x.masked_fill(~seen, -float("inf")), -1)
    mag = float((q.double().abs() @ k.double().abs().t()).max()) * abs(scale)
    n, d = k.shape[0], q.shape[1]
    rel = 2 * (d + 4) * 2.0 ** -23 * mag + 4 * 2.0 ** -21 + (2 * n + 64) * 2.0 ** -23
    out, size = p @ v.double(), p @ v.double().abs()
    if umma:
        rel += EPS[dtype]
        size = size + LOW[dtype] * n * float(v.double().abs().max()) / rel
    return out, rel * size + EPS[dtype] * out.abs() * (1 + rel) + LOW[dtype]


def latent_exact(b, q, cu, scale, causal, umma):
    """q [T, H, lat + rot] on the CPU; cu None: one query per sequence."""
    T, H, _ = q.shape
    out = torch.zeros((T, H, b.lat), dtype=torch.float64)
    bound = torch.zeros((T, H, b.lat), dtype=torch.float64)
    for s, L in enumerate(b.lens):
        lo, hi = (s, s + 1) if cu is None else (cu[s], cu[s + 1])
        if hi == lo or L == 0:
            continue
        rows = b.rows(0, s, 0)
        seen = torch.ones((hi - lo, L), dtype=torch.bool)
        if causal:
            seen = torch.arange(L - (hi - lo), L)[:, None] >= torch.arange(L)
        seen = seen.repeat_interleave(H, 0)
        o, e = attention(q[lo:hi].reshape(-1, q.shape[2]), rows, rows[:, : b.lat], scale, seen, b.dtype, umma)
        out[lo:hi], bound[lo:hi] = o.view(hi - lo, H, -1), e.expand(-1, b.lat).reshape(hi - lo, H, -1)
    return out, bound


class SharedBatch(Batch):
    """Groups (members, prefix, tails) of sequences whose tables begin alike; members 0 tails on their own: loners."""

    def __init__(self, groups, hkv, hd, bs, dtype, seed, loners=()):
        lens, starts, prefix = [], [0], []
        for pre, tails in groups:
            lens += [pre + t for t in tails]
            starts.append(len(lens))
            prefix.append(pre)
        lens += list(loners)
        super().__init__(lens, hkv, hd, bs, dtype, seed)
        self.starts, self.prefix = starts, prefix
        for g, pre in enumerate(prefix):
            for s in range(starts[g], starts[g + 1]):
                self.tables[s, : pre // bs] = self.tables[starts[g], : pre // bs]

    def to(self, dev):
        super().to(dev)
        self.dstarts = torch.tensor(self.starts, dtype=torch.int32, device=dev)
        self.dprefix = torch.tensor(self.prefix, dtype=torch.int32, device=dev)
        return self


def shared_exact(b, q, scale, umma):
    S, hq, hd = q.shape
    G = hq // b.hkv
    out, bound = (torch.zeros((S, hq, hd), dtype=torch.float64) for _ in range(2))
    for s, L in enumerate(b.lens):
        for h in range(b.hkv):
            g = slice(h * G, (h + 1) * G)
            o, e = attention(q[s, g], b.rows(0, s, h), b.rows(1, s, h), scale, torch.ones((G, L), dtype=torch.bool),
                             b.dtype, umma)
            out[s, g], bound[s, g] = o, e
    return out, bound


def rand(shape, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * spread).to(DTYPES[dtype])


def close(got, exact, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    err = (got - exact).abs() - bound
    assert (err <= 0).all(), "over by %g (bound there %g)" % (float(err.max()), float(bound.flatten()[err.argmax()]))
