"""Plain 64-bit forms of the cache-side operators (rotary write, attention
weights, eviction) and the inputs their tests share.  Written from the
definitions in include/pa.h, on CPU tensors; the product never imports this."""
import numpy as np
import torch

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
EPS = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}  # half a step, relative


def rope(x, positions, inv_freq, pair_axis, interleaved):
    """x [n, heads, hd] rotated, in 64 bits."""
    x = x.double().clone()
    half = inv_freq.numel()
    axis = pair_axis.long() if pair_axis is not None else torch.zeros(half, dtype=torch.long)
    # whole turns taken out in integers: positions times the frequency's turns, exact to 2^-50 of a turn here
    angle = positions.double()[axis].t() * inv_freq.double()
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    a, b = x[..., i0].clone(), x[..., i1].clone()
    x[..., i0], x[..., i1] = a * c - b * s, b * c + a * s
    return x


def rope_bound(x, half, interleaved):
    """|x1| + |x2| of each element's pair (0 past the rotated part)."""
    b = torch.zeros_like(x, dtype=torch.float64)
    i0 = torch.arange(half) * 2 if interleaved else torch.arange(half)
    i1 = i0 + 1 if interleaved else i0 + half
    s = x[..., i0].double().abs() + x[..., i1].double().abs()
    b[..., i0], b[..., i1] = s, s
    return b


class Batch:
    """A paged batch: pools with NaN in every unused slot, random block order."""

    def __init__(self, lens, hkv, hd, bs, dtype, seed, fp8=False, extra_blocks=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hkv, self.hd, self.bs, self.dtype, self.fp8 = list(lens), hkv, hd, bs, dtype, fp8
        need = [-(-L // bs) for L in lens]
        self.num_blocks = sum(need) + 2 + extra_blocks
        perm = torch.randperm(sum(need) + 2, generator=g).to(torch.int32)
        self.tables = torch.full((len(lens), max(1, max(need, default=0)) + 1), -1, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = perm[at:at + n]
            at += n
        shape = (self.num_blocks, bs, hkv, hd)
        used = torch.zeros((self.num_blocks, bs), dtype=torch.bool)
        for s, L in enumerate(lens):
            for j in range(need[s]):
                used[self.tables[s, j].long(), : min(bs, L - j * bs)] = True
        self.scales = None
        if fp8:
            k, v = (torch.randn(shape, generator=g).mul(100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                    for _ in range(2))
            k[~used], v[~used] = 0x7F, 0x7F
            ks, vs = (torch.rand((self.num_blocks, hkv, bs), generator=g) * 0.01 + 0.005 for _ in range(2))
            self.scales = []
            for sc in (ks, vs):
                sc.transpose(1, 2)[~used] = float("nan")
                self.scales.append(sc.contiguous())
        else:
            k, v = ((torch.randn(shape, generator=g) * spread).to(DTYPES[dtype]) for _ in range(2))
            k[~used], v[~used] = float("nan"), float("nan")
        self.k, self.v = k, v
        self.max_context = max(max(lens, default=0), 1)

    def rows(self, which, s, h, L=None, tables=None):
        """[L, hd] in 64 bits: K (which 0) or V rows of head h of sequence s."""
        L = self.lens[s] if L is None else L
        pool = (self.k, self.v)[which]
        t = (self.tables if tables is None else tables)[s, : -(-L // self.bs)].long()
        x = pool[t, :, h]
        if self.fp8:
            x = x.view(torch.float8_e4m3fn).double() * self.scales[which][t, h].double()[..., None]
        return x.double().reshape(-1, self.hd)[:L]

    def to(self, dev):
        self.dk, self.dv = self.k.to(dev), self.v.to(dev)
        self.dtables = self.tables.to(dev)
        self.dlens = torch.tensor(self.lens, dtype=torch.int32, device=dev)
        self.dscales = [s.to(dev) for s in self.scales] if self.fp8 else None
        return self


def softmax_rows(q, k, scale, seen):
    """Softmax over the keys each row sees (seen [rows, keys]), in 64 bits, and the largest sum |q_d k_d| scale."""
    x = q.double() @ k.double().t() * scale
    p = torch.softmax(x.masked_fill(~seen, -float("inf")), -1)
    mag = float((q.double().abs() @ k.double().abs().t()).max()) * scale if k.shape[0] else 0.0
    return p, mag


def weight_rtol(hd, mag, keys, rows):
    """Relative error a fp32-accumulated weight may have.

    A score is a sum of hd exact products accumulated in fp32: off by at most hd 2^-23 mag (2^-23 rather than 2^-24:
    the tensor cores cut where fp32 addition rounds), and two more roundings for the scale and log2 e; it enters the
    weight's exponential and the row's sum, so twice.  exp2 is good to 2^-21, a sum of n positive terms to n 2^-24,
    for the row's keys and for the weight's rows."""
    return 2 * (hd + 4) * 2.0 ** -23 * max(mag, 1.0) + 2 * 2.0 ** -21 + (keys + rows + 8) * 2.0 ** -24


def decode_exact(b, q, scale, weights):
    """(out, weights, rtol of the added weights) of one decode step, q [S, Hq, hd] on the CPU."""
    S, hq, hd = q.shape
    G = hq // b.hkv
    out = torch.zeros((S, hq, hd), dtype=torch.float64)
    w = weights.double().clone()
    rtol = 0.0
    for s, L in enumerate(b.lens):
        if L == 0:
            continue
        for h in range(b.hkv):
            k = b.rows(0, s, h)
            p, mag = softmax_rows(q[s, h * G:(h + 1) * G], k, scale, torch.ones((G, L), dtype=torch.bool))
            out[s, h * G:(h + 1) * G] = p @ b.rows(1, s, h)
            add = p.sum(0)
            w[s, h, : L - 1] += add[: L - 1]
            w[s, h, L - 1] = add[L - 1]
            rtol = max(rtol, weight_rtol(hd, mag, L, G))
    return out, w, rtol


def prompt_exact(b, q, cu, window, scale, causal, weights):
    S, (T, hq, hd) = len(b.lens), q.shape
    G = hq // b.hkv
    w = weights.double().clone()
    rtol = 0.0
    for s, L in enumerate(b.lens):
        n = cu[s + 1] - cu[s]
        r = n if window == 0 else min(n, window)
        if r == 0 or L == 0:
            continue
        seen = torch.ones((r, L), dtype=torch.bool)
        if causal:
            seen = torch.arange(L - r, L)[:, None] >= torch.arange(L)
        for h in range(b.hkv):
            k = b.rows(0, s, h)
            add = torch.zeros(L, dtype=torch.float64)
            for g in range(G):
                p, mag = softmax_rows(q[cu[s + 1] - r: cu[s + 1], h * G + g], k, scale, seen)
                add += p.sum(0)
                rtol = max(rtol, weight_rtol(hd, mag, L, r * G))
            w[s, h, : L - n] += add[: L - n]
            w[s, h, L - n: L] = add[L - n:]
    return w, rtol


def evict_exact(w, pos, L, n, c, keep, sink, recent):
    """Source index of each destination index, and the kept tokens' positions: one (sequence, head).  w, pos numpy."""
    p = np.arange(L, dtype=np.int64) + n - L
    if c:
        p[:c] = pos[:c]
    if L <= keep:
        return np.arange(L), p
    held = (p < sink) | (p >= n - recent)
    rank = []
    for j in range(L):
        x = float(w[j])
        # held first, then NaN, then larger weights, then the lower index; 0.0 == -0.0
        rank.append((0 if held[j] else 1, 0 if x != x else 1, 0.0 if x != x else -x, j))
    kept = np.zeros(L, dtype=bool)
    kept[[r[3] for r in sorted(rank)[:keep]]] = True
    late = [j for j in range(keep, L) if kept[j]]
    src = [i if kept[i] else late.pop(0) for i in range(keep)]
    assert not late
    return np.array(src), p[src]
