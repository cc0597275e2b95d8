"""Cases of the library's latent-cache and shared-prefix operators, with their plain forms.

Attention that reads few cached bytes for many query rows:

* ``write``:  normalise the latent vector of each new token, rotate its position part and the queries' position
  parts, and write one row a token [latent | position part] to its slot of the paged latent pool.
* ``decode``: one query token per sequence over the latent pool: every head's key is the whole row, its value the
  row's latent part.
* ``varlen``: the same for prompts and chunks of them (causal, new tokens at the end of their context).
* ``shared``: decode over a paged K/V pool in which groups of sequences share the leading blocks of their tables.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the library's calls.
"""
import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELT = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one generation step of a 64-sequence batch: 64 rows into the pool, 64 tokens' queries rotated
        {"name": "write step 64", "op": "write", "dtype": "bf16", "n": 64, "h": 16, "lat": 512, "rot": 64, "bs": 16,
         "norm": True, "interleaved": True, "far": 4096},
        # a long prompt of many heads
        {"name": "write prompt 8192", "op": "write", "dtype": "bf16", "n": 8192, "h": 128, "lat": 512, "rot": 64,
         "bs": 16, "norm": True, "interleaved": True, "far": 131072},
        # one short conversation: latency counts
        {"name": "decode 1 x 1999", "op": "decode", "dtype": "bf16", "seqs": 1, "lo": 1999, "hi": 1999, "h": 16,
         "lat": 512, "rot": 64, "bs": 16},
        # the ragged 64-sequence batch, all heads on one GPU
        {"name": "decode 64 h128", "op": "decode", "dtype": "bf16", "seqs": 64, "lo": 120, "hi": 3480, "h": 128,
         "lat": 512, "rot": 64, "bs": 16},
        # few long sequences, a slice of the heads: the work is split along each of them
        {"name": "decode 8 x 32768 h16", "op": "decode", "dtype": "bf16", "seqs": 8, "lo": 32768, "hi": 32768,
         "h": 16, "lat": 512, "rot": 64, "bs": 64},
        # chunks of 64 to 1024 new tokens behind 0 to 1024 cached ones
        {"name": "varlen chunks 16", "op": "varlen", "dtype": "bf16", "seqs": 16, "new_lo": 64, "new_hi": 1024,
         "old_lo": 0, "old_hi": 1024, "h": 16, "lat": 512, "rot": 64, "bs": 16},
        # a whole prompt
        {"name": "varlen whole 8192", "op": "varlen", "dtype": "f16", "seqs": 1, "new_lo": 8192, "new_hi": 8192,
         "old_lo": 0, "old_hi": 0, "h": 16, "lat": 512, "rot": 64, "bs": 16},
        # 60 prompts of 300 tokens, four samples of each: 18 blocks shared, the rest of each sample its own
        {"name": "shared 60 x 4 samples", "op": "shared", "dtype": "bf16", "groups": 60, "members": 4, "prefix": 288,
         "lo": 13, "hi": 256, "hq": 12, "hkv": 2, "hd": 128, "bs": 16},
        # 64 requests behind one long instruction
        {"name": "shared 64 behind 8192", "op": "shared", "dtype": "bf16", "groups": 1, "members": 64,
         "prefix": 8192, "lo": 20, "hi": 1500, "hq": 32, "hkv": 8, "hd": 128, "bs": 16},
        # several instructions of one KV head per query head, odd members
        {"name": "shared 5 x 13 mha", "op": "shared", "dtype": "f16", "groups": 5, "members": 13, "prefix": 2048,
         "lo": 1, "hi": 480, "hq": 40, "hkv": 40, "hd": 128, "bs": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("write", "decode", "varlen", "shared"))
    dtype = rng.choice(("bf16", "bf16", "bf16", "f16", "f16", "f32"))
    bs = rng.choice((16, 16, 8, 32, 64))
    if op == "shared":
        hq, hkv = rng.choice(((32, 8), (12, 2), (8, 8), (16, 1), (40, 40), (28, 4)))
        hd = rng.choice((128, 128, 64))
        groups = _log_int(rng, 1, 40)
        members = _log_int(rng, 1, max(2, 160 // groups))
        room = 300 if dtype == "f32" else 8000
        prefix = _log_int(rng, bs, max(bs, min(room, 80000 // groups))) // bs * bs
        hi = _log_int(rng, 1, max(2, min(room // 4, 40000 // (groups * members))))
        if hkv > 8:
            prefix, hi = max(bs, prefix // 4 // bs * bs), max(1, hi // 4)
        return {"op": op, "dtype": dtype, "groups": groups, "members": members, "prefix": prefix,
                "lo": rng.randint(0, hi), "hi": hi, "hq": hq, "hkv": hkv, "hd": hd, "bs": bs}
    lat, rot, h = 512, 64, rng.choice((16, 16, 128, 64, 32, 8, 20))
    if op == "write":
        return {"op": op, "dtype": dtype, "n": _log_int(rng, 1, 6000), "h": h, "lat": lat, "rot": rot, "bs": bs,
                "norm": rng.random() < 0.7, "interleaved": rng.random() < 0.5, "far": _log_int(rng, 100, 1 << 20)}
    if op == "decode":
        if dtype == "f32":
            seqs, hi = rng.randint(1, 6), _log_int(rng, 3, 1000)
        else:
            seqs = _log_int(rng, 1, 96)
            hi = _log_int(rng, 20, min(40000, 200000 // seqs))
        return {"op": op, "dtype": dtype, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "h": h, "lat": lat,
                "rot": rot, "bs": bs}
    seqs = _log_int(rng, 1, 12)
    if dtype == "f32":
        new_hi, old_hi = _log_int(rng, 1, 60), rng.randint(0, 300)
    else:
        new_hi, old_hi = _log_int(rng, 1, 2400 // seqs + 300), rng.randint(0, 4000 // seqs + 300)
    return {"op": op, "dtype": dtype, "seqs": seqs, "new_lo": rng.randint(1, new_hi), "new_hi": new_hi,
            "old_lo": rng.randint(0, old_hi), "old_hi": old_hi, "h": min(h, 32), "lat": lat, "rot": rot, "bs": bs}


# ---------------------------------------------------------------- inputs

def _spread(lo, hi, count):
    """`count` lengths from lo to hi, evenly: the same ones for every seed."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _lengths(case):
    """New tokens and context of every sequence."""
    if case["op"] == "varlen":
        new = _spread(case["new_lo"], case["new_hi"], case["seqs"])
        old = _spread(case["old_lo"], case["old_hi"], case["seqs"])
        old = old[1::2] + old[0::2]
        return new, [a + b for a, b in zip(new, old)]
    if case["op"] == "shared":
        tails = _spread(case["lo"], case["hi"], case["groups"] * case["members"])
        return None, [case["prefix"] + x for x in tails]
    return None, _spread(case["lo"], case["hi"], case["seqs"])


def _randn(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device=DEV).to(dtype)


def _tables(gen, lens, bs, first, width):
    """Block tables over a random permutation of the blocks first, first + 1, ...; padding is block 0."""
    need = [-(-x // bs) for x in lens]
    total = sum(need)
    perm = torch.randperm(total, generator=gen, device=DEV, dtype=torch.int64) + first
    n = torch.tensor(need, device=DEV)
    start = torch.cumsum(n, 0) - n
    col = torch.arange(width, device=DEV)
    at = (start[:, None] + col[None, :]).clamp(max=max(0, total - 1))
    return torch.where(col[None, :] < n[:, None], perm[at] if total else at, torch.zeros_like(at)).to(torch.int32), total


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    order = random.Random(seed)
    s = {"case": case, "op": case["op"]}
    dt, bs = DTYPES[case["dtype"]], case["bs"]
    if case["op"] == "write":
        n, h, lat, rot = (case[k] for k in ("n", "h", "lat", "rot"))
        # rows of the down projection; the queries' position parts lie behind 128 other elements of each head
        s["kv"] = (torch.randn((n, lat + rot), generator=gen, device=DEV) * 0.7).to(dt)
        s["q"] = _randn(gen, (n, h, 128 + rot), dt)[..., 128:]
        s["q_out"] = torch.zeros((n, h, lat + rot), dtype=dt, device=DEV)
        s["norm"] = (1 + 0.2 * torch.randn(lat, generator=gen, device=DEV)).to(dt) if case["norm"] else None
        s["eps"] = 1e-6
        s["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=DEV)
        pairs = rot // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
        blocks = -(-n // bs) + 1
        s["slots"] = torch.randperm(blocks * bs, generator=gen, device=DEV)[:n].contiguous()
        s["slots"][torch.rand(n, generator=gen, device=DEV) < 0.01] = -1  # padding tokens of the batch
        s["cache"] = torch.zeros((blocks, bs, lat + rot), dtype=dt, device=DEV)
        return s
    new, lens = _lengths(case)
    S = len(lens)
    at = list(range(S))
    order.shuffle(at)
    lens = [lens[i] for i in at]
    s["max_context"] = max(lens)
    s["lens"] = _ints(lens)
    width = max(1, -(-max(lens) // bs))
    if case["op"] == "shared":
        hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
        lead = case["prefix"] // bs
        heads, first = _tables(gen, [case["prefix"]] * case["groups"], bs, 1, lead)
        own_blocks, total = _tables(gen, [x - case["prefix"] for x in lens], bs, first + 1, max(1, width - lead))
        s["tables"] = torch.cat((heads.repeat_interleave(case["members"], 0), own_blocks), 1).contiguous()
        shape = (first + total + 1, bs, hkv, hd)
        s["k_cache"], s["v_cache"] = _randn(gen, shape, dt), _randn(gen, shape, dt)
        s["q"] = _randn(gen, (S, hq, hd), dt)
        s["out"] = torch.zeros_like(s["q"])
        s["starts"] = _ints([g * case["members"] for g in range(case["groups"] + 1)])
        s["prefix_lens"] = _ints([case["prefix"]] * case["groups"])
        s["scale"] = hd ** -0.5
        if own:  # scratch that a user's program allocates once
            import paged_kv_cache_116_gb300 as pa

            s["ws"] = torch.empty(max(16, pa.pa_decode_shared_workspace_size(S, case["groups"], hq, hkv, hd, bs,
                                                                             s["max_context"], dt)),
                                  dtype=torch.uint8, device=DEV)
        return s
    h, lat, rot = case["h"], case["lat"], case["rot"]
    s["tables"], blocks = _tables(gen, lens, bs, 1, width)
    s["cache"] = _randn(gen, (blocks + 1, bs, lat + rot), dt)
    s["scale"] = (128 + rot) ** -0.5  # of the heads before the key's projection went into the query
    rows = S
    if case["op"] == "varlen":
        new = [new[i] for i in at]
        rows = sum(new)
        cu = [0]
        for x in new:
            cu.append(cu[-1] + x)
        s["cu"], s["max_q"], s["new"] = _ints(cu), max(new), _ints(new)
    s["q"] = _randn(gen, (rows, h, lat + rot), dt)
    s["out"] = torch.zeros((rows, h, lat), dtype=dt, device=DEV)
    if own:
        import paged_kv_cache_116_gb300 as pa

        if case["op"] == "decode":
            size = pa.pa_latent_decode_workspace_size(S, h, lat, rot, bs, s["max_context"], dt)
        else:
            size = pa.pa_latent_varlen_workspace_size(S, rows, s["max_q"], h, lat, rot, bs, s["max_context"], dt)
        s["ws"] = torch.empty(max(16, size), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"write": _write_plain, "decode": _decode_plain, "varlen": _varlen_plain, "shared": _shared_plain}[s["op"]](s)


def _outputs(s):
    if s["op"] == "write":
        return {"cache": s["cache"], "q": s["q_out"]}
    return {"out": s["out"]}


def _run_own(s):
    import paged_kv_cache_116_gb300 as pa

    case = s["case"]
    if s["op"] == "write":
        pa.pa_latent_write(s["kv"], s["positions"], s["inv_freq"], s["slots"], s["cache"], norm_weight=s["norm"],
                           eps=s["eps"], q=s["q"], q_out=s["q_out"][..., case["lat"]:],
                           interleaved=case["interleaved"])
    elif s["op"] == "decode":
        pa.pa_latent_decode(s["out"], s["q"], s["cache"], s["tables"], s["lens"], s["max_context"], s["scale"],
                            workspace=s["ws"])
    elif s["op"] == "varlen":
        pa.pa_latent_varlen(s["out"], s["q"], s["cache"], s["tables"], s["lens"], s["cu"], s["max_q"],
                            s["max_context"], s["scale"], workspace=s["ws"])
    else:
        pa.pa_decode_shared(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["starts"],
                            s["prefix_lens"], s["max_context"], s["scale"], workspace=s["ws"])
    return _outputs(s)


def _turn(x, cos, sin, interleaved):
    half = x.shape[-1] // 2
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    a, b = x[..., :half], x[..., half:]
    return torch.cat((a * cos - b * sin, b * cos + a * sin), -1)


def _write_plain(s):
    case = s["case"]
    lat = case["lat"]
    angle = s["positions"].double()[:, None] * s["inv_freq"]  # far positions lose their angle in 32 bits
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    s["q_out"][..., lat:] = _turn(s["q"].float(), cos[:, None], sin[:, None], case["interleaved"]).to(s["q"].dtype)
    kv = s["kv"].float()
    c = kv[:, :lat]
    if s["norm"] is not None:
        c = c / torch.sqrt((c * c).mean(-1, keepdim=True) + s["eps"]) * s["norm"].float()
    row = torch.cat((c, _turn(kv[:, lat:], cos, sin, case["interleaved"])), -1).to(s["cache"].dtype)
    fine = s["slots"] >= 0
    s["cache"].view(-1, row.shape[1])[s["slots"][fine]] = row[fine]
    return _outputs(s)


def _gathered(s, pool):
    """The sequences' rows [S, T, ...] through their block tables, in 32 bits."""
    return pool[s["tables"].long()].flatten(1, 2)[:, : s["max_context"]].float()


def _softmax(x):
    p = torch.exp(x - x.amax(-1, keepdim=True))
    return p / p.sum(-1, keepdim=True)


def _decode_plain(s):
    rows = _gathered(s, s["cache"])
    x = torch.einsum("shd,std->sht", s["q"].float(), rows) * s["scale"]
    t = torch.arange(s["max_context"], device=DEV)
    p = _softmax(x.masked_fill(t >= s["lens"][:, None, None], -math.inf))
    s["out"].copy_(torch.einsum("sht,std->shd", p, rows[..., : s["case"]["lat"]]))
    return _outputs(s)


def _varlen_plain(s):
    rows = _gathered(s, s["cache"])
    cu, n = s["cu"].long(), s["new"].long()
    j = torch.arange(s["max_q"], device=DEV)
    there = j < n[:, None]
    q = s["q"].float()[(cu[:-1, None] + j).clamp(max=s["q"].shape[0] - 1)]
    x = torch.einsum("sjhd,std->shjt", q, rows) * s["scale"]
    pos = (s["lens"].long() - n)[:, None] + j
    t = torch.arange(s["max_context"], device=DEV)
    x.masked_fill_((t > pos[..., None])[:, None], -math.inf)
    o = torch.einsum("shjt,std->sjhd", _softmax(x), rows[..., : s["case"]["lat"]])
    s["out"].copy_(o[there])
    return _outputs(s)


def _shared_plain(s):
    case = s["case"]
    S, hkv, hd = s["q"].shape[0], case["hkv"], case["hd"]
    k, v = _gathered(s, s["k_cache"]), _gathered(s, s["v_cache"])
    x = torch.einsum("shgd,sthd->shgt", s["q"].float().view(S, hkv, -1, hd), k) * s["scale"]
    t = torch.arange(s["max_context"], device=DEV)
    p = _softmax(x.masked_fill(t >= s["lens"][:, None, None, None], -math.inf))
    s["out"].copy_(torch.einsum("shgt,sthd->shgd", p, v).reshape(S, -1, hd))
    return _outputs(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    elt, bs = ELT[case["dtype"]], case["bs"]
    if case["op"] == "write":
        n, h, lat, rot = (case[k] for k in ("n", "h", "lat", "rot"))
        return {"bytes": n * (2 * (lat + rot) * elt + 2 * h * rot * elt + 16),
                "flops": n * (4 * lat + 3 * (h + 1) * rot)}
    new, lens = _lengths(case)
    total = sum(lens)
    if case["op"] == "shared":
        hq, hkv, hd = case["hq"], case["hkv"], case["hd"]
        read = total - case["prefix"] * (len(lens) - case["groups"])
        return {"bytes": read * hkv * 2 * hd * elt + 2 * len(lens) * hq * hd * elt + 4 * (total // bs + len(lens)),
                "flops": 4 * total * hq * hd}
    h, lat, rot = case["h"], case["lat"], case["rot"]
    rows = len(lens) if new is None else sum(new)
    seen = total if new is None else sum(n * L - n * (n - 1) // 2 for n, L in zip(new, lens))
    return {"bytes": total * (lat + rot) * elt + rows * h * (2 * lat + rot) * elt + 4 * (total // bs + len(lens)),
            "flops": 2 * seen * h * (2 * lat + rot)}


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"write": _write_exact, "decode": _decode_exact, "varlen": _varlen_exact, "shared": _shared_exact}[s["op"]](s)


def _write_exact(s):
    case = s["case"]
    lat, rot = case["lat"], case["rot"]
    first = slice(0, rot, 2) if case["interleaved"] else slice(0, rot // 2)
    second = slice(1, rot, 2) if case["interleaved"] else slice(rot // 2, rot)

    def rotated(x, angle):
        z = torch.complex(x[..., first], x[..., second]) * torch.polar(torch.ones_like(angle), angle)
        y = x.clone()
        y[..., first], y[..., second] = z.real, z.imag
        return y

    angle = s["positions"][:, None].double() * s["inv_freq"][None]
    q = torch.zeros(s["q_out"].shape, dtype=torch.float64, device=DEV)
    q[..., lat:] = rotated(s["q"].double(), angle[:, None])
    kv = s["kv"].double()
    c = kv[:, :lat]
    if s["norm"] is not None:
        c = c * torch.rsqrt(c.square().sum(-1, keepdim=True) / lat + s["eps"]) * s["norm"].double()
    rows = torch.cat((c, rotated(kv[:, lat:], angle)), 1)
    cache = torch.zeros(s["cache"].shape, dtype=torch.float64, device=DEV).view(-1, lat + rot)
    for i, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            cache[slot] = rows[i]
    return {"cache": cache.view(s["cache"].shape), "q": q}


def _rows64(s, pool, i, L):
    ids = s["tables"][i, : -(-L // s["case"]["bs"])].long()
    return pool[ids].flatten(0, 1)[:L].double()


def _decode_exact(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for i, L in enumerate(s["lens"].tolist()):
        rows = _rows64(s, s["cache"], i, L)
        p = torch.softmax(s["q"][i].double() @ rows.t() * s["scale"], -1)
        out[i] = p @ rows[:, : s["case"]["lat"]]
    return {"out": out}


def _varlen_exact(s):
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    cu = s["cu"].tolist()
    for i, L in enumerate(s["lens"].tolist()):
        rows = _rows64(s, s["cache"], i, L)
        n = cu[i + 1] - cu[i]
        blind = torch.arange(L - n, L, device=DEV)[:, None] < torch.arange(L, device=DEV)
        for h in range(s["case"]["h"]):
            x = s["q"][cu[i]: cu[i + 1], h].double() @ rows.t() * s["scale"]
            p = torch.softmax(x.masked_fill(blind, -math.inf), -1)
            out[cu[i]: cu[i + 1], h] = p @ rows[:, : s["case"]["lat"]]
    return {"out": out}


def _shared_exact(s):
    case = s["case"]
    G = case["hq"] // case["hkv"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    for i, L in enumerate(s["lens"].tolist()):
        k, v = (_rows64(s, s[name], i, L) for name in ("k_cache", "v_cache"))
        q = s["q"][i].double().view(case["hkv"], G, -1)
        p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * s["scale"], -1)
        out[i] = torch.einsum("hgt,thd->hgd", p, v).flatten(0, 1)
    return {"out": out}
