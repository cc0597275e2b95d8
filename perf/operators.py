"""Cases of the library's cache-side operators, with their plain forms.

The path of a long-context server around the paged attention:

* ``rope``:   rotate q and k by their positions (one axis, or time / height / width) and write K and V to
  their slots of the paged pool (16-bit rows, or E4M3 codes with a scale per row).
* ``decode``: attention of one new token per sequence over the paged pool, adding each cached token's
  attention weight (summed over the query heads of a KV head) to the sequence's weight row.
* ``prompt``: the weights that the last ``window`` new queries of each request (all of them where window is 0)
  give to the request's cached tokens.
* ``evict``:  keep the tokens with the largest weights, besides the first few and the most recent, and move the
  kept rows to the front of the sequence's blocks (or into other blocks).

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the library's calls.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
ELT = {"f32": 4, "bf16": 2, "f16": 2}


# ---------------------------------------------------------------- cases

def listed():
    return [
        # one generation step of a 64-sequence batch, positions on three axes
        {"name": "rope step 64", "op": "rope", "dtype": "bf16", "fp8": False, "n": 64, "hq": 32, "hkv": 8, "hd": 128,
         "bs": 16, "axes": 3, "rot": 128, "interleaved": False, "far": 4096},
        # a long prompt straight from a fused q/k/v projection (rows of one wide matrix)
        {"name": "rope prompt 8192", "op": "rope", "dtype": "bf16", "fp8": False, "n": 8192, "hq": 32, "hkv": 8,
         "hd": 128, "bs": 16, "axes": 3, "rot": 128, "interleaved": False, "far": 131072},
        # an odd number of tokens into a quantized cache, half of the head rotated, interleaved pairs
        {"name": "rope fp8 1999", "op": "rope", "dtype": "f16", "fp8": True, "n": 1999, "hq": 12, "hkv": 2, "hd": 128,
         "bs": 16, "axes": 1, "rot": 64, "interleaved": True, "far": 32768},
        # the ragged 64-sequence GQA batch
        {"name": "decode gqa 64", "op": "decode", "dtype": "bf16", "fp8": False, "seqs": 64, "lo": 120, "hi": 3480,
         "hq": 32, "hkv": 8, "hd": 128, "bs": 16},
        # few long sequences: the work is split along each of them
        {"name": "decode 8 x 32768", "op": "decode", "dtype": "bf16", "fp8": False, "seqs": 8, "lo": 32768,
         "hi": 32768, "hq": 32, "hkv": 8, "hd": 128, "bs": 16},
        # the GQA batch over a quantized cache
        {"name": "decode fp8 64", "op": "decode", "dtype": "bf16", "fp8": True, "seqs": 64, "lo": 120, "hi": 3480,
         "hq": 32, "hkv": 8, "hd": 128, "bs": 16},
        # weights of long prompts from their last 32 queries
        {"name": "prompt 4 x 32768 w32", "op": "prompt", "dtype": "bf16", "fp8": False, "seqs": 4, "new_lo": 64,
         "new_hi": 64, "old_lo": 32704, "old_hi": 32704, "window": 32, "hq": 32, "hkv": 8, "hd": 128, "bs": 16},
        # chunks of 64 to 1024 new tokens behind 0 to 1024 cached ones, every query counted
        {"name": "prompt chunks 16", "op": "prompt", "dtype": "bf16", "fp8": False, "seqs": 16, "new_lo": 64,
         "new_hi": 1024, "old_lo": 0, "old_hi": 1024, "window": 0, "hq": 12, "hkv": 2, "hd": 128, "bs": 16},
        # a whole prompt, every query counted
        {"name": "prompt whole 8192", "op": "prompt", "dtype": "f16", "fp8": False, "seqs": 1, "new_lo": 8192,
         "new_hi": 8192, "old_lo": 0, "old_hi": 0, "window": 0, "hq": 32, "hkv": 8, "hd": 128, "bs": 16},
        # steady state: 16 tokens over the budget, dropped in place
        {"name": "evict 64 x 1040 to 1024", "op": "evict", "dtype": "bf16", "fp8": False, "seqs": 64, "lo": 1040,
         "hi": 1040, "recorded": 1024, "keep": 1024, "sink": 4, "recent": 512, "fresh": False, "hkv": 8, "hd": 128,
         "bs": 16},
        # long prompts pruned into fresh blocks (the prompt's own blocks stay shared)
        {"name": "evict 8 x 32768 to 4096", "op": "evict", "dtype": "bf16", "fp8": False, "seqs": 8, "lo": 32768,
         "hi": 32768, "recorded": 0, "keep": 4096, "sink": 4, "recent": 1024, "fresh": True, "hkv": 8, "hd": 128,
         "bs": 16},
        # a ragged batch of a quantized cache, some sequences under the budget
        {"name": "evict fp8 ragged", "op": "evict", "dtype": "bf16", "fp8": True, "seqs": 48, "lo": 100, "hi": 3480,
         "recorded": 0, "keep": 1000, "sink": 3, "recent": 100, "fresh": False, "hkv": 8, "hd": 128, "bs": 16},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("rope", "decode", "prompt", "evict"))
    hq, hkv = rng.choice(((32, 8), (12, 2), (8, 8), (16, 1), (40, 40), (28, 4)))
    bs = rng.choice((16, 16, 8, 32, 64))
    hd = rng.choice((128, 128, 64))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    fp8 = rng.random() < 0.25
    if fp8:
        hd, dtype = 128, rng.choice(("bf16", "f16"))
    if op == "rope":
        rot = rng.choice((hd, hd // 2))
        return {"op": op, "dtype": dtype, "fp8": fp8, "n": _log_int(rng, 1, 4000), "hq": hq, "hkv": hkv, "hd": hd,
                "bs": bs, "axes": rng.choice((1, 2, 3)), "rot": rot, "interleaved": rng.random() < 0.5,
                "far": _log_int(rng, 100, 1 << 20)}
    if op == "decode":
        if dtype == "f32":
            seqs, hi = rng.randint(1, 6), _log_int(rng, 3, 2000)
        else:
            seqs = _log_int(rng, 1, 96)
            hi = _log_int(rng, 20, min(40000, 200000 // seqs))
        if hkv > 8:
            hi = min(hi, max(1, 48000 // seqs))
        return {"op": op, "dtype": dtype, "fp8": fp8, "seqs": seqs, "lo": rng.randint(1, hi), "hi": hi, "hq": hq,
                "hkv": hkv, "hd": hd, "bs": bs}
    if op == "prompt":
        seqs = _log_int(rng, 1, 12)
        if dtype == "f32":
            new_hi, old_hi, window = _log_int(rng, 1, 160), rng.randint(0, 500), rng.choice((0, 16))
        elif rng.random() < 0.5:
            new_hi, old_hi, window = _log_int(rng, 1, 100), _log_int(rng, 100, 50000 // seqs), rng.randint(8, 64)
        else:
            new_hi, old_hi, window = _log_int(rng, 60, 2400 // seqs + 300), rng.randint(0, 900), 0
        if hkv > 8:
            old_hi = old_hi // 4
        return {"op": op, "dtype": dtype, "fp8": fp8, "seqs": seqs, "new_lo": rng.randint(1, new_hi),
                "new_hi": new_hi, "old_lo": rng.randint(0, old_hi), "old_hi": old_hi, "window": window, "hq": hq,
                "hkv": hkv, "hd": hd, "bs": bs}
    seqs = _log_int(rng, 1, 64)
    hi = _log_int(rng, 30, min(30000, 150000 // seqs))
    if hkv > 8:
        hi = max(30, hi // 8)
    keep = max(8, int(hi * rng.uniform(0.1, 0.98)))
    sink = rng.randint(0, 4)
    recorded = keep if rng.random() < 0.5 else 0
    return {"op": op, "dtype": dtype, "fp8": fp8, "seqs": seqs, "lo": rng.randint(1, hi) if not recorded else hi,
            "hi": hi, "recorded": recorded, "keep": keep, "sink": sink, "recent": rng.randint(0, keep - sink),
            "fresh": rng.random() < 0.5, "hkv": hkv, "hd": hd, "bs": bs}


# ---------------------------------------------------------------- inputs

def _spread(lo, hi, count):
    """`count` lengths from lo to hi, evenly: the same ones for every seed."""
    if count == 1:
        return [hi]
    return [lo + (hi - lo) * i // (count - 1) for i in range(count)]


def _lengths(case):
    if case["op"] == "prompt":
        new = _spread(case["new_lo"], case["new_hi"], case["seqs"])
        old = _spread(case["old_lo"], case["old_hi"], case["seqs"])
        old = old[1::2] + old[0::2]
        return new, [a + b for a, b in zip(new, old)]
    return None, _spread(case["lo"], case["hi"], case["seqs"])


def _sections(pairs, axes):
    """The axis of each rotary pair: contiguous sections, the first the smallest."""
    first = pairs // (axes + 1) if axes > 1 else pairs
    rest = (pairs - first) // max(1, axes - 1)
    return [0 if i < first else min(axes - 1, 1 + (i - first) // max(1, rest)) for i in range(pairs)]


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


def _pools(gen, case, blocks):
    shape = (blocks, case["bs"], case["hkv"], case["hd"])
    if case["fp8"]:
        k, v = (_randn(gen, shape, torch.float32).mul_(120).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
                for _ in range(2))
        ks, vs = (torch.rand((blocks, case["hkv"], case["bs"]), generator=gen, device=DEV) * 0.004 + 0.006
                  for _ in range(2))
        return k, v, ks, vs
    # some tokens draw much more attention than the rest
    k, v = _randn(gen, shape, torch.float32), _randn(gen, shape, DTYPES[case["dtype"]])
    heavy = torch.rand((blocks, case["bs"], 1, 1), generator=gen, device=DEV) < 0.02
    return (k * torch.where(heavy, 2.5, 1.0)).to(DTYPES[case["dtype"]]), v, None, None


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    order = random.Random(seed)
    s = {"case": case, "op": case["op"]}
    if case["op"] == "rope":
        n, hq, hkv, hd, bs = (case[k] for k in ("n", "hq", "hkv", "hd", "bs"))
        qkv = _randn(gen, (n, (hq + 2 * hkv) * hd), DTYPES[case["dtype"]])
        s["q"] = qkv[:, : hq * hd].view(n, hq, hd)
        s["k"] = qkv[:, hq * hd: (hq + hkv) * hd].view(n, hkv, hd)
        s["v"] = qkv[:, (hq + hkv) * hd:].view(n, hkv, hd)
        s["positions"] = torch.randint(0, case["far"], (case["axes"], n), generator=gen, device=DEV)
        pairs = case["rot"] // 2
        s["inv_freq"] = 10000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
        s["pair_axis"] = _ints(_sections(pairs, case["axes"]))
        blocks = -(-n // bs) + 1
        s["slots"] = torch.randperm(blocks * bs, generator=gen, device=DEV)[:n].contiguous()
        s["slots"][torch.rand(n, generator=gen, device=DEV) < 0.01] = -1  # padding tokens of the batch
        s["q_out"] = torch.zeros((n, hq, hd), dtype=s["q"].dtype, device=DEV)
        pool = torch.uint8 if case["fp8"] else s["q"].dtype
        s["k_cache"], s["v_cache"] = (torch.zeros((blocks, bs, hkv, hd), dtype=pool, device=DEV) for _ in range(2))
        if case["fp8"]:
            s["ks"], s["vs"] = (torch.zeros((blocks, hkv, bs), device=DEV) for _ in range(2))
        return s
    new, lens = _lengths(case)
    S, bs, hkv, hd = case["seqs"], case["bs"], case["hkv"], case["hd"]
    at = list(range(S))
    order.shuffle(at)
    lens = [lens[i] for i in at]
    s["max_context"] = max(lens)
    s["lens"] = _ints(lens)
    s["tables"], blocks = _tables(gen, lens, bs, 1, -(-max(lens) // bs))
    s["stride"] = -(-max(lens) // 4) * 4
    weights = torch.exp(2.0 * torch.randn((S, hkv, s["stride"]), generator=gen, device=DEV)) * 0.01
    if case["op"] == "evict":
        fresh = [min(x, case["keep"]) for x in lens]
        width = -(-max(fresh) // bs)
        s["new_tables"] = s["tables"][:, :width].contiguous()
        total = blocks + 1
        if case["fresh"]:
            s["new_tables"], more = _tables(gen, fresh, bs, total, width)
            total += more
        s["k_cache"], s["v_cache"], s["ks"], s["vs"] = _pools(gen, case, total)
        s["weights"] = weights
        s["weights_out"] = torch.zeros_like(weights)
        s["positions_out"] = torch.zeros((S, hkv, s["stride"]), dtype=torch.int32, device=DEV)
        s["new_lens"] = torch.zeros(S, dtype=torch.int32, device=DEV)
        s["recorded"] = s["seen"] = s["positions"] = None
        if case["recorded"]:  # evicted before: the first tokens' positions are what that left
            c = case["recorded"]
            seen = [x + 500 for x in lens]
            before = min(seen) - max(lens) + c
            pos = torch.rand((S, hkv, before), generator=gen, device=DEV).argsort(-1)[..., :c]
            s["positions"] = torch.zeros_like(s["positions_out"])
            s["positions"][..., :c] = pos.to(torch.int32)
            s["recorded"], s["seen"] = _ints([c] * S), _ints(seen)
        if own:  # scratch that a user's program allocates once
            import paged_kv_cache_116_gb300 as pa

            s["ws"] = torch.empty(max(16, pa.pa_evict_workspace_size(S, hkv, s["max_context"], case["keep"])),
                                  dtype=torch.uint8, device=DEV)
        return s
    s["k_cache"], s["v_cache"], s["ks"], s["vs"] = _pools(gen, case, blocks + 1)
    s["weights"] = weights
    s["scale"] = hd ** -0.5
    if case["op"] == "decode":
        s["q"] = _randn(gen, (S, case["hq"], hd), DTYPES[case["dtype"]])
        s["out"] = torch.zeros_like(s["q"])
        if own:
            import paged_kv_cache_116_gb300 as pa

            size = pa.pa_decode_weights_fp8_workspace_size if case["fp8"] else pa.pa_decode_weights_workspace_size
            s["ws"] = torch.empty(max(16, size(S, case["hq"], hkv, hd, bs, s["max_context"], s["q"].dtype)),
                                  dtype=torch.uint8, device=DEV)
        return s
    new = [new[i] for i in at]
    total = sum(new)
    s["q"] = _randn(gen, (total, case["hq"], hd), DTYPES[case["dtype"]])
    s["cu"] = _ints([0] + list(np.cumsum(new)))
    s["max_q"] = max(new)
    if own:
        import paged_kv_cache_116_gb300 as pa

        size = pa.pa_prompt_weights_fp8_workspace_size if case["fp8"] else pa.pa_prompt_weights_workspace_size
        s["ws"] = torch.empty(max(16, size(S, total, s["max_q"], case["hq"], hkv, hd, bs, s["max_context"],
                                           case["window"], s["q"].dtype)), dtype=torch.uint8, device=DEV)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    if own:
        return _run_own(s)
    return {"rope": _rope_plain, "decode": _decode_plain, "prompt": _prompt_plain, "evict": _evict_plain}[s["op"]](s)


def _outputs(s):
    fp8 = s["case"]["fp8"]
    if s["op"] == "rope":
        k, v = s["k_cache"], s["v_cache"]
        if fp8:
            return {"q": s["q_out"], "k": k.view(torch.float8_e4m3fn), "v": v.view(torch.float8_e4m3fn),
                    "k_scales": s["ks"], "v_scales": s["vs"]}
        return {"q": s["q_out"], "k": k, "v": v}
    if s["op"] == "decode":
        return {"out": s["out"], "weights": s["weights"]}
    if s["op"] == "prompt":
        return {"weights": s["weights"]}
    got = {"lens": s["new_lens"], "weights": s["weights_out"], "positions": s["positions_out"], "k": s["k_cache"],
           "v": s["v_cache"]}
    if fp8:
        got.update(k=s["k_cache"].view(torch.float8_e4m3fn), v=s["v_cache"].view(torch.float8_e4m3fn),
                   k_scales=s["ks"], v_scales=s["vs"])
    return got


def _run_own(s):
    import paged_kv_cache_116_gb300 as pa

    case, fp8 = s["case"], s["case"]["fp8"]
    if s["op"] == "rope":
        if fp8:
            pa.pa_rope_write_kv_fp8(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"],
                                    s["k_cache"], s["v_cache"], s["ks"], s["vs"], pair_axis=s["pair_axis"],
                                    interleaved=case["interleaved"])
        else:
            pa.pa_rope_write_kv(s["q_out"], s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["slots"],
                                s["k_cache"], s["v_cache"], pair_axis=s["pair_axis"],
                                interleaved=case["interleaved"])
    elif s["op"] == "decode":
        if fp8:
            pa.pa_decode_weights_fp8(s["out"], s["weights"], s["q"], s["k_cache"], s["v_cache"], s["ks"], s["vs"],
                                     s["tables"], s["lens"], s["max_context"], s["scale"], workspace=s["ws"])
        else:
            pa.pa_decode_weights(s["out"], s["weights"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                 s["max_context"], s["scale"], workspace=s["ws"])
    elif s["op"] == "prompt":
        if fp8:
            pa.pa_prompt_weights_fp8(s["weights"], s["q"], s["k_cache"], s["ks"], s["tables"], s["lens"], s["cu"],
                                     s["max_q"], s["max_context"], case["window"], s["scale"], workspace=s["ws"])
        else:
            pa.pa_prompt_weights(s["weights"], s["q"], s["k_cache"], s["tables"], s["lens"], s["cu"], s["max_q"],
                                 s["max_context"], case["window"], s["scale"], workspace=s["ws"])
    else:
        pa.pa_evict(s["new_lens"], s["weights_out"], s["positions_out"], s["weights"], s["k_cache"], s["v_cache"],
                    s["tables"], s["new_tables"], s["lens"], s["max_context"], case["keep"], case["sink"],
                    case["recent"], positions=s["positions"], recorded_lens=s["recorded"], seen_lens=s["seen"],
                    k_scales=s["ks"], v_scales=s["vs"], workspace=s["ws"])
    return _outputs(s)


def _turn(x, cos, sin, rot, interleaved):
    """x [n, heads, hd] rotated by the angles of cos, sin [n, 1, rot / 2]."""
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., rot:]), -1)


def _rope_plain(s):
    case = s["case"]
    angle = s["positions"][s["pair_axis"]].t().double() * s["inv_freq"]  # far positions lose their angle in 32 bits
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    s["q_out"].copy_(_turn(s["q"].float(), cos, sin, case["rot"], case["interleaved"]))
    k = _turn(s["k"].float(), cos, sin, case["rot"], case["interleaved"])
    v = s["v"].float()
    slots = s["slots"]
    fine = slots >= 0
    to = slots[fine]
    hkv, hd, bs = case["hkv"], case["hd"], case["bs"]
    for x, pool, scales in ((k, s["k_cache"], s.get("ks")), (v, s["v_cache"], s.get("vs"))):
        x = x[fine]
        if case["fp8"]:
            top = x.abs().amax(-1, keepdim=True)
            scale = torch.where(top > 0, top / 448, torch.ones_like(top))
            scales.transpose(1, 2)[to // bs, to % bs] = scale[..., 0]
            pool.view(-1, hkv, hd)[to] = (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            pool.view(-1, hkv, hd)[to] = x.to(pool.dtype)
    return _outputs(s)


def _gathered(s, pool, scales, dtype=torch.float32):
    """The sequences' rows [S, T, hkv, hd] through their block tables."""
    case = s["case"]
    at = s["tables"].long()
    x = pool[at]
    if case["fp8"]:
        x = x.view(torch.float8_e4m3fn).to(dtype) * scales[at].transpose(2, 3)[..., None].to(dtype)
    else:
        x = x.to(dtype)
    return x.flatten(1, 2)[:, : s["max_context"]]


def _decode_plain(s):
    case = s["case"]
    S, hkv, hd = case["seqs"], case["hkv"], case["hd"]
    k = _gathered(s, s["k_cache"], s["ks"])
    q = s["q"].float().view(S, hkv, -1, hd)
    x = torch.einsum("shgd,sthd->shgt", q, k) * s["scale"]
    t = torch.arange(s["max_context"], device=DEV)
    x = x.masked_fill(t >= s["lens"][:, None, None, None], -math.inf)
    p = torch.exp(x - x.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    v = _gathered(s, s["v_cache"], s["vs"])
    s["out"].copy_(torch.einsum("shgt,sthd->shgd", p, v).reshape(S, -1, hd))
    _add_weights(s, p.sum(2), (s["lens"] - 1))
    return _outputs(s)


def _add_weights(s, w, first_new):
    """weights += w on the tokens before first_new, = w on the others of the sequence."""
    t = torch.arange(s["max_context"], device=DEV)
    old = s["weights"][..., : s["max_context"]]
    sums = torch.where(t < first_new[:, None, None], old + w, w)
    old.copy_(torch.where(t < s["lens"][:, None, None], sums, old))


def _prompt_plain(s):
    case = s["case"]
    S, hkv, hd = case["seqs"], case["hkv"], case["hd"]
    k = _gathered(s, s["k_cache"], s["ks"])
    cu = s["cu"].long()
    n = cu[1:] - cu[:-1]
    rows = s["max_q"] if case["window"] == 0 else min(s["max_q"], case["window"])
    r = torch.arange(rows, device=DEV)
    j = n[:, None] - rows + r  # the request's last `rows` new tokens; negative: it has fewer
    q = s["q"].float()[(cu[:-1, None] + j).clamp(min=0)].view(S, rows, hkv, -1, hd)
    x = torch.einsum("srhgd,sthd->shgrt", q, k) * s["scale"]
    t = torch.arange(s["max_context"], device=DEV)
    pos = s["lens"][:, None] - n[:, None] + j
    x.masked_fill_((t > pos[..., None])[:, None, None], -math.inf)
    x -= x.amax(-1, keepdim=True)
    p = x.exp_()
    p /= p.sum(-1, keepdim=True)
    p.masked_fill_((j < 0)[:, None, None, :, None], 0.0)
    _add_weights(s, p.sum((2, 3)), s["lens"] - n)
    return _outputs(s)


def _evict_plain(s):
    case = s["case"]
    S, hkv, hd, bs, keep = (case[k] for k in ("seqs", "hkv", "hd", "bs", "keep"))
    T = s["max_context"]
    t = torch.arange(T, device=DEV)
    L = s["lens"].long()[:, None, None]
    seen = L if s["seen"] is None else s["seen"].long()[:, None, None]
    pos = (seen - L + t).expand(S, hkv, T)
    if s["recorded"] is not None:
        pos = torch.where(t < s["recorded"].long()[:, None, None], s["positions"][..., :T].long(), pos)
    held = (pos < case["sink"]) | (pos >= seen - case["recent"])
    w = s["weights"][..., :T]
    key = torch.where(held, torch.full_like(w, math.inf), w)
    key = torch.where(t < L, key, torch.full_like(w, -math.inf))
    first = key.sort(dim=-1, descending=True, stable=True).indices
    rank = torch.empty_like(first).scatter_(-1, first, t.expand_as(first).contiguous())
    kept = (rank < keep) & (t < L)
    m = min(keep, T)
    late = kept & (t >= keep)
    movers = torch.cat(((~late).to(torch.int8).sort(dim=-1, stable=True).indices,
                        torch.zeros((S, hkv, 1), dtype=torch.int64, device=DEV)), -1)
    hole = ~kept[..., :m]
    nth = (hole.cumsum(-1) - 1).clamp(min=0, max=T)
    new = torch.minimum(L, torch.full_like(L, keep))
    i = t[:m].expand(S, hkv, m)
    real = i < new
    src = torch.where(hole, movers.gather(-1, nth), i)
    src = torch.where(real, src, src[..., :1])
    dst = torch.where(real, i, torch.zeros_like(i))
    seq = torch.arange(S, device=DEV)[:, None, None]
    head = torch.arange(hkv, device=DEV)[None, :, None].expand(S, hkv, m)
    from_ = s["tables"].long()[seq, src // bs] * bs + src % bs
    to = s["new_tables"].long()[seq, dst // bs] * bs + dst % bs
    for pool in (s["k_cache"], s["v_cache"]):
        rows = pool.view(-1, hkv, hd)
        rows[to, head] = rows[from_, head]
    if case["fp8"]:
        for pool in (s["ks"], s["vs"]):
            pool[to // bs, head, to % bs] = pool[from_ // bs, head, from_ % bs]
    s["weights_out"][..., :m] = torch.where(real, w.gather(-1, src), s["weights_out"][..., :m])
    s["positions_out"][..., :m] = torch.where(real, pos.gather(-1, src).int(), s["positions_out"][..., :m])
    s["new_lens"].copy_(new[:, 0, 0])
    return _outputs(s)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    hkv, hd, bs = case["hkv"], case["hd"], case["bs"]
    elt = ELT[case["dtype"]]
    row = hd + 4 if case["fp8"] else hd * elt  # one cached K (or V) row of one head
    if case["op"] == "rope":
        n, hq = case["n"], case["hq"]
        moved = n * (2 * hq * hd * elt + 2 * hkv * (hd * elt + row) + 8 + 8 * case["axes"])
        return {"bytes": moved, "flops": 3 * n * (hq + hkv) * case["rot"]}
    new, lens = _lengths(case)
    total = sum(lens)
    if case["op"] == "decode":
        moved = total * hkv * (2 * row + 8) + 2 * len(lens) * case["hq"] * hd * elt + 4 * (total // bs + len(lens))
        return {"bytes": moved, "flops": 4 * total * case["hq"] * hd}
    if case["op"] == "prompt":
        rows = [min(n, case["window"] or n) for n in new]
        seen = sum(r * L - r * (r - 1) // 2 for r, L in zip(rows, lens))
        moved = (total * hkv * row + sum(rows) * case["hq"] * hd * elt
                 + hkv * (8 * (total - sum(new)) + 4 * sum(new)) + 4 * (total // bs))
        return {"bytes": moved, "flops": 2 * seen * case["hq"] * hd}
    kept = [min(x, case["keep"]) for x in lens]
    if case["fresh"]:
        rows = sum(kept)
    else:  # in place, only the kept tokens past the budget move: all of the recent ones, a share of the others
        rows = sum(max(0, x - case["keep"]) if x - case["keep"] <= case["recent"]
                   else (x - case["keep"]) * case["keep"] // x for x in lens)
    moved = hkv * (4 * total + 4 * case["recorded"] * len(lens) + 8 * sum(kept) + 4 * row * rows)
    return {"bytes": moved, "flops": 0}


# ---------------------------------------------------------------- 64 bits, from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _rope_exact, "decode": _decode_exact, "prompt": _prompt_exact, "evict": _evict_exact}[s["op"]](s)


def _rope_exact(s):
    case = s["case"]
    rot = case["rot"]
    half = rot // 2
    angle = torch.stack([s["positions"][a].double() * s["inv_freq"][i]
                         for i, a in enumerate(s["pair_axis"].tolist())], 1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, None]

    def rotated(x):
        x = x.double().clone()
        first = slice(0, rot, 2) if case["interleaved"] else slice(0, half)
        second = slice(1, rot, 2) if case["interleaved"] else slice(half, rot)
        z = torch.complex(x[..., first], x[..., second]) * turn
        x[..., first], x[..., second] = z.real, z.imag
        return x

    bs, hkv, hd = case["bs"], case["hkv"], case["hd"]
    got = {"q": rotated(s["q"])}
    blocks = s["k_cache"].shape[0]
    for name, x in (("k", rotated(s["k"])), ("v", s["v"].double())):
        rows = torch.zeros((blocks * bs, hkv, hd), dtype=torch.float64, device=DEV)
        scales = torch.zeros((blocks * bs, hkv), dtype=torch.float64, device=DEV)
        fine = s["slots"] >= 0
        x = x[fine]
        if case["fp8"]:
            # the quantizer's own values: the scale and the codes' nearest values, from 64-bit rows
            scale = x.abs().amax(-1) / 448
            scale = torch.where(scale > 0, scale, torch.ones_like(scale))
            scales[s["slots"][fine]] = scale
            y = x / scale[..., None]
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            x = (torch.round(y / step) * step).clamp(-448, 448)
        rows[s["slots"][fine]] = x
        got[name] = rows.view(blocks, bs, hkv, hd)
        if case["fp8"]:
            got[name + "_scales"] = scales.view(blocks, bs, hkv).transpose(1, 2).contiguous()
    return got


def _sequence(s, pool, scales, i, L, h):
    """Rows [L, hd] of KV head h of sequence i, in 64 bits."""
    case = s["case"]
    bs = case["bs"]
    ids = s["tables"][i, : -(-L // bs)].long()
    x = pool[ids, :, h]
    if case["fp8"]:
        x = x.view(torch.float8_e4m3fn).double() * scales[ids, h].double()[..., None]
    return x.double().reshape(-1, case["hd"])[:L]


def _decode_exact(s):
    case = s["case"]
    hkv = case["hkv"]
    G = case["hq"] // hkv
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    weights = s["weights"].double()
    for i, L in enumerate(s["lens"].tolist()):
        for h in range(hkv):
            k = _sequence(s, s["k_cache"], s["ks"], i, L, h)
            p = torch.softmax(s["q"][i, h * G:(h + 1) * G].double() @ k.t() * s["scale"], -1)
            out[i, h * G:(h + 1) * G] = p @ _sequence(s, s["v_cache"], s["vs"], i, L, h)
            w = p.sum(0)
            weights[i, h, : L - 1] += w[: L - 1]
            weights[i, h, L - 1] = w[L - 1]
    return {"out": out, "weights": weights}


def _prompt_exact(s):
    case = s["case"]
    hkv = case["hkv"]
    G = case["hq"] // hkv
    weights = s["weights"].double()
    cu = s["cu"].tolist()
    for i, L in enumerate(s["lens"].tolist()):
        n = cu[i + 1] - cu[i]
        rows = n if case["window"] == 0 else min(n, case["window"])
        seen = torch.arange(L - rows, L, device=DEV)[:, None] >= torch.arange(L, device=DEV)
        for h in range(hkv):
            k = _sequence(s, s["k_cache"], s["ks"], i, L, h)
            w = torch.zeros(L, dtype=torch.float64, device=DEV)
            for g in range(G):
                x = s["q"][cu[i + 1] - rows: cu[i + 1], h * G + g].double() @ k.t() * s["scale"]
                w += torch.softmax(x.masked_fill(~seen, -math.inf), -1).sum(0)
            weights[i, h, : L - n] += w[: L - n]
            weights[i, h, L - n: L] = w[L - n:]
    return {"weights": weights}


def _evict_exact(s):
    case = s["case"]
    bs, keep = case["bs"], case["keep"]
    lens = s["lens"].tolist()
    seen = lens if s["seen"] is None else s["seen"].tolist()
    recorded = [0] * len(lens) if s["recorded"] is None else s["recorded"].tolist()
    old_w = s["weights"].cpu().numpy()
    old_p = None if s["positions"] is None else s["positions"].cpu().numpy()
    tables, new_tables = s["tables"].cpu().numpy(), s["new_tables"].cpu().numpy()
    weights = np.zeros(old_w.shape)
    positions = np.zeros(old_w.shape, dtype=np.int64)
    moves = []
    for i, L in enumerate(lens):
        for h in range(case["hkv"]):
            pos = np.arange(L) + seen[i] - L
            if recorded[i]:
                pos[: recorded[i]] = old_p[i, h, : recorded[i]]
            w = old_w[i, h, :L]
            held = (pos < case["sink"]) | (pos >= seen[i] - case["recent"])
            best = np.lexsort((np.arange(L), -w, ~held))[:keep]
            kept = np.zeros(L, dtype=bool)
            kept[best] = True
            src = np.arange(min(L, keep))
            src[~kept[:keep]] = np.flatnonzero(kept[keep:])[: (~kept[:keep]).sum()] + keep
            weights[i, h, : len(src)] = w[src]
            positions[i, h, : len(src)] = pos[src]
            dst = np.arange(len(src))
            moves.append(np.stack((tables[i, src // bs] * bs + src % bs, new_tables[i, dst // bs] * bs + dst % bs,
                                   np.full(len(src), h))))
    move = torch.from_numpy(np.concatenate(moves, 1).astype(np.int64)).to(DEV)
    got = {"lens": torch.tensor([min(x, keep) for x in lens], dtype=torch.int32),
           "weights": torch.from_numpy(weights), "positions": torch.from_numpy(positions).int()}
    for name, pool in (("k", s["k_cache"]), ("v", s["v_cache"])):
        rows = pool.view(-1, case["hkv"], case["hd"])
        after = rows.clone()
        after[move[1], move[2]] = rows[move[0], move[2]]
        got[name] = (after.view(torch.float8_e4m3fn) if case["fp8"] else after).double().view(pool.shape)
        if case["fp8"]:
            scales = s["ks" if name == "k" else "vs"]
            flat = scales.transpose(1, 2).reshape(-1, case["hkv"])
            moved = flat.clone()
            moved[move[1], move[2]] = flat[move[0], move[2]]
            got[name + "_scales"] = moved.view(-1, bs, case["hkv"]).transpose(1, 2).contiguous().double()
    return got
