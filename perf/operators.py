"""The serving operators around the paged cache, as they are measured.

Six operators of one decode step or prompt chunk, each in a plain form (elementary torch
operations) and as the library's call:

  norm_rope   per-head RMS norm of q and k, position rotation, append of K and V to the cache
  append      rows into an 8-bit cache with one power-of-two scale for each block and KV head
  decode      attention of one query per sequence over such a cache
  bounds      per-block, per-head minima and maxima of the keys a call appended
  select      the blocks each KV head's queries may need most, by the bounds' upper bound of q.k
  sparse      attention of one query per sequence over the selected blocks only
"""
import math

import torch

own = False

QMAX = {"e4m3": 448.0, "e5m2": 57344.0, "int8": 127.0}
CODES = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2, "int8": torch.int8}
ELEMENT = {"bf16": 2, "f32": 4, "e4m3": 1, "e5m2": 1, "int8": 1}
ROWS = {"bf16": torch.bfloat16, "f32": torch.float32}
# exponents a block's scale may take
SCALE_LO, SCALE_HI = -50, 50
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a few running sequences take one token each: latency is all that counts
        {"name": "norm_rope_step_4", "op": "norm_rope", "tokens": 4, "heads": 32, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "rows": "bf16", "cache": "bf16", "block": 16, "prompt": False},
        # one large chunk of prompts, 40 query heads
        {"name": "norm_rope_chunk_8192", "op": "norm_rope", "tokens": 8192, "heads": 40, "kv_heads": 8, "dim": 128,
         "rotary": 128, "interleaved": False, "rows": "bf16", "cache": "bf16", "block": 16, "prompt": True},
        # the append of a decode step of 128 sequences into an E4M3 cache
        {"name": "append_step_128_e4m3", "op": "append", "seqs": 128, "len_lo": 1024, "len_hi": 1280, "new_lo": 1,
         "new_hi": 1, "kv_heads": 8, "dim": 128, "block": 16, "rows": "bf16", "cache": "e4m3"},
        # ragged prompt chunks behind older tokens into an INT8 cache
        {"name": "append_chunks_16_int8", "op": "append", "seqs": 16, "len_lo": 2100, "len_hi": 4099, "new_lo": 801,
         "new_hi": 2047, "kv_heads": 8, "dim": 128, "block": 16, "rows": "bf16", "cache": "int8"},
        # a full batch of short sequences, 40 query heads on 8 KV heads, E4M3
        {"name": "decode_128x1280_e4m3", "op": "decode", "seqs": 128, "len_lo": 1024, "len_hi": 1280, "heads": 40,
         "kv_heads": 8, "dim": 128, "block": 16, "cache": "e4m3"},
        # few long sequences of unequal length, INT8
        {"name": "decode_16x32768_int8", "op": "decode", "seqs": 16, "len_lo": 24001, "len_hi": 32768, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "cache": "int8"},
        # the key bounds of a decode step of 64 sequences
        {"name": "bounds_step_64", "op": "bounds", "seqs": 64, "len_lo": 1024, "len_hi": 1280, "new_lo": 1,
         "new_hi": 1, "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16"},
        # the key bounds of whole prompts
        {"name": "bounds_prompts_16x8192", "op": "bounds", "seqs": 16, "len_lo": 8192, "len_hi": 8192,
         "new_lo": 8192, "new_hi": 8192, "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16"},
        # long-context decode: an eighth of the blocks is kept
        {"name": "select_16x8192", "op": "select", "seqs": 16, "len_lo": 8192, "len_hi": 8192, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "keep": 64},
        # a full batch of long sequences
        {"name": "select_64x32768", "op": "select", "seqs": 64, "len_lo": 20001, "len_hi": 32768, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "keep": 128},
        # one very long sequence: little is read, the latency of one stream counts
        {"name": "sparse_1x131072", "op": "sparse", "seqs": 1, "len_lo": 131071, "len_hi": 131071, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16", "keep": 64, "block_scales": False},
        # a full batch of long sequences
        {"name": "sparse_64x16384", "op": "sparse", "seqs": 64, "len_lo": 9001, "len_hi": 16384, "heads": 32,
         "kv_heads": 8, "dim": 128, "block": 16, "cache": "bf16", "keep": 128, "block_scales": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append", "decode", "bounds", "select", "sparse"])
    kv_heads = rng.choice([2, 4, 8, 8, 5, 1])
    case = {"op": op, "kv_heads": kv_heads, "dim": 128, "block": rng.choice([16, 16, 32])}
    if op == "norm_rope":
        case |= {"tokens": _log(rng, 1, 8192), "heads": kv_heads * rng.choice([1, 2, 4, 5]), "dim": rng.choice([64, 128]),
                 "rows": rng.choice(["bf16", "bf16", "f32"]), "prompt": rng.random() < 0.5,
                 "interleaved": rng.random() < 0.3}
        case["rotary"] = rng.choice([case["dim"], case["dim"], case["dim"] // 2])
        case["cache"] = rng.choice([case["rows"], case["rows"], "e4m3", "none"])
        return case
    if op == "append":
        step = rng.random() < 0.5
        seqs = _log(rng, 1, 256) if step else _log(rng, 1, 16)
        hi = _log(rng, 17, 8000) if step else _log(rng, 40, 4099)
        new_hi = 1 if step else rng.randint(2, min(hi, 2047))
        return case | {"seqs": seqs, "len_lo": max(new_hi, hi // 2), "len_hi": hi, "new_lo": max(1, new_hi // 3),
                       "new_hi": new_hi, "rows": rng.choice(["bf16", "bf16", "f32"]),
                       "cache": rng.choice(["e4m3", "e5m2", "int8"])}
    if op == "bounds":
        step = rng.random() < 0.5
        seqs = _log(rng, 1, 256) if step else _log(rng, 1, 16)
        hi = _log(rng, 17, 8192)
        new_hi = 1 if step else rng.randint(2, hi)
        return case | {"seqs": seqs, "len_lo": max(new_hi, hi // 2), "len_hi": hi, "new_lo": max(1, new_hi // 3),
                       "new_hi": new_hi, "cache": rng.choice(["bf16", "bf16", "e4m3", "int8"])}
    case["heads"] = kv_heads * rng.choice([1, 2, 4, 5, 8])
    hi = _log(rng, 33 if op != "select" else 700, 32768)   # where there is something to select from
    case |= {"len_lo": max(1, hi // rng.choice([2, 3, 8])), "len_hi": hi}
    if op == "decode":
        case |= {"seqs": max(1, min(_log(rng, 1, 256), 400000 // hi)), "cache": rng.choice(["e4m3", "e5m2", "int8"])}
        return case
    case |= {"seqs": max(1, min(_log(rng, 1, 64), 1000000 // hi)), "keep": _log(rng, 2, 128)}
    if op == "select":
        case["keep"] = _log(rng, 6, min(128, hi // case["block"] // 2))
    if op == "sparse":
        case["cache"] = rng.choice(["bf16", "bf16", "e4m3", "int8"])
        case["block_scales"] = case["cache"] != "bf16" and rng.random() < 0.5
    return case


def _lens(case):
    """The sequences' lengths and the number of each one's newest tokens: fixed by the case, spread over its range."""
    n, lo, hi = case["seqs"], case["len_lo"], case["len_hi"]
    at = [(i * 617 + 401) % 997 / 996 for i in range(n)]
    lens = [lo + round((hi - lo) * x) for x in at]
    lens[0] = hi
    if "new_lo" not in case:
        return lens, None
    new = [case["new_lo"] + round((case["new_hi"] - case["new_lo"]) * (1 - x)) for x in at]
    return lens, [min(a, b) for a, b in zip(new, lens)]


def _touched(case):
    """(sequence, logical block) of every block that holds a new token."""
    lens, new = _lens(case)
    b = case["block"]
    return [(s, j) for s, (n, w) in enumerate(zip(lens, new)) for j in range((n - w) // b, -(-n // b))]


def work(case):
    d, hkv = case["dim"], case["kv_heads"]
    if case["op"] == "norm_rope":
        t, hq, e = case["tokens"], case["heads"], ELEMENT[case["rows"]]
        v = 0 if case["cache"] == "none" else hkv
        out = e if case["cache"] == "none" else ELEMENT[case["cache"]]
        return {"bytes": t * d * (e * (hq + hkv + v) + e * hq + out * (hkv + v)) + t * (16 + 4 * case["rotary"]),
                "flops": t * (hq + hkv) * d * 8}
    b = case["block"]
    lens, new = _lens(case)
    if case["op"] == "append":
        rows = sum(new) * hkv * d * 2
        return {"bytes": rows * (ELEMENT[case["rows"]] + 1) + 16 * hkv * len(_touched(case)), "flops": 3 * rows}
    if case["op"] == "bounds":
        # the keys of every touched block, once; its minima and maxima
        tokens = sum(min(lens[s] - j * b, b) for s, j in _touched(case))
        return {"bytes": tokens * hkv * d * ELEMENT[case["cache"]] + len(_touched(case)) * hkv * 4 * d,
                "flops": 2 * tokens * hkv * d}
    hq, blocks = case["heads"], [-(-n // b) for n in lens]
    if case["op"] == "select":
        scored = sum(n for n in blocks if n > case["keep"])
        return {"bytes": scored * hkv * 4 * d + len(lens) * (2 * hq * d + 4 * hkv * case["keep"]) + 4 * sum(blocks),
                "flops": scored * hq * 4 * d}
    if case["op"] == "decode":
        tokens, scales = sum(lens), 8 * hkv * sum(blocks)
    else:
        tokens = sum(n if m <= case["keep"] else (case["keep"] - 1) * b + n - (m - 1) * b for n, m in zip(lens, blocks))
        scales = 8 * hkv * sum(min(m, case["keep"]) for m in blocks) if case["block_scales"] else 0
    return {"bytes": tokens * hkv * d * 2 * ELEMENT[case["cache"]] + scales + 4 * len(lens) * hq * d,
            "flops": 4 * tokens * hq * d}


# ------------------------------------------------------------------ inputs

def _tables(case, lens, gen):
    """A pool a little larger than the batch needs and each sequence's blocks, scattered over it."""
    b = case["block"]
    blocks = [-(-n // b) for n in lens]
    width, pool = max(blocks), sum(blocks) + 3
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    held = torch.arange(width, device="cuda") < torch.tensor(blocks, device="cuda")[:, None]
    table[held] = order[:sum(blocks)]
    return table, pool


def _pool(case, pool, gen, spread=1.0):
    """One cache of `pool` blocks: values about as large as keys and values are, 8-bit ones as codes."""
    shape = (pool, case["kv_heads"], case["block"], case["dim"])
    kind = case["cache"]
    if kind in ROWS:
        return torch.randn(shape, generator=gen, device="cuda", dtype=ROWS[kind]).mul_(spread)
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)
    if kind == "int8":
        return x.mul_(36).round_().clamp_(-127, 127).to(torch.int8)
    return x.mul_(100 if kind == "e4m3" else 12000).clamp_(-QMAX[kind], QMAX[kind]).to(CODES[kind])


def _block_scales(case, pool, gen):
    """A positive scale for each block and head that brings the codes back to ordinary values."""
    unit = {"e4m3": 0.01, "e5m2": 1 / 12000, "int8": 1 / 36}[case["cache"]]
    return unit * (0.5 + torch.rand(pool, case["kv_heads"], generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case}
    if case["op"] == "norm_rope":
        t, hq, hkv, d, r, b = (case[x] for x in ("tokens", "heads", "kv_heads", "dim", "rotary", "block"))
        rows = ROWS[case["rows"]]
        # one projection's output: q, k and v are views of it
        qkv = torch.randn(t, (hq + 2 * hkv) * d, generator=gen, device="cuda", dtype=rows)
        q, k, v = qkv.split([hq * d, hkv * d, hkv * d], dim=1)
        state |= {"q": q.unflatten(1, (hq, d)), "k": k.unflatten(1, (hkv, d)), "v": v.unflatten(1, (hkv, d))}
        state["q_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda", dtype=rows)
        state["k_weight"] = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda", dtype=rows)
        far = 32768
        angle = torch.arange(far, device="cuda", dtype=torch.float64)[:, None] * THETA ** (
            -torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        state["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
        if case["prompt"]:
            state["positions"] = torch.arange(t, device="cuda") + int(torch.randint(0, far - t + 1, (1,), generator=gen, device="cuda"))
        else:
            state["positions"] = torch.randint(0, far, (t,), generator=gen, device="cuda")
        state["q_out"] = torch.empty(t, hq, d, device="cuda", dtype=rows)
        if case["cache"] == "none":
            state["k_out"] = torch.empty(t, hkv, d, device="cuda", dtype=rows)
            return state
        pool = -(-t // b) + 3
        if case["prompt"]:   # whole blocks in the order of the prompt
            order = torch.randperm(pool, generator=gen, device="cuda")
            at = torch.arange(t, device="cuda")
            state["slots"] = order[at // b] * b + at % b
        else:
            state["slots"] = torch.randperm(pool * b, generator=gen, device="cuda")[:t]
        if t > 8:
            state["slots"][5] = -1   # a padding row
        state["scale"] = 0.01 if case["cache"] == "e4m3" else 1.0
        kind = ROWS.get(case["cache"], torch.float8_e4m3fn)
        state["k_cache"] = torch.zeros(pool, hkv, b, d, device="cuda", dtype=kind)
        state["v_cache"] = torch.zeros(pool, hkv, b, d, device="cuda", dtype=kind)
        return state

    lens, new = _lens(case)
    table, pool = _tables(case, lens, gen)
    state |= {"tables": table, "lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    hkv, d, b, n = case["kv_heads"], case["dim"], case["block"], len(lens)
    if new is not None:
        state["offsets"] = torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32)
        state["rows"] = sum(new)
        # what a scheduler knows of the call: the blocks it appends to
        state["touched"] = torch.tensor(_touched(case), device="cuda")
    if case["op"] == "append":
        state["k_cache"], state["v_cache"] = _pool(case, pool, gen), _pool(case, pool, gen)
        unit = {"e4m3": -7, "e5m2": -14, "int8": -6}[case["cache"]] - SCALE_LO
        # the powers of two a scale may be, from a table: exp2 on the GPU need not give them exactly
        state["powers"] = torch.tensor([2.0 ** e for e in range(SCALE_LO, SCALE_HI + 1)], device="cuda")
        for x in ("k_scales", "v_scales"):
            state[x] = state["powers"][torch.randint(unit - 1, unit + 2, (pool, hkv), generator=gen, device="cuda")]
        for x, size in (("k", 1.5), ("v", 0.6)):
            y = torch.randn(sum(new), hkv, d, generator=gen, device="cuda")
            # some tokens are larger than what their block has held
            y *= size * torch.exp(0.5 * torch.randn(sum(new), hkv, 1, generator=gen, device="cuda"))
            state[x] = y.to(ROWS[case["rows"]])
        return state
    if case["op"] == "bounds":
        state["k_cache"] = _pool(case, pool, gen)
        state["bounds"] = torch.zeros(pool, hkv, 2, d, device="cuda", dtype=torch.bfloat16)
        if case["cache"] != "bf16":
            state["k_scales"] = _block_scales(case, pool, gen)
        return state

    hq = case["heads"]
    state["q"] = torch.randn(n, hq, d, generator=gen, device="cuda").to(torch.bfloat16)
    if case["op"] == "select":
        # the minima and maxima of a block's keys: near -1.7 and 1.7 for ordinary ones
        mid = torch.randn(pool, hkv, 1, d, generator=gen, device="cuda", dtype=torch.bfloat16) * 0.5
        half = 1.7 + 0.3 * torch.randn(pool, hkv, 1, d, generator=gen, device="cuda", dtype=torch.bfloat16).abs()
        state["bounds"] = torch.cat([mid + half, mid - half], 2)
        state["selected"] = torch.empty(n, hkv, case["keep"], dtype=torch.int32, device="cuda")
        return state
    state["k_cache"], state["v_cache"] = _pool(case, pool, gen), _pool(case, pool, gen)
    state["out"] = torch.empty_like(state["q"])
    state["scale"] = d ** -0.5
    if case["cache"] != "bf16":
        if case["op"] == "decode" or case["block_scales"]:
            state["k_scales"], state["v_scales"] = _block_scales(case, pool, gen), _block_scales(case, pool, gen)
        else:
            state["k_scale"], state["v_scale"] = 0.011, 0.009
    if case["op"] == "sparse":
        # distinct blocks of each head in ascending order, the last one always among them; -1 behind
        keep, width = case["keep"], table.shape[1]
        score = torch.rand(n, hkv, width, generator=gen, device="cuda")
        j = torch.arange(width, device="cuda")
        blocks = ((state["lens"] + b - 1) // b)[:, None, None]
        score = torch.where(j == blocks - 1, 2.0, torch.where(j < blocks, score, -1.0))
        best, at = score.topk(min(keep, width), dim=2)
        at = torch.where(best >= 0, at, width).sort(2).values
        sel = torch.full((n, hkv, keep), -1, dtype=torch.int32, device="cuda")
        sel[:, :, :at.shape[2]] = torch.where(at < width, at, -1).to(torch.int32)
        state["selected"] = sel
    return state


# ------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return {"norm_rope": _norm_rope, "append": _append, "decode": _decode, "bounds": _bounds, "select": _select,
            "sparse": _sparse}[case["op"]](state, case)


def _own(s, case):
    import paged_kv_cache_462_b200 as pkv
    if case["op"] == "norm_rope":
        if case["cache"] == "none":
            pkv.qk_norm_rope(s["q_out"], s["k_out"], s["q"], s["k"], s["q_weight"], s["k_weight"], EPS, s["cos_sin"],
                             s["positions"], interleaved=case["interleaved"])
            return s["q_out"], s["k_out"]
        pkv.qk_norm_rope_and_cache(s["q_out"], s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], EPS,
                                   s["cos_sin"], s["positions"], s["k_cache"], s["v_cache"], s["slots"],
                                   interleaved=case["interleaved"], k_scale=s["scale"], v_scale=s["scale"])
        return s["q_out"], s["k_cache"], s["v_cache"]
    if case["op"] == "append":
        pkv.reshape_and_cache_block_scales(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"],
                                           s["tables"], s["lens"], s["offsets"])
        return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]
    if case["op"] == "decode":
        pkv.paged_attention_decode_block_scales(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                                s["scale"], s["k_scales"], s["v_scales"])
        return s["out"]
    if case["op"] == "bounds":
        pkv.update_key_bounds(s["bounds"], s["k_cache"], s["tables"], s["lens"], s["offsets"], s["rows"],
                              k_block_scales=s.get("k_scales"))
        return s["bounds"]
    if case["op"] == "select":
        pkv.select_blocks(s["selected"], s["q"], s["bounds"], s["tables"], s["lens"], case["block"])
        return s["selected"]
    pkv.paged_attention_decode_sparse(s["out"], s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                      s["selected"], s["scale"], s.get("k_scale", 1.0), s.get("v_scale", 1.0),
                                      k_block_scales=s.get("k_scales"), v_block_scales=s.get("v_scales"))
    return s["out"]


def _rotate(x, cos, sin, interleaved):
    if interleaved:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


def _norm_rotate(x, weight, s, case):
    r = case["rotary"]
    x = x.float()
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    cos, sin = s["cos_sin"][s["positions"]][:, None].chunk(2, -1)
    return torch.cat([_rotate(x[..., :r], cos, sin, case["interleaved"]), x[..., r:]], -1)


def _norm_rope(s, case):
    q = _norm_rotate(s["q"], s["q_weight"], s, case)
    k = _norm_rotate(s["k"], s["k_weight"], s, case)
    s["q_out"].copy_(q)
    if case["cache"] == "none":
        s["k_out"].copy_(k)
        return s["q_out"], s["k_out"]
    # padding rows write what their neighbour writes too
    at = s["slots"]
    row = torch.arange(at.shape[0], device=at.device)
    row = torch.where(at < 0, (row + 1) % at.shape[0], row)
    at = at[row]
    for cache, x in ((s["k_cache"], k), (s["v_cache"], s["v"].float())):
        if case["cache"] == "e4m3":
            x = (x / s["scale"]).clamp(-448, 448)
        cache.view(torch.uint8 if case["cache"] == "e4m3" else cache.dtype)[at // case["block"], :, at % case["block"]] = (
            x[row].to(cache.dtype).view(torch.uint8) if case["cache"] == "e4m3" else x[row].to(cache.dtype))
    return s["q_out"], s["k_cache"], s["v_cache"]


def _encode(x, kind):
    if kind == "int8":
        return x.round().clamp(-127, 127).to(torch.int8)
    return x.clamp(-QMAX[kind], QMAX[kind]).to(CODES[kind])


def _append(s, case):
    b, kind = case["block"], case["cache"]
    seq, j = s["touched"].unbind(1)
    phys = s["tables"][seq, j].long()
    end = s["lens"].long()[seq, None]
    pos = j[:, None] * b + torch.arange(b, device=j.device)
    off = s["offsets"].long()
    first = end - (off[seq + 1] - off[seq])[:, None]
    old, fresh = pos < first, (pos >= first) & (pos < end)
    row = torch.where(fresh, off[seq, None] + pos - first, 0)
    old, fresh = old[:, None, :, None], fresh[:, None, :, None]
    for cache, scales, x in ((s["k_cache"], s["k_scales"], s["k"]), (s["v_cache"], s["v_scales"], s["v"])):
        x = x.float()[row].transpose(1, 2)                                    # [touched, heads, block, dim]
        mantissa, exponent = torch.frexp((x * fresh).abs().amax((2, 3)))
        top, power = math.frexp(QMAX[kind])
        need = (exponent - power + (mantissa > top)).clamp(SCALE_LO, SCALE_HI)
        need = s["powers"][torch.where(mantissa == 0, SCALE_LO, need) - SCALE_LO]
        before = scales[phys]
        after = torch.where(old.any(2)[..., 0], torch.maximum(before, need), need)
        held = cache.view(torch.uint8)[phys]
        moved = _encode(held.view(cache.dtype).float() * (before / after)[:, :, None, None], kind)
        written = _encode(x / after[:, :, None, None], kind)
        held = torch.where(old, moved.view(torch.uint8), torch.where(fresh, written.view(torch.uint8), held))
        cache.view(torch.uint8)[phys] = held
        scales[phys] = after
    return s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"]


def _values(cache, phys, scales, const):
    """[..., heads, block, dim] of the blocks `phys` as 32-bit values."""
    x = cache.view(torch.uint8)[phys].view(cache.dtype).float() if cache.element_size() == 1 else cache[phys].float()
    return x * (const if scales is None else scales[phys][..., None, None])


def _attend(q, k, v, held, scale):
    """q [n, heads, group, d]; k, v [n, heads, tokens, d]; held [n, 1 or heads, tokens]"""
    score = (q @ k.transpose(2, 3)) * scale
    score = score.masked_fill(~held[:, :, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    return (p @ v) / p.sum(-1, keepdim=True)


def _decode(s, case):
    n, hkv, d = case["seqs"], case["kv_heads"], case["dim"]
    phys = s["tables"].long().clamp(min=0)
    k = _values(s["k_cache"], phys, s["k_scales"], 1.0).transpose(1, 2).reshape(n, hkv, -1, d)
    v = _values(s["v_cache"], phys, s["v_scales"], 1.0).transpose(1, 2).reshape(n, hkv, -1, d)
    held = torch.arange(k.shape[2], device=k.device) < s["lens"][:, None]
    q = s["q"].float().reshape(n, hkv, -1, d)
    s["out"].copy_(_attend(q, k, v, held[:, None], s["scale"]).reshape(n, -1, d))
    return s["out"]


def _bounds(s, case):
    seq, j = s["touched"].unbind(1)
    phys = s["tables"][seq, j].long()
    pos = j[:, None] * case["block"] + torch.arange(case["block"], device=j.device)
    held = (pos < s["lens"][seq, None])[:, None, :, None]
    x = _values(s["k_cache"], phys, s.get("k_scales"), 1.0)
    s["bounds"][phys, :, 0] = x.masked_fill(~held, -math.inf).amax(2).to(torch.bfloat16)
    s["bounds"][phys, :, 1] = x.masked_fill(~held, math.inf).amin(2).to(torch.bfloat16)
    return s["bounds"]


def _select(s, case):
    n, hkv, d, keep = case["seqs"], case["kv_heads"], case["dim"], case["keep"]
    # in 64 bits: which of two blocks is kept hangs on sums that lie close together
    q = s["q"].double().reshape(n, hkv, -1, d)
    x = s["bounds"][s["tables"].long().clamp(min=0)].double().permute(0, 2, 3, 4, 1)   # [n, heads, 2, d, blocks]
    score = (q.clamp(min=0) @ x[:, :, 0] + q.clamp(max=0) @ x[:, :, 1]).amax(2)
    blocks = ((s["lens"] + case["block"] - 1) // case["block"])[:, None, None]
    j = torch.arange(score.shape[2], device=score.device)
    score = score.masked_fill((j == 0) | (j == blocks - 1), math.inf).masked_fill(j >= blocks, -math.inf)
    at = score.sort(dim=2, descending=True, stable=True).indices[:, :, :keep]
    at = torch.where(at < blocks, at, score.shape[2]).sort(2).values
    s["selected"].fill_(-1)
    s["selected"][:, :, :at.shape[2]] = torch.where(at < score.shape[2], at, -1).to(torch.int32)
    return s["selected"]


def _sparse(s, case):
    n, hkv, d, b = case["seqs"], case["kv_heads"], case["dim"], case["block"]
    sel = s["selected"].long()
    phys = s["tables"].long()[torch.arange(n, device=sel.device)[:, None, None], sel.clamp(min=0)]
    head = torch.arange(hkv, device=sel.device)[None, :, None]

    def values(cache, scales, const):
        x = cache.view(torch.uint8)[phys, head].view(cache.dtype) if cache.element_size() == 1 else cache[phys, head]
        factor = const if scales is None else scales[phys, head][..., None, None]
        return (x.float() * factor).reshape(n, hkv, -1, d)

    k = values(s["k_cache"], s.get("k_scales"), s.get("k_scale", 1.0))
    v = values(s["v_cache"], s.get("v_scales"), s.get("v_scale", 1.0))
    pos = sel[..., None] * b + torch.arange(b, device=sel.device)
    held = ((pos < s["lens"].long()[:, None, None, None]) & (sel >= 0)[..., None]).reshape(n, hkv, -1)
    q = s["q"].float().reshape(n, hkv, -1, d)
    s["out"].copy_(_attend(q, k, v, held, s["scale"]).reshape(n, -1, d))
    return s["out"]


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm_rope":
        return _exact_norm_rope(s, case)
    if op == "append":
        return _exact_append(s, case)
    if op == "bounds":
        out = s["bounds"].double()
        lens = s["lens"].tolist()
        for i, j in s["touched"].tolist():
            p = int(s["tables"][i, j])
            x = s["k_cache"][p, :, :lens[i] - j * case["block"]].double()
            if "k_scales" in s:
                x = x * s["k_scales"][p].double()[:, None, None]
            out[p, :, 0], out[p, :, 1] = x.max(1).values, x.min(1).values
        return out
    if op == "select":
        return _exact_select(s, case)
    n, hq, hkv, d, b = case["seqs"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    out = torch.zeros(n, hq, d, dtype=torch.float64, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        count = -(-length // b)
        for h in range(hkv):
            if op == "sparse":
                blocks = s["selected"][i, h]
                blocks = blocks[blocks >= 0].long()
            else:
                blocks = torch.arange(count, device="cuda")
            phys = s["tables"][i].long()[blocks]
            pos = (blocks[:, None] * b + torch.arange(b, device="cuda")).flatten()
            kv = []
            for x in ("k", "v"):
                c = s[x + "_cache"]
                c = c.view(torch.uint8)[phys, h].view(c.dtype) if c.element_size() == 1 else c[phys, h]
                f = s[x + "_scales"].double()[phys, h][:, None, None] if x + "_scales" in s else s.get(x + "_scale", 1.0)
                kv.append((c.double() * f).reshape(-1, d)[pos < length])
            group = slice(h * hq // hkv, (h + 1) * hq // hkv)
            p = torch.softmax((s["q"][i, group].double() @ kv[0].T) * s["scale"], -1)
            out[i, group] = p @ kv[1]
    return out


def _exact_norm_rope(s, case):
    r = case["rotary"]
    table = s["cos_sin"].double()[s["positions"]]

    def turned(x, w):
        x = x.double()
        x = x / ((x ** 2).sum(-1, keepdim=True) / case["dim"] + EPS).sqrt() * w.double()
        y = x.clone()
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
            c, t = table[:, i, None], table[:, i + r // 2, None]
            y[..., a] = x[..., a] * c - x[..., b] * t
            y[..., b] = x[..., b] * c + x[..., a] * t
        return y

    q, k = turned(s["q"], s["q_weight"]), turned(s["k"], s["k_weight"])
    if case["cache"] == "none":
        return q, k
    # codes stand for their value over the scale: what is rounded to them
    k_cache, v_cache = s["k_cache"].double(), s["v_cache"].double()
    at = s["slots"][s["slots"] >= 0]
    k_cache[at // case["block"], :, at % case["block"]] = k[s["slots"] >= 0] / s["scale"]
    v_cache[at // case["block"], :, at % case["block"]] = s["v"].double()[s["slots"] >= 0] / s["scale"]
    return q, k_cache, v_cache


def _exact_append(s, case):
    """The codes of touched blocks by definition: nearest, ties to even, of value over scale."""
    if len(_touched(case)) > 6000:
        return None
    kind, b, qmax = case["cache"], case["block"], QMAX[case["cache"]]

    def nearest(x):
        x = x.clamp(-qmax, qmax)
        if kind == "int8":
            return x.round()
        bits, low = (4, -6) if kind == "e4m3" else (3, -14)
        step = powers[torch.frexp(x)[1].clamp(min=low + 1).long() - bits - SCALE_LO]
        return (x / step).round() * step

    lens, new = _lens(case)
    at = s["offsets"].tolist()
    powers = s["powers"].double()
    done = []
    for x in ("k", "v"):
        cache, scales, rows = s[x + "_cache"], s[x + "_scales"].double(), s[x].double()
        codes = cache.double()
        for i, j in _touched(case):
            p = int(s["tables"][i, j])
            first, end = max(lens[i] - new[i] - j * b, 0), min(lens[i] - j * b, b)
            row = at[i] + j * b + first - (lens[i] - new[i])
            fresh = rows[row:row + end - first].transpose(0, 1)
            size = fresh.abs().amax((1, 2))
            need = powers[torch.searchsorted(powers * qmax, size).clamp(max=powers.numel() - 1)]
            after = torch.maximum(need, scales[p]) if first else need
            codes[p, :, :first] = nearest(codes[p, :, :first] * (scales[p] / after)[:, None, None])
            codes[p, :, first:end] = nearest(fresh / after[:, None, None])
            scales[p] = after
        done.append((codes.to(torch.int8) if kind == "int8" else codes, scales))
    return done[0][0], done[1][0], done[0][1], done[1][1]


def _exact_select(s, case):
    n, hkv, keep = case["seqs"], case["kv_heads"], case["keep"]
    out = torch.full((n, hkv, keep), -1, dtype=torch.int32, device="cuda")
    for i, length in enumerate(s["lens"].tolist()):
        count = -(-length // case["block"])
        x = s["bounds"][s["tables"][i, :count].long()].double()
        for h in range(hkv):
            group = case["heads"] // hkv
            score = torch.full((count,), -math.inf, dtype=torch.float64, device="cuda")
            for g in range(group):
                q = s["q"][i, h * group + g].double()
                score = torch.maximum(score, torch.maximum(q * x[:, h, 0], q * x[:, h, 1]).sum(1))
            score[0] = score[-1] = math.inf
            best = torch.argsort(score, descending=True, stable=True)[:keep].sort().values
            out[i, h, :best.numel()] = best.to(torch.int32)
    return out
