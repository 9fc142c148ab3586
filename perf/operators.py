"""Measured cases of the paged FP8 KV cache: writing keys and values into it,
reading them back, and attention of new tokens over it.

The cache holds pages of ``page`` tokens of every KV head: E4M3 codes
``[pages, heads, page, 128]`` and one power-of-two scale (E8M0 byte e, value
2^(e-127)) for each token and head, ``[pages, heads, page]``.  Quantising a
vector x: e is the smallest exponent with max|x| <= 448 * 2^(e-127), clamped
to 0..254 (127 for a zero vector), and code = E4M3(x * 2^(127-e)), rounded to
the nearest even.  The scaling is exact, so codes, scales and the values read
back are the same in every precision; only attention rounds.

A case is one call.  ``run`` gives its outputs in the plain form (elementary
torch operations in 32 bits), or with ``own`` from the package's operators;
``exact`` gives them from the definition in 64 bits.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128
_TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _write(name, tokens, heads, page, dtype, fused, padded):
    return {"name": name, "op": "write", "tokens": tokens, "heads": heads, "page": page, "dtype": dtype,
            "fused": fused, "padded": padded}


def _read(name, tokens, heads, page, dtype):
    return {"name": name, "op": "read", "tokens": tokens, "heads": heads, "page": page, "dtype": dtype}


def _attend(name, batch, q_max, kv_max, heads, group, page, dtype, *, ragged=0, window=0, lse=False, causal=True):
    """ragged: 0 for equal lengths, else the seed that the lengths are drawn with."""
    return {"name": name, "op": "attend", "batch": batch, "q_max": q_max, "kv_max": kv_max, "heads": heads,
            "group": group, "page": page, "dtype": dtype, "ragged": ragged, "window": window, "lse": lse,
            "causal": causal}


def listed():
    return [
        # The cache write of one decode step of 64 sequences: 64 tokens, one
        # each, two of them padding; the smallest call, latency counts.
        _write("write_step_64", 64, 8, 16, "bf16", True, True),
        # One prefill chunk, K and V views of a fused QKV projection.
        _write("write_chunk_8192", 8192, 8, 64, "bf16", True, False),
        # A whole prompt of the long workload's length, FP16.
        _write("write_prompt_73397", 73397, 8, 128, "fp16", False, False),
        # A short cached prefix read back for a program that wants it dense.
        _read("read_1000", 1000, 7, 16, "fp16"),
        # A long sequence read back (offload, or a change of format).
        _read("read_65536", 65536, 8, 64, "bf16"),
        # One decode step of one short sequence: latency.
        _attend("decode_b1_1k", 1, 1, 1024, 2, 7, 16, "bf16"),
        # One decode step of a serving batch with ragged contexts and an empty
        # (padded) entry; 56 query heads over 8 KV heads.
        _attend("decode_b32_ragged_16k", 32, 1, 16384, 8, 7, 64, "bf16", ragged=1, lse=True),
        # One decode step over long contexts: bound by the cache's bytes.
        _attend("decode_b8_128k", 8, 1, 131072, 8, 4, 64, "fp16"),
        # Verification of four drafted tokens per sequence, shared KV head.
        _attend("verify_b16_8k", 16, 4, 8191, 1, 8, 32, "bf16", lse=True),
        # Chunked prefill of one sequence: a chunk over a moderate context.
        _attend("chunk_512_8k", 1, 512, 8192, 8, 7, 64, "bf16"),
        # A mixed batch of chunks and single tokens with a sliding window.
        _attend("chunk_mixed_window", 8, 500, 8000, 4, 8, 16, "fp16", ragged=2, window=4096, lse=True),
        # A large chunk over a long context: bound by the tensor cores.
        _attend("chunk_4k_64k", 1, 4096, 65536, 8, 4, 128, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(("write", "read", "decode", "verify", "chunk", "chunk"))
    page = rng.choice((16, 32, 48, 64, 128, 256))
    dtype = rng.choice(("bf16", "fp16"))
    if op == "write":
        return {k: v for k, v in _write("", _log(rng, 1, 73397), rng.randint(1, 8), page, dtype,
                                        rng.random() < 0.5, rng.random() < 0.5).items() if k != "name"}
    if op == "read":
        return {k: v for k, v in _read("", _log(rng, 1, 65536), rng.randint(1, 8), page, dtype).items()
                if k != "name"}
    heads = rng.randint(1, 8)
    group = rng.choice((1, 2, 3, 4, 5, 7, 8, 16) if heads <= 4 else (1, 2, 4, 7))
    ragged = rng.randint(1, 10 ** 6) if rng.random() < 0.6 else 0
    lse = rng.random() < 0.5
    causal = rng.random() < 0.85
    if op == "chunk":
        batch = _log(rng, 1, 8)
        q_max = _log(rng, 17, 4096 // batch)
        kv_max = _log(rng, q_max, max(q_max, 61440 // batch))
        group = min(group, 32 // heads)
    else:
        batch = _log(rng, 1, 64)
        q_max = 1 if op == "decode" else rng.randint(2, 8)
        kv_max = _log(rng, 16, 1048576 // batch)
    window = _log(rng, 16, kv_max) if causal and rng.random() < 0.3 else 0
    return {k: v for k, v in _attend("", batch, q_max, kv_max, heads, group, page, dtype, ragged=ragged,
                                     window=window, lse=lse, causal=causal).items() if k != "name"}


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of every sequence."""
    b, qm, km = case["batch"], case["q_max"], case["kv_max"]
    if not case["ragged"]:
        return [qm] * b, [km] * b
    rng = random.Random(case["ragged"])
    ql = [qm if qm == 1 else _log(rng, 1, qm) for _ in range(b)]
    ql[rng.randrange(b)] = qm
    kl = [_log(rng, max(1, q), max(q, km)) for q in ql]
    kl[rng.randrange(b)] = km
    if b > 4:
        kl[rng.randrange(b)] = 0     # a padded entry: rows that see no key
    return ql, kl


def _pairs(case):
    """Query-key pairs that the mask leaves, for one query head, and the keys read."""
    pairs = keys = 0
    for ql, kl in zip(*_lengths(case)):
        if not case["causal"]:
            pairs, keys = pairs + ql * kl, keys + kl
            continue
        pos = np.arange(kl - ql, kl, dtype=np.int64)
        seen = np.clip(pos + 1, 0, None)
        if case["window"]:
            seen = np.minimum(seen, case["window"])
        pairs += int(seen.sum())
        keys += min(kl, case["window"] + ql - 1) if case["window"] else kl
    return pairs, keys


def work(case):
    if case["op"] == "attend":
        pairs, keys = _pairs(case)
        hq = case["heads"] * case["group"]
        rows = sum(_lengths(case)[0]) * hq
        return {"bytes": keys * case["heads"] * 2 * (D + 1) + rows * (4 * D + (4 if case["lse"] else 0)),
                "flops": 4 * D * hq * pairs}
    n = case["tokens"] * case["heads"] * 2
    return {"bytes": n * (D + 1 + 2 * D) + 4 * case["tokens"], "flops": 2 * n * D}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _quantise(x):
    """E4M3 codes (float8 tensor) and E8M0 bytes of the vectors x [..., 128]."""
    x = x.float()
    amax = x.abs().amax(-1)
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(-127, 127)
    e = torch.where(amax == 0, torch.zeros_like(e), e)
    inverse = ((127 - e) << 23).view(torch.float32)    # 2^-e by its bits: exact
    return (x * inverse.unsqueeze(-1)).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _scale(byte):
    """2^(byte - 127) in 32 bits by its bits: exact."""
    e = byte.int()
    return torch.where(e == 0, 1 << 22, e << 23).to(torch.int32).view(torch.float32)


def _tokens(gen, shape, dtype, biased):
    """Activations: normal, with a per-(head, channel) offset where keys have one."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    if biased:
        x += torch.randn(shape[-2:], generator=gen, device="cuda", dtype=torch.float32) * math.sqrt(2.0)
    return x.to(dtype)


def _empty_cache(pages, heads, page):
    return {"k": torch.zeros((pages, heads, page, D), dtype=torch.uint8, device="cuda"),
            "v": torch.zeros((pages, heads, page, D), dtype=torch.uint8, device="cuda"),
            "k_scale": torch.full((pages, heads, page), 127, dtype=torch.uint8, device="cuda"),
            "v_scale": torch.full((pages, heads, page), 127, dtype=torch.uint8, device="cuda")}


def _filled_cache(gen, pages, heads, page):
    c = {}
    for n in ("k", "v"):
        x = _tokens(gen, (pages, page, heads, D), torch.bfloat16, n == "k")
        codes, scale = _quantise(x)
        c[n] = codes.view(torch.uint8).transpose(1, 2).contiguous()
        c[n + "_scale"] = scale.transpose(1, 2).contiguous()
    return c


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    heads, page = case["heads"], case["page"]
    if case["op"] != "attend":
        n = case["tokens"]
        pages = -(-n // page) + 3
        order = torch.randperm(pages, generator=gen, device="cuda")
        t = torch.arange(n, device="cuda")
        slots = (order[t // page] * page + t % page).to(torch.int32)
        s = {"case": case, "slots": slots}
        if case["op"] == "read":
            s.update(_filled_cache(gen, pages, heads, page))
            return s
        dtype = _TYPES[case["dtype"]]
        if case["padded"]:
            slots[torch.randperm(n, generator=gen, device="cuda")[:n // 32]] = -1
        x = _tokens(gen, (n, 3 * heads if case["fused"] else 2 * heads, D), dtype, True)
        if case["fused"]:
            s["new_k"], s["new_v"] = x[:, heads:2 * heads], x[:, 2 * heads:]
        else:
            s["new_k"], s["new_v"] = x[:, :heads].contiguous(), x[:, heads:].contiguous()
        s.update(_empty_cache(pages, heads, page))
        return s
    ql, kl = _lengths(case)
    width = max(1, -(-max(kl) // page))
    used = [-(-k // page) for k in kl]
    pages = sum(used) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros((len(kl), width), dtype=torch.int32, device="cuda")
    col = torch.arange(width, device="cuda")
    held = col.unsqueeze(0) < torch.tensor(used, device="cuda").unsqueeze(1)
    table[held] = order[:sum(used)]
    s = {"case": case, "table": table, "kv_lens": torch.tensor(kl, dtype=torch.int32, device="cuda"), "q_max": max(ql)}
    s["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(ql)]), dtype=torch.int32, device="cuda")
    s["q"] = _tokens(gen, (sum(ql), heads * case["group"], D), _TYPES[case["dtype"]], True)
    s.update(_filled_cache(gen, pages, heads, page))
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _fp8(x):
    return x.view(torch.float8_e4m3fn)


def _plain_write(s):
    page = s["case"]["page"]
    keep = s["slots"] >= 0
    slots = s["slots"][keep].long()
    for n in ("k", "v"):
        codes, scale = _quantise(s["new_" + n])
        s[n][slots // page, :, slots % page] = codes.view(torch.uint8)[keep]
        s[n + "_scale"][slots // page, :, slots % page] = scale[keep]
    return {"k": _fp8(s["k"]), "v": _fp8(s["v"]), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _values(s, n):
    """The cache's values in 32 bits, [pages, heads, page, 128]."""
    return _fp8(s[n]).float() * _scale(s[n + "_scale"]).unsqueeze(-1)


def _plain_read(s):
    page, dtype = s["case"]["page"], _TYPES[s["case"]["dtype"]]
    slots = s["slots"].long()
    at = (slots // page, slice(None), slots % page)
    out = {}
    for n in ("k", "v"):
        out[n] = (_fp8(s[n][at]).float() * _scale(s[n + "_scale"][at]).unsqueeze(-1)).to(dtype)
    return out


def _plain_attend(s):
    case = s["case"]
    heads, group, page = case["heads"], case["group"], case["page"]
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    ql = cu[1:] - cu[:-1]
    batch, length = s["table"].shape[0], s["table"].shape[1] * page
    # the sequences padded to one length: queries [B, H, g * T, 128], keys and values [B, H, L, 128]
    i = torch.arange(s["q_max"], device="cuda")
    row = (cu[:-1].unsqueeze(1) + i).clamp_(max=max(0, s["q"].shape[0] - 1))
    q = s["q"][row].float().view(batch, s["q_max"], heads, group, D).permute(0, 2, 3, 1, 4)
    q = q.reshape(batch, heads, group * s["q_max"], D)
    j = torch.arange(length, device="cuda")
    there = (j < kv.unsqueeze(1)).view(batch, 1, length, 1)
    k, v = (_values({n: s[n][s["table"].long()], n + "_scale": s[n + "_scale"][s["table"].long()]}, n)
            .transpose(1, 2).reshape(batch, heads, length, D).masked_fill_(~there, 0.0) for n in ("k", "v"))
    score = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    seen = (j < kv.unsqueeze(1)).unsqueeze(1)
    if case["causal"]:
        pos = (kv - ql).unsqueeze(1) + i
        seen = seen & (j <= pos.unsqueeze(2))
        if case["window"]:
            seen = seen & (j > (pos - case["window"]).unsqueeze(2))
    score = score.view(batch, heads, group, s["q_max"], length)
    score.masked_fill_(~seen.view(batch, 1, 1, seen.shape[1], length), -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(batch, heads, group * s["q_max"], length), v)
    o = o.view(batch, heads, group, s["q_max"], D) / torch.where(total == 0, torch.ones_like(total), total)
    lse = (total.log() + top).squeeze(-1)
    held = i < ql.unsqueeze(1)
    out = {"o": o.permute(0, 3, 1, 2, 4).reshape(batch, s["q_max"], heads * group, D)[held].to(torch.bfloat16)}
    if case["lse"]:
        out["lse"] = lse.permute(0, 3, 1, 2).reshape(batch, s["q_max"], heads * group)[held]
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        import fp8_bit_attention_gb300 as ovc

        if "cache" not in state:    # the handle a program keeps beside its cache's memory
            state["cache"] = ovc.KVCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
        cache, case = state["cache"], state["case"]
        if op == "write":
            ovc.kv_cache_write(cache, state["new_k"], state["new_v"], state["slots"])
            return {"k": _fp8(cache.k), "v": _fp8(cache.v), "k_scale": cache.k_scale, "v_scale": cache.v_scale}
        if op == "read":
            k, v = ovc.kv_cache_read(cache, state["slots"], dtype=_TYPES[case["dtype"]])
            return {"k": k, "v": v}
        ragged = {} if state["q_max"] == 1 else {"cu_q": state["cu_q"], "max_q": state["q_max"]}
        o = ovc.paged_attention(state["q"], cache, state["table"], state["kv_lens"], causal=case["causal"],
                                window=case["window"] or None, return_lse=case["lse"], **ragged)
        return {"o": o[0], "lse": o[1]} if case["lse"] else {"o": o}
    return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](state)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def _e4m3_grid():
    """The value of each E4M3 byte (the two NaN bytes as NaN)."""
    b = np.arange(256)
    sign, exp, man = np.where(b & 128, -1.0, 1.0), (b >> 3) & 15, b & 7
    val = sign * np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
    val[[127, 255]] = np.nan
    return val


def _powers():
    """The value of each scale byte."""
    return np.ldexp(1.0, np.arange(255) - 127)


def _e4m3_round(x):
    """Values of |x| <= 448 rounded to the nearest E4M3 value, ties to the even byte."""
    values = _e4m3_grid()[:127]
    middle = torch.tensor((values[:-1] + values[1:]) / 2, dtype=torch.float64, device="cuda")
    y = x.abs()
    i = torch.searchsorted(middle, y)
    tie = y == middle[i.clamp(max=125)]
    i = torch.where(tie & (i % 2 == 1), i + 1, i)
    return torch.copysign(torch.tensor(values, dtype=torch.float64, device="cuda")[i], x)


def exact(case, seed):
    s = prepare(case, seed)
    page = case["page"]
    grid = torch.tensor(_e4m3_grid(), dtype=torch.float64, device="cuda")
    power = torch.tensor(_powers(), dtype=torch.float64, device="cuda")
    if case["op"] == "write":
        out = {}
        for n in ("k", "v"):
            x = s["new_" + n].double()
            amax = x.abs().amax(-1)
            byte = torch.searchsorted(448.0 * power, amax)    # the first scale that reaches amax
            byte = torch.where(amax == 0, torch.full_like(byte, 127), byte)
            val = _e4m3_round(x / power[byte].unsqueeze(-1))
            cache = torch.zeros(s[n].shape, dtype=torch.float64, device="cuda")
            scale = s[n + "_scale"].clone()
            for t in torch.nonzero(s["slots"] >= 0).flatten().split(4096):
                slot = s["slots"][t].long()
                p, r = torch.div(slot, page, rounding_mode="floor"), torch.remainder(slot, page)
                cache[p, :, r] = val[t]
                scale[p, :, r] = byte[t].to(torch.uint8)
            out[n], out[n + "_scale"] = cache, scale
        return out
    if case["op"] == "read":
        out = {}
        p, r = s["slots"].long() // page, s["slots"].long() % page
        for n in ("k", "v"):
            out[n] = grid[s[n][p, :, r].long()] * power[s[n + "_scale"][p, :, r].long()].unsqueeze(-1)
        return out
    group, at, o, lse = case["group"], 0, [], []
    for b, (ql, kl) in enumerate(zip(*_lengths(case))):
        q = s["q"][at:at + ql].double()
        at += ql
        ob = torch.zeros((ql, case["heads"] * group, D), dtype=torch.float64, device="cuda")
        lb = torch.full((ql, case["heads"] * group), -math.inf, dtype=torch.float64, device="cuda")
        held = s["table"][b, :-(-kl // page)].long()
        for h in range(case["heads"] if kl else 0):
            k, v = (grid[s[n][held, h].reshape(-1, D)[:kl].long()] *
                    power[s[n + "_scale"][held, h].reshape(-1)[:kl].long()].unsqueeze(-1)
                    for n in ("k", "v"))
            for hq in range(h * group, (h + 1) * group):
                for i0 in range(0, ql, 1024):
                    sc = (q[i0:i0 + 1024, hq] @ k.T) / math.sqrt(D)
                    if case["causal"]:
                        pos = torch.arange(kl - ql + i0, kl - ql + i0 + sc.shape[0], device="cuda").unsqueeze(1)
                        j = torch.arange(kl, device="cuda").unsqueeze(0)
                        hide = j > pos
                        if case["window"]:
                            hide |= j + case["window"] <= pos
                        sc[hide] = -math.inf
                    lt = torch.logsumexp(sc, -1)
                    w = torch.exp(sc - torch.where(lt == -math.inf, torch.zeros_like(lt), lt).unsqueeze(-1))
                    ob[i0:i0 + 1024, hq] = w @ v
                    lb[i0:i0 + 1024, hq] = lt
        o.append(ob)
        lse.append(lb)
    return {"o": torch.cat(o), "lse": torch.cat(lse)} if case["lse"] else {"o": torch.cat(o)}
