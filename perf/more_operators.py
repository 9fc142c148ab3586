"""Measured cases of the steps between two attention calls over a paged FP8 KV
cache: who holds which page (``step``: pages given back and taken; ``branch``:
sequences forked into candidates), what moves inside the cache (``copy`` of
pages, ``compact`` of the tokens that are kept), and which drafted tokens stay
(``verify``).

Pages.  Row b of the page table holds ceil(lens[b] / page) pages, entries behind
them are -1, and refs[p] counts the entries that name page p.  Releasing to a
smaller length drops the pages behind it.  Reserving to a larger one takes the
lowest free pages, in the order of the rows and then of the columns; a row whose
last, partly filled page others hold too takes a page in its place and lists the
copy that has to follow, unless all holders of the page grow in the call: then
the highest of them keeps it.  A row grows if the rows up to it need no more
pages than are free.

Drafts.  Drafted token x of row i stays if all before it did and u * q[x] < p[x];
at the first that does not, the next token is drawn from max(p - q, 0) (from p
where that is zero everywhere), and after the last from its row of p: the least
index whose running sum exceeds u times the total.  Drafts without probabilities
were certain: q is 1 at the draft.

A case is one pass.  ``run`` gives its outputs in the plain form (elementary
torch operations; sums that are compared in 64 bits), or with ``own`` from the
package's operators; ``exact`` gives them from the definition.
"""
import math

import numpy as np
import torch

own = False

D = 128
_TYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def _step(name, rows, len_max, page, pool, *, churn=0.0, tight=False):
    """churn: the share of rows that give all up and take in a new prompt."""
    return {"name": name, "op": "step", "rows": rows, "len_max": len_max, "page": page, "pool": pool, "churn": churn,
            "tight": tight}


def _branch(name, parents, children, len_max, drafts, page, pool):
    return {"name": name, "op": "branch", "parents": parents, "children": children, "len_max": len_max, "drafts": drafts,
            "page": page, "pool": pool}


def _copy(name, copies, heads, page, *, partial):
    return {"name": name, "op": "copy", "copies": copies, "heads": heads, "page": page, "partial": partial}


def _compact(name, batch, kv_max, heads, page, kind, *, per_head=False, ragged=0):
    """kind: the last few tokens thinned out ("reject"), a random half kept
    ("evict"), the first four and the last three quarters kept ("window").
    ragged: 0 for equal lengths, else the seed that the lengths are drawn with."""
    return {"name": name, "op": "compact", "batch": batch, "kv_max": kv_max, "heads": heads, "page": page, "kind": kind,
            "per_head": per_head, "ragged": ragged}


def _verify(name, batch, drafts, vocab, dtype, *, lookup=False, ragged=0):
    """lookup: the drafts came without probabilities (found in the text).
    ragged: 0 for equal numbers of drafts, else the seed that they are drawn with."""
    return {"name": name, "op": "verify", "batch": batch, "drafts": drafts, "vocab": vocab, "dtype": dtype, "lookup": lookup,
            "ragged": ragged}


def listed():
    return [
        # One decode step of 64 sequences, rejected drafts' pages given back
        # and room made for the next ones: latency.
        _step("step_64", 64, 8192, 16, 32768),
        # A large server: half of 256 sequences are done and new prompts of up
        # to 128k tokens come in their place.
        _step("step_prompts_256", 256, 131072, 64, 600000, churn=0.5),
        # Four candidates for each of 8 sequences, each to be grown by its own
        # drafts: latency.
        _branch("branch_8x4", 8, 4, 4096, 5, 16, 8192),
        # Wide sampling from long prompts: 64 prompts, 15 more rows each.
        _branch("branch_64x15", 64, 15, 65536, 64, 64, 131072),
        # The copies of forked rows' last pages, partly filled: latency.
        _copy("copy_tails_32", 32, 8, 16, partial=True),
        # Whole pages, as a cache is spread anew: bound by memory.
        _copy("copy_pages_2048", 2048, 8, 64, partial=False),
        # The accepted path of a tree of drafts at the end of 16 sequences
        # moves together; nearly all tokens stay where they are: latency.
        _compact("compact_reject_16", 16, 8192, 8, 16, "reject", ragged=1),
        # The better half of each head's tokens, by that head's own choice.
        _compact("compact_evict_8x32k", 8, 32768, 8, 64, "evict", per_head=True, ragged=2),
        # A window slides on over one long sequence.
        _compact("compact_window_64k", 1, 65536, 8, 128, "window"),
        # Four drafts of one sequence: latency.
        _verify("verify_b1_32k", 1, 4, 32000, "fp32"),
        # A serving batch with up to eight drafts, some with none.
        _verify("verify_b64_128k", 64, 8, 131072, "fp32", ragged=3),
        # Drafts found in the text, an odd vocabulary, probabilities in 16 bits.
        _verify("verify_b256_lookup", 256, 4, 100003, "bf16", lookup=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    op = rng.choice(("step", "branch", "copy", "compact", "compact", "verify", "verify"))
    page = rng.choice((16, 32, 48, 64, 128, 256))
    if op == "step":
        rows = _log(rng, 1, 512)
        len_max = _log(rng, 16, min(131072, 524288 // rows * page))
        least = rows * -(-len_max // page)
        c = _step("", rows, len_max, page, _log(rng, least, max(least, min(4 * least, 600000))),
                  churn=rng.choice((0.0, 0.25, 0.5)), tight=rng.random() < 0.3)
    elif op == "branch":
        parents, children = _log(rng, 1, 64), rng.randint(1, 15)
        len_max, drafts = _log(rng, 1, 65536), _log(rng, 1, 64)
        least = parents * (-(-len_max // page) + (children + 1) * (-(-drafts // page) + 1))
        c = _branch("", parents, children, len_max, drafts, page, _log(rng, least, 2 * least))
    elif op == "copy":
        heads = rng.randint(1, 8)
        c = _copy("", _log(rng, 1, 2048 * 8 * 64 // (heads * page)), heads, page, partial=rng.random() < 0.5)
    elif op == "compact":
        heads, batch = rng.randint(1, 8), _log(rng, 1, 32)
        c = _compact("", batch, _log(rng, 1, 131072 // batch), heads, page, rng.choice(("reject", "evict", "window")),
                     per_head=rng.random() < 0.4, ragged=rng.randint(1, 10 ** 6) if rng.random() < 0.6 else 0)
    else:
        vocab, drafts = _log(rng, 100, 200001), _log(rng, 1, 8)
        c = _verify("", _log(rng, 1, min(256, 60_000_000 // (vocab * (drafts + 1)))), drafts, vocab,
                    rng.choice(("fp32", "bf16", "fp16")), lookup=rng.random() < 0.3, ragged=rng.randint(1, 10 ** 6) if rng.random() < 0.6 else 0)
    return {k: v for k, v in c.items() if k != "name"}


# ---------------------------------------------------------------------------
# Lengths and tables, made on the host
# ---------------------------------------------------------------------------
def _up(n, page):
    return -(-n // page)


def _host_rng(seed):
    return np.random.default_rng(int(seed) * 7919 + 17)


def _some_lengths(rng, n, most, least=1):
    v = np.exp(rng.uniform(math.log(least), math.log(most + 0.99), n)).astype(np.int64).clip(least, most)
    v[rng.integers(n)] = most
    return v


def _held_rows(rng, lens, page, pool, share):
    """A table whose rows hold random pages (with `share`, groups of four rows
    have the first half of their whole pages in common), and refs."""
    rows, n = len(lens), _up(lens, page)
    table = np.full((rows, max(1, int(n.max()))), -1, np.int32)
    held = np.arange(table.shape[1]) < n[:, None]
    table[held] = rng.permutation(pool)[:n.sum()]
    common = np.zeros(rows, np.int64)
    for g in range(0, rows - 3 if share else 0, 4):
        k = int((lens[g:g + 4] // page).min()) // 2
        table[g + 1:g + 4, :k] = table[g, :k]
        common[g:g + 4] = k
    return table, np.bincount(table[held], minlength=pool).astype(np.int32), common


def _step_inputs(case, seed):
    rng = _host_rng(seed)
    rows, page, pool, most = case["rows"], case["page"], case["pool"], case["len_max"]
    lens = _some_lengths(rng, rows, most, max(1, most // 16))
    table, refs, common = _held_rows(rng, lens, page, pool, True)
    low = np.maximum(0, lens - rng.integers(0, 5, rows))
    for g in range(0, rows - 3, 16):              # a group that goes back into what it shares
        if common[g]:
            low[g:g + 4] = common[g] * page - rng.integers(1, page)
    new = rng.random(rows) < case["churn"]
    low = np.where(new, 0, low)
    high = np.minimum(most, np.where(new, _some_lengths(rng, rows, most, max(1, most // 16)), low + rng.integers(1, 9, rows)))
    if case["tight"]:                              # others hold most of what is free
        need = int((_up(high, page) - _up(low, page)).sum())
        free = rng.permutation(np.nonzero(refs == 0)[0])
        back = int((_up(lens, page) - _up(low, page)).sum())
        refs[free[max(0, need // 2 - back):]] = 1
    return table, lens, refs, low, high


def _branch_inputs(case, seed):
    rng = _host_rng(seed)
    p, c, page = case["parents"], case["children"], case["page"]
    rows = rng.permutation(p * (c + 1))
    parents, children = rows[:p], rows[p:]
    lens = np.zeros(p * (c + 1), np.int64)
    lens[parents] = _some_lengths(rng, p, case["len_max"], max(1, case["len_max"] // 16))
    table, refs, _ = _held_rows(rng, lens, page, case["pool"], False)
    wide = np.full((len(lens), _up(case["len_max"] + case["drafts"], page)), -1, np.int32)
    wide[:, :table.shape[1]] = table
    origin = np.repeat(parents, c)
    high = np.zeros(len(lens), np.int64)
    high[children] = lens[origin] + rng.integers(1, case["drafts"] + 1, len(children))
    # half of the parents go on as candidates themselves, the others only lend their pages
    grow = np.where(rng.random(p) < 0.5, 1, 0)
    high[parents] = lens[parents] + grow * rng.integers(1, case["drafts"] + 1, p)
    return wide, lens, refs, origin, children, high


def _compact_lengths(case):
    rng = _host_rng(case["ragged"])
    n, most = case["batch"], case["kv_max"]
    lens = _some_lengths(rng, n, most, max(1, most // 16)) if case["ragged"] else np.full(n, most)
    if case["kind"] == "reject":
        kept = lens - np.minimum(lens, rng.integers(0, 7, n))
    elif case["kind"] == "evict":
        kept = (lens + 1) // 2
    else:
        kept = np.minimum(lens, 4 + lens * 3 // 4)
    return lens, kept


def _draft_lengths(case):
    n, most = case["batch"], case["drafts"]
    if not case["ragged"]:
        return np.full(n, most)
    rng = _host_rng(case["ragged"])
    v = rng.integers(0, most + 1, n)
    v[rng.integers(n)] = most
    return v


def work(case):
    op = case["op"]
    if op == "step":
        _, lens, _, low, high = _step_inputs(case, 1)
        moved = int((_up(lens, case["page"]) - _up(low, case["page"])).sum() + (_up(high, case["page"]) - _up(low, case["page"])).sum())
        return {"bytes": 4 * case["pool"] + 12 * moved + 28 * case["rows"], "flops": case["pool"] + moved}
    if op == "branch":
        _, lens, _, origin, _, _ = _branch_inputs(case, 1)
        shared = int(_up(lens[origin], case["page"]).sum())
        return {"bytes": 4 * case["pool"] + 24 * shared + 28 * len(lens), "flops": case["pool"] + 2 * shared}
    if op == "copy":
        tokens = case["copies"] * (case["page"] if not case["partial"] else (case["page"] + 1) / 2)
        return {"bytes": int(tokens * case["heads"] * 4 * (D + 1)) + 12 * case["copies"], "flops": 0}
    if op == "compact":
        lens, kept = _compact_lengths(case)
        lists = case["heads"] if case["per_head"] else 1
        moved = int({"reject": np.minimum(kept, 8), "evict": kept, "window": np.maximum(0, kept - 4)}[case["kind"]].sum())
        return {"bytes": moved * (case["heads"] * 4 * (D + 1) + 4 * lists) + 8 * case["batch"], "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    lines = case["batch"] * case["vocab"]
    return {"bytes": lines * size * (1 if case["lookup"] else 2) + case["batch"] * (case["drafts"] * (12 + 2 * size) + 12),
            "flops": lines * (2 if case["lookup"] else 3)}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _ints(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _filled_cache(gen, pages, heads, page):
    c = {}
    for n in ("k", "v"):
        codes = torch.randint(0, 256, (pages, heads, page, D), generator=gen, device="cuda", dtype=torch.uint8)
        c[n] = torch.where((codes & 127) == 127, codes ^ 1, codes)       # any code but NaN
        c[n + "_scale"] = torch.randint(100, 140, (pages, heads, page), generator=gen, device="cuda", dtype=torch.uint8)
    return c


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 17)
    if op == "step":
        table, lens, refs, low, high = _step_inputs(case, seed)
        return {"case": case, "table": _ints(table), "lens": _ints(lens), "refs": _ints(refs), "low": _ints(low), "high": _ints(high)}
    if op == "branch":
        table, lens, refs, origin, children, high = _branch_inputs(case, seed)
        return {"case": case, "table": _ints(table), "lens": _ints(lens), "refs": _ints(refs), "low": _ints(lens),
                "origin": _ints(origin), "children": _ints(children), "high": _ints(high)}
    if op == "copy":
        n, page = case["copies"], case["page"]
        pages = 2 * n + 256
        order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
        tokens = torch.randint(1, page + 1, (n,), generator=gen, device="cuda", dtype=torch.int32)
        src, dst = order[:n].clone(), order[n:2 * n].clone()
        src[2::64] = -1                                                  # rows that copy nothing
        return {"case": case, "src": src, "dst": dst, "tokens": tokens if case["partial"] else None,
                **_filled_cache(gen, pages, case["heads"], page)}
    if op == "compact":
        page, heads = case["page"], case["heads"]
        lens, kept = _compact_lengths(case)
        rng = _host_rng(seed)
        n = _up(lens, page)
        table, refs, _ = _held_rows(rng, lens, page, int(n.sum()) + 2, False)
        lists = heads if case["per_head"] else 1
        keep = []
        for length, k in zip(lens, kept):
            i = torch.arange(length, device="cuda")
            if case["kind"] == "window":
                first = min(4, int(k))
                one = torch.cat([i[:first], i[length - k + first:]]).expand(lists, -1)
            else:                                                        # the tokens that may go, and a random choice of them
                fixed = max(0, int(length) - 8) if case["kind"] == "reject" else 0
                luck = torch.rand((lists, int(length) - fixed), generator=gen, device="cuda")
                some = luck.topk(max(0, int(k) - fixed), dim=1).indices.sort(1).values + fixed
                one = torch.cat([i[:fixed].expand(lists, -1), some], 1)[:, :int(k)]
            keep.append(one)
        keep = torch.cat(keep, 1).to(torch.int32)
        return {"case": case, "table": _ints(table), "lens": _ints(lens), "refs": _ints(refs),
                "keep": keep if case["per_head"] else keep[0].contiguous(),
                "cu": _ints(np.concatenate([[0], np.cumsum(kept)])), **_filled_cache(gen, len(refs), heads, page)}
    dtype, v = _TYPES[case["dtype"]], case["vocab"]
    nd = _draft_lengths(case)
    rows, n = int(nd.sum()) + len(nd), int(nd.sum())
    of = torch.tensor(np.arange(n) + np.repeat(np.arange(len(nd)), nd), device="cuda")     # target row of each draft
    logits = torch.randn((rows, v), generator=gen, device="cuda") * 4.5
    s = {"case": case, "cu": _ints(np.concatenate([[0], np.cumsum(nd)])), "most": int(nd.max())}
    q = torch.softmax(logits[of] + 0.6 * torch.randn((n, v), generator=gen, device="cuda"), -1)
    drafts = torch.multinomial(q, 1, generator=gen).flatten() if n else torch.zeros(0, device="cuda")
    p = torch.softmax(logits, -1)
    # every other row is cut to its likely tokens, as a sampler does
    p[::2] = torch.where(p[::2] < 0.01 * p[::2].amax(-1, keepdim=True), 0.0, p[::2])
    p /= p.sum(-1, keepdim=True)
    if case["lookup"]:                             # mostly what the target would say
        likely = torch.multinomial(p[of].sqrt(), 1, generator=gen).flatten()
        drafts = torch.where(torch.rand(n, generator=gen, device="cuda") < 0.8, p[of].argmax(-1), likely)
    s.update(p=p.to(dtype), q=None if case["lookup"] else q.to(dtype), drafts=drafts.to(torch.int32),
             u=torch.rand(n, generator=gen, device="cuda"), us=torch.rand(len(nd), generator=gen, device="cuda"))
    if not case["ragged"]:
        s["drafts"] = s["drafts"].view(len(nd), -1)
        s["u"] = s["u"].view(len(nd), -1)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------
def _fp8(x):
    return x.view(torch.float8_e4m3fn)


def _ceil(n, page):
    return torch.div(n + page - 1, page, rounding_mode="floor")


def _plain_release(s, to):
    page, col = s["case"]["page"], torch.arange(s["table"].shape[1], device="cuda")
    to = torch.minimum(torch.where(to < 0, s["lens"], to), s["lens"])
    drop = (col >= _ceil(to, page).unsqueeze(1)) & (col < _ceil(s["lens"], page).unsqueeze(1))
    s["refs"].index_add_(0, s["table"].clamp(min=0).view(-1).long(), -drop.view(-1).int())
    s["table"].masked_fill_(drop, -1)
    s["lens"].copy_(to)


def _plain_fork(s):
    child, origin = s["children"].long(), s["origin"].long()
    line = s["table"][origin]
    s["refs"].index_add_(0, line.clamp(min=0).view(-1).long(), (line >= 0).view(-1).int())
    s["table"][child] = line
    s["lens"][child] = s["lens"][origin]


def _plain_reserve(s, to):
    table, lens, refs, page = s["table"], s["lens"], s["refs"], s["case"]["page"]
    rows, width = table.shape
    row, grow = torch.arange(rows, device="cuda"), to > lens
    have, want = _ceil(lens, page).long(), _ceil(to, page).long()
    last = table.gather(1, (have - 1).clamp(min=0).unsqueeze(1)).squeeze(1).clamp(min=0).long()
    shared = grow & (lens % page != 0) & (refs[last] > 1)
    left = refs.index_add(0, last, -shared.int())
    empty = shared & (left[last] == 0)
    highest = torch.full_like(refs, -1).scatter_reduce_(0, last, torch.where(empty, row, -1).int(), "amax")
    moves = shared & ~(empty & (highest[last] == row))
    fresh = torch.where(grow, want - have, 0) + moves
    upto, rank = fresh.cumsum(0), (refs == 0).long().cumsum(0)
    fits = upto <= rank[-1]
    grow, moves, fresh = grow & fits, moves & fits, torch.where(fits, fresh, 0)
    # the free page of rank r goes to the row within whose share of the ranks r lies
    upto = fresh.cumsum(0)
    take = (refs == 0) & (rank <= upto[-1])
    to_row = torch.searchsorted(upto, rank - 1, right=True).clamp(max=rows - 1)
    first = have - moves.long()
    col = first[to_row] + (rank - 1) - (upto - fresh)[to_row]
    flat = torch.cat([table.view(-1), table.new_zeros(1)])
    flat[torch.where(take, to_row * width + col, rows * width)] = torch.arange(refs.shape[0], device="cuda", dtype=torch.int32)
    refs.index_add_(0, last, -moves.int())
    refs.add_(take.int())
    table.copy_(flat[:-1].view(rows, width))
    copies = {"src": torch.where(moves, last, -1).int(),
              "dst": torch.where(moves, table.gather(1, first.clamp(0, width - 1).unsqueeze(1)).squeeze(1), -1).int(),
              "tokens": torch.where(moves, lens % page, 0).int()}
    lens.copy_(torch.where(grow, to, lens))
    return copies


def _state(s, copies):
    return {"table": s["table"], "lens": s["lens"], "refs": s["refs"], **copies}


def _plain_step(s):
    _plain_release(s, s["low"])
    return _state(s, _plain_reserve(s, s["high"]))


def _plain_branch(s):
    _plain_release(s, s["low"])
    _plain_fork(s)
    return _state(s, _plain_reserve(s, s["high"]))


def _cache(s):
    return {"k": _fp8(s["k"]), "v": _fp8(s["v"]), "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _plain_copy(s):
    there = s["src"] >= 0
    src, dst = s["src"][there].long(), s["dst"][there].long()
    for n in ("k", "v", "k_scale", "v_scale"):
        new = s[n][src]
        if s["tokens"] is not None:
            kept = torch.arange(s["case"]["page"], device="cuda") < s["tokens"][there].unsqueeze(1)
            kept = kept.view(len(src), 1, -1, *([1] * (new.dim() - 3)))
            new = torch.where(kept, new, s[n][dst])
        s[n][dst] = new
    return _cache(s)


def _plain_compact(s):
    page, cu = s["case"]["page"], s["cu"].long()
    keep = s["keep"].long()
    n = keep.shape[-1]
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    to = i - cu[b]
    head = torch.arange(s["case"]["heads"], device="cuda").unsqueeze(1)
    at = (s["table"][b, keep // page].long(), head, keep % page)
    into = (s["table"][b, to // page].long(), head, to % page)
    for x in ("k", "v", "k_scale", "v_scale"):
        s[x][into] = s[x][at]
    return _cache(s)


def _plain_verify(s):
    cu, drafts, u = s["cu"].long(), s["drafts"].reshape(-1).long(), s["u"].reshape(-1)
    batch, n = cu.shape[0] - 1, drafts.shape[0]
    i = torch.arange(n, device="cuda")
    b = torch.searchsorted(cu, i, right=True) - 1
    count = cu[1:] - cu[:-1]
    p = s["p"][i + b, drafts].double()
    q = torch.ones_like(p) if s["q"] is None else s["q"][i, drafts].double()
    stays = u.double() * q < p
    accepted = count.scatter_reduce(0, b, torch.where(stays, n, i - cu[b]), "amin")
    rejected = accepted < count
    w = s["p"][cu[:-1] + torch.arange(batch, device="cuda") + accepted].double()
    if n:
        at = (cu[:-1] + accepted).clamp(max=n - 1)
        if s["q"] is None:
            rest = w.scatter(1, drafts[at].unsqueeze(1), 0.0)
        else:
            rest = (w - s["q"][at].double()).clamp_(min=0.0)
        usable = rejected & (rest.sum(-1) > 0)
        w = torch.where(usable.unsqueeze(1), rest, w)
    c = w.cumsum(-1)
    token = (c <= (s["us"].double() * c[:, -1]).unsqueeze(1)).sum(-1)
    last = torch.where(w > 0, torch.arange(w.shape[1], device="cuda"), -1).amax(-1)
    token = torch.minimum(token, last)
    r = torch.arange(n + batch, device="cuda")
    start = cu + torch.arange(batch + 1, device="cuda")
    rb = torch.searchsorted(start, r, right=True) - 1
    place = r - start[rb]
    draft = drafts[(r - rb).clamp(max=max(0, n - 1))] if n else torch.zeros_like(r)
    out = torch.where(place < accepted[rb], draft, torch.where(place == accepted[rb], token[rb], -1))
    return {"tokens": out.int(), "accepted": accepted.int()}


def run(state):
    s, op = state, state["case"]["op"]
    if own:
        import fp8_bit_attention_gb300 as ovc

        if "handles" not in s:      # what a program keeps beside the memory itself
            s["handles"] = (ovc.KVPages(s["table"], s["lens"], s["refs"], s["case"]["page"]) if "table" in s else None,
                            ovc.KVCache(s["k"], s["v"], s["k_scale"], s["v_scale"]) if "k" in s else None)
        pages, cache = s["handles"]
        if op in ("step", "branch"):
            ovc.kv_pages_release(pages, s["low"])
            if op == "branch":
                ovc.kv_pages_fork(pages, s["origin"], s["children"])
            src, dst, tokens = ovc.kv_pages_reserve(pages, s["high"])
            return _state(s, {"src": src, "dst": dst, "tokens": tokens})
        if op == "copy":
            ovc.kv_cache_copy(cache, s["src"], s["dst"], s["tokens"])
            return _cache(s)
        if op == "compact":
            ovc.kv_cache_compact(cache, pages, s["keep"], s["cu"])
            return _cache(s)
        tokens, accepted = ovc.verify_drafts(s["p"], s["drafts"], s["u"], s["us"], draft_probs=s["q"],
                                             cu_drafts=s["cu"] if s["case"]["ragged"] else None)
        return {"tokens": tokens, "accepted": accepted}
    return {"step": _plain_step, "branch": _plain_branch, "copy": _plain_copy, "compact": _plain_compact,
            "verify": _plain_verify}[op](s)


# ---------------------------------------------------------------------------
# The definition, row by row
# ---------------------------------------------------------------------------
def _e4m3_grid():
    """The value of each E4M3 byte (the two NaN bytes as NaN)."""
    b = np.arange(256)
    sign, exp, man = np.where(b & 128, -1.0, 1.0), (b >> 3) & 15, b & 7
    val = sign * np.where(exp == 0, man * 2.0 ** -9, (8 + man) * 2.0 ** (exp - 10.0))
    val[[127, 255]] = np.nan
    return val


def _exact_pages(s):
    page = s["case"]["page"]
    table, lens, refs = (s[n].cpu().numpy().astype(np.int64) for n in ("table", "lens", "refs"))
    low, high = s["low"].cpu().numpy(), s["high"].cpu().numpy()
    rows = range(len(lens))
    for b in rows:
        for c in range(_up(low[b], page), _up(lens[b], page)):
            refs[table[b, c]] -= 1
            table[b, c] = -1
        lens[b] = min(lens[b], low[b])
    if "origin" in s:
        for a, b in zip(s["origin"].tolist(), s["children"].tolist()):
            table[b], lens[b] = table[a], lens[a]
            np.add.at(refs, table[a][table[a] >= 0], 1)
    holders = {}
    for b in rows:
        if high[b] > lens[b] and lens[b] % page and refs[table[b, lens[b] // page]] > 1:
            holders.setdefault(int(table[b, lens[b] // page]), []).append(b)
    mover = {b: p for p, bs in holders.items() for b in (bs[:-1] if len(bs) == refs[p] else bs)}
    free = np.nonzero(refs == 0)[0].tolist()[::-1]
    copies = {"src": np.full(len(lens), -1), "dst": np.full(len(lens), -1), "tokens": np.zeros(len(lens), np.int64)}
    for b in rows:
        cols = list(range(_up(lens[b], page), _up(high[b], page)))
        if b in mover:
            cols.insert(0, int(lens[b] // page))
        if len(cols) > len(free):
            break
        if b in mover:
            refs[mover[b]] -= 1
            copies["src"][b], copies["dst"][b], copies["tokens"][b] = mover[b], free[-1], lens[b] % page
        for c in cols:
            table[b, c] = free.pop()
            refs[table[b, c]] = 1
        lens[b] = max(lens[b], high[b])
    return {n: _ints(x) for n, x in {"table": table, "lens": lens, "refs": refs, **copies}.items()}


def _exact_cache(s):
    """Pages or kept tokens moved one by one, values in 64 bits."""
    grid = torch.tensor(_e4m3_grid(), device="cuda")
    old = {n: (grid[s[n].int()] if s[n].dim() == 4 else s[n]) for n in ("k", "v", "k_scale", "v_scale")}
    new = {n: x.clone() for n, x in old.items()}
    page = s["case"]["page"]
    if s["case"]["op"] == "copy":
        tokens = [page] * len(s["src"]) if s["tokens"] is None else s["tokens"].tolist()
        for a, b, t in zip(s["src"].tolist(), s["dst"].tolist(), tokens):
            for n in old if a >= 0 else ():
                new[n][b, :, :t] = old[n][a, :, :t]
        return new
    cu = s["cu"].tolist()
    for b in range(len(cu) - 1):
        pages = s["table"][b].long()
        for h in range(s["case"]["heads"]):
            at = (s["keep"][h] if s["case"]["per_head"] else s["keep"])[cu[b]:cu[b + 1]].long()
            to = torch.arange(len(at), device="cuda")
            for n in old:
                new[n][pages[to // page], h, to % page] = old[n][pages[at // page], h, at % page]
    return new


def _exact_verify(s):
    cu, u, us = s["cu"].tolist(), s["u"].flatten().double().tolist(), s["us"].double().tolist()
    drafts = s["drafts"].flatten().tolist()
    tokens, accepted = [], []
    for b in range(len(cu) - 1):
        a, n = cu[b], cu[b + 1] - cu[b]
        at = 0
        while at < n:
            x = drafts[a + at]
            if not u[a + at] * (1.0 if s["q"] is None else float(s["q"][a + at, x])) < float(s["p"][a + b + at, x]):
                break
            at += 1
        p = s["p"][a + b + at].cpu().to(torch.float64).numpy()
        w = p
        if at < n:
            q = np.zeros_like(p)
            if s["q"] is None:
                q[drafts[a + at]] = np.inf
            else:
                q = s["q"][a + at].cpu().to(torch.float64).numpy()
            w = np.where(p > q, p - q, 0.0)
            w = w if w.any() else p
        upto = np.cumsum(w.astype(np.longdouble))
        over = np.nonzero((upto > np.longdouble(us[b]) * upto[-1]) & (w > 0))[0]
        held = np.nonzero(w > 0)[0]
        token = int(over[0]) if len(over) else int(held[-1]) if len(held) else -1
        tokens += drafts[a:a + at] + [token] + [-1] * (n - at)
        accepted.append(at)
    return {"tokens": _ints(tokens), "accepted": _ints(accepted)}


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_pages, "branch": _exact_pages, "copy": _exact_cache, "compact": _exact_cache, "verify": _exact_verify}[case["op"]](s)
