"""GPU tests of the verification of drafted tokens, against its definition in 64
bits (pages_util), and of a loop of drafts over a paged cache."""
import numpy as np
import pytest
import torch

import fp8_bit_attention_gb300 as ovc

from pages_util import check_verified, verify

pytestmark = pytest.mark.gpu

BAD_INDEX = 7
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module", autouse=True)
def _build():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    ovc.device_status()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _f32(x):
    return torch.tensor(np.asarray(x), dtype=torch.float32, device="cuda")


def _probs(g, rows, vocab, dtype, sharp, cut):
    p = torch.softmax(sharp * torch.randn((rows, vocab), generator=g, device="cuda"), -1)
    if cut:
        p = torch.where(p < 0.05 * p.amax(-1, keepdim=True), 0.0, p)
    return (p / p.sum(-1, keepdim=True)).to(dtype)


class Case:
    def __init__(self, counts, vocab, dtype, *, lookup=False, sharp=2.0, cut=True, seed=0, near=True):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.cu = np.r_[0, np.cumsum(counts)]
        n, batch = int(self.cu[-1]), len(counts)
        of = torch.tensor(np.arange(n) + np.repeat(np.arange(batch), counts), device="cuda")
        self.p = _probs(g, n + batch, vocab, dtype, sharp, cut)
        q = _probs(g, n, vocab, dtype, sharp, False)
        if near and n:
            q = (0.7 * self.p[of].float() + 0.3 * q.float()).to(dtype)
        self.drafts = torch.multinomial(q.float(), 1, generator=g).flatten().int() if n else _i32([])
        self.q = None if lookup else q
        self.u = torch.rand(n, generator=g, device="cuda")
        self.us = torch.rand(batch, generator=g, device="cuda")

    def run(self, **kw):
        kw = {"draft_probs": self.q, **kw}
        if "cu_drafts" not in kw:
            kw["cu_drafts"] = _i32(self.cu)
        return ovc.verify_drafts(self.p, self.drafts, self.u, self.us, **kw)

    def check(self, tokens, accepted):
        host = [None if x is None else x.double().cpu().numpy() for x in (self.p, self.q)]
        drafts, us = self.drafts.cpu().numpy().reshape(-1), self.us.double().cpu().numpy()
        want = verify(*host, drafts, self.cu, self.u.double().cpu().numpy().reshape(-1), us)
        check_verified(tokens.cpu().numpy(), accepted.cpu().numpy(), drafts, self.cu, us, want)
        return want


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("counts, vocab", [([1], 1), ([0], 7), ([3, 0, 5], 31), ([4] * 5, 32), ([2, 1, 7, 0], 1000), ([8] * 20, 1024),
                                           ([600, 3], 101), ([1, 5], 1025), ([4], 32000), ([3, 4, 0, 1] * 40, 5003),
                                           ([2] * 3, 131072), ([1], 262147), ([2, 0], 1200007)], ids=str)
@pytest.mark.parametrize("lookup", [False, True])
def test_verified_drafts(dtype, counts, vocab, lookup):
    for seed, sharp in ((1, 2.0), (2, 0.2)):
        c = Case(counts, vocab, dtype, lookup=lookup, sharp=sharp, cut=seed == 1, seed=seed + vocab)
        c.check(*c.run())
    assert ovc.device_status() == 0


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("offset, extra", [(0, 0), (0, 8), (8, 8), (1, 0), (3, 5), (0, 1)])
def test_rows_of_any_alignment(dtype, offset, extra):
    """Views into wider rows, at every place of the 16 bytes of a load."""
    c = Case([3, 2, 4, 0], 4099, dtype, seed=5)
    whole = c.run()
    for name in ("p", "q"):
        x = getattr(c, name)
        wide = torch.full((x.shape[0], x.shape[1] + extra + offset), 7.0, dtype=dtype, device="cuda")
        wide[:, offset:offset + x.shape[1]] = x
        setattr(c, name, wide[:, offset:offset + x.shape[1]])
        got = c.run()
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])
    c.check(*whole)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [3, 70, 2047, 2049, 9001])
def test_rows_of_different_alignment(dtype, vocab):
    """The draft's rows at every place relative to the target's."""
    c = Case([2, 1], vocab, dtype, seed=vocab)
    whole = c.run()
    c.check(*whole)
    q = c.q
    for offset in range(9):
        wide = torch.full((3, vocab + 16), 7.0, dtype=dtype, device="cuda")[:, offset:offset + vocab]
        wide.copy_(q)
        c.q = wide
        got = c.run()
        assert torch.equal(got[0], whole[0]) and torch.equal(got[1], whole[1])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("batch", [33, 36, 42, 50, 60, 80, 100, 140])
@pytest.mark.parametrize("lookup", [False, True])
def test_clusters_of_every_size(dtype, batch, lookup):
    """8, 7, 6, 5, 4, 3, 2 CTAs and one a sequence (on 152 SMs), each with drafts, in
    any number, or none."""
    counts = [1 + b % 2 if b % 5 else 0 for b in range(batch)]
    c = Case(counts, 33001 + batch, dtype, lookup=lookup, sharp=0.5, cut=batch % 4 == 0, seed=batch)
    c.check(*c.run())
    assert ovc.device_status() == 0


@pytest.mark.parametrize("drafted", [False, True])
def test_large_vocabularies_of_many_sequences(drafted):
    """Tiles of several lines: one row of the target (and of the draft) for all, no two random numbers alike."""
    vocab, batch = 2200003, 160
    g = torch.Generator(device="cuda").manual_seed(13)
    p, q = _probs(g, 1, vocab, torch.float32, 1.0, False), _probs(g, 1, vocab, torch.float32, 1.0, False)
    us = torch.rand(batch, generator=g, device="cuda")
    w = p[0].double().cpu().numpy()
    if drafted:
        x = torch.full((batch, 1), int((p[0] / q[0]).argmin()), dtype=torch.int32, device="cuda")
        u = torch.full((batch, 1), 0.999, device="cuda")
        tokens, accepted = ovc.verify_drafts(p.expand(2 * batch, -1), x, u, us, draft_probs=q.expand(batch, -1))
        w = np.maximum(w - q[0].double().cpu().numpy(), 0.0)
        cu = np.arange(batch + 1)
    else:
        cu = np.zeros(batch + 1, int)
        tokens, accepted = ovc.verify_drafts(p.expand(batch, -1), _i32([]), _f32([]), us, cu_drafts=_i32(cu))
    check_verified(tokens.cpu().numpy(), accepted.cpu().numpy(), [], cu, us.double().cpu().numpy(), [(0, w)] * batch)


def test_equal_numbers_of_drafts_need_no_starts():
    c = Case([5] * 7, 777, torch.float32, seed=3)
    a = c.run()
    b = ovc.verify_drafts(c.p, c.drafts.view(7, 5), c.u.view(7, 5), c.us, draft_probs=c.q)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_padded_drafts_end_a_sequence():
    """A negative draft: what comes after it is not looked at, and the next token is
    drawn from its row of the target."""
    c = Case([4] * 30, 500, torch.bfloat16, seed=4)
    d = c.drafts.view(30, 4)
    for b in range(30):
        d[b, b % 5:] = -1
    c.q.view(30, 4, -1)[d < 0] = float("nan")
    got = c.run()
    want = c.check(*got)
    assert {i for i, _ in want} >= {0, 1, 2} and ovc.device_status() == 0


def test_every_token_of_a_row():
    """Random numbers in each token's share give that token."""
    vocab = 2000
    w = np.random.default_rng(1).integers(0, 4, vocab) / 4096.0       # sums exact in any order
    upto = np.cumsum(w)
    some = np.nonzero(w)[0]
    mid = (upto[some] - w[some] / 2) / upto[-1]
    p = _f32(np.broadcast_to(w, (len(some), vocab)))
    none = torch.zeros((len(some), 0), device="cuda")
    tokens, accepted = ovc.verify_drafts(p, none.int(), none, _f32(mid))
    assert np.array_equal(tokens.cpu().numpy(), some) and not accepted.any()


@pytest.mark.parametrize("lookup", [False, True])
def test_random_numbers_at_their_ends(lookup):
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, float("nan")):
        c = Case([2] * 9, 3001, torch.float32, lookup=lookup, seed=6)
        c.us.fill_(u)
        tokens, accepted = c.run()
        host = [None if x is None else x.double().cpu().numpy() for x in (c.p, c.q)]
        want = verify(*host, c.drafts.cpu().numpy(), c.cu, c.u.double().cpu().numpy(), None)
        for b, (i, w) in enumerate(want):
            some = np.nonzero(w)[0]
            t = int(tokens[3 * b + i])
            assert accepted[b] == i and (t == some[0] if u == 0 else t == some[-1] if u >= 1 else t in some)


def test_borders_of_acceptance():
    """u * q < p is decided without rounding."""
    g = np.random.default_rng(7)
    q = g.random(4000).astype(np.float32) * 0.5 + 0.25
    u = g.random(4000).astype(np.float32)
    near = (u.astype(np.float64) * q).astype(np.float32)               # nearest FP32 value of the product
    for p in (near, np.nextafter(near, np.float32(1)), np.nextafter(near, np.float32(0))):
        probs = np.zeros((8000, 3), np.float32)
        probs[0::2, 1] = p
        probs[:, 0] = 0.5
        qs = np.zeros((4000, 3), np.float32)
        qs[:, 1] = q
        one = torch.ones((4000, 1), device="cuda")
        _, accepted = ovc.verify_drafts(_f32(probs), one.int(), _f32(u)[:, None], torch.zeros(4000, device="cuda"), draft_probs=_f32(qs))
        assert np.array_equal(accepted.cpu().numpy() == 1, u.astype(np.float64) * q < p)


def test_rejected_where_nothing_is_left_of_the_difference():
    """p = q but for what was drafted, which p does not have: drawn from p itself."""
    p = _f32(np.random.default_rng(8).random((2, 900)))
    q = p[:1].clone()
    p[0, 5], q[0, 5] = 0.0, 0.3
    tokens, accepted = ovc.verify_drafts(p, _i32([[5]]), _f32([[0.5]]), _f32([0.4]), draft_probs=q)
    w = p[0].double().cpu().numpy()
    check_verified(tokens.cpu().numpy(), accepted.cpu().numpy(), [5], [0, 1], [float(np.float32(0.4))], [(0, w)])
    tokens, _ = ovc.verify_drafts(torch.eye(9, device="cuda")[[4, 4]], _i32([[3]]), _f32([[0.5]]), _f32([0.4]))
    assert tokens.tolist() == [4, -1]


@pytest.mark.parametrize("vocab", [5, 3000])
def test_rows_that_leave_nothing(vocab):
    p = torch.zeros((3, vocab), device="cuda")
    p[1] = float("nan")
    q = torch.full((1, vocab), 0.1, device="cuda")
    for draft_probs in (q, None):
        tokens, accepted = ovc.verify_drafts(p, _i32([2]), _f32([0.0]), _f32([0.5, 0.5]), draft_probs=draft_probs, cu_drafts=_i32([0, 1, 1]))
        assert tokens.tolist() == [-1, -1, -1] and accepted.tolist() == [0, 0]
    p[1, 3], p[2, 1:4] = 0.2, float("nan")          # a NaN leaves its token without weight
    p[2, 4] = 1e-30
    tokens, _ = ovc.verify_drafts(p[1:], _i32([]), _f32([]), _f32([0.9, 0.9]), cu_drafts=_i32([0, 0, 0]))
    assert tokens.tolist() == [3, 4]
    p = torch.full((2, vocab), 0.25, device="cuda")
    q[0], q[0, 1], q[0, 2] = float("nan"), 0.125, 0.5
    for x, u in ((2, 0.9), (0, 0.0)):               # rejected by its probabilities, or by a NaN among them
        tokens, accepted = ovc.verify_drafts(p, _i32([[x]]), _f32([[u]]), _f32([0.99]), draft_probs=q)
        assert tokens.tolist() == [1, -1] and accepted.tolist() == [0]
    assert ovc.device_status() == 0


def test_very_small_and_large_probabilities():
    """Rows need not sum to 1: subnormal and large ones, and both in one row."""
    g = np.random.default_rng(9)
    w = np.stack([g.random(3000) * s for s in (1e-42, 1e30, 1.0)]).astype(np.float32)
    w[2] *= (2.0 ** g.integers(-140, 100, 3000)).astype(np.float32)
    us = [0.3, 0.7, 0.5]
    tokens, accepted = ovc.verify_drafts(_f32(w), _i32([]), _f32([]), _f32(us), cu_drafts=_i32([0] * 4))
    check_verified(tokens.cpu().numpy(), accepted.cpu().numpy(), [], [0] * 4, np.float32(us).astype(float), [(0, r.astype(float)) for r in w])


def test_bad_drafts_and_starts_are_reported():
    c = Case([2, 2], 50, torch.float32, seed=10)
    c.drafts[2] = 50
    tokens, accepted = c.run()
    assert ovc.device_status() == BAD_INDEX
    c.check(tokens, accepted)                           # as if it had ended there
    c.drafts[2] = 0
    for cu in ([0, 3, 2], [-1, 2, 4], [0, 2, 5]):
        tokens, accepted = c.run(cu_drafts=_i32(cu))
        assert ovc.device_status() == BAD_INDEX
        bad = 0 if cu[0] < 0 else 1
        assert accepted[bad] == 0 and ovc.device_status() == 0


@pytest.mark.parametrize("cu", [[0, 3, 2], [-1, 2, 4], [0, 2, 5], [1, 2, 4], [2, 2, 2], [0, 2, 3], [0, 0, 0], [5, 2, 4], [0, 4, 3], [3, 2, 1],
                                [0, -1, -1, 1, 3, 9, 4, 4], [2, 2, 7, 2, 3, -5], [9, 9, 9, 9], [-1, 0, 0, 4], [3, 4, 5], [4], [1, 3],
                                [-1] * 700 + [2, 3] + [9] * 700, [0] * 3 + [-7] * 1400 + [3, 4, 4], [-1] * 600], ids=lambda x: str(x[:9]))
@pytest.mark.parametrize("vocab", [50, 40000])
def test_rows_of_no_sequence_hold_no_token(cu, vocab):
    """Starts that do not begin at 0, do not reach N, or are none."""
    n, batch = 4, len(cu) - 1
    c = Case([n], vocab, torch.float32, seed=14)
    p = c.p.repeat(-(-(n + batch) // (n + 1)), 1)[:n + batch].contiguous()
    us = torch.rand(batch, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    starts = _i32(cu)
    ovc.device_status()
    held = [torch.full((n + batch,), 12345, dtype=torch.int32, device="cuda") for _ in range(4)]
    del held                                            # what a new tensor is likely to hold
    tokens, accepted = ovc.verify_drafts(p, c.drafts, c.u, us, draft_probs=c.q, cu_drafts=starts)
    good = [b for b in range(batch) if 0 <= cu[b] <= cu[b + 1] <= n]
    assert ovc.device_status() == (0 if len(good) == batch else BAD_INDEX)
    rows = sorted(r for b in good for r in range(cu[b] + b, cu[b + 1] + b + 1))
    assert len(rows) == len(set(rows))
    got, kept = tokens.cpu().numpy(), accepted.cpu().numpy()
    assert (np.delete(got, rows) == -1).all() and not np.delete(kept, good).any()
    host = [x.double().cpu().numpy() for x in (p, c.q, c.u, us)]
    drafts = c.drafts.cpu().numpy()
    for b in good[:8] + good[-8:]:
        want = verify(host[0][b:], host[1], drafts, cu[b:b + 2], host[2], None)
        check_verified(got[b:], kept[b:], drafts, cu[b:b + 2], host[3][b:], want)


def test_long_strides():
    """Rows beyond 32-bit offsets."""
    wide = torch.empty((3, 1 << 31), dtype=torch.bfloat16, device="cuda")[:, :1000]
    c = Case([1, 0], 1000, torch.bfloat16, seed=11)
    wide.copy_(c.p)
    a = c.run()
    c.p = wide
    assert all(torch.equal(x, y) for x, y in zip(a, c.run()))


def test_captured_calls_follow_new_inputs_and_streams():
    cases = [Case([3, 0, 5, 2], 9000, torch.float32, seed=s) for s in range(3)]
    c = Case([3, 0, 5, 2], 9000, torch.float32, seed=20)
    cu = _i32(c.cu)
    c.run(cu_drafts=cu)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = c.run(cu_drafts=cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for x in cases:
        for name in ("p", "q", "drafts", "u", "us"):
            getattr(c, name).copy_(getattr(x, name))
        graph.replay()
        eager = x.run(stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager))
        x.check(*eager)


def test_empty_batch_and_refusals():
    tokens, accepted = ovc.verify_drafts(torch.zeros((0, 9), device="cuda"), _i32([]), _f32([]), _f32([]), cu_drafts=_i32([0]))
    assert tokens.shape == accepted.shape == (0,)
    c = Case([2, 2], 50, torch.float32, seed=12)
    with pytest.raises(TypeError):
        ovc.verify_drafts(c.p.double(), c.drafts, c.u, c.us, cu_drafts=_i32(c.cu))
    with pytest.raises(ValueError, match="draft_probs"):
        c.run(draft_probs=c.q.half())
    with pytest.raises(ValueError, match="draft_probs"):
        c.run(draft_probs=c.q[:3])
    with pytest.raises(ValueError, match="target_probs"):
        ovc.verify_drafts(c.p[:5], c.drafts, c.u, c.us, cu_drafts=_i32(c.cu))
    with pytest.raises(ValueError, match="column stride"):
        ovc.verify_drafts(c.p.t().contiguous().t(), c.drafts, c.u, c.us, cu_drafts=_i32(c.cu))
    with pytest.raises(ValueError, match="accept_u"):
        ovc.verify_drafts(c.p, c.drafts, c.u[:3], c.us, cu_drafts=_i32(c.cu))
    with pytest.raises(ValueError, match="sample_u"):
        ovc.verify_drafts(c.p, c.drafts, c.u, c.us[:1], cu_drafts=_i32(c.cu))
    with pytest.raises(ValueError, match="cu_drafts"):
        ovc.verify_drafts(c.p, c.drafts, c.u, c.us)


def test_a_loop_of_drafts_over_shared_pages():
    """Two prompts, each continued by a second sequence that shares its pages.
    Every step drafts tokens, writes and attends them, verifies, and gives back what
    was not accepted; sometimes a sequence drops old tokens.  The attention of each
    step equals that of a cache of its own which holds the same tokens."""
    heads, page, vocab, width = 2, 16, 64, 20
    g = torch.Generator(device="cuda").manual_seed(30)
    r = np.random.default_rng(31)
    table_k, table_v = (torch.randn((vocab, heads, 128), generator=g, device="cuda").bfloat16() for _ in range(2))
    head = torch.randn((heads * 128, vocab), generator=g, device="cuda") * 0.2
    pages, cache = ovc.kv_pages(60, 4, width, page), ovc.kv_cache(60, heads, page)
    text = [list(r.integers(0, vocab, n)) for n in (45, 17, 0, 0)]          # the tokens whose keys a sequence holds

    def slots(b, t):
        return pages.page_table[b, t // page] * page + t % page

    def write(b, start, tokens):
        t = torch.arange(start, start + len(tokens), device="cuda")
        x = torch.tensor(np.array(tokens, np.int64), device="cuda")
        ovc.kv_cache_write(cache, table_k[x], table_v[x], slots(b, t).int())

    def grow(lens):
        src, dst, tokens = ovc.kv_pages_reserve(pages, _i32(lens))
        ovc.kv_cache_copy(cache, src, dst, tokens)
        assert pages.kv_lens.tolist() == list(lens)

    grow([45, 17, 0, 0])
    for b in (0, 1):
        write(b, 0, text[b])
    ovc.kv_pages_fork(pages, _i32([0, 1]), _i32([2, 3]))
    text[2:] = [list(text[0]), list(text[1])]
    last = [1, 2, 3, 4]                                                     # committed, not yet in the cache
    accepted_once = moved_once = 0
    for step in range(12):
        n = [int(r.integers(0, 4)) for _ in range(4)]
        drafts = [list(r.integers(0, vocab, k)) for k in n]
        old = [len(t) for t in text]
        grow([o + 1 + k for o, k in zip(old, n)])
        rows = [[x] + d for x, d in zip(last, drafts)]
        for b in range(4):
            write(b, old[b], rows[b])
            text[b] += rows[b]
        cu_q = _i32(np.r_[0, np.cumsum([len(x) for x in rows])])
        q = torch.randn((sum(n) + 4, heads, 128), generator=g, device="cuda").bfloat16()
        o = ovc.paged_attention(q, cache, pages.page_table, pages.kv_lens, cu_q=cu_q, max_q=4)
        own = ovc.kv_cache(4 * width, heads, page)                          # the same tokens, nothing shared
        own_table = torch.arange(4 * width, dtype=torch.int32, device="cuda").view(4, width)
        for b in range(4):
            t = torch.arange(len(text[b]), device="cuda")
            x = torch.tensor(np.array(text[b], np.int64), device="cuda")
            ovc.kv_cache_write(own, table_k[x], table_v[x], (own_table[b, t // page] * page + t % page).int())
        assert torch.equal(o, ovc.paged_attention(q, own, own_table, pages.kv_lens, cu_q=cu_q, max_q=4))
        p = torch.softmax(o.float().flatten(1) @ head, -1)
        cu = np.r_[0, np.cumsum(n)]
        u, us = torch.rand(sum(n), generator=g, device="cuda") * 0.05, torch.rand(4, generator=g, device="cuda")
        flat = np.array([x for d in drafts for x in d], np.int64)
        tokens, accepted = ovc.verify_drafts(p, _i32(flat), u, us, cu_drafts=_i32(cu))
        check_verified(tokens.cpu().numpy(), accepted.cpu().numpy(), flat, cu, us.double().cpu().numpy(),
                       verify(p.double().cpu().numpy(), None, flat, cu, u.double().cpu().numpy(), None))
        got, accepted = tokens.tolist(), accepted.tolist()
        accepted_once += sum(accepted)
        for b in range(4):
            text[b] = text[b][:old[b] + 1 + accepted[b]]
            last[b] = got[cu[b] + b + accepted[b]]
        ovc.kv_pages_release(pages, pages.kv_lens - _i32(n) + _i32(accepted))
        assert pages.kv_lens.tolist() == [len(t) for t in text]
        if step % 3 == 2:                                                   # every sequence drops a token behind what is shared
            keep = [[i for i in range(len(t)) if i != max(len(t) - 3, 48)] for t in text]
            ovc.kv_cache_compact(cache, pages, _i32(np.concatenate(keep)), _i32(np.r_[0, np.cumsum([len(k) for k in keep])]))
            text = [[t[i] for i in k] for t, k in zip(text, keep)]
            ovc.kv_pages_release(pages, _i32([len(t) for t in text]))
            moved_once += 1
    assert accepted_once and moved_once and ovc.device_status() == 0
    ovc.kv_pages_release(pages, torch.zeros_like(pages.kv_lens))
    assert not pages.refs.any() and (pages.page_table == -1).all()
