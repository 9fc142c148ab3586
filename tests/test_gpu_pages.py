"""GPU tests of the pages that sequences hold and of moves inside a paged cache,
against their definitions (pages_util)."""
import numpy as np
import pytest
import torch

import fp8_bit_attention_gb300 as ovc

from pages_util import Pages, compacted, copied

pytestmark = pytest.mark.gpu

BAD_INDEX = 7


@pytest.fixture(scope="module", autouse=True)
def _build():
    import __graft_entry__
    __graft_entry__.build()
    assert torch.cuda.is_available()
    ovc.device_status()


def _i32(x):
    return torch.tensor(np.ascontiguousarray(x), dtype=torch.int32, device="cuda")


def _state(table, lens, refs, page):
    return ovc.KVPages(_i32(table), _i32(lens), _i32(refs), page)


def _reserve(p, lens):
    return [x.cpu().numpy() for x in ovc.kv_pages_reserve(p, _i32(lens))]


def _filled(pages, heads, page, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, heads, page)
    return ovc.KVCache(*(torch.randint(0, 256, s, generator=g, device="cuda", dtype=torch.uint8)
                         for s in (shape + (128,), shape + (128,), shape, shape)))


def _arrays(c):
    return [x.cpu() for x in (c.k, c.v, c.k_scale, c.v_scale)]


def _holds(c, want):
    return all(torch.equal(x, y) for x, y in zip(_arrays(c), want))


# ------------------------------------------------------------------ the pages
@pytest.mark.parametrize("rows, width, pages, page", [(1, 1, 1, 16), (1, 40, 33, 16), (3, 5, 9, 48), (40, 9, 300, 64),
                                                      (33, 700, 20000, 16), (1025, 6, 3000, 1024), (64, 3000, 70001, 16),
                                                      (8192, 4, 20000, 32), (5, 200000, 300007, 16)])
def test_steps_follow_the_definition(rows, width, pages, page):
    """Random rows grow, shrink and are forked; the pool is short at times."""
    g = np.random.default_rng(rows * 7 + pages)
    p = ovc.kv_pages(pages, rows, width, page)
    want = Pages.of(p)
    for step in range(9):
        most = min(width * page, 2 * page * pages // rows + 40)
        lens = np.where(g.random(rows) < 0.3, -1, want.lens + g.integers(-5, most, rows)).clip(-1, width * page)
        for x, y in zip(_reserve(p, lens), want.reserve(lens)):
            assert np.array_equal(x, y)
        assert want.same_as(p) and want.sound()
        empty, full = np.nonzero(want.lens == 0)[0], np.nonzero(want.lens)[0]
        if len(empty) and len(full):
            parents, children = g.choice(full, len(empty)), g.permutation(empty)
            parents[::5] = children[::5] = -1
            ovc.kv_pages_fork(p, _i32(parents), _i32(children))
            want.fork(parents, children)
            assert want.same_as(p) and want.sound()
            lens = want.lens + g.integers(0, 20, rows)          # forked rows grow, and page by page all holders of one
            lens = lens.clip(0, width * page)
            for x, y in zip(_reserve(p, lens), want.reserve(lens)):
                assert np.array_equal(x, y)
            assert want.same_as(p) and want.sound()
        lens = np.where(g.random(rows) < 0.5, want.lens - g.integers(0, 3 * page, rows), want.lens * (g.random(rows) < 0.5)).clip(-1)
        ovc.kv_pages_release(p, _i32(lens))
        want.release(lens)
        assert want.same_as(p) and want.sound()
    assert ovc.device_status() == 0


@pytest.mark.parametrize("grow, copies", [([1, 1, 1], [1, 1, 0]), ([1, 0, 1], [1, 0, 1]), ([0, 0, 1], [0, 0, 1]), ([1, 1, 0], [1, 1, 0])])
def test_holders_of_a_partly_filled_page(grow, copies):
    p = ovc.kv_pages(20, 3, 4, 16)
    _reserve(p, [20, 0, 0])
    ovc.kv_pages_fork(p, _i32([0, 0]), _i32([1, 2]))
    src, dst, tokens = _reserve(p, 20 + np.array(grow))
    assert list(src) == [1 if c else -1 for c in copies] and list(tokens) == [4 if c else 0 for c in copies]
    assert [d >= 0 for d in dst] == [bool(c) for c in copies] and len(set(dst[dst >= 0])) == sum(copies)
    assert p.refs[0] == 3 and p.refs[1] == 3 - sum(copies) and ovc.device_status() == 0


def test_a_page_that_the_program_keeps_is_replaced():
    """refs raised by hand: no holder writes to that page."""
    p = ovc.kv_pages(9, 1, 4, 16)
    _reserve(p, [10])
    p.refs[0] += 1
    src, dst, tokens = _reserve(p, [11])
    assert (src[0], dst[0], tokens[0]) == (0, 1, 10) and p.refs[:3].tolist() == [1, 1, 0]


def test_full_pages_stay_shared():
    p = ovc.kv_pages(9, 2, 4, 16)
    _reserve(p, [32, 0])
    ovc.kv_pages_fork(p, _i32([0]), _i32([1]))
    src, _, _ = _reserve(p, [33, 40])
    assert (src == -1).all() and p.page_table.tolist() == [[0, 1, 2, -1], [0, 1, 3, -1]]


def test_rows_that_do_not_fit_stay():
    p = ovc.kv_pages(5, 4, 9, 16)
    _reserve(p, [16, 10, 0, 0])
    _reserve(p, [33, 12, 17, 1])             # 2 + 0 + 2 + 1 of 3 free ones
    assert p.kv_lens.tolist() == [33, 12, 0, 0] and (p.refs == 0).sum() == 1
    _reserve(p, [-1, 16, -1, 16])
    assert p.kv_lens.tolist() == [33, 16, 0, 16]


def test_a_row_may_hold_every_page():
    """Tokens up to the end of 31 bits."""
    n = (2 ** 31 - 1024) // 1024
    p = ovc.kv_pages(n, 2, n, 1024)
    _reserve(p, [0, n * 1024 - 5])
    assert torch.equal(p.page_table[1], torch.arange(n, dtype=torch.int32, device="cuda")) and (p.refs == 1).all()
    assert p.kv_lens.tolist() == [0, n * 1024 - 5]
    _reserve(p, [1, -1])
    assert p.kv_lens.tolist() == [0, n * 1024 - 5]
    ovc.kv_pages_release(p, _i32([-1, 1024 * (n - 1)]))
    _reserve(p, [1, n * 1024])
    assert p.kv_lens.tolist() == [1, 1024 * (n - 1)] and p.page_table[0, 0] == n - 1 and ovc.device_status() == 0


def test_wishes_beyond_32_bits():
    """Rows that together want more than 2^32 pages: only the first fits."""
    rows, n = 1026, 1 << 22
    if torch.cuda.mem_get_info()[0] < 4 * rows * n + (8 << 30):
        pytest.skip("needs 25 GB")
    p = ovc.kv_pages(n, rows, n, 16)
    src, dst, tokens = _reserve(p, np.full(rows, 16 * n))
    assert (src == -1).all() and (dst == -1).all() and not tokens.any()
    assert p.kv_lens[0] == 16 * n and not p.kv_lens[1:].any() and (p.refs == 1).all()
    assert torch.equal(p.page_table[0], torch.arange(n, dtype=torch.int32, device="cuda"))
    assert all((row == -1).all() for row in p.page_table[1:].split(128)) and ovc.device_status() == 0


def test_bad_rows_are_reported_and_left_alone():
    def state():
        return _state([[0, 1, -1], [2, 77, -1], [3, -1, -1], [4, -1, -1]], [20, 20, 60, 16], [1, 1, 1, 1, 1, 0, 0, 0], 16)

    p = state()
    _reserve(p, [21, 21, 70, 49])            # row 1's last page, row 2's length, row 3's wish are out of range
    assert ovc.device_status() == BAD_INDEX and ovc.device_status() == 0
    assert p.kv_lens.tolist() == [21, 20, 60, 16] and p.refs.tolist() == [1, 1, 1, 1, 1, 0, 0, 0]
    p = state()
    ovc.kv_pages_release(p, _i32([0, 0, 0, 0]))
    assert ovc.device_status() == BAD_INDEX
    assert p.kv_lens.tolist() == [0, 0, 60, 0] and p.refs.tolist() == [0, 0, 0, 1, 0, 0, 0, 0]
    ovc.kv_pages_release(p, _i32([-1, -1, -1, -1]))      # rows that stay are not looked at
    assert ovc.device_status() == 0
    p.kv_lens[0] = 5                         # a page that nobody holds
    p.page_table[0, 0] = 6
    ovc.kv_pages_release(p, _i32([0, 0, -1, 0]))
    assert ovc.device_status() == BAD_INDEX and p.refs[6] == 0


def test_pages_with_too_few_holders_are_reported():
    """More entries name a page than refs counts: given back, or left for one of their
    own, by more rows than hold it, its count stays 0, or as it is."""
    rows = 500
    p = _state(np.zeros((rows, 1), int), [5] * rows, [rows - 100, 0], 16)
    ovc.kv_pages_release(p, _i32([0] * rows))
    assert ovc.device_status() == BAD_INDEX and p.refs.tolist() == [0, 0]
    assert not p.kv_lens.any() and (p.page_table == -1).all()
    p = _state([[0, 1, -1], [0, 1, -1], [2, 1, -1], [3, -1, -1]], [20, 20, 20, 10], [2, 2, 1, 1, 0, 0, 0, 0, 0], 16)
    src, dst, tokens = _reserve(p, [24, 24, 34, 40])
    assert ovc.device_status() == BAD_INDEX and p.kv_lens.tolist() == [20, 20, 20, 40] and p.refs.tolist() == [2, 2, 1, 1, 1, 1, 0, 0, 0]
    assert (src == -1).all() and (dst == -1).all() and not tokens.any() and p.page_table.tolist()[2:] == [[2, 1, -1], [3, 4, 5]]


@pytest.mark.parametrize("parents, children, done", [([0, 0], [2, 2], []), ([0, 2], [2, 3], [3]), ([0, 1], [1, 2], [2]),
                                                     ([0, 9], [2, 3], [2]), ([0, -1], [2, -1], [2]), ([0, -1], [2, 3], [2]),
                                                     ([0, 0], [2, 4], [2]), ([0, 3], [2, 3], [2]), ([4, 0], [2, 3], [3])], ids=str)
def test_bad_forks_are_reported_and_skipped(parents, children, done):
    """Rows 0 and 1 hold pages, 2 and 3 are empty, 4 has a length that is none; a
    child named twice or as a parent is no child."""
    p = _state(np.array([[0, 1], [2, -1], [-1, -1], [-1, -1], [3, -1]]), [20, 5, 0, 0, 99], [1, 1, 1, 1, 0], 16)
    ovc.kv_pages_fork(p, _i32(parents), _i32(children))
    assert ovc.device_status() == (0 if (parents[1], children[1]) == (-1, -1) else BAD_INDEX)
    lens = [20, 5, 0, 0, 99]
    for a, b in zip(parents, children):
        if b in done:
            lens[b] = lens[a]
    assert p.kv_lens.tolist() == lens
    want = Pages(p.page_table.cpu().numpy(), lens, p.refs.cpu().numpy(), 16)
    want.lens[4], want.refs[3] = 0, 0
    want.table[4] = -1
    assert want.sound()


# --------------------------------------------------------------------- copies
@pytest.mark.parametrize("pages, heads, page", [(5, 1, 16), (40, 3, 48), (30, 8, 64), (7, 9, 1024), (300, 2, 32)])
@pytest.mark.parametrize("partial", [False, True])
def test_copies(pages, heads, page, partial):
    g = np.random.default_rng(pages)
    c = _filled(pages, heads, page, 1)
    order = g.permutation(pages)
    n = pages // 2
    src, dst = order[g.integers(0, n, n)], order[n:2 * n].copy()
    src[1::5] = -1
    dst[2::7] = -3
    tokens = g.integers(0, page + 1, n) if partial else None
    if partial:
        tokens[:3] = [page, 0, 1][:n]
    want = copied(_arrays(c), src, dst, tokens)
    ovc.kv_cache_copy(c, _i32(src), _i32(dst), _i32(tokens) if partial else None)
    assert _holds(c, want) and ovc.device_status() == 0


def test_copies_between_caches():
    a, b = _filled(12, 3, 32, 1), _filled(5, 3, 32, 2)
    src, dst = [11, 0, 7], [4, 2, 0]
    old, into = _arrays(a), _arrays(b)
    ovc.kv_cache_copy(b, _i32(src), _i32(dst), source=a)
    for x, y in zip(old, into):
        y[dst] = x[src]
    assert _holds(b, into) and _holds(a, old)


def test_bad_copies_are_reported_and_skipped():
    c = _filled(6, 2, 16, 3)
    for src, dst, tokens in (([6], [0], [3]), ([0], [6], [3]), ([0], [1], [17]), ([0], [1], [-1])):
        old = _arrays(c)
        ovc.kv_cache_copy(c, _i32(src + [2]), _i32(dst + [3]), _i32(tokens + [5]))
        assert ovc.device_status() == BAD_INDEX and _holds(c, copied(old, [2], [3], [5]))


def test_copies_beyond_32_bit_offsets():
    c = ovc.kv_cache(70000, 4, 128)           # 4.6 GB of codes each
    c.k[69990].fill_(5)
    c.v[69990].fill_(6)
    c.k_scale[69990].fill_(7)
    c.v_scale[69990].fill_(8)
    ovc.kv_cache_copy(c, _i32([69990, 69990]), _i32([69999, 1]), _i32([128, 127]))
    for x, v in zip((c.k, c.v, c.k_scale, c.v_scale), (5, 6, 7, 8)):
        assert (x[69999] == v).all() and (x[1, :, :127] == v).all()
    assert ovc.device_status() == 0


# ----------------------------------------------------------------- compaction
def _held(lens, page, seed, spare=2):
    """Rows of random pages: table, refs."""
    g = np.random.default_rng(seed)
    n = -(-np.asarray(lens) // page)
    pages = int(n.sum()) + spare
    table = np.full((len(lens), max(1, int(n.max()))), -1)
    order, at = g.permutation(pages), 0
    for b, k in enumerate(n):
        table[b, :k] = order[at:at + k]
        at += k
    refs = np.zeros(pages, int)
    refs[order[:at]] = 1
    return table, refs


def _keep(lens, kind, heads, seed):
    """Kept positions of each row, [n] or [heads, n], and their starts."""
    g = np.random.default_rng(seed)
    out = []
    for n in lens:
        if kind == "all":
            k = n
        elif kind == "none":
            k = 0
        else:
            k = int(g.integers(0, n + 1))
        one = np.stack([np.sort(g.permutation(n)[:k]) for _ in range(heads)])
        if kind == "window" and n:
            one = np.broadcast_to(np.r_[np.arange(min(4, k)), np.arange(n - k + min(4, k), n)], (heads, k))
        if kind == "late" and n:
            one = np.broadcast_to(np.delete(np.arange(n), n // 2), (heads, n - 1))
        out.append(one)
    cu = np.r_[0, np.cumsum([x.shape[1] for x in out])]
    return np.concatenate(out, 1), cu


@pytest.mark.parametrize("lens, heads, page", [([1], 1, 16), ([2, 0, 37], 3, 16), ([700, 64, 255, 256, 257], 2, 48),
                                               ([5000], 1, 64), ([40000], 2, 128), ([3000, 17, 2047], 5, 1024), ([90] * 70, 8, 32)])
@pytest.mark.parametrize("kind", ["some", "window", "late", "all", "none"])
@pytest.mark.parametrize("per_head", [False, True])
def test_compaction(lens, heads, page, kind, per_head):
    table, refs = _held(lens, page, len(lens))
    c = _filled(len(refs), heads, page, 4)
    p = _state(table, lens, refs, page)
    keep, cu = _keep(lens, kind, heads if per_head else 1, 5)
    old = _arrays(c)
    want = compacted(old, table, page, keep if per_head else keep[0], cu)
    ovc.kv_cache_compact(c, p, _i32(keep if per_head else keep[0]), _i32(cu))
    for b in range(len(lens)):                # the kept tokens are in place
        i = np.arange(cu[b + 1] - cu[b])
        for got, x in zip(_arrays(c), want):
            assert torch.equal(got[table[b, i // page], :, i % page], x[table[b, i // page], :, i % page])
    free = np.nonzero(refs == 0)[0]
    for got, x in zip(_arrays(c), old):       # and no other page has changed
        assert torch.equal(got[free], x[free])
        for b, n in enumerate(lens):
            behind = table[b, -(-int(cu[b + 1] - cu[b]) // page):-(-n // page)]
            assert torch.equal(got[behind], x[behind])
    assert Pages(table, lens, refs, page).same_as(p) and ovc.device_status() == 0


def test_compaction_of_many_chunks_is_repeatable():
    """A long row, every cluster at work, ten times the same."""
    n, page = 200000, 64
    table, refs = _held([n], page, 6)
    keep = np.sort(np.random.default_rng(7).permutation(n)[:n // 2])
    p = _state(table, [n], refs, page)
    c = _filled(len(refs), 1, page, 8)
    old = _arrays(c)
    i = np.arange(len(keep))
    want = [x[table[0, keep // page], :, keep % page] for x in old]
    for _ in range(10):
        for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), old):
            x.copy_(y)
        ovc.kv_cache_compact(c, p, _i32(keep), _i32([0, len(keep)]))
        assert all(torch.equal(x[table[0, i // page], :, i % page], y) for x, y in zip(_arrays(c), want))


@pytest.mark.parametrize("rows, heads, most, page", [(5, 4, 40000, 64), (9, 5, 27000, 16), (11, 6, 16000, 48), (8, 9, 12000, 128),
                                                     (10, 5, 24000, 64), (13, 7, 5000, 16), (70, 3, 4000, 32), (6, 3, 40000, 64)])
@pytest.mark.parametrize("kind", ["some", "window", "late"])
@pytest.mark.parametrize("per_head", [False, True])
def test_compaction_by_clusters_of_every_size(rows, heads, most, page, kind, per_head):
    """Ragged rows of many chunks: 8, 6, 4, 3, 5 CTAs a sequence and head, one
    (twice), and 7 with half of the channels each (on 152 SMs)."""
    g = np.random.default_rng(rows)
    lens = g.integers(1, most // 8, rows)
    lens[::3] = g.integers(most // 2, most, len(lens[::3]))
    lens[rows // 2] = most
    table, refs = _held(lens, page, rows)
    c = _filled(len(refs), heads, page, rows + 1)
    p = _state(table, lens, refs, page)
    keep, cu = _keep(lens, kind, heads if per_head else 1, 5)
    all_keep = torch.tensor(np.broadcast_to(keep, (heads, keep.shape[1])), device="cuda")
    of = torch.tensor(np.repeat(np.arange(rows), np.diff(cu)), device="cuda")
    i = torch.arange(keep.shape[1], device="cuda") - torch.tensor(cu, device="cuda")[of]
    pages, head = p.page_table.long(), torch.arange(heads, device="cuda").unsqueeze(1)
    free = torch.tensor(np.nonzero(refs == 0)[0], device="cuda")
    want = [(x[pages[of, all_keep // page], head, all_keep % page], x[free]) for x in (c.k, c.v, c.k_scale, c.v_scale)]
    ovc.kv_cache_compact(c, p, _i32(keep if per_head else keep[0]), _i32(cu))
    for x, (kept, unheld) in zip((c.k, c.v, c.k_scale, c.v_scale), want):
        assert torch.equal(x[pages[of, i // page], head, i % page], kept) and torch.equal(x[free], unheld)
    assert Pages(table, lens, refs, page).same_as(p) and ovc.device_status() == 0


def test_lists_of_heads_may_be_views():
    n, heads, page = 100, 4, 16
    table, refs = _held([n], page, 1)
    g = np.random.default_rng(2)
    wide = _i32(np.stack([np.sort(g.permutation(n)[:60]) for _ in range(heads)]))
    for keep in (wide[:, :40], wide[:1, :40].expand(heads, -1), wide[:3:2].repeat_interleave(2, 0)[:, :60]):
        p, c = _state(table, [n], refs, page), _filled(len(refs), heads, page, 3)
        want = compacted(_arrays(c), table, page, keep.cpu().numpy(), [0, keep.shape[1]])
        ovc.kv_cache_compact(c, p, keep, _i32([0, keep.shape[1]]))
        i = np.arange(keep.shape[1])
        assert all(torch.equal(x[table[0, i // page], :, i % page], y[table[0, i // page], :, i % page]) for x, y in zip(_arrays(c), want))
    assert ovc.device_status() == 0


def test_shared_pages_are_not_written():
    """Row 1 shares row 0's first two pages: it may keep them and move what lies
    behind, but not move tokens into them."""
    page = 16
    table = np.array([[0, 1, 2], [0, 1, 3]])
    p = _state(table, [40, 44], [2, 2, 1, 1, 0], page)
    c = _filled(5, 2, page, 9)
    old = _arrays(c)
    ok = np.r_[np.arange(32), 35, 40]
    ovc.kv_cache_compact(c, p, _i32(np.r_[np.arange(40), ok]), _i32([0, 40, 40 + len(ok)]))
    assert ovc.device_status() == 0 and _holds(c, compacted(old, table, page, np.r_[np.arange(40), ok], [0, 40, 40 + len(ok)]))
    old = _arrays(c)
    bad = np.r_[np.arange(31), 35, 40]
    ovc.kv_cache_compact(c, p, _i32(np.r_[np.arange(39), bad]), _i32([0, 39, 39 + len(bad)]))
    assert ovc.device_status() == BAD_INDEX and _holds(c, old)


@pytest.mark.parametrize("heads, length, page", [(3, 44, 16), (1, 90, 16), (2, 300, 48), (8, 700, 16), (5, 3001, 64), (9, 5000, 1024),
                                                 (2, 40000, 16), (300, 100, 16), (4, 20000, 128)])
@pytest.mark.parametrize("pairs", [1, 4, 20])
def test_a_sequence_with_shared_pages_is_left_alone_in_all_heads(heads, length, page, pairs):
    """A list for each head.  The second row of each pair shares whole pages of the
    first's and drops seven tokens a head: behind them in all heads, within them in
    one, in some or in all, or only at the end, where nothing moves."""
    pairs = max(1, min(pairs, 900000 // (heads * length)))
    g = np.random.default_rng(heads + length)
    held = -(-length // page)
    table = np.arange(2 * pairs * held).reshape(2 * pairs, held)
    keep, refused = [], []
    for i in range(pairs):
        shared = [held, held // 2, 1, held - 1][i % 4] if held > 1 else 1
        table[2 * i + 1, :shared] = table[2 * i, :shared]
        end = shared * page
        inside = {0: [], 1: [int(g.integers(heads))], 2: g.choice(heads, heads // 2, replace=False), 3: range(heads)}[int(g.integers(4))]
        behind = np.arange(min(end, length - 7), length)
        lists = []
        for h in range(heads):
            drop = g.choice(min(end, length) if h in inside else behind, 7, replace=False)
            if h not in inside and g.random() < 0.3:
                drop = np.arange(length - 7, length)
            lists.append(np.delete(np.arange(length), drop))
        lists = np.stack(lists)
        kept = -(-(length - 7) // page)                       # columns of the kept tokens
        moved = [np.nonzero(k != np.arange(length - 7))[0] for k in lists]
        refused.append(any(len(m) and m[0] // page < min(shared, kept) for m in moved))
        keep += [np.broadcast_to(np.arange(length), (heads, length)), lists]
    pages, refs = 2 * pairs * held, np.bincount(table.ravel(), minlength=2 * pairs * held)
    cu = np.r_[0, np.cumsum([k.shape[1] for k in keep])]
    c, p = _filled(pages, heads, page, 1), _state(table, [length] * (2 * pairs), refs, page)
    old = [x.clone() for x in (c.k, c.v, c.k_scale, c.v_scale)]
    ovc.kv_cache_compact(c, p, _i32(np.concatenate(keep, 1)), _i32(cu))
    assert ovc.device_status() == (BAD_INDEX if any(refused) else 0)
    changed = np.zeros(pages, bool)
    head, i = torch.arange(heads, device="cuda").unsqueeze(1), torch.arange(length - 7, device="cuda")
    for b, no in enumerate(refused):
        if not no:
            row, k = p.page_table[2 * b + 1].long(), torch.tensor(keep[2 * b + 1], device="cuda")
            own = refs[table[2 * b + 1]] == 1
            changed[table[2 * b + 1][own]] = True
            for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), old):
                assert torch.equal(x[row[i // page], head, i % page], y[row[k // page], head, k % page])
    same = torch.tensor(np.nonzero(~changed)[0], device="cuda")
    assert all(torch.equal(x[same], y[same]) for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), old))


@pytest.mark.parametrize("keep, cu", [([0, 2, 2, 5], [0, 4, 4]), ([0, 3, 2], [0, 3, 3]), ([0, 30], [0, 2, 2]), ([-1, 3], [0, 2, 2]),
                                      ([0, 1], [0, 3, 3]), ([0, 1], [1, 0, 0]), ([0, 1], [-1, 0, 0]), (list(range(1, 25)), [0, 24, 24])], ids=str)
def test_bad_positions_are_reported(keep, cu):
    """Row 0 has 20 tokens; row 1's pages and the free one stay as they are."""
    table = np.array([[0, 1], [2, 3]])
    p = _state(table, [20, 32], [1, 1, 1, 1, 0], 16)
    c = _filled(5, 2, 16, 10)
    old = _arrays(c)
    ovc.kv_cache_compact(c, p, _i32(keep), _i32(cu))
    assert ovc.device_status() == BAD_INDEX
    assert all(torch.equal(x[2:], y[2:]) for x, y in zip(_arrays(c), old))


def test_a_bad_position_before_those_that_move():
    """A long list that goes wrong among the positions that stay, at one that the
    search for the first that moves does not look at: its page, which others hold
    too, is not written."""
    page, n, at, kept = 16, 66100, 258 * 100, 66000
    table, refs = _held([n], page, 3)
    keep = np.arange(kept)
    keep[at + 101:] += 1
    for wrong in range(at, at + 6):
        bad = keep.copy()
        bad[wrong] = wrong + 40
        shared = table[0, wrong // page]
        r = refs.copy()
        r[shared] = 2
        c, p = _filled(len(refs), 1, page, 4), _state(table, [n], r, page)
        old = [x[shared].clone() for x in (c.k, c.v, c.k_scale, c.v_scale)]
        ovc.kv_cache_compact(c, p, _i32(bad), _i32([0, kept]))
        assert all(torch.equal(x[shared], y) for x, y in zip((c.k, c.v, c.k_scale, c.v_scale), old))
    ovc.device_status()


# --------------------------------------------------------- streams and graphs
def test_captured_step_follows_new_lengths_and_lists():
    """Release, fork, reserve, copy and compact in one graph, replayed as lengths
    and lists change, beside an eager copy of everything."""
    page, rows = 16, 6

    def make():
        p = ovc.kv_pages(200, rows, 12, page)
        ovc.kv_pages_reserve(p, _i32([90, 40, 17, 0, 0, 0]))
        return p, _filled(200, 3, page, 11)

    io = {"to": _i32([80, 40, 17, 0, 0, 0]), "parents": _i32([0, 1, 2]), "children": _i32([3, 4, 5]),
          "lens": _i32([90, 41, 20, 85, 47, 17]), "keep": _i32(np.zeros(300)), "cu": _i32(np.zeros(rows + 1))}

    def step(p, c):
        ovc.kv_pages_release(p, io["to"])
        ovc.kv_pages_fork(p, io["parents"], io["children"])
        src, dst, tokens = ovc.kv_pages_reserve(p, io["lens"])
        ovc.kv_cache_copy(c, src, dst, tokens)
        ovc.kv_cache_compact(c, p, io["keep"], io["cu"])

    p, c = make()
    q, d = make()
    step(p, c)
    step(q, d)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(p, c)                            # not run: recorded
    g = np.random.default_rng(12)
    for i in range(6):
        lens = q.kv_lens.cpu().numpy()
        to = np.where(np.arange(rows) < 3, lens - g.integers(0, 9, rows), 0).clip(0)
        children = g.permutation([3, 4, 5])
        grown = np.r_[to[:3], np.zeros(3, int)]
        grown[children] = to[:3]
        grown = grown + g.integers(0, 20, rows)
        kept = np.array([int(g.integers(0, n + 1)) if b % 2 else 0 for b, n in enumerate(grown)])
        # rows whose pages are shared keep all: others drop tokens behind the shared ones only by luck, and are reported
        keep = np.concatenate([np.sort(g.permutation(n)[:k]) for n, k in zip(grown, kept)])
        for name, v in (("to", to), ("children", children), ("lens", grown), ("keep", np.r_[keep, np.zeros(300 - len(keep), int)]),
                        ("cu", np.r_[0, np.cumsum(kept)])):
            io[name].copy_(_i32(v))
        graph.replay()
        step(q, d)
        assert Pages.of(q).same_as(p) and all(torch.equal(x, y) for x, y in zip(_arrays(c), _arrays(d)))
    ovc.device_status()


def test_captured_compactions_at_the_same_time():
    """Two graphs, of caches of their own, on two streams, replayed as lists change:
    many chunks, several CTAs a sequence and head."""
    rows, heads, page, most = 5, 4, 64, 30000
    g = np.random.default_rng(1)
    parts = []
    for i in range(2):
        lens = g.integers(most // 2, most, rows)
        table, refs = _held(lens, page, i)
        s = {"p": _state(table, lens, refs, page), "c": _filled(len(refs), heads, page, i), "lens": lens, "refs": refs, "table": table,
             "keep": _i32(np.zeros((heads, int(lens.sum())))), "cu": _i32(np.zeros(rows + 1)), "stream": torch.cuda.Stream(),
             "graph": torch.cuda.CUDAGraph()}
        ovc.kv_cache_compact(s["c"], s["p"], s["keep"], s["cu"])
        with torch.cuda.graph(s["graph"]):
            ovc.kv_cache_compact(s["c"], s["p"], s["keep"], s["cu"])
        parts.append(s)
    for step in range(4):
        for s in parts:
            keep, cu = _keep(s["lens"], ["some", "window", "late", "some"][step], heads, step)
            s["keep"][:, :keep.shape[1]].copy_(_i32(keep))
            s["cu"].copy_(_i32(cu))
            of = torch.tensor(np.repeat(np.arange(rows), np.diff(cu)), device="cuda")
            k, i = torch.tensor(keep, device="cuda"), torch.arange(keep.shape[1], device="cuda") - _i32(cu).long()[of]
            t, head = s["p"].page_table.long(), torch.arange(heads, device="cuda").unsqueeze(1)
            s["at"] = (t[of, i // page], head, i % page)
            s["want"] = [x[t[of, k // page], head, k % page] for x in (s["c"].k, s["c"].v, s["c"].k_scale, s["c"].v_scale)]
        torch.cuda.synchronize()
        for s in parts:
            with torch.cuda.stream(s["stream"]):
                s["graph"].replay()
        torch.cuda.synchronize()
        for s in parts:
            assert all(torch.equal(x[s["at"]], y) for x, y in zip((s["c"].k, s["c"].v, s["c"].k_scale, s["c"].v_scale), s["want"]))
            assert Pages(s["table"], s["lens"], s["refs"], page).same_as(s["p"])
        assert ovc.device_status() == 0


def test_calls_on_a_stream_and_side_by_side():
    side = torch.cuda.Stream()
    states = []
    for i in range(2):
        lens = [300 + i, 129]
        table, refs = _held(lens, 16, i)
        keep, cu = _keep(lens, "some", 1, i)
        states.append((_state(table, lens, refs, 16), _filled(len(refs), 4, 16, 20 + i), _i32(keep[0]), _i32(cu), table, keep[0], cu))
    torch.cuda.synchronize()
    want = [compacted(_arrays(s[1]), s[4], 16, s[5], s[6]) for s in states]
    for s, stream in zip(states, (side, None)):
        ovc.kv_cache_compact(s[1], s[0], s[2], s[3], stream=stream)
        ovc.kv_pages_release(s[0], s[3][1:] - s[3][:-1] if stream is None else _on(side, lambda s=s: s[3][1:] - s[3][:-1]), stream=stream)
        src, _, _ = ovc.kv_pages_reserve(s[0], _on(side, lambda: torch.full((2,), 100, dtype=torch.int32, device="cuda"))
                                         if stream else torch.full((2,), 100, dtype=torch.int32, device="cuda"), stream=stream)
    torch.cuda.synchronize()
    for s, w in zip(states, want):
        for b in range(2):
            i = np.arange(s[6][b + 1] - s[6][b])
            for x, y in zip(_arrays(s[1]), w):
                assert torch.equal(x[s[4][b, i // 16], :, i % 16], y[s[4][b, i // 16], :, i % 16])
            assert s[0].kv_lens[b] == max(100, len(i))
    assert ovc.device_status() == 0


def _on(stream, fn):
    with torch.cuda.stream(stream):
        return fn()


def test_empty_calls_do_nothing():
    p, c = ovc.kv_pages(4, 2, 2, 16), _filled(4, 1, 16, 1)
    none = _i32(np.zeros(0, int))
    old = _arrays(c)
    ovc.kv_pages_fork(p, none, none)
    ovc.kv_cache_copy(c, none, none)
    ovc.kv_cache_compact(c, p, none, _i32([0, 0, 0]))
    assert _holds(c, old) and ovc.device_status() == 0


def test_refusals():
    p, c = ovc.kv_pages(4, 2, 2, 16), ovc.kv_cache(4, 2, 16)
    two, three = _i32([0, 0]), _i32([0, 0, 0])
    with pytest.raises(ValueError, match="lens"):
        ovc.kv_pages_reserve(p, three)
    with pytest.raises(ValueError, match="int32"):
        ovc.kv_pages_release(p, two.long())
    with pytest.raises(ValueError, match="up to 2"):
        ovc.kv_pages_fork(p, three, three)
    with pytest.raises(ValueError, match="parents"):
        ovc.kv_pages_fork(p, three, two)
    with pytest.raises(ValueError, match="dst"):
        ovc.kv_cache_copy(c, two, three)
    with pytest.raises(ValueError, match="tokens"):
        ovc.kv_cache_copy(c, two, two, three)
    with pytest.raises(ValueError, match="source"):
        ovc.kv_cache_copy(c, two, two, source=ovc.kv_cache(4, 2, 32))
    with pytest.raises(ValueError, match="keep"):
        ovc.kv_cache_compact(c, p, torch.zeros((3, 2), dtype=torch.int32, device="cuda"), three)
    with pytest.raises(ValueError, match="cu_keep"):
        ovc.kv_cache_compact(c, p, two, two)
    with pytest.raises(ValueError, match="pages and page size"):
        ovc.kv_cache_compact(ovc.kv_cache(5, 2, 16), p, two, three)
    with pytest.raises(ValueError, match="CUDA device"):
        ovc.kv_pages_release(p, two.cpu())
    for bad in (dict(page_size=20), dict(page_size=2048), dict(num_pages=0), dict(num_sequences=0), dict(num_sequences=8193)):
        with pytest.raises(ValueError):
            ovc.kv_pages(**{**dict(num_pages=4, num_sequences=2, pages_per_sequence=2, page_size=16), **bad})
    refs = torch.zeros(9, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="aligned"):
        ovc.KVPages(p.page_table, p.kv_lens, refs[1:], 16)
