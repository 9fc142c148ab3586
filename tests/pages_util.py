"""Definitions, for the tests, of the pages that sequences hold, of moves inside
a paged cache, and of verifying drafted tokens: row by row, on the host."""
import numpy as np
import torch


class Pages:
    """page_table, kv_lens and refs as numpy arrays, changed by the definition."""

    def __init__(self, table, lens, refs, page):
        self.table, self.lens, self.refs, self.page = (np.array(table, np.int64), np.array(lens, np.int64),
                                                       np.array(refs, np.int64), page)

    @classmethod
    def of(cls, p):
        return cls(p.page_table.cpu().numpy(), p.kv_lens.cpu().numpy(), p.refs.cpu().numpy(), p.page)

    def same_as(self, p):
        return (np.array_equal(self.table, p.page_table.cpu().numpy()) and np.array_equal(self.lens, p.kv_lens.cpu().numpy())
                and np.array_equal(self.refs, p.refs.cpu().numpy()))

    def held(self, n):
        return -(-int(n) // self.page)

    def sound(self):
        """Every entry of a row names a page, what lies behind is -1, and refs counts the entries."""
        count = np.zeros_like(self.refs)
        for b, n in enumerate(self.lens):
            row, k = self.table[b], self.held(n)
            if (row[:k] < 0).any() or (row[:k] >= len(self.refs)).any() or (row[k:] != -1).any() or len(set(row[:k])) != k:
                return False
            np.add.at(count, row[:k], 1)
        return np.array_equal(count, self.refs)

    def release(self, lens):
        for b, to in enumerate(lens):
            if 0 <= to < self.lens[b]:
                for c in range(self.held(to), self.held(self.lens[b])):
                    self.refs[self.table[b, c]] -= 1
                    self.table[b, c] = -1
                self.lens[b] = to

    def fork(self, parents, children):
        for a, b in zip(parents, children):
            if a < 0 and b < 0:
                continue
            k = self.held(self.lens[a])
            self.table[b, :k] = self.table[a, :k]
            np.add.at(self.refs, self.table[a, :k], 1)
            self.lens[b] = self.lens[a]

    def reserve(self, lens):
        rows, most = range(len(self.lens)), self.table.shape[1] * self.page
        grow = [self.lens[b] < lens[b] <= most for b in rows]
        writers = {}
        for b in rows:
            if grow[b] and self.lens[b] % self.page:
                p = self.table[b, self.lens[b] // self.page]
                if self.refs[p] > 1:
                    writers.setdefault(int(p), []).append(b)
        moves = {b: p for p, bs in writers.items() for b in (bs[:-1] if len(bs) == self.refs[p] else bs)}
        free = [int(p) for p in np.nonzero(self.refs == 0)[0]]
        src, dst, tokens = (np.full(len(self.lens), v, np.int64) for v in (-1, -1, 0))
        for b in rows:
            if not grow[b]:
                continue
            cols = list(range(self.held(self.lens[b]), self.held(lens[b])))
            if b in moves:
                cols = [self.lens[b] // self.page] + cols
            if len(cols) > len(free):
                break
            got, free = free[:len(cols)], free[len(cols):]
            if b in moves:
                self.refs[moves[b]] -= 1
                src[b], dst[b], tokens[b] = moves[b], got[0], self.lens[b] % self.page
            self.table[b, cols] = got
            self.refs[got] += 1
            self.lens[b] = lens[b]
        return src, dst, tokens


def copied(old, src, dst, tokens):
    """The arrays [pages, heads, page, ...] after a copy within themselves."""
    new = [x.clone() for x in old]
    for i, (a, b) in enumerate(zip(src, dst)):
        for x, y in zip(old, new):
            if a >= 0 and b >= 0:
                t = x.shape[2] if tokens is None else tokens[i]
                y[b, :, :t] = x[a, :, :t]
    return new


def compacted(old, table, page, keep, cu):
    """The arrays after each sequence's kept tokens moved together; keep is a list
    for all heads, or one for each."""
    new = [x.clone() for x in old]
    for b in range(len(cu) - 1):
        for h in range(old[0].shape[1]):
            k = torch.as_tensor(keep[h] if np.ndim(keep) == 2 else keep)[cu[b]:cu[b + 1]].long()
            i = torch.arange(len(k))
            t = torch.as_tensor(table[b]).long()
            for x, y in zip(old, new):
                y[t[i // page], h, i % page] = x[t[k // page], h, k % page]
    return new


def verify(p, q, drafts, cu, accept_u, sample_u):
    """Accepted drafts of each sequence, and the weights (64 bits) that its next
    token is drawn by.  p, q: float64 arrays (q None: drafts were certain)."""
    out = []
    for b in range(len(cu) - 1):
        a, n = cu[b], cu[b + 1] - cu[b]
        i, rejected = 0, False
        while i < n:
            x = drafts[a + i]
            if x < 0 or x >= p.shape[1]:
                break
            if not accept_u[a + i] * (1.0 if q is None else q[a + i, x]) < p[a + b + i, x]:
                rejected = True
                break
            i += 1
        w = np.where(p[a + b + i] > 0, p[a + b + i], 0.0)
        if rejected:
            if q is None:
                rest = w.copy()
                rest[drafts[a + i]] = 0.0
            else:
                with np.errstate(invalid="ignore"):
                    rest = np.where(p[a + b + i] > q[a + i], p[a + b + i] - q[a + i], 0.0)
            if rest.any():
                w = rest
        out.append((i, w))
    return out


def check_verified(tokens, accepted, drafts, cu, sample_u, want):
    """The outputs against :func:`verify`'s.  The drawn token t has a weight, and
    u * total lies between the sums before and up to it, where sums may be off by
    V * 2^-46 of the total.  The kernel's sums are pairs of FP32 numbers at every
    level; drafts.cuh derives K^2 + 40 K + 380 units of 2^-48 for a running sum and
    the total together, with K <= 3 up to V = 248: less than 4 V units from V = 128
    on, with what the FP64 sums here are off by (V * 2^-52).  Below that one tile has
    sums of few lanes, and adding 0 is exact: K = 3 weights a sum 17, merges within
    the lane and over l lanes 2 (4 m + m (m + 1) / 2), m = 2 + log2(l), the search
    24 + 3 log2(l), a product 3: 123 of 124 at V = 31, l = 8.  Shorter rows are held to the
    same, tighter than the kernel's bound of (V + 128) * 2^-46."""
    for b, (i, w) in enumerate(want):
        a, n = cu[b], cu[b + 1] - cu[b]
        got = tokens[a + b:a + b + n + 1]
        assert accepted[b] == i, (b, accepted[b], i)
        assert list(got[:i]) == list(drafts[a:a + i]) and (got[i + 1:] == -1).all()
        t = got[i]
        if not w.any():
            assert t == -1
            continue
        assert 0 <= t < len(w) and w[t] > 0, (b, t)
        upto = np.cumsum(w)
        slack = upto[-1] * len(w) * 2.0 ** -46
        goal = sample_u[b] * upto[-1]
        last = not (w[t + 1:] > 0).any()
        assert upto[t] - w[t] <= goal + slack and (last or goal <= upto[t] + slack), (b, t, goal, upto[t] - w[t], upto[t])
