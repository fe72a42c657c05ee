"""Plain forms of the page calls and of beam search's selection, and inputs.

Pages: Python lists and loops over the definitions in include/qgemv.h, sharing
no code with the library. Selection: every candidate's score in 64 bits.
"""
from __future__ import annotations

import numpy as np


class Pages:
    """A page record on the host: table [n][wide], lens, held, refs."""

    def __init__(self, n, wide, pool, page):
        self.n, self.wide, self.pool, self.page = n, wide, pool, page
        self.table = np.full((n, wide), -7, np.int32)        # entries that no row holds: anything
        self.lens, self.held = np.zeros(n, np.int32), np.zeros(n, np.int32)
        self.refs = np.zeros(pool, np.int32)

    def need(self, tokens):
        return -(-int(tokens) // self.page)

    def fits(self, b):
        return 0 <= self.lens[b] <= 2 ** 30 and 0 <= self.held[b] <= self.wide and self.need(self.lens[b]) <= self.held[b]

    def row(self, b):
        """(tokens, entries) of row b, none if they do not fit."""
        return (int(self.lens[b]), int(self.held[b])) if self.fits(b) else (0, 0)

    def counts(self):
        """How often the table names each page."""
        c = np.zeros(self.pool, np.int64)
        for b in range(self.n):
            for e in self.table[b, :self.held[b]]:
                c[e] += 1
        return c

    def fork(self, parent):
        """Whether something did not fit."""
        bad = False
        rows = [self.row(b) for b in range(self.n)]
        old = self.table.copy()
        for b in range(self.n):
            bad = bad or not self.fits(b)
            for e in old[b, :rows[b][1]]:
                if 0 <= e < self.pool:
                    self.refs[e] -= 1
                else:
                    bad = True
        for i in range(self.n):
            p = int(parent[i])
            if not -1 <= p < self.n:
                p, bad = i, True
            tokens = rows[p][0] if p >= 0 else 0
            k = self.need(tokens)
            self.table[i, :k] = old[p, :k]
            for e in old[p, :k]:
                if 0 <= e < self.pool:
                    self.refs[e] += 1
            self.lens[i], self.held[i] = tokens, k
        return bad

    def reserve(self, new):
        """(moves, free pages left, whether something did not fit)."""
        bad, plans, writers = False, [], {}
        for b in range(self.n):
            (tokens, held), add = self.row(b), int(new[b])
            end = tokens + add
            if not self.fits(b) or add < 0 or end > min(self.wide * self.page, 2 ** 30):
                bad = True
                continue
            if add == 0:
                continue
            first, last = tokens // self.page, self.need(end)
            tail = int(self.table[b, first]) if tokens % self.page else None
            ahead = [int(e) for e in self.table[b, first + (tail is not None):max(first, min(held, last))]]
            ok = tail is None or (0 <= tail < self.pool and self.refs[tail] >= 1)
            ok = ok and all(0 <= e < self.pool and self.refs[e] == 1 for e in ahead)
            if not ok:
                bad = True
                continue
            plans.append((b, tokens, held, first, last, tail))
            if tail is not None:
                writers.setdefault(tail, []).append(b)
        free = [p for p in range(self.pool) if self.refs[p] == 0]
        want = []                                            # (row, column, page to copy from, tokens)
        for b, tokens, held, first, last, tail in plans:
            if tail is not None and self.refs[tail] > 1:
                w = writers[tail]
                if not (len(w) == self.refs[tail] and w[0] == b):
                    want.append((b, first, tail, tokens % self.page))
            want += [(b, c, None, 0) for c in range(held, last)]
        left = len(free) - len(want)
        if left < 0:
            return [], left, bad
        moves = []
        for page, (b, c, tail, tokens) in zip(free, want):
            self.table[b, c] = page
            self.refs[page] = 1
            if tail is not None:
                self.refs[tail] -= 1
                moves.append((tail, page, tokens, 0))
        for b, tokens, held, first, last, tail in plans:
            self.held[b] = max(held, last)
        return moves, left, bad

    def compact(self, capacity):
        """(moves, map, pages in use, whether something did not fit)."""
        live = [p for p in range(self.pool) if self.refs[p] != 0]
        L = len(live)
        holes = [p for p in range(L) if self.refs[p] == 0]
        movers = [p for p in live if p >= L][::-1]
        where = np.full(self.pool, -1, np.int32)
        where[live] = live
        moves = []
        for src, dst in list(zip(movers, holes))[:capacity]:
            moves.append((src, dst, self.page, 0))
            where[src] = dst
            self.refs[dst], self.refs[src] = self.refs[src], 0
        bad = False
        for b in range(self.n):
            bad = bad or not self.fits(b)
            for c in range(self.row(b)[1]):
                e = self.table[b, c]
                if 0 <= e < self.pool and where[e] >= 0:
                    self.table[b, c] = where[e]
                else:
                    bad = True
        return moves, where, L, bad

    # ------------------------------------------------------------------ the device's
    def device(self, torch, q):
        dev = [torch.from_numpy(x.copy()).cuda() for x in (self.table, self.lens, self.held, self.refs)]
        return q.KVPages(*dev, self.page)

    def same(self, rec):
        for name, mine, theirs in (("page_table", self.table, rec.page_table), ("seq_lens", self.lens, rec.seq_lens),
                                   ("n_pages", self.held, rec.n_pages), ("refs", self.refs, rec.refs)):
            assert np.array_equal(mine, theirs.cpu().numpy()), name


def random_pages(r, n, wide, pool, page, fill=0.6, outside=0.05):
    """Rows that share some pages with the row before them, hold some ahead, and have lengths next to page borders."""
    P = Pages(n, wide, pool, page)
    order = list(r.permutation(pool))
    budget = int(pool * fill)
    for b in range(n):
        most = min(wide - 2, budget) if n < 3 else min(wide - 2, max(0, budget // (n - b)) * 2)
        k = int(r.integers(0, max(1, most + 1)))
        share = 0
        if b and r.random() < 0.6:
            share = int(r.integers(0, min(k, P.need(P.lens[b - 1])) + 1))
        k = min(k, share + budget, share + len(order))
        own = [order.pop() for _ in range(k - share)]
        budget -= len(own)
        P.table[b, :share] = P.table[b - 1, :share]
        P.table[b, share:k] = own
        P.held[b] = k
        if k:
            ahead = int(r.integers(0, 2)) if k - share > 1 else 0
            P.lens[b] = max(0, (k - ahead) * page - int(r.choice([0, 1, page - 1, r.integers(0, page)])))
        for e in P.table[b, :k]:
            P.refs[e] += 1
    for p in range(pool):
        if r.random() < outside:
            P.refs[p] += 1
    return P


# ------------------------------------------------------------------ selection
def log_sums(x):
    """ln sum exp of each row (float64), -inf for a row of -infinities, NaN where it has no sum."""
    with np.errstate(all="ignore"):
        top = x.max(1)
        safe = np.where(np.isfinite(top), top, 0.0)
        out = safe + np.log(np.exp(x - safe[:, None]).sum(1))
        out = np.where(top == -np.inf, -np.inf, out)
        return np.where(np.isnan(x).any(1) | (top == np.inf), np.nan, out)


def sum_bound(x):
    """How far a row's ln sum may be off. A term's argument v - top is rounded,
    multiplied by a rounded log2(e) and rounded: 3 half steps, 3 * 2^-24 |v -
    top| of the term, and so for the factor that brings a piece to the row's
    maximum; the hardware's 2^x is off by 2^-22 of it (its documented bound is
    below that). A lane adds 16 pairs, their two halves and, of the pieces of
    1,024, every 32nd, each of these with a factor; 10 steps join the lanes. One
    addition is a half step of the sum, one with a factor 7 at most. The
    logarithm is off by less than 2^-23, of which a half step is its rounding."""
    with np.errstate(all="ignore"):
        top = x.max(1, keepdims=True)
        w = np.exp(x - top)
        p = w / w.sum(1, keepdims=True)
        far = np.where(p > 0, p * np.where(np.isfinite(x), top - x, 0.0), 0.0).sum(1)
        n = x.shape[1] / 32768 + 16 + 1 + 10 + 4
        return 3 * 2.0 ** -24 * far + 2.0 ** -22 + 7 * n * 2.0 ** -24 + 2.0 ** -23


def check_selection(x, scores, finished, eos, pad, got, n_out):
    """got = (scores, tokens, parents, finished) [lanes][n_out] against every
    candidate. Within a row the order is exact: the first of the row's tokens
    by (logit, lower token). Between rows it holds up to the sums' bounds."""
    L, B = scores.shape
    V = x.shape[1]
    x = x.astype(np.float64)
    z, off = log_sums(x), sum_bound(x)
    gs, gt, gp, gf = got
    for lane in range(L):
        rows = range(lane * B, lane * B + B)
        take = {}
        lists = {}
        for r in rows:
            s = float(scores.reshape(-1)[r])
            if np.isnan(s) or s == np.inf or s == -np.inf:
                continue
            if finished is not None and finished.reshape(-1)[r]:
                lists[r] = [(s, pad, 0.0)]
                continue
            if not np.isfinite(z[r]):
                continue
            order = np.lexsort((np.arange(V), -x[r]))[:n_out + 1]
            lists[r] = [(s + (x[r, t] - z[r]), int(t), off[r]) for t in order if x[r, t] > -np.inf]
        want = min(n_out, sum(len(v) for v in lists.values()))
        prev = None
        for o in range(n_out):
            s, t, p, f = float(gs[lane, o]), int(gt[lane, o]), int(gp[lane, o]), bool(gf[lane, o])
            if o >= want:
                assert (s, t, p, f) == (-np.inf, pad, lane * B, False), (lane, o, s, t, p, f)
                continue
            assert p in lists, (lane, o, p)
            k = take.get(p, 0)
            assert k < len(lists[p]), (lane, o, p)
            true, token, b = lists[p][k]
            assert t == token, (lane, o, p, t, token)
            # a score of fp32's range or beyond rounds to -infinity: nearest rounding overflows from (2 - 2^-24) 2^127 on
            if true - b <= -(2 - 2.0 ** -24) * 2.0 ** 127:
                assert s == -np.inf, (lane, o, s, true)
            else:
                assert abs(s - true) <= b + 2.0 ** -24 * abs(true) + 1e-45, (lane, o, s, true, b)
            done = finished is not None and bool(finished.reshape(-1)[p])
            assert f == (done or t == eos), (lane, o)
            take[p] = k + 1
            # nothing that is left may be better, and equal exact candidates come in the order of rows
            for r, c in lists.items():
                j = take.get(r, 0) if r != p else None
                if j is not None and j < len(c):
                    slack = c[j][2] + b + 2.0 ** -50 * (abs(true) + abs(c[j][0]))
                    assert c[j][0] <= true + slack, (lane, o, r, c[j], true)
            prev = s if prev is None else prev
            assert o == 0 or s <= float(gs[lane, o - 1]), (lane, o)
