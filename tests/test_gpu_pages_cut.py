"""Cutting sequences that share pages: rows stay free to be appended to, and what their branches
hold stays as it was."""
import random

import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK, DIM, HEADS, Pages, Seq, attend64
from tests.test_gpu_paged import _gen, _no_error
from tests.test_gpu_pages import Pool, _error, _ints

pytestmark = pytest.mark.gpu


class CutPages(Pages):
    """The plain bookkeeping of a resize that copies partly used shared pages."""

    def resize_copy(self, entries):
        """Page copies (from, to), and whether every row has its last page to itself."""
        want = [len(r) if e < 0 else min(self.width, -(-e // self.P))
                for r, e in zip(self.rows, entries)]
        for r, w in zip(self.rows, want):
            for p in r[w:]:
                self.ref[p] -= 1
            del r[w:]
        free, copies, fine = self.free(), [], True
        for r, e in zip(self.rows, entries):
            c = e // self.P
            if e > 0 and e % self.P and c < len(r) and self.ref[r[c]] > 1:
                if not free:
                    fine = False
                    continue
                copies.append((r[c], free[0]))
                self.ref[r[c]] -= 1
                r[c] = free.pop(0)
                self.ref[r[c]] = 1
        for r, w in zip(self.rows, want):
            while len(r) < w and free:
                r.append(free.pop(0))
                self.ref[r[-1]] = 1
        return copies, fine


class CutPool(Pool):
    def __init__(self, rows, width, num, P, seed):
        super().__init__(rows, width, num, P, seed)
        self.plain = CutPages(self.table.tolist(), [0] * rows, [0] * num, P)

    def cut(self, entries):
        want = [x.clone() for x in self.pools]
        hca.resize_pages(self.table, self.n, self.ref, _ints(entries), self.P, pools=self.pools)
        copies, fine = self.plain.resize_copy(entries)
        for x, y in zip(want, self.pools):
            for s, d in copies:
                x[d] = x[s]
            assert torch.equal(x, y)
        self.check()
        assert _error() == (0 if fine else 5)
        return copies


def test_rows_that_share_a_page():
    need_gpu()
    p = CutPool(5, 4, 9, 16, seed=1)
    p.resize([48, 0, 0, 0, 0])
    p.fork([0, 0], [1, 2], [48, 32])          # pages 0 and 1 in three rows, 2 in two
    assert p.cut([-1, -1, 20, 0, 0]) == [(1, 3)]       # a branch cut below where it left
    assert p.cut([20, 20, -1, 0, 0]) == [(1, 2)]       # both others: the second keeps the page
    assert p.cut([20, 18, 30, 0, 0]) == []             # nothing left to copy
    assert p.cut([32, 32, 16, 0, 0]) == []             # whole pages may be shared
    p.fork([0], [3], [32])
    p.resize([-1, -1, -1, -1, 16 * 4])
    assert p.cut([3, 3, 3, 3, 60]) == [(0, 1), (0, 2), (0, 7)]   # four rows: the last keeps it


def test_no_page_is_free():
    need_gpu()
    p = CutPool(3, 4, 3, 16, seed=2)
    p.resize([48, 0, 0])
    p.fork([0], [1], [48])
    assert p.cut([-1, 40, 0]) == []                    # the shared page is kept, and reported
    assert p.table[1].tolist() == [0, 1, 2, -1] and p.ref.tolist() == [2, 2, 2]
    assert p.cut([32, 40, 0]) == []                    # now it is the branch's own


@pytest.mark.parametrize("rows,width,num,P", [(5, 7, 24, 32), (40, 30, 700, 16),
                                              (1500, 20, 12000, 128), (9, 600, 5000, 64)])
def test_random_histories_with_cuts(rows, width, num, P):
    need_gpu()
    r = random.Random(rows)
    p = CutPool(rows, width, num, P, seed=rows)
    for step in range(10):
        p.cut([r.choice([-1, -1, 0, r.randint(0, width * P), r.randint(0, P)])
               for _ in range(rows)])
        live = [i for i in range(rows) if p.plain.rows[i]]
        empty = [i for i in range(rows) if not p.plain.rows[i]]
        if live and empty:
            n = r.randint(1, min(len(empty), 300))
            a = [r.choice(live) for _ in range(n)]
            p.fork(a, r.sample(empty, n), [r.randint(0, len(p.plain.rows[x]) * P) for x in a])
            assert _error() == 0
        if step % 4 == 3:
            p.compact()


@pytest.mark.parametrize("who", ["branch", "parent", "both"])
def test_append_after_a_cut(who):
    """A branch, or its parent, goes back to an earlier token and goes on from there: the entries
    of the other are untouched, and both answer from their own history."""
    need_gpu()
    P, num = 16, 12
    gen = _gen(len(who))
    hist = [Seq(BLOCK * 40, gen, "cuda")]
    table = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    n_pages, ref = _ints([0, 0]), _ints([0] * num)
    ck = torch.full((num, P, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
    cv = ck.clone()
    wk = torch.full((2, BLOCK, DIM), float("nan"), dtype=torch.bfloat16, device="cuda")
    wv, ws = wk.clone(), torch.full((2, BLOCK), float("nan"), dtype=torch.bfloat16, device="cuda")
    L = BLOCK * 32 + 5                                  # 32 entries: two whole pages
    hca.resize_pages(table, n_pages, ref, _ints([32, 0]), P, pools=(ck, cv))
    s = hist[0]
    hca.paged_append(s.k[:L], s.v[:L], s.s[:L].clone(), _ints([0, L, L]), _ints([L, 0]), wk, wv, ws,
                     ck, cv, table)
    assert hca.fork_pages(table, n_pages, ref, _ints([0]), _ints([1]), _ints([32]), (ck, cv), P,
                          rings=(wk, wv, ws)).tolist() == [1]
    # back to 21 entries and 7 tokens; the ring is the caller's to set
    back = BLOCK * 21 + 7
    cut = {"branch": [1], "parent": [0], "both": [0, 1]}[who]
    rows = [(s.k[:L], s.v[:L], s.s[:L])] * 2
    hca.resize_pages(table, n_pages, ref, _ints([21 if i in cut else -1 for i in range(2)]), P,
                     pools=(ck, cv))
    for i in cut:
        rows[i] = tuple(x[:back] for x in rows[i])
        for ring, x in zip((wk, wv, ws), rows[i]):
            ring[i] = s.ring(x, back, float("nan"))
    n = [150 + 300 * (i in cut) for i in range(2)]
    new = [Seq(m, gen, "cuda") for m in n]
    rows = [tuple(torch.cat([a, b]) for a, b in zip(x, (y.k, y.v, y.s))) for x, y in zip(rows, new)]
    lens = [len(x[0]) for x in rows]
    hca.resize_pages(table, n_pages, ref, _ints([x // BLOCK for x in lens]), P, pools=(ck, cv))
    k, v, sc = (torch.cat([getattr(y, f) for y in new]) for f in "kvs")
    q, g = (torch.randn((sum(n), HEADS, DIM), generator=gen, device="cuda").bfloat16() for _ in "qg")
    out = hca.paged_prefill(q, g, k, v, sc, _ints([0, n[0], sum(n)]), _ints(lens), wk, wv, ws, ck,
                            cv, table)
    _no_error()
    for i in range(2):
        e = lens[i] // BLOCK
        want = hca.compress(*(x[None] for x in rows[i]))
        pages = table[i, :-(-e // P)].long()
        ek, ev = (x[pages].reshape(-1, DIM)[:e] for x in (ck, cv))
        assert torch.equal(ek, want[0][0]) and torch.equal(ev, want[1][0]), i
        for r in (0, n[i] // 2, n[i] - 1):
            at = i * n[0] + r
            ref_o, bound = attend64(q[at], g[at], ek, ev, rows[i][0], rows[i][1], lens[i] - n[i] + r)
            assert ((out[at].double() - ref_o).abs() <= bound).all(), (i, r)
