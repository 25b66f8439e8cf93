"""Page bookkeeping and page copies against the plain model (tests/paged_ref.py),
and a serving run that uses everything together."""
import random

import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK, DIM, HEADS, Pages, Seq, attend64, pages_for

pytestmark = pytest.mark.gpu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Pool:
    def __init__(self, rows, width, num, P, seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.table = torch.full((rows, width + 3), -1, dtype=torch.int32, device="cuda")[:, :width]
        self.n, self.ref = _ints([0] * rows), _ints([0] * num)
        self.pools = [torch.randint(0, 256, (num, P, 16 * w), generator=gen, device="cuda",
                                    dtype=torch.uint8) for w in (1, 3, 64)]
        self.rings = [torch.randint(0, 9999, (rows, 128, w), generator=gen, device="cuda",
                                    dtype=torch.int16) for w in (1, 512)]
        self.P = P
        self.plain = Pages(self.table.tolist(), [0] * rows, [0] * num, P)

    def check(self):
        assert self.table.tolist() == self.plain.table()
        assert self.n.tolist() == [len(r) for r in self.plain.rows]
        assert self.ref.tolist() == self.plain.ref

    def resize(self, entries):
        hca.resize_pages(self.table, self.n, self.ref, _ints(entries), self.P)
        self.plain.resize(entries)
        self.check()

    def fork(self, a, b, e):
        want = [x.clone() for x in self.pools + self.rings]
        ok = hca.fork_pages(self.table, self.n, self.ref, _ints(a), _ints(b), _ints(e), self.pools,
                            self.P, rings=self.rings)
        good, pages, rows = self.plain.fork(a, b, e)
        assert ok.tolist() == good
        for x in want[:3]:
            for s, d in pages:
                x[d] = x[s]
        for x in want[3:]:
            for s, d in rows:
                x[d] = x[s]
        self.check()
        assert all(torch.equal(x, y) for x, y in zip(self.pools + self.rings, want))
        return good

    def compact(self):
        want = [x.clone() for x in self.pools]
        live = hca.compact_pages(self.table, self.n, self.ref, self.pools)
        for s, d in self.plain.compact():
            for x in want:
                x[d] = x[s]
        assert live.tolist() == [sum(c > 0 for c in self.plain.ref)]
        self.check()
        assert all(torch.equal(x, y) for x, y in zip(self.pools, want))


def _error():
    torch.cuda.synchronize()
    return hca.device_error()[0]


@pytest.mark.parametrize("rows,width,num,P", [(1, 1, 1, 16), (5, 7, 20, 32), (40, 30, 500, 16),
                                              (1500, 20, 9000, 128), (9, 600, 4097, 64)])
def test_random_histories(rows, width, num, P):
    """Grow, cut, fork and compact at random; the pool runs out now and then."""
    need_gpu()
    r = random.Random(rows + num)
    p = Pool(rows, width, num, P, seed=rows)
    for step in range(12):
        entries = [r.choice([-1, -1, 0, r.randint(0, width * P), r.randint(0, P)])
                   for _ in range(rows)]
        p.resize(entries)
        assert _error() == 0
        live = [i for i in range(rows) if p.plain.rows[i]]
        empty = [i for i in range(rows) if not p.plain.rows[i]]
        if live and empty:
            n = r.randint(1, min(len(empty), 300))
            a = [r.choice(live) for _ in range(n)]
            e = [r.randint(0, len(p.plain.rows[x]) * P) for x in a]
            e[0] = len(p.plain.rows[a[0]]) * P       # nothing partly filled
            p.fork(a, r.sample(empty, n), e)
            assert _error() == 0
        if step % 3 == 2:
            p.compact()
            assert _error() == 0
    p.resize([0] * rows)
    assert p.plain.free() == list(range(num))
    p.compact()


def test_growth_stops_when_the_pool_is_empty():
    need_gpu()
    p = Pool(4, 8, 10, 16, seed=1)
    p.resize([64, 100, 0, 50])      # 4 + 7 + 0 + 4 pages wanted, 10 there
    assert p.n.tolist() == [4, 6, 0, 0]
    p.resize([16, -1, 48, -1])      # the first gives 3 back, the third takes them
    assert p.n.tolist() == [1, 6, 3, 0]
    assert p.fork([1], [3], [90]) == [0]         # no page for the partly filled one
    assert p.fork([1], [3], [80]) == [1]
    assert _error() == 0


def test_refused_forks_and_lengths():
    need_gpu()
    p = Pool(6, 8, 40, 16, seed=2)
    p.resize([40, 60, 0, 0, 0, 16])
    good = p.fork([0, 0, 1, 7, -1, 0, 1, 0, 2], [2, 2, 5, 3, 3, 9, 3, 0, 4],
                  [40, 40, 60, 10, 10, 10, 65, 10, 0])
    # the row of the last pair's parent is a child of the first: that one is refused, and
    # with it nothing is left of row 2 but its second mention, refused as a repetition
    assert good == [0, 0, 0, 0, 0, 0, 0, 0, 1]
    assert _error() == 5
    p.fork([0, 1, 0], [2, 3, 2], [33, 64, 1])
    assert _error() == 5
    # a row that would need more columns than there are is cut and reported
    p.resize([-1, 16 * 9, -1, -1, -1, -1])
    assert p.n.tolist()[1] == 8 and _error() == 5


def test_counts_that_do_not_fit_are_reported():
    need_gpu()
    p = Pool(2, 4, 8, 16, seed=3)
    p.resize([64, 0])
    p.ref[1] = 0                     # lost count
    p.table[0, 2] = 99               # no such page
    hca.resize_pages(p.table, p.n, p.ref, _ints([0, -1]), 16)
    assert _error() == 5
    assert p.ref.tolist() == [0, 0, 1, 0, 0, 0, 0, 0] and p.n.tolist() == [0, 0]


@pytest.mark.parametrize("n", [1, 33, 1500])
def test_copy(n):
    need_gpu()
    r = random.Random(n)
    items = 3 * n + 5
    gen = torch.Generator(device="cuda").manual_seed(n)
    arrays = [torch.randint(0, 256, (items, b), generator=gen, device="cuda", dtype=torch.uint8)
              for b in (16, 48, 16384, 16400, 40000)]
    src = [r.randrange(n) for _ in range(n)]
    dst = r.sample(range(n, items), n)
    want = [x.clone() for x in arrays]
    for a, b in zip(src, dst):
        for x in want:
            x[b] = x[a]
    hca.copy_pages(arrays, _ints(src), _ints(dst))
    assert _error() == 0
    assert all(torch.equal(x, y) for x, y in zip(arrays, want))


def test_copy_refuses_what_depends_on_timing():
    need_gpu()
    x = torch.arange(10 * 32, device="cuda", dtype=torch.int32).view(10, 32)
    want = x.clone()
    want[9] = want[0]
    # 3 named twice, 5 is a source, 12 and -1 out of range, 4 onto itself, 0 -> 9 is fine
    hca.copy_pages([x], _ints([1, 2, 5, 0, 1, 4, -1, 0]), _ints([3, 3, 6, 5, 12, 4, 7, 9]))
    torch.cuda.synchronize()
    want[6] = want[5]
    assert torch.equal(x, want) and hca.device_error()[0] == 5


def test_serving_run():
    """Prompts enter, branch, take chunks and single tokens, some end, the pool closes up: every
    output is that of the whole history, and equal before and after the pool is compacted."""
    need_gpu()
    P, rows, num = 16, 6, 60
    gen = torch.Generator(device="cuda").manual_seed(77)
    base = [Seq(9000, gen, "cuda") for _ in range(3)]
    table = torch.full((rows, 12), -1, dtype=torch.int32, device="cuda")
    n_pages, ref = _ints([0] * rows), _ints([0] * num)
    nan = float("nan")
    ck = torch.full((num, P, DIM), nan, dtype=torch.bfloat16, device="cuda")
    cv = ck.clone()
    wk = torch.full((rows, BLOCK, DIM), nan, dtype=torch.bfloat16, device="cuda")
    wv, ws = wk.clone(), torch.full((rows, BLOCK), nan, dtype=torch.bfloat16, device="cuda")
    cache = (wk, wv, ws, ck, cv, table)
    hist = [(x.k[:0], x.v[:0], x.s[:0]) for x in base] + [None] * 3

    def feed(n, attend):
        """n[i] new tokens of each row, drawn anew; checks the outputs of some."""
        ks, lens = [], []
        for i in range(rows):
            m = n[i]
            fresh = Seq(m, gen, "cuda") if m else None
            if m:
                hist[i] = tuple(torch.cat([a, b]) for a, b in zip(hist[i], (fresh.k, fresh.v, fresh.s)))
                ks.append(fresh)
            lens.append(len(hist[i][0]) if hist[i] is not None else 0)
        k, v, s = (torch.cat([getattr(x, f) for x in ks]) for f in "kvs")
        start = _ints([sum(n[:i]) for i in range(rows + 1)])
        ctx = _ints(lens)
        hca.resize_pages(table, n_pages, ref, _ints([x // BLOCK for x in lens]), P)
        if not attend:
            hca.paged_append(k, v, s, start, ctx, *cache)
            assert _error() == 0
            return
        N = sum(n)
        q, g = (torch.randn((N, HEADS, DIM), generator=gen, device="cuda").bfloat16() for _ in "qg")
        out = hca.paged_prefill(q, g, k, v, s, start, ctx, *cache)
        assert _error() == 0
        for i in range(rows):
            for r in {0, n[i] // 2, n[i] - 1} if n[i] else ():
                at = sum(n[:i]) + r
                e = lens[i] // BLOCK
                pages = table[i, :pages_for(lens[i], P)].long()
                ref_o, bound = attend64(q[at], g[at], ck[pages].reshape(-1, DIM)[:e],
                                        cv[pages].reshape(-1, DIM)[:e], hist[i][0], hist[i][1],
                                        lens[i] - n[i] + r)
                assert ((out[at].double() - ref_o).abs() <= bound).all(), (i, r)

    feed([8000, 3000, 130, 0, 0, 0], attend=False)
    feed([40, 1, 5, 0, 0, 0], attend=True)
    # rows 3 and 4 branch off row 0, row 5 off row 1
    par, chi = [0, 0, 1], [3, 4, 5]
    ok = hca.fork_pages(table, n_pages, ref, _ints(par), _ints(chi),
                        _ints([len(hist[a][0]) // BLOCK for a in par]), (ck, cv), P,
                        rings=(wk, wv, ws))
    assert ok.tolist() == [1, 1, 1] and _error() == 0
    for a, b in zip(par, chi):
        hist[b] = hist[a]
    feed([1, 200, 3, 300, 1, 0], attend=True)
    feed([1, 1, 1, 1, 1, 1], attend=True)
    # rows 0 and 1 end; their branches live on through the shared pages
    hist[0] = hist[1] = (base[0].k[:0], base[0].v[:0], base[0].s[:0])
    hca.resize_pages(table, n_pages, ref, _ints([0, 0, -1, -1, -1, -1]), P)
    ctx = _ints([max(1, len(h[0])) for h in hist])
    q, g = (torch.randn((rows, HEADS, DIM), generator=gen, device="cuda").bfloat16() for _ in "qg")
    before = hca.paged_decode(q, ck, cv, table, wk, wv, ctx, g)
    live = hca.compact_pages(table, n_pages, ref, (ck, cv))
    ck[int(live):], cv[int(live):] = nan, nan
    after = hca.paged_decode(q, ck, cv, table, wk, wv, ctx, g)
    assert torch.equal(before[2:], after[2:]) and torch.isfinite(after[2:]).all()
    assert sorted(set(table[table >= 0].tolist())) == list(range(int(live)))
    assert _error() == 0
    feed([300, 1, 1, 129, 64, 2], attend=True)
