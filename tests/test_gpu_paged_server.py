"""Random runs of a server on the paged cache: prompts, chunks, single tokens, branches, sequences
that go back to an earlier token, ends and compaction, on shared workspaces.  Every step is checked
against the raw history of each row: rings and entries bit for bit, outputs against 64 bits."""
import random

import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK, DIM, HEADS, Seq, attend64

pytestmark = pytest.mark.gpu
NAN = float("nan")


class Server:
    def __init__(self, seed, rows, P, num, width):
        self.r = random.Random(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.P = rows, P
        self.limit = width * P * BLOCK
        full = lambda *s: torch.full(s, NAN, dtype=torch.bfloat16, device="cuda")  # noqa: E731
        self.table = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        self.n_pages = torch.zeros(rows, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(num, dtype=torch.int32, device="cuda")
        self.ck, self.cv = full(num, P, DIM), full(num, P, DIM)
        self.wk, self.wv, self.ws = full(rows, BLOCK, DIM), full(rows, BLOCK, DIM), full(rows, BLOCK)
        self.hist = [None] * rows                 # (k, v, s) of each row in use
        self.base = Seq(60000, self.gen, "cuda")
        self.room_p = hca.paged_prefill_workspace(rows, 700, "cuda")
        self.room_d = hca.paged_decode_workspace(rows, "cuda")

    def ints(self, x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")

    def cache(self):
        return self.wk, self.wv, self.ws, self.ck, self.cv, self.table

    def length(self, i):
        return 0 if self.hist[i] is None else len(self.hist[i][0])

    def no_error(self):
        torch.cuda.synchronize()
        code, where = hca.device_error()
        assert code == 0, (code, where)

    def resize(self, lens):
        """Pages for lens[i] tokens; False if there are not enough."""
        want = [x // BLOCK for x in lens]
        hca.resize_pages(self.table, self.n_pages, self.ref, self.ints(want), self.P,
                         pools=(self.ck, self.cv))
        return self.n_pages.tolist() == [-(-e // self.P) for e in want]

    def fresh(self, n):
        at = self.r.randrange(0, (60000 - n) // 8 + 1) * 8
        return self.base.k[at:at + n], self.base.v[at:at + n], self.base.s[at:at + n]

    def feed(self, n, how):
        lens = [self.length(i) + m for i, m in enumerate(n)]
        if not self.resize(lens):
            self.resize([self.length(i) for i in range(self.rows)])
            return
        parts = [self.fresh(m) for m in n]
        for i, (m, x) in enumerate(zip(n, parts)):
            if m:
                old = self.hist[i] or tuple(y[:0] for y in x)
                self.hist[i] = tuple(torch.cat([a, b]) for a, b in zip(old, x))
        k, v, s = (torch.cat([x[j] for x in parts]) for j in range(3))
        N = sum(n)
        ctx = self.ints([max(x, 1) if how == "step" else x for x in lens])
        start = self.ints([sum(n[:i]) for i in range(self.rows + 1)])
        q, g = (torch.randn((N, HEADS, DIM), generator=self.gen, device="cuda").bfloat16()
                for _ in "qg")
        vha = None
        if self.r.random() < 0.25:
            vha = tuple((torch.randn((HEADS, self.r.randint(1, 64)), generator=self.gen,
                                     device="cuda") / 16).bfloat16() for _ in range(1)) * 2
        if how == "append":
            hca.paged_append(k, v, s, start, ctx, *self.cache())
        elif how == "step":
            out = hca.paged_decode_step(q, g, k, v, s, ctx, *self.cache(), workspace=self.room_d,
                                        vha=vha)
        else:
            given = self.room_p if N <= 700 else None
            out = hca.paged_prefill(q, g, k, v, s, start, ctx, *self.cache(), workspace=given,
                                    vha=vha)
        self.no_error()
        if how != "append":
            for i, m in enumerate(n):
                for t in {0, m - 1, self.r.randrange(m), self.r.randrange(m)} if m else ():
                    at = sum(n[:i]) + t
                    ek, ev = self.stored(i)
                    ref, bound = attend64(q[at], g[at], ek, ev, self.hist[i][0], self.hist[i][1],
                                          lens[i] - m + t, vha)
                    assert ((out[at].double() - ref).abs() <= bound).all(), (how, n, i, t, lens[i])

    def stored(self, i):
        e = self.length(i) // BLOCK
        pages = self.table[i, :-(-e // self.P)].long()
        return self.ck[pages].reshape(-1, DIM)[:e], self.cv[pages].reshape(-1, DIM)[:e]

    def check(self):
        for i in range(self.rows):
            L = self.length(i)
            if not L:
                continue
            k, v, s = self.hist[i]
            slots = torch.arange(max(0, L - BLOCK), L, device="cuda")
            for ring, x in ((self.wk, k), (self.wv, v), (self.ws, s)):
                assert torch.equal(ring[i][slots % BLOCK], x[slots]), i
            if L >= BLOCK:
                want = hca.compress(k[None], v[None], s[None])
                got = self.stored(i)
                assert torch.equal(got[0], want[0][0]) and torch.equal(got[1], want[1][0]), i
        named = torch.zeros_like(self.ref)
        for i in range(self.rows):
            p = self.table[i, :int(self.n_pages[i])].long()
            named.index_add_(0, p, torch.ones_like(p, dtype=torch.int32))
        assert torch.equal(named, self.ref)

    def fork(self):
        live = [i for i in range(self.rows) if self.length(i)]
        empty = [i for i in range(self.rows) if not self.length(i)]
        if not live or not empty:
            return
        n = self.r.randint(1, len(empty))
        a, b = [self.r.choice(live) for _ in range(n)], self.r.sample(empty, n)
        ok = hca.fork_pages(self.table, self.n_pages, self.ref, self.ints(a), self.ints(b),
                            self.ints([self.length(x) // BLOCK for x in a]), (self.ck, self.cv),
                            self.P, rings=(self.wk, self.wv, self.ws))
        for x, y, good in zip(a, b, ok.tolist()):
            if good:
                self.hist[y] = self.hist[x]

    def back(self):
        """Some rows return to an earlier token (the caller sets their rings)."""
        lens = [self.length(i) for i in range(self.rows)]
        rows = [i for i in range(self.rows) if lens[i] and self.r.random() < 0.4]
        if len(self.ref) - int((self.ref > 0).sum()) < len(rows):
            return                                 # each may need a page
        for i in rows:
            lens[i] = self.r.randint(1, lens[i])
            self.hist[i] = tuple(x[:lens[i]] for x in self.hist[i])
            slots = torch.arange(max(0, lens[i] - BLOCK), lens[i], device="cuda")
            for ring, x in zip((self.wk, self.wv, self.ws), self.hist[i]):
                ring[i] = NAN
                ring[i][slots % BLOCK] = x[slots]
        assert self.resize(lens)

    def run(self, steps):
        for _ in range(steps):
            what = self.r.choice(["step", "step", "chunk", "chunk", "draft", "append", "fork", "back",
                                  "end", "compact"])
            room = [self.limit - self.length(i) for i in range(self.rows)]
            if what == "step":
                if min(room) > 0:
                    self.feed([1] * self.rows, "step")
            elif what in ("chunk", "append", "draft"):
                top = 12 if what == "draft" else 700
                n = [self.r.choice([0, 0, 1, self.r.randint(1, top), 128]) for _ in range(self.rows)]
                n = [min(m, x) for m, x in zip(n, room)]
                if sum(n):
                    self.feed(n, "append" if what == "append" else "chunk")
            elif what == "fork":
                self.fork()
            elif what == "back":
                self.back()
            elif what == "end":
                for i in range(self.rows):
                    if self.r.random() < 0.3:
                        self.hist[i] = None
                assert self.resize([self.length(i) for i in range(self.rows)])
            else:
                live = int(hca.compact_pages(self.table, self.n_pages, self.ref, (self.ck, self.cv)))
                self.ck[live:], self.cv[live:] = NAN, NAN
            self.no_error()
            self.check()


@pytest.mark.parametrize("seed,rows,P,num,width", [(1, 3, 16, 9, 4), (2, 8, 16, 40, 5),
                                                   (3, 20, 32, 60, 4), (4, 5, 64, 12, 3),
                                                   (5, 6, 128, 14, 2), (6, 70, 16, 150, 2)])
def test_random_runs(seed, rows, P, num, width):
    need_gpu()
    Server(seed, rows, P, num, width).run(25)
