"""Plain 64-bit models of the paged cache, used by its tests.

`Seq` keeps a sequence's whole raw history; everything the paged operators are
to hold or return follows from it: entries (softmax-weighted sums over blocks),
the ring, and the attention of any position over the entries as they are
stored (bf16) and the raw window.  `Pages` is the bookkeeping, page by page."""
import math

import torch

BLOCK, DIM, HEADS = 128, 512, 64
SCALE = DIM ** -0.5


def visible(L):
    """Entries that the newest of L tokens sees."""
    return max(0, (L - 128) // 128)


def entries64(k, v, s):
    """Entries of every complete block of [T, 512] rows in 64 bits."""
    nb = k.shape[0] // BLOCK
    w = torch.softmax(s[:nb * BLOCK].double().view(nb, BLOCK), 1)
    f = lambda x: torch.einsum("bi,bid->bd", w, x[:nb * BLOCK].double().view(nb, BLOCK, DIM))  # noqa: E731
    return f(k), f(v)


def attend64(q, g, ek, ev, k, v, t, vha=None):
    """One position t: q, g [64, 512]; stored entries ek, ev; raw history k, v.

    Returns (out, bound): the output and, per element, how far a kernel may be
    from it.  With a = sum p |v| the result o carries at most half a step of
    bf16 (2^-8) on each probability, the same once more where splits are joined
    (their partial results are held in bf16), both times the gate; the output
    is rounded once (2^-8 of itself); the gate's own approximation is below
    2^-11 of a.  Half a step more covers the 32-bit scores, exponentials and
    sums (below 2^-12 for the magnitudes used here)."""
    nc = max(0, (t - 127) // 128)
    lo = max(0, t - 127)
    keys = torch.cat([ek[:nc], k[lo:t + 1]]).double()
    vals = torch.cat([ev[:nc], v[lo:t + 1]]).double()
    p = torch.softmax(q.double() @ keys.T * SCALE, 1)
    o, a = p @ vals, p @ vals.abs()
    gate = torch.sigmoid(g.double())
    out = gate * o
    bound = out.abs() * 2 ** -8 + a * (gate * 2.5 * 2 ** -8 + 2 ** -11)
    if vha is not None:
        # y = x + up down^T x on x rounded to bf16; up down^T rounded to bf16 in one of
        # the two forms (half a step of each term), the sums in 32 bits
        m = vha[1].double() @ vha[0].double().T
        y = out + m @ out
        spread = (vha[1].double().abs() @ vha[0].double().abs().T) @ out.abs()
        bound = bound + m.abs() @ bound + (out.abs() + spread) * 2 ** -8 + y.abs() * 2 ** -8
        out = y
    return out, bound


class Seq:
    """A sequence's raw history (bf16 rows on a device) and its length."""

    def __init__(self, T, gen, device, scale=1.0):
        r = lambda *s: torch.randn(s, generator=gen, device=device).bfloat16()  # noqa: E731
        self.k, self.v, self.s = (r(T, DIM) * scale).bfloat16(), r(T, DIM), r(T)

    def ring(self, x, L, fill):
        """Ring of the first L tokens of x; slots without a token hold `fill`."""
        out = torch.full((BLOCK,) + tuple(x.shape[1:]), fill, dtype=x.dtype, device=x.device)
        p = torch.arange(max(0, L - BLOCK), L, device=x.device)
        out[p % BLOCK] = x[p]
        return out


class Pages:
    """The page bookkeeping in plain Python."""

    def __init__(self, table, n_pages, ref, P):
        self.rows = [list(r[:n]) for r, n in zip(table, n_pages)]
        self.width, self.ref, self.P = len(table[0]), list(ref), P

    def free(self):
        return [p for p, c in enumerate(self.ref) if c <= 0]

    def resize(self, entries):
        want = [len(r) if e < 0 else min(self.width, -(-e // self.P))
                for r, e in zip(self.rows, entries)]
        for r, w in zip(self.rows, want):
            for p in r[w:]:
                self.ref[p] -= 1
            del r[w:]
        free = self.free()
        for r, w in zip(self.rows, want):
            while len(r) < w and free:
                r.append(free.pop(0))
                self.ref[r[-1]] = 1

    def fork(self, parents, children, entries):
        """(ok, page copies, row copies)."""
        empty = [not r for r in self.rows]
        n = len(self.rows)
        good = []
        for i, (a, b, e) in enumerate(zip(parents, children, entries)):
            good.append(0 <= a < n and 0 <= b < n and e >= 0 and empty[b] and b not in parents
                        and b not in children[:i] and -(-e // self.P) <= len(self.rows[a]))
        free = self.free()
        ok, pages, rows = [], [], []
        for a, b, e, fine in zip(parents, children, entries, good):
            if fine and e % self.P and not free:
                fine = False
            ok.append(int(fine))
            if not fine:
                continue
            full = e // self.P
            self.rows[b] = self.rows[a][:full]
            for p in self.rows[b]:
                self.ref[p] += 1
            if e % self.P:
                new = free.pop(0)
                pages.append((self.rows[a][full], new))
                self.rows[b].append(new)
                self.ref[new] = 1
            rows.append((a, b))
        return ok, pages, rows

    def compact(self):
        """Page moves (from, to)."""
        used = [p for p, c in enumerate(self.ref) if c > 0]
        live = len(used)
        holes = [p for p in range(live) if self.ref[p] <= 0]
        moves = list(zip([p for p in used if p >= live], holes))
        to = dict(moves)
        self.rows = [[to.get(p, p) for p in r] for r in self.rows]
        for a, b in moves:
            self.ref[b], self.ref[a] = self.ref[a], 0
        return moves

    def table(self):
        return [r + [-1] * (self.width - len(r)) for r in self.rows]


def pages_for(L, P):
    return math.ceil((L // BLOCK) / P)
