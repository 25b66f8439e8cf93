"""The paged cache against plain 64-bit models (tests/paged_ref.py): appends,
chunks, single tokens, and runs of them as a server makes them.  Storage that
belongs to no token of a sequence is filled with NaN throughout."""
import numpy as np
import pytest
import torch

import compressed_sliding_window_b200 as hca
from oracle import hca_oracle as O
from tests.gpu_util import need_gpu, to64
from tests.paged_ref import (BLOCK, DIM, HEADS, Pages, Seq, attend64, entries64, pages_for,
                             visible)

pytestmark = pytest.mark.gpu
NAN = float("nan")


class Cache:
    """Sequences in a paged cache whose unused storage is NaN; the pages of the
    rows are scattered over the pool, the table is a view with wide rows."""

    def __init__(self, seqs, lens, P, seed=0, room=0, extra=3):
        dev = seqs[0].k.device
        self.P, self.lens, self.seqs = P, list(lens), seqs
        counts = [pages_for(L + room, P) for L in lens]
        total = sum(counts) + extra
        order = torch.randperm(total, generator=torch.Generator().manual_seed(seed)).tolist()
        width = max(counts) + 1
        wide = torch.full((len(seqs), width + 5), -7, dtype=torch.int32, device=dev)
        self.table = wide[:, :width]
        self.ck = torch.full((total, P, DIM), NAN, dtype=torch.bfloat16, device=dev)
        self.cv = self.ck.clone()
        at = 0
        for i, c in enumerate(counts):
            self.table[i, :c] = torch.tensor(order[at:at + c], dtype=torch.int32, device=dev)
            at += c
        for i, (s, L) in enumerate(zip(seqs, lens)):
            if L >= BLOCK:
                ek, ev = hca.compress(s.k[None, :L], s.v[None, :L], s.s[None, :L])
                for j in range(L // BLOCK):
                    p = int(self.table[i, j // P])
                    self.ck[p, j % P], self.cv[p, j % P] = ek[0, j], ev[0, j]
        self.wk = torch.stack([s.ring(s.k, L, NAN) for s, L in zip(seqs, lens)])
        self.wv = torch.stack([s.ring(s.v, L, NAN) for s, L in zip(seqs, lens)])
        self.ws = torch.stack([s.ring(s.s, L, NAN) for s, L in zip(seqs, lens)])

    def args(self):
        return self.wk, self.wv, self.ws, self.ck, self.cv, self.table

    def chunk(self, n):
        """Inputs of the next n[i] tokens of each sequence (advances the lengths)."""
        dev = self.wk.device
        take = lambda x: torch.cat([getattr(s, x)[L:L + m] for s, L, m in zip(self.seqs, self.lens, n)])  # noqa: E731
        k, v, s = take("k"), take("v"), take("s")
        self.lens = [L + m for L, m in zip(self.lens, n)]
        start = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=dev)
        return k, v, s, start, torch.tensor(self.lens, dtype=torch.int32, device=dev)

    def stored(self, i):
        """Entries of sequence i as the pool holds them."""
        e = self.lens[i] // BLOCK
        pages = self.table[i, :pages_for(self.lens[i], self.P)].long()
        return (self.ck[pages].reshape(-1, DIM)[:e], self.cv[pages].reshape(-1, DIM)[:e])

    def check_state(self):
        """Rings exactly, entries bit-identical to the whole-sequence compressor, the rest of
        the pool untouched."""
        used = torch.zeros(self.ck.shape[:2], dtype=torch.bool, device=self.ck.device)
        for i, (s, L) in enumerate(zip(self.seqs, self.lens)):
            for ring, x in ((self.wk, s.k), (self.wv, s.v), (self.ws, s.s)):
                assert torch.equal(ring[i].nan_to_num(7.0), s.ring(x, L, 7.0)), f"ring {i}"
            e = L // BLOCK
            if e:
                ek, ev = hca.compress(s.k[None, :L], s.v[None, :L], s.s[None, :L])
                gk, gv = self.stored(i)
                assert torch.equal(gk, ek[0]) and torch.equal(gv, ev[0]), f"entries {i}"
                j = torch.arange(e, device=used.device)
                used[self.table[i, j // self.P].long(), j % self.P] = True
        assert self.ck[~used].isnan().all() and self.cv[~used].isnan().all()

    def check_out(self, out, q, g, n, vha=None, picks=None):
        at = 0
        for i, m in enumerate(n):
            s, L = self.seqs[i], self.lens[i]
            ek, ev = self.stored(i)
            rows = range(m) if picks is None else [r for r in picks if r < m]
            for r in rows:
                ref, bound = attend64(q[at + r], g[at + r], ek, ev, s.k, s.v, L - m + r, vha)
                far = (out[at + r].double() - ref).abs()
                assert torch.isfinite(out[at + r]).all(), f"sequence {i} token {r}"
                assert (far <= bound).all(), \
                    f"sequence {i} token {r}: {(far / bound).max().item():.3f} of the bound"
            at += m


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _qg(N, gen):
    f = lambda: torch.randn((N, HEADS, DIM), generator=gen, device="cuda").bfloat16()  # noqa: E731
    return f(), f()


def _no_error():
    torch.cuda.synchronize()
    code, where = hca.device_error()
    assert code == 0, f"device error {code} at {where}"


def test_model_agrees_with_the_oracle():
    """The 64-bit model is the oracle's prefill, entry rounding apart (bf16 2^-8)."""
    need_gpu()
    gen = _gen(1)
    s = Seq(400, gen, "cuda")
    q, g = _qg(400, gen)
    ref = O.prefill_forward(to64(q)[None], to64(s.k)[None], to64(s.v)[None], to64(s.s)[None],
                            to64(g)[None])
    ek, ev = entries64(s.k, s.v, s.s)
    for t in (0, 5, 127, 128, 254, 255, 256, 383, 399):
        out, _ = attend64(q[t], g[t], ek, ev, s.k, s.v, t)
        assert np.abs(out.cpu().numpy() - ref[0, t]).max() < 1e-12


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_append_pieces_make_the_whole(P):
    """Ragged pieces, one token to several blocks, some sequences resting."""
    need_gpu()
    gen = _gen(P)
    pieces = [[1, 0, 128, 300, 5, 127], [0, 640, 1, 2, 129, 1], [130, 1, 126, 0, 1000, 128],
              [1, 1, 1, 1, 1, 1]]
    L0 = [0, 0, 127, 128, 1000, 4095]
    room = 2600
    seqs = [Seq(L + room, gen, "cuda") for L in L0]
    c = Cache(seqs, L0, P, seed=P, room=room)
    for n in pieces:
        k, v, s, start, ctx = c.chunk(n)
        hca.paged_append(k, v, s, start, ctx, *c.args())
        _no_error()
        c.check_state()
    for _ in range(3):   # one token each, without offsets
        k, v, s, start, ctx = c.chunk([1] * 6)
        hca.paged_append(k, v, s, None, ctx, *c.args())
        _no_error()
        c.check_state()


CHUNKS = [
    ("first tokens", [0, 0, 0], [1, 2, 127]),
    ("a first chunk over blocks", [0, 0], [300, 129]),
    ("one resting, one of one", [500, 131072 // 8, 77], [0, 1, 9]),
    ("around block borders", [127, 128, 255, 256, 383, 1151], [1, 1, 2, 130, 5, 258]),
    ("drafts on long contexts", [40000, 70001], [4, 7]),
    ("a long chunk", [2500], [700]),
]


@pytest.mark.parametrize("P", [16, 64])
@pytest.mark.parametrize("name,L0,n", CHUNKS, ids=[c[0] for c in CHUNKS])
def test_chunk_attention(name, L0, n, P):
    need_gpu()
    gen = _gen(len(name) + P)
    seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
    c = Cache(seqs, L0, P, seed=P, room=max(n))
    k, v, s, start, ctx = c.chunk(n)
    N = sum(n)
    q, g = _qg(N, gen)
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
    _no_error()
    c.check_state()
    c.check_out(out, q, g, n, picks=None if N < 400 else range(0, max(n), 3))


@pytest.mark.parametrize("P", [32, 128])
def test_chunk_of_many_tokens(P):
    """More tokens than one-query-a-CTA serves, ragged, with rows behind the last sequence."""
    need_gpu()
    gen = _gen(3)
    L0, n = [1000, 0, 20000, 5, 300], [517, 129, 803, 1, 66]
    seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
    c = Cache(seqs, L0, P, room=max(n))
    k, v, s, start, ctx = c.chunk(n)
    N, tail = sum(n), 7
    pad = lambda x: torch.cat([x, torch.full((tail,) + tuple(x.shape[1:]), NAN, dtype=x.dtype, device="cuda")])  # noqa: E731
    q, g = _qg(N, gen)
    out = torch.full((N + tail, HEADS, DIM), 3.0, dtype=torch.bfloat16, device="cuda")
    hca.paged_prefill(pad(q), pad(g), pad(k), pad(v), pad(s), start, ctx, *c.args(), out=out)
    _no_error()
    assert (out[N:] == 3.0).all()
    c.check_state()
    c.check_out(out, q, g, n, picks=[0, 1, 2, 3, 4, 5, 64, 65, 126, 127, 128, 129, 130, 255, 256,
                                     400, 512, 513, 514, 515, 516, 700, 799, 800, 801, 802])


@pytest.mark.parametrize("P", [16, 32, 64, 128])
def test_decode_step(P):
    need_gpu()
    gen = _gen(P + 50)
    L0 = [0, 1, 126, 127, 128, 254, 255, 383, 2047, 2048 * 9 + 127, 131071]
    seqs = [Seq(L + 1, gen, "cuda") for L in L0]
    c = Cache(seqs, L0, P, seed=P, room=1)
    n = [1] * len(L0)
    k, v, s, _, ctx = c.chunk(n)
    q, g = _qg(len(L0), gen)
    out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args())
    _no_error()
    c.check_state()
    c.check_out(out, q, g, n)
    # the step left the cache as the attention alone finds it
    again = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g)
    assert torch.equal(again, out)
    # a chunk of one token each is the same step
    c2 = Cache(seqs, L0, P, seed=P, room=1)
    start = torch.arange(len(L0) + 1, dtype=torch.int32, device="cuda")
    out2 = hca.paged_prefill(q, g, k, v, s, start, ctx, *c2.args())
    _no_error()
    c2.lens = c.lens
    c2.check_state()
    c2.check_out(out2, q, g, n)


FORMS = [[56], [57], [0, 40, 0, 16], [1] * 64, [2] * 37, [2] * 38, [1, 0] * 60, [1] * 127, [1] * 128,
         [0, 3, 1] * 31]


@pytest.mark.parametrize("n", FORMS, ids=[f"{sum(n)} of {len(n)}" for n in FORMS])
def test_chunks_on_both_sides_of_the_forms(n):
    """Numbers of tokens and sequences where a chunk changes from one query at a time to four
    positions at a time, on one workspace of the largest size among them."""
    need_gpu()
    gen = _gen(len(n) + sum(n))
    base = Seq(2700, gen, "cuda")
    L0 = [int(x) for x in np.random.default_rng(len(n)).integers(0, 2600, len(n))]
    L0[0] = 2600 - 2600 % 128 - 1
    c = Cache([base] * len(n), L0, 16, room=max(n), seed=len(n))
    ws = hca.paged_prefill_workspace(128, 128, "cuda")
    k, v, s, start, ctx = c.chunk(n)
    q, g = _qg(sum(n), gen)
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(), workspace=ws)
    _no_error()
    c.check_state()
    c.check_out(out, q, g, n)


SPLITS = [(1, 40, 300, 16), (1, 50000, 50000, 32), (1, 110000, 110000, 64), (3, 1000, 140000, 16),
          (9, 90000, 140000, 128), (37, 1, 33000, 16), (38, 1, 40000, 64), (74, 1, 70000, 32),
          (75, 1, 20000, 16)]


@pytest.mark.parametrize("S,lo,hi,P", SPLITS, ids=[f"{c[0]}x{c[1]}-{c[2]}" for c in SPLITS])
def test_decode_splits(S, lo, hi, P):
    """Numbers of sequences and lengths at which the work is split in other ways: whole queries,
    with 4, 2 or all column groups a CTA, and parts of queries with them."""
    need_gpu()
    gen = _gen(S + hi)
    base = Seq(hi + 2, gen, "cuda")
    L0 = [int(x) for x in np.random.default_rng(S).integers(lo, hi + 1, S)]
    L0[-1] = hi - hi % 128 - 1                      # the step completes a block
    c = Cache([base] * S, L0, P, room=2, seed=S)
    n = [1] * S
    ws = hca.paged_decode_workspace(S, "cuda")
    k, v, s, _, ctx = c.chunk(n)
    q, g = _qg(S, gen)
    out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ws)
    _no_error()
    c.check_state()
    c.check_out(out, q, g, n)
    assert torch.equal(hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g, workspace=ws), out)
    vha = tuple((torch.randn((HEADS, 5), generator=gen, device="cuda") / 8).bfloat16()
                for _ in range(2))
    k, v, s, _, ctx = c.chunk(n)                    # the entry just written becomes visible later
    out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ws, vha=vha)
    _no_error()
    c.check_state()
    c.check_out(out, q, g, n, vha)


def test_decode_many_sequences():
    """More sequences than each CTA plans for itself."""
    need_gpu()
    gen = _gen(9)
    S = 1100
    base = Seq(700, gen, "cuda")
    L0 = [int(x) for x in np.random.default_rng(2).integers(0, 699, S)]
    c = Cache([base] * S, L0, 16, room=1)
    k, v, s, _, ctx = c.chunk([1] * S)
    q, g = _qg(S, gen)
    out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args())
    _no_error()
    c.check_out(out, q, g, [1] * S)


@pytest.mark.parametrize("rank", [1, 16, 64])
def test_head_mix(rank):
    need_gpu()
    gen = _gen(rank)
    L0, n = [260, 5000, 0], [3, 1, 6]
    seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
    vha = tuple((torch.randn((HEADS, rank), generator=gen, device="cuda") / 8).bfloat16()
                for _ in range(2))
    c = Cache(seqs, L0, 32, room=8)
    k, v, s, start, ctx = c.chunk(n)
    q, g = _qg(sum(n), gen)
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(), vha=vha)
    _no_error()
    c.check_out(out, q, g, n, vha)
    last = start[1:].long() - 1
    one = hca.paged_decode(q[last].contiguous(), c.ck, c.cv, c.table, c.wk, c.wv, ctx,
                           g[last].contiguous(), vha=vha)
    _no_error()
    at = 0
    for i, m in enumerate(n):
        ek, ev = c.stored(i)
        ref, bound = attend64(q[at + m - 1], g[at + m - 1], ek, ev, seqs[i].k, seqs[i].v,
                              c.lens[i] - 1, vha)
        assert ((one[i].double() - ref).abs() <= bound).all()
        at += m


def test_many_calls_on_one_workspace_and_scaled_scores():
    """Ten steps on one workspace, chunks and single tokens in turn, sharp softmaxes."""
    need_gpu()
    gen = _gen(4)
    L0 = [900, 10, 3000, 127]
    seqs = [Seq(L + 200, gen, "cuda", scale=6.0) for L in L0]
    c = Cache(seqs, L0, 16, room=200)
    ws = hca.paged_prefill_workspace(4, 64, "cuda")
    ds = hca.paged_decode_workspace(4, "cuda")
    for step, n in enumerate([[3, 1, 16, 2], [1] * 4, [0, 40, 0, 1], [1] * 4, [20, 20, 20, 1],
                              [1] * 4, [1] * 4, [0, 0, 1, 0], [10, 1, 1, 7], [1] * 4]):
        k, v, s, start, ctx = c.chunk(n)
        q, g = _qg(sum(n), gen)
        if n == [1] * 4:
            out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ds)
        else:
            out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(), workspace=ws)
        _no_error()
        c.check_state()
        c.check_out(out, q, g, n)


def test_capture_and_replay():
    """A chunk and a step in one graph, replayed on new inputs in the same buffers, sharing
    workspaces with a second graph; on a stream of its own."""
    need_gpu()
    gen = _gen(6)
    L0, n = [250, 1300], [6, 3]
    seqs = [Seq(L + 100, gen, "cuda") for L in L0]
    stream = torch.cuda.Stream()
    ws = hca.paged_prefill_workspace(2, 9, "cuda")
    ds = hca.paged_decode_workspace(2, "cuda")
    c = Cache(seqs, L0, 16, room=100)
    first = c.chunk(n)
    second = c.chunk([1, 1])
    q, g = _qg(9, gen)
    q1, g1 = _qg(2, gen)
    buf = [x.clone() for x in first + second]

    def both():
        a = hca.paged_prefill(q, g, *buf[:5], *c.args(), workspace=ws)
        b = hca.paged_decode_step(q1, g1, *buf[5:8], buf[9], *c.args(), workspace=ds)
        return a, b

    keep = [x.clone() for x in c.args()[:5]]
    with torch.cuda.stream(stream):
        both()
        stream.synchronize()
        graphs = []
        for _ in range(2):
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                outs = both()
            graphs.append((graph, outs))
    torch.cuda.synchronize()
    for x, y in zip(c.args()[:5], keep):
        x.copy_(y)
    for graph, outs in graphs:
        graph.replay()
        torch.cuda.synchronize()
        c.check_state()
        c.check_out(outs[1], q1, g1, [1, 1])
        c.lens = [L - 1 for L in c.lens]
        c.check_out(outs[0], q, g, n)
        c.lens = [L + 1 for L in c.lens]
        for b, x in zip(buf, c.chunk(n) + c.chunk([1, 1])):
            b.copy_(x)
    del graphs
    _no_error()


def test_bad_pages_and_offsets_are_reported():
    """Pages outside of the pool read as zeros and take no entry; falling offsets are clamped."""
    need_gpu()
    gen = _gen(8)
    s = Seq(128 * 40, gen, "cuda")
    L = 128 * 40 - 1
    c = Cache([s], [L], 16, room=1)
    k, v, sc, start, ctx = c.chunk([1])
    c.table[0, 1], c.table[0, 2] = 10 ** 9, -3
    q, g = _qg(1, gen)
    before = c.ck.clone(), c.cv.clone()
    out = hca.paged_decode_step(q, g, k, v, sc, ctx, *c.args())
    torch.cuda.synchronize()
    assert hca.device_error()[0] == 5 and hca.device_error()[0] == 0
    assert torch.equal(c.ck.nan_to_num(9.0), before[0].nan_to_num(9.0))
    ek, ev = entries64(s.k, s.v, s.s)
    ek[:16], ev[:16] = c.ck[c.table[0, 0].long()].double(), c.cv[c.table[0, 0].long()].double()
    ek[16:], ev[16:] = 0, 0
    ref, bound = attend64(q[0], g[0], ek, ev, s.k, s.v, L)
    assert ((out[0].double() - ref).abs() <= bound).all()
    # offsets that fall: clamped, reported, nothing faults
    c = Cache([s, s], [300, 300], 16, room=10)
    bad = torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda")
    lens = torch.tensor([304, 300], dtype=torch.int32, device="cuda")
    q, g = _qg(4, gen)
    out = hca.paged_prefill(q, g, s.k[300:304], s.v[300:304], s.s[300:304].clone(), bad, lens,
                            *c.args())
    torch.cuda.synchronize()
    assert hca.device_error()[0] == 5
    # a context shorter than the tokens it counts
    short = torch.tensor([2, 300], dtype=torch.int32, device="cuda")
    ok = torch.tensor([0, 4, 4], dtype=torch.int32, device="cuda")
    hca.paged_append(s.k[300:304], s.v[300:304], s.s[300:304].clone(), ok, short, *c.args())
    torch.cuda.synchronize()
    assert hca.device_error()[0] == 5
    # a completed block past the table
    c = Cache([s], [127], 16)
    k, v, sc, start, ctx = c.chunk([1])
    hca.paged_append(k, v, sc, start, ctx, *c.args())
    torch.cuda.synchronize()
    assert hca.device_error()[0] == 5 and c.ck.isnan().all()


def test_agrees_with_the_contiguous_decode():
    """Same lengths, split and sums as decode on a contiguous cache; that one also rounds the
    split partials to bf16 (half a step of each), and both round the output."""
    need_gpu()
    gen = _gen(12)
    L = [131072, 5000, 1, 300, 128 * 77 + 5]
    seqs = [Seq(x, gen, "cuda") for x in L]
    c = Cache(seqs, L, 32)
    q, g = _qg(5, gen)
    nc = max(visible(x) for x in L)
    ck = torch.zeros((5, nc, DIM), dtype=torch.bfloat16, device="cuda")
    cv = torch.zeros_like(ck)
    for i, x in enumerate(L):
        e = visible(x)
        if e:
            ck[i, :e], cv[i, :e] = (t[:e] for t in c.stored(i))
    ctx = torch.tensor(L, dtype=torch.int32, device="cuda")
    a = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g)
    b = hca.decode(q, ck, cv, c.wk.nan_to_num(0.0), c.wv.nan_to_num(0.0), ctx, g)
    _no_error()
    for i, x in enumerate(L):
        ref, bound = attend64(q[i], g[i], ck[i], cv[i], seqs[i].k, seqs[i].v, x - 1)
        assert ((a[i].double() - b[i].double()).abs() <= bound).all()
