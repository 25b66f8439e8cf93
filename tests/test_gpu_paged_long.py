"""Contexts of millions of tokens: a query split over more CTAs than one batch of the merge takes,
alone, beside others, and where the tiles of all queries are cut evenly."""
import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK, DIM, Seq, pages_for
from tests.test_gpu_paged import NAN, Cache, _gen, _no_error, _qg

pytestmark = pytest.mark.gpu


class LongCache(Cache):
    """Cache, its pages in ascending order and filled a sequence at a time."""

    def __init__(self, seqs, lens, P, room):
        dev = seqs[0].k.device
        self.P, self.lens, self.seqs = P, list(lens), seqs
        counts = [pages_for(L + room, P) for L in lens]
        self.table = torch.full((len(seqs), max(counts) + 1), -1, dtype=torch.int32, device=dev)
        self.ck = torch.full((sum(counts) + 1, P, DIM), NAN, dtype=torch.bfloat16, device=dev)
        self.cv = self.ck.clone()
        at = 0
        for i, (s, L, m) in enumerate(zip(seqs, lens, counts)):
            self.table[i, :m] = torch.arange(at, at + m, device=dev, dtype=torch.int32)
            if L >= BLOCK:
                for pool, x in zip((self.ck, self.cv), hca.compress(s.k[None, :L], s.v[None, :L],
                                                                    s.s[None, :L])):
                    pool[at:at + m].view(-1, DIM)[:L // BLOCK] = x[0]
            at += m
        self.wk, self.wv, self.ws = (
            torch.stack([s.ring(getattr(s, f), L, NAN) for s, L in zip(seqs, lens)]) for f in "kvs")


# 16384 tokens a tile of 128 entries
LONG = [[1_100_000], [2_200_000], [4_000_000], [1_500_000, 300], [2_500_000, 1_200_000, 5],
        [300] * 149 + [6_000_000]]


@pytest.mark.parametrize("rank", [0, 3])
@pytest.mark.parametrize("L0", LONG, ids=[f"{len(x)} to {max(x)}" for x in LONG])
def test_single_tokens(L0, rank):
    need_gpu()
    S, gen = len(L0), _gen(len(L0) + rank)
    base = Seq(max(L0) + 2, gen, "cuda")
    c = LongCache([base] * S, L0, 128, 2)
    ws = hca.paged_decode_workspace(S, "cuda")
    vha = tuple((torch.randn((64, rank), generator=gen, device="cuda") / 8).bfloat16()
                for _ in range(2)) if rank else None
    n = [1] * S
    for _ in range(2):
        k, v, s, _, ctx = c.chunk(n)
        q, g = _qg(S, gen)
        out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ws, vha=vha)
        _no_error()
        c.check_out(out, q, g, n, vha)
        again = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g, workspace=ws, vha=vha)
        assert torch.equal(again, out)
    c.check_state()


@pytest.mark.parametrize("n", [[3], [60], [2, 1]])
def test_chunks(n):
    need_gpu()
    gen = _gen(sum(n))
    L0 = [2_200_000, 1_100_000][:len(n)]
    base = Seq(max(L0) + max(n), gen, "cuda")
    c = LongCache([base] * len(n), L0, 64, max(n))
    k, v, s, start, ctx = c.chunk(n)
    q, g = _qg(sum(n), gen)
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
    _no_error()
    c.check_state()
    c.check_out(out, q, g, n, picks=[0, 1, 2, 33, 59])
