"""Serving steps of many sequences: blocks that many of them complete at once, work that is cut
in every way over the CTAs, and the state that each step leaves."""
import numpy as np
import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK, Seq
from tests.test_gpu_paged import Cache, _gen, _no_error, _qg

pytestmark = pytest.mark.gpu


def _windows(S, T, gen):
    """S sequences of T tokens that share storage but not their tokens."""
    base = Seq(T + 8 * (S - 1), gen, "cuda")
    out = []
    for i in range(S):
        s = Seq.__new__(Seq)
        s.k, s.v, s.s = (x[8 * i:8 * i + T] for x in (base.k, base.v, base.s))
        out.append(s)
    return out


@pytest.mark.parametrize("S", [16, 64, 200, 512, 1100])
def test_every_sequence_completes_a_block(S):
    """Each step completes a block of every sequence (with up to 512 of them inside the attention
    kernel, several to a CTA): outputs, rings and all entries, bit for bit."""
    need_gpu()
    gen = _gen(S)
    steps = 2
    L0 = [BLOCK * int(x) - 1 for x in np.random.default_rng(S).integers(1, 9, S)]
    L0[0], L0[-1] = BLOCK - 1, BLOCK * 20 - 1
    seqs = _windows(S, max(L0) + 1 + BLOCK * steps, gen)
    c = Cache(seqs, L0, 16, room=1 + BLOCK * steps, seed=S)
    ws = hca.paged_decode_workspace(S, "cuda")
    n = [1] * S
    for step in range(steps):
        if step:
            k, v, s, start, ctx = c.chunk([BLOCK - 1] * S)
            hca.paged_append(k, v, s, start, ctx, *c.args())
        k, v, s, _, ctx = c.chunk(n)
        assert (ctx % BLOCK == 0).all()
        q, g = _qg(S, gen)
        out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ws)
        _no_error()
        c.check_state()
        c.check_out(out, q, g, n)


def _long_among_short(S, rng):
    L = [300] * S
    L[S // 3], L[-1] = 200000, 90000 - 90000 % BLOCK - 1
    return L


def _mixed(S, rng):
    return [int(x) for x in np.exp(rng.uniform(0, np.log(20000), S))]


# with 148 CTAs: parts of queries below, all tiles cut evenly from 148 on where lengths differ;
# above 512 the plan is a kernel of its own and the append another
CUTS = [(147, _long_among_short), (150, _long_among_short), (150, _mixed), (200, _mixed),
        (512, _long_among_short), (512, _mixed), (513, _mixed), (700, _long_among_short)]


@pytest.mark.parametrize("rank", [0, 7])
@pytest.mark.parametrize("S,lens", CUTS, ids=[f"{c[0]}{c[1].__name__}" for c in CUTS])
def test_unequal_lengths(S, lens, rank):
    """Steps of many sequences of unequal lengths on one workspace: outputs, state, the same bits
    from the attention alone and from every repetition."""
    need_gpu()
    gen = _gen(S + rank)
    L0 = lens(S, np.random.default_rng(S + 1))
    L0[5] = BLOCK * 7 - 1                               # the first step completes a block
    seqs = _windows(S, max(L0) + 3, gen)
    c = Cache(seqs, L0, 32, room=3, seed=S)
    ws = hca.paged_decode_workspace(S, "cuda")
    vha = tuple((torch.randn((64, rank), generator=gen, device="cuda") / 8).bfloat16()
                for _ in range(2)) if rank else None
    n = [1] * S
    for step in range(2):
        k, v, s, _, ctx = c.chunk(n)
        q, g = _qg(S, gen)
        out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ws, vha=vha)
        _no_error()
        c.check_state()
        c.check_out(out, q, g, n, vha)
        for _ in range(3):
            again = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g, workspace=ws,
                                     vha=vha)
            assert torch.equal(again, out)
    _no_error()


def test_even_cut_in_a_graph():
    """Captured and replayed on new tokens, in turn with a call outside of the graph on the same
    workspace."""
    need_gpu()
    S, gen = 170, _gen(5)
    L0 = _long_among_short(S, None)
    seqs = _windows(S, max(L0) + 8, gen)
    c = Cache(seqs, L0, 16, room=8)
    ws = hca.paged_decode_workspace(S, "cuda")
    n = [1] * S
    take = lambda: [x for j, x in enumerate(c.chunk(n)) if j != 3]  # noqa: E731
    buf = take()
    q, g = _qg(S, gen)
    hca.paged_decode_step(q, g, *buf, *c.args(), workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = hca.paged_decode_step(q, g, *buf, *c.args(), workspace=ws)
    for _ in range(3):
        for b, x in zip(buf, take()):
            b.copy_(x)
        graph.replay()
        _no_error()
        c.check_state()
        c.check_out(out, q, g, n)
        assert torch.equal(hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, buf[3], g,
                                            workspace=ws), out)
    del graph
