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
