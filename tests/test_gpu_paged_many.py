"""Ragged batches of many sequences: appends and chunks whose sequences are found among hundreds
and thousands of offsets."""
import numpy as np
import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK
from tests.test_gpu_paged import Cache, _gen, _no_error, _qg
from tests.test_gpu_paged_steps import _windows

pytestmark = pytest.mark.gpu


def _tokens(S, rng):
    """Mostly a token or two, some none, a few blocks of them."""
    n = rng.integers(0, 3, S)
    n[rng.integers(0, S, max(1, S // 20))] = rng.integers(1, 300, max(1, S // 20))
    n[: S // 8] = 0                                     # a run of resting ones in front
    return [int(x) for x in n]


@pytest.mark.parametrize("S", [127, 128, 129, 300, 1025, 4096])
def test_appends_and_chunks(S):
    need_gpu()
    gen, rng = _gen(S), np.random.default_rng(S)
    L0 = [int(x) for x in rng.integers(0, 700, S)]
    seqs = _windows(S, 700 + 3 * 300, gen)
    c = Cache(seqs, L0, 16, room=900, seed=S)
    for attend in (False, True, False):
        n = _tokens(S, rng)
        k, v, s, start, ctx = c.chunk(n)
        if not attend:
            hca.paged_append(k, v, s, start, ctx, *c.args())
            _no_error()
            c.check_state()
            continue
        q, g = _qg(sum(n), gen)
        out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
        _no_error()
        c.check_state()
        c.check_out(out, q, g, n, picks=[0, 1, 3, 4, 130, 255])
    if S > 1025:
        return
    k, v, s, start, ctx = c.chunk([1] * S)              # without offsets
    hca.paged_append(k, v, s, None, ctx, *c.args())
    _no_error()
    c.check_state()


def test_append_to_more_sequences_than_a_chunk_takes():
    """The append has no limit of 4096 sequences."""
    need_gpu()
    S, gen = 6000, _gen(1)
    L0 = [(7 * i) % 255 for i in range(S)]
    seqs = _windows(S, 258, gen)
    c = Cache(seqs, L0, 16, room=3)
    k, v, s, start, ctx = c.chunk([i % 3 for i in range(S)])
    hca.paged_append(k, v, s, start, ctx, *c.args())
    _no_error()
    c.check_state()
    assert sum(L // BLOCK > L1 // BLOCK for L, L1 in zip(c.lens, L0)) > 20
