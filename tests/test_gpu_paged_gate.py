"""Gates that are nearly shut: the gate is exact relative to itself, however a query's work is
split, so a channel that the model closes stays closed.

With a = sum p |v|, the result before the gate carries half a step of bf16 on each probability
(2^-8) and 32-bit scores, exponentials, sums and merges (below 2^-11 for these magnitudes); the
gate is a 32-bit 1 / (1 + exp(-g)) (exponential and division, below 2^-19 of itself up to
|g| = 12); the output is rounded once (2^-8)."""
import numpy as np
import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import HEADS, SCALE, Seq
from tests.test_gpu_paged import Cache, _gen, _no_error, _qg

pytestmark = pytest.mark.gpu


def check_gated(c, out, q, g, n):
    """Outputs of the last n[i] tokens of each sequence, relative to the gate."""
    at = 0
    for i, m in enumerate(n):
        s, L = c.seqs[i], c.lens[i]
        ek, ev = c.stored(i)
        for t in range(L - m, L):
            nc, lo = max(0, (t - 127) // 128), max(0, t - 127)
            keys = torch.cat([ek[:nc], s.k[lo:t + 1]]).double()
            vals = torch.cat([ev[:nc], s.v[lo:t + 1]]).double()
            p = torch.softmax(q[at].double() @ keys.T * SCALE, 1)
            gate = torch.sigmoid(g[at].double())
            ref = gate * (p @ vals)
            bound = ref.abs() * 2 ** -8 + gate * (p @ vals.abs()) * (2 ** -8 + 2 ** -11)
            far = ((out[at].double() - ref).abs() / bound).max().item()
            assert far <= 1, f"sequence {i} position {t}: {far:.2f} of the bound"
            at += 1


def _gates(N, gen):
    """bf16 gates from -12 to 12, most of them shut."""
    g = torch.rand((N, HEADS, 512), generator=gen, device="cuda") * 8 - 12
    g[:, ::16] *= -1
    return g.bfloat16()


# sequences, shortest and longest: whole queries in four, two and one column groups; parts of a
# query with and without column groups; an even cut of unequal queries
SPLITS = [(1, 300, 300), (70, 100, 400), (200, 200, 400), (1, 50000, 50000), (9, 90000, 140000),
          (150, 300, 60000)]


@pytest.mark.parametrize("S,lo,hi", SPLITS, ids=[f"{c[0]}x{c[1]}-{c[2]}" for c in SPLITS])
def test_single_tokens(S, lo, hi):
    need_gpu()
    gen = _gen(S + hi)
    base = Seq(hi, gen, "cuda")
    L0 = [int(x) for x in np.random.default_rng(S).integers(lo, hi + 1, S)]
    L0[-1] = hi
    if S == 150:                      # few long ones among short ones
        L0[:140] = [lo] * 140
    c = Cache([base] * S, L0, 64, seed=S)
    ctx = torch.tensor(L0, dtype=torch.int32, device="cuda")
    q, g = _qg(S, gen)[0], _gates(S, gen)
    out = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g)
    _no_error()
    check_gated(c, out, q, g, [1] * S)


@pytest.mark.parametrize("L0,n", [([40000, 300], [4, 3]), ([700, 0, 20000], [30, 20, 6])],
                         ids=["drafts", "56 tokens"])
def test_chunks_one_query_at_a_time(L0, n):
    need_gpu()
    gen = _gen(sum(n))
    seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
    c = Cache(seqs, L0, 32, room=max(n))
    k, v, s, start, ctx = c.chunk(n)
    q, g = _qg(sum(n), gen)[0], _gates(sum(n), gen)
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
    _no_error()
    check_gated(c, out, q, g, n)


@pytest.mark.parametrize("L0,n", [([300], [60]), ([700, 0, 5000, 129], [100, 3, 57, 1])],
                         ids=["60 tokens", "ragged"])
def test_chunks_four_positions_at_a_time(L0, n):
    need_gpu()
    gen = _gen(sum(n))
    seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
    c = Cache(seqs, L0, 32, room=max(n))
    k, v, s, start, ctx = c.chunk(n)
    q, g = _qg(sum(n), gen)[0], _gates(sum(n), gen)
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
    _no_error()
    check_gated(c, out, q, g, n)


ALL = torch.arange(-(1 << 15), 1 << 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
GATES = torch.where(ALL.isnan(), torch.zeros_like(ALL), ALL)      # every gate, infinities included


def _flat(L, gen):
    """A history whose every key gives the score 0 and whose values are 1: before the gate every
    output is exactly 1 (up to 2^-23 for 1 / l), in any form."""
    s = Seq(L, gen, "cuda")
    s.k.zero_()
    s.v.fill_(1.0)
    return s


def _every_gate(out, first):
    """Rows of `out` hold the gates from pattern 32768 * first on, row after row."""
    g = GATES.cuda().view(2, HEADS, 512)
    for i in range(out.shape[0]):
        gate = torch.sigmoid(g[(first + i) % 2].double())
        far = (out[i].double() - gate).abs()
        bound = gate * (2 ** -8 + 2 ** -11) + 2 ** -126      # rounded once; tiny ones may be 0
        bad = far > bound
        assert not bad.any(), (i, g[(first + i) % 2][bad][:8], out[i][bad][:8])


# lengths: alone; whole queries; in parts; in parts by column groups; cut evenly
FLAT = [[1, 1], [300] * 70, [200] * 200, [50000] * 2, [120000] * 9, [300] * 140 + [50000] * 10]


@pytest.mark.parametrize("L", FLAT, ids=[f"{len(x)} to {max(x)}" for x in FLAT])
def test_every_gate_of_single_tokens(L):
    need_gpu()
    base = _flat(max(L), _gen(1))
    S = len(L)
    c = Cache([base] * S, L, 64)
    q = _qg(S, _gen(2))[0]
    g = GATES.cuda().view(2, HEADS, 512).repeat((S + 1) // 2, 1, 1)[:S].contiguous()
    ctx = torch.tensor(L, dtype=torch.int32, device="cuda")
    out = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g)
    _no_error()
    _every_gate(out, 0)


@pytest.mark.parametrize("n", [[1, 3], [2] * 64, [300, 0, 51]], ids=["4", "128", "351"])
def test_every_gate_of_chunks(n):
    need_gpu()
    S, N = len(n), sum(n)
    base = _flat(2000, _gen(3))
    c = Cache([base] * S, [1000] * S, 32, room=max(n))
    k, v, s, start, ctx = c.chunk(n)
    q = _qg(N, _gen(4))[0]
    g = GATES.cuda().view(2, HEADS, 512).repeat((N + 1) // 2, 1, 1)[:N].contiguous()
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
    _no_error()
    _every_gate(out, 0)
