"""Paged cache and pages at their edges: both bindings, padded batches, shared and oversized
workspaces, streams at the same time, pools past 32-bit offsets, values that no softmax likes."""
import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import BLOCK, DIM, HEADS, Seq, attend64
from tests.test_gpu_paged import NAN, Cache, _gen, _no_error, _qg

pytestmark = pytest.mark.gpu


class _Refuse:
    """A compiled module that leaves every call to the checks behind it."""

    def __getattr__(self, name):
        return lambda *a: False


def _run_all(seed):
    """Chunks in both forms, steps, branches and compaction; every result in order."""
    gen = _gen(seed)
    L0 = [300, 0, 4000]
    seqs = [Seq(L + 200, gen, "cuda") for L in L0]
    c = Cache(seqs, L0, 16, room=200)
    out = []
    for n in ([3, 5, 1], [60, 1, 30]):
        k, v, s, start, ctx = c.chunk(n)
        q, g = _qg(sum(n), gen)
        ws = hca.paged_prefill_workspace(3, sum(n), "cuda")
        out.append(hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(), workspace=ws))
    k, v, s, start, ctx = c.chunk([40, 2, 0])
    hca.paged_append(k, v, s, start, ctx, *c.args())
    k, v, s, _, ctx = c.chunk([1, 1, 1])
    q, g = _qg(3, gen)
    ws = hca.paged_decode_workspace(3, "cuda")
    out.append(hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), workspace=ws, scale=0.05))
    out.append(hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g, workspace=ws,
                                out=torch.empty_like(q)))
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table, count, ref = torch.full((4, 6), -1, dtype=torch.int32, device="cuda"), ints(0, 0, 0, 0), \
        torch.zeros(len(c.ck), dtype=torch.int32, device="cuda")
    hca.resize_pages(table, count, ref, ints(20, 0, 33, 0), 16)
    out.append(hca.fork_pages(table, count, ref, ints(0), ints(1), ints(18), [c.ck, c.cv], 16))
    hca.resize_pages(table, count, ref, ints(0, -1, -1, -1), 16)
    out.append(hca.compact_pages(table, count, ref, [c.ck, c.cv]))
    _no_error()
    return out + [table, count, ref] + [x.nan_to_num(3.0) for x in (c.ck, c.cv, c.wk, c.wv, c.ws)]


def test_both_bindings_give_the_same(monkeypatch):
    need_gpu()
    a = _run_all(21)
    monkeypatch.setattr(hca, "_CALLS", _Refuse())
    b = _run_all(21)
    assert len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


def test_wrong_tensors_are_refused_on_the_device():
    need_gpu()
    gen = _gen(1)
    seqs = [Seq(400, gen, "cuda"), Seq(300, gen, "cuda")]
    c = Cache(seqs, [300, 200], 16, room=20)
    k, v, s, start, ctx = c.chunk([2, 3])
    q, g = _qg(5, gen)
    ws = hca.paged_prefill_workspace(2, 5, "cuda")
    good = dict(q=q, g=g, k_new=k, v_new=v, s_new=s, q_start=start, ctx_len=ctx, wk=c.wk, wv=c.wv,
                ws=c.ws, ck_pages=c.ck, cv_pages=c.cv, page_table=c.table, workspace=ws)
    state = [x.clone() for x in c.args()]
    wide = torch.empty(5, HEADS, 2 * DIM, dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=q.float()), dict(g=g[:4]), dict(q=wide[:, :, :DIM]), dict(k_new=k[:, :256]),
                dict(v_new=v[:4]), dict(s_new=s.float()), dict(q_start=start.long()),
                dict(q_start=None), dict(ctx_len=ctx.cpu()), dict(wk=c.wk[:1]), dict(ws=c.ws.T),
                dict(ck_pages=c.ck[:, :8]), dict(cv_pages=c.cv[:1]), dict(page_table=c.table[:1]),
                dict(page_table=c.table.long()), dict(out=q[:4]), dict(out=q.cpu()),
                dict(vha=(q, g))):
        with pytest.raises((ValueError, TypeError)):
            hca.paged_prefill(**{**good, **bad})
    for bad, code in ((dict(scale=-1.0), 1), (dict(workspace=ws[:-1].clone()), 1),
                      (dict(workspace=ws[16:]), 1), (dict(scale=float("nan")), 1)):
        with pytest.raises(hca.HCAError) as e:
            hca.paged_prefill(**{**good, **bad})
        assert e.value.code == code
    torch.cuda.synchronize()
    assert all(torch.equal(x.nan_to_num(5.0), y.nan_to_num(5.0)) for x, y in zip(c.args(), state))
    out = hca.paged_prefill(**good)
    _no_error()
    c.check_state()
    c.check_out(out, q, g, [2, 3])


@pytest.mark.parametrize("n,pad", [([2, 0, 3], 4), ([30, 9, 40], 6), ([0, 0, 0], 3), ([0, 0, 0], 50)])
def test_rows_behind_the_last_sequence(n, pad):
    """Inputs behind q_start[S] are not looked at, outputs there stay as they were."""
    need_gpu()
    gen = _gen(3)
    L0 = [200, 77, 1500]
    seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
    c = Cache(seqs, L0, 32, room=64)
    k, v, s, start, ctx = c.chunk(n)
    N = sum(n)
    q, g = _qg(N, gen)
    more = lambda x: torch.cat([x, torch.full((pad,) + x.shape[1:], NAN, dtype=x.dtype,  # noqa: E731
                                              device="cuda")])
    out = torch.full((N + pad, HEADS, DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    hca.paged_prefill(more(q), more(g), more(k), more(v), more(s), start, ctx, *c.args(), out=out)
    _no_error()
    assert (out[N:] == 7.0).all()
    c.check_state()
    c.check_out(out, q, g, n, picks=[0, 1, 2, 8, 29, 39])


def test_one_workspace_for_every_size_and_form():
    """A workspace for more sequences and tokens serves smaller calls of either form in turn."""
    need_gpu()
    gen = _gen(5)
    ws = hca.paged_prefill_workspace(5, 300, "cuda")
    for i, (L0, n) in enumerate([([0], [1]), ([500, 20], [200, 60]), ([9000], [4]),
                                 ([130] * 5, [60] * 5), ([130] * 5, [8] * 5), ([70000], [41]),
                                 ([70000], [40])]):
        seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
        c = Cache(seqs, L0, (16, 64)[i % 2], room=max(n))
        k, v, s, start, ctx = c.chunk(n)
        q, g = _qg(sum(n), gen)
        out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(), workspace=ws)
        _no_error()
        c.check_state()
        c.check_out(out, q, g, n, picks=[0, 1, 3, 7, 39, 40, 59, 199])


def test_calls_on_two_streams_at_once():
    """Two chunks and two steps in flight together, a workspace each: what they give alone."""
    need_gpu()
    gen = _gen(13)
    runs = []
    for L0, n in (([20000, 300], [50, 7]), ([9000, 127], [3, 1])):
        seqs = [Seq(L + m + 1, gen, "cuda") for L, m in zip(L0, n)]
        c = Cache(seqs, L0, 32, room=64)
        k, v, s, start, ctx = c.chunk(n)
        k1, v1, s1, _, ctx1 = c.chunk([1, 1])
        q, g = _qg(sum(n), gen)
        q1, g1 = _qg(2, gen)
        runs.append((c, n, (q, g, k, v, s, start, ctx), (q1, g1, k1, v1, s1, ctx1),
                     hca.paged_prefill_workspace(2, sum(n), "cuda"),
                     hca.paged_decode_workspace(2, "cuda"), torch.cuda.Stream(),
                     [x.clone() for x in c.args()[:5]]))
    torch.cuda.synchronize()

    def go(run):
        c, _, a, b, ws, ds = run[:6]
        return [hca.paged_prefill(*a, *c.args(), workspace=ws),
                hca.paged_decode_step(*b, *c.args(), workspace=ds)]

    alone = []
    for run in runs:
        alone.append(go(run))
        torch.cuda.synchronize()
    for _ in range(3):
        for run in runs:
            for x, y in zip(run[0].args(), run[7]):
                x.copy_(y)
        torch.cuda.synchronize()
        both = []
        for run in runs:
            with torch.cuda.stream(run[6]):
                both.append(go(run))
        torch.cuda.synchronize()
        _no_error()
        for x, y in zip(alone, both):
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    for run in runs:
        run[0].check_state()


def test_pool_past_32_bit_offsets():
    """Pools of 9 GB each (over 2^32 elements): entries written and read at their far end, pages
    copied there and moved from there."""
    need_gpu()
    P, num = 128, 70000
    gen = _gen(17)
    L = 128 * 300 + 100
    seq = Seq(L + 60, gen, "cuda")
    small = Cache([seq], [L], P, room=60)
    ck = torch.empty((num, P, DIM), dtype=torch.bfloat16, device="cuda")
    cv = torch.empty_like(ck)
    far = [num - 1, 3, num - 5]
    table = torch.tensor([far + [-1]], dtype=torch.int32, device="cuda")
    for j in range(3):
        p = int(small.table[0, j])
        ck[far[j]], cv[far[j]] = small.ck[p], small.cv[p]
    k, v, s, start, ctx = small.chunk([50])       # completes a block: entry 300, page num - 5
    q, g = _qg(50, gen)
    rings = [x.clone() for x in (small.wk, small.wv, small.ws)]
    want = hca.paged_prefill(q, g, k, v, s, start, ctx, *small.args())
    got = hca.paged_prefill(q, g, k, v, s, start, ctx, *rings, ck, cv, table)
    assert torch.equal(want, got)
    assert torch.equal(ck[num - 5, 300 - 256], small.stored(0)[0][300])
    for n in (3, 1):
        k, v, s, start, ctx = small.chunk([n])
        q, g = _qg(n, gen)
        want = hca.paged_prefill(q, g, k, v, s, start, ctx, *small.args())
        got = hca.paged_prefill(q, g, k, v, s, start, ctx, *rings, ck, cv, table)
        assert torch.equal(want, got)
    small.check_state()
    # pages: the last one in part to a fresh page, then everything down to the front
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ref = torch.zeros(num, dtype=torch.int32, device="cuda")
    ref[table[0, :3].long()] = 1
    rows = torch.cat([table, torch.full_like(table, -1)])
    count = ints(3, 0)
    hca.copy_pages([ck, cv], ints(num - 1), ints(num - 3))
    assert torch.equal(ck[num - 3].nan_to_num(1.0), ck[num - 1].nan_to_num(1.0))
    ok = hca.fork_pages(rows, count, ref, ints(0), ints(1), ints(299), [ck, cv], P)
    assert ok.tolist() == [1] and rows[1].tolist() == [num - 1, 3, 0, -1]
    assert torch.equal(cv[0].nan_to_num(1.0), cv[num - 5].nan_to_num(1.0))
    keep = ck[num - 1].clone(), ck[num - 5].clone()
    live = hca.compact_pages(rows, count, ref, [ck, cv])
    assert live.tolist() == [4] and rows[0].tolist() == [2, 3, 1, -1]
    assert torch.equal(ck[2].nan_to_num(1.0), keep[0].nan_to_num(1.0))
    assert torch.equal(ck[1].nan_to_num(1.0), keep[1].nan_to_num(1.0))
    _no_error()


@pytest.mark.parametrize("n", [1, 60])
def test_extreme_values(n):
    """Block scores of the type's lowest value and of -infinity beside a finite one, equal scores
    far from zero, query rows that spread a softmax over 60 powers of two."""
    need_gpu()
    gen = _gen(n + 100)
    L = 128 * 9 - 1
    seq = Seq(L + n, gen, "cuda")
    low = torch.finfo(torch.bfloat16).min
    seq.s[:128] = low                  # all equal: the mean
    seq.s[128:256] = float("-inf")
    seq.s[200] = low                   # the only one that counts
    seq.s[256:384] = 3e38
    seq.s[L - 127:L] = low             # the block that this call completes
    c = Cache([seq], [L], 16, room=n)
    k, v, s, start, ctx = c.chunk([n])
    q, g = _qg(n, gen)
    q[:, ::2] *= 8
    g[:, 1], g[:, 2], g[:, 3] = 80.0, -80.0, float("-inf")
    out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
    _no_error()
    c.check_state()
    assert (out[:, 3] == 0).all()
    g[:, 3] = -1e30
    c.check_out(out, q, g, [n], picks=[0, 59])
    assert torch.equal(c.stored(0)[0][1], seq.k[200])


def test_non_finite_tokens_stay_in_their_sequence():
    """A token with an infinite value reaches its own and later outputs (and may reach others of
    its sequence: a weight of zero does not hold it back); its neighbours in the batch are not
    touched, nor are the rings and entries of theirs."""
    need_gpu()
    gen = _gen(31)
    for n in ([8, 8, 8], [64, 64, 64]):
        L0 = [900, 2000, 300]
        seqs = [Seq(L + m, gen, "cuda") for L, m in zip(L0, n)]
        c = Cache(seqs, L0, 32, room=64)
        k, v, s, start, ctx = c.chunk(n)
        q, g = _qg(sum(n), gen)
        bad = n[0] + 40 if n[0] == 64 else n[0] + 4
        v = v.clone()
        v[bad] = float("inf")
        out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
        _no_error()
        finite = torch.isfinite(out.float()).all(-1).all(-1)
        assert finite[:n[0]].all() and finite[2 * n[0]:].all()
        assert not finite[bad:2 * n[0]].any()
        assert torch.isfinite(c.wv[0].float()).all() and torch.isfinite(c.wv[2].float()).all()
        for i in (0, 2):
            for r in (0, n[0] - 1):
                ek, ev = c.stored(i)
                ref, bound = attend64(q[i * n[0] + r], g[i * n[0] + r], ek, ev, seqs[i].k,
                                      seqs[i].v, L0[i] + r)
                assert ((out[i * n[0] + r].double() - ref).abs() <= bound).all()


def test_output_over_an_input_is_refused():
    """Before anything is launched: the cache stays as it was."""
    need_gpu()
    gen = _gen(51)
    for n in ([1], [60]):
        seq = Seq(400, gen, "cuda")
        c = Cache([seq], [300], 16, room=n[0])
        k, v, s, start, ctx = c.chunk(n)
        qg = torch.randn((2 * n[0] + 1, HEADS, DIM), generator=gen, device="cuda").bfloat16()
        q, g = qg[:n[0]], qg[n[0]:2 * n[0]]
        before = [x.clone().nan_to_num(3.0) for x in c.args()[:5]]
        for out in (q, g, qg[1:n[0] + 1]):
            for given in (None, hca.paged_prefill_workspace(1, n[0], "cuda")):
                with pytest.raises(hca.HCAError):
                    hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(), workspace=given, out=out)
                if n == [1]:
                    with pytest.raises(hca.HCAError):
                        hca.paged_decode_step(q, g, k, v, s, ctx, *c.args(), out=out)
        assert all(torch.equal(a, b.nan_to_num(3.0)) for a, b in zip(before, c.args()))
        out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args(),
                                out=torch.empty_like(qg)[:n[0]])
        _no_error()
        c.check_out(out, q, g, n, picks=[0, 59])


def test_no_pages_and_one_page():
    """Sequences too short for an entry need no pool; a pool of one page holds sixteen."""
    need_gpu()
    gen = _gen(41)
    empty = torch.empty((0, 16, DIM), dtype=torch.bfloat16, device="cuda")
    none = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    L0, n = [0, 50], [60, 70]
    seqs = [Seq(L + m + 1, gen, "cuda") for L, m in zip(L0, n)]
    c = Cache(seqs, L0, 16)
    c.ck, c.cv, c.table = empty, empty.clone(), none
    for n in ([5, 3], [55, 67], [1, 1]):
        k, v, s, start, ctx = c.chunk(n)
        q, g = _qg(sum(n), gen)
        out = hca.paged_prefill(q, g, k, v, s, start, ctx, *c.args())
        _no_error()
        c.check_out(out, q, g, n, picks=[0, 2, 54, 66])
    one = hca.paged_decode(q, c.ck, c.cv, c.table, c.wk, c.wv, ctx, g)
    _no_error()
    c.check_out(one, q, g, [1, 1])
    seq = Seq(128 * 16, gen, "cuda")
    c = Cache([seq], [0], 16, room=128 * 16, extra=0)
    assert len(c.ck) == 1
    for m in (1000, 1047):
        k, v, s, start, ctx = c.chunk([m])
        hca.paged_append(k, v, s, start, ctx, *c.args())
    k, v, s, _, ctx = c.chunk([1])
    q, g = _qg(1, gen)
    out = hca.paged_decode_step(q, g, k, v, s, ctx, *c.args())
    _no_error()
    c.check_state()
    c.check_out(out, q, g, [1])
    assert BLOCK * 16 == c.lens[0]
