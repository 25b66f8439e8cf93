"""Host side of the resize that copies shared pages, without a GPU: its refusals (none reaches a
kernel) and the plain model of tests/test_gpu_pages_cut.py against page contents."""
import ctypes
import random

import pytest
import torch

import compressed_sliding_window_b200 as hca
from compressed_sliding_window_b200 import build as B
from tests.test_gpu_pages_cut import CutPages
from tests.test_paged_cpu import F, INVALID, UNSUPPORTED, CArray, CTable, f32, i32, sz, vp  # noqa: F401


def test_resize_copy_refuses():
    lib = ctypes.CDLL(B.build())
    fn = lib.hca_pages_resize_copy
    fn.argtypes, fn.restype = [vp, vp, vp, i32, vp, sz, vp], i32
    size = lib.hca_pages_workspace_size
    size.argtypes, size.restype = [i32] * 3, sz
    need = size(4, 9, 0)
    assert need >= 4 * (9 + 3 * 4 + 2)

    def call(pools=((F, 64),), n=None, entries=F, ws=F, room=need, **kw):
        t = CTable(F, 8, 4, 8, F, F, 9, 16)
        for k, v in kw.items():
            setattr(t, k, v)
        arrays = (CArray * max(1, len(pools)))(*[CArray(*p) for p in pools])
        return fn(ctypes.addressof(t), entries, ctypes.addressof(arrays),
                  len(pools) if n is None else n, ws, room, None)

    assert call(pools=()) == INVALID
    assert call(n=-1) == INVALID
    assert call(pools=((None, 64),)) == INVALID
    assert call(pools=((F + 8, 64),)) == INVALID
    assert call(pools=((F, 24),)) == INVALID
    assert call(pools=((F, 0),)) == INVALID
    assert call(pools=((F, 64),) * 9) == UNSUPPORTED
    assert call(pools=((F, 1 << 46),)) == UNSUPPORTED
    assert call(entries=None) == INVALID
    assert call(ws=None) == INVALID and call(ws=F + 8) == INVALID
    assert call(room=need - 1) == INVALID
    assert call(rows=0) == INVALID and call(page_size=24) == UNSUPPORTED
    assert call(ref=None) == INVALID
    assert fn(None, F, None, 1, F, need, None) == INVALID


def test_pools_are_checked():
    t = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        hca.resize_pages(t.view(2, 2), t[:2], t, t[:2], 16, pools=[torch.zeros(4, 16)])


@pytest.mark.parametrize("seed", range(6))
def test_model_keeps_every_history(seed):
    """Random cuts, forks and appends on the model's pages: each row always reads back what its own
    history holds, although pages are shared."""
    r = random.Random(seed)
    P, rows, width, num = 4, 6, 8, 60
    m = CutPages([[-1] * width] * rows, [0] * rows, [0] * num, P)
    store = [[None] * P for _ in range(num)]
    hist = [[] for _ in range(rows)]
    fresh = 0
    for _ in range(200):
        keep = [r.randint(0, len(h)) if r.random() < 0.4 else len(h) for h in hist]
        copies, fine = m.resize_copy(keep)
        assert fine
        for s, d in copies:
            store[d] = list(store[s])
        hist = [h[:n] for h, n in zip(hist, keep)]
        live, empty = [i for i in range(rows) if hist[i]], [i for i in range(rows) if not hist[i]]
        if live and empty and r.random() < 0.5:
            a, b = r.choice(live), r.choice(empty)
            e = r.randint(0, len(hist[a]))
            ok, pages, _ = m.fork([a], [b], [e])
            assert ok == [1]
            for s, d in pages:
                store[d] = list(store[s])
            hist[b] = hist[a][:e]
        add = [r.randint(0, 6) if len(h) < 20 else 0 for h in hist]
        copies, fine = m.resize_copy([len(h) + n for h, n in zip(hist, add)])
        assert fine and not copies
        for i, n in enumerate(add):
            for _ in range(n):
                j = len(hist[i])
                store[m.rows[i][j // P]][j % P] = fresh
                hist[i].append(fresh)
                fresh += 1
        for i in range(rows):
            assert [store[m.rows[i][j // P]][j % P] for j in range(len(hist[i]))] == hist[i]
