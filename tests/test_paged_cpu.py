"""Host side of the paged cache, without a GPU: refusals of the C ABI (none of these calls
reaches a kernel), of the Python functions, and the plain models that the GPU tests use."""
import ctypes
import random

import numpy as np
import pytest
import torch

import compressed_sliding_window_b200 as hca
from compressed_sliding_window_b200 import build as B
from oracle import hca_oracle as O
from tests.paged_ref import BLOCK, DIM, HEADS, Pages, Seq, attend64, entries64

OK, INVALID, UNSUPPORTED = 0, 1, 2
F = 1 << 20        # aligned fake device address
vp, i32, f32, sz, i64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t,
                         ctypes.c_longlong)


class CCache(ctypes.Structure):
    _fields_ = [(n, vp) for n in ("wk", "wv", "ws", "ck", "cv", "page_table")] + [
        ("table_stride", i64), ("max_pages", i32), ("num_pages", i32), ("page_size", i32)]


class CTable(ctypes.Structure):
    _fields_ = [("page_table", vp), ("table_stride", i64), ("rows", i32), ("max_pages", i32),
                ("n_pages", vp), ("ref", vp), ("num_pages", i32), ("page_size", i32)]


class CArray(ctypes.Structure):
    _fields_ = [("data", vp), ("item_bytes", i64)]


@pytest.fixture(scope="module")
def lib():
    return ctypes.CDLL(B.build())


def cache(**kw):
    c = CCache(F, F, F, F, F, F, 8, 8, 32, 16)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


BAD_CACHE = [(dict(wk=None), INVALID), (dict(wv=F + 8), INVALID), (dict(ck=None), INVALID),
             (dict(cv=F + 2), INVALID), (dict(page_table=None), INVALID),
             (dict(page_table=F + 2), INVALID), (dict(table_stride=7), INVALID),
             (dict(max_pages=-1), INVALID), (dict(num_pages=-1), INVALID),
             (dict(page_size=0), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
             (dict(page_size=48), UNSUPPORTED), (dict(page_size=256), UNSUPPORTED),
             (dict(max_pages=1 << 21, table_stride=1 << 21), UNSUPPORTED)]


def caller(lib, name, names, args, types):
    """name(**changes): the call with valid arguments but for the changed ones."""
    fn = getattr(lib, name)
    fn.argtypes = types

    def call(**kw):
        a = dict(zip(names, args))
        assert not set(kw) - set(a)
        a.update(kw)
        c = a.get("cache")
        if isinstance(c, ctypes.Structure):
            a["cache"] = ctypes.addressof(c)
        return fn(*a.values())
    return call


def append(lib):
    return caller(lib, "hca_paged_append", "k v s start len S N cache stream".split(),
                  [F, F, F, F, F, 4, 9, cache(), None], [vp] * 5 + [i32, i32, vp, vp])


def prefill(lib):
    return caller(lib, "hca_paged_prefill",
                  "q g k v s start len S N H scale down up rank cache out ws bytes stream".split(),
                  [F] * 7 + [4, 9, 64, 0.04, None, None, 0, cache(), F, F, 1 << 40, None],
                  [vp] * 7 + [i32] * 3 + [f32, vp, vp, i32, vp, vp, vp, sz, vp])


def decode(lib):
    return caller(lib, "hca_paged_decode",
                  "q g len S H scale down up rank cache out ws bytes stream".split(),
                  [F] * 3 + [4, 64, 0.04, None, None, 0, cache(), F, F, 1 << 40, None],
                  [vp] * 3 + [i32] * 2 + [f32, vp, vp, i32, vp, vp, vp, sz, vp])


def step(lib):
    return caller(lib, "hca_paged_decode_step",
                  "q g k v s len S H scale down up rank cache out ws bytes stream".split(),
                  [F] * 6 + [4, 64, 0.04, None, None, 0, cache(), F, F, 1 << 40, None],
                  [vp] * 6 + [i32] * 2 + [f32, vp, vp, i32, vp, vp, vp, sz, vp])


@pytest.mark.parametrize("kw,code", BAD_CACHE, ids=[str(c[0]) for c in BAD_CACHE])
def test_every_call_refuses_a_bad_cache(lib, kw, code):
    for call in (append, prefill, decode, step):
        assert call(lib)(cache=cache(**kw)) == code
    for call in (append, prefill, step):          # a score ring is needed to append
        assert call(lib)(cache=cache(ws=None)) == INVALID
        assert call(lib)(cache=None) == INVALID


def test_append_refuses(lib):
    call = append(lib)
    for kw in (dict(S=0), dict(S=-1), dict(N=-1), dict(k=None), dict(v=None), dict(s=None),
               dict(len=None), dict(k=F + 8), dict(v=F + 2), dict(len=F + 2), dict(start=F + 1),
               dict(start=None)):                 # without offsets there are S tokens, not 9
        assert call(**kw) == INVALID, kw
    assert call(S=1 << 25) == UNSUPPORTED         # ring rows are 32-bit
    assert call(N=0) == OK                        # nothing to do, nothing launched
    assert call(N=0, cache=cache(max_pages=0, num_pages=0, ck=None, cv=None,
                                 page_table=None)) == OK


ATTEND = [(dict(H=63), UNSUPPORTED), (dict(H=128), UNSUPPORTED), (dict(q=None), INVALID),
          (dict(g=None), INVALID), (dict(out=None), INVALID), (dict(q=F + 8), INVALID),
          (dict(g=F + 4), INVALID), (dict(out=F + 2), INVALID), (dict(ws=None), INVALID),
          (dict(ws=F + 128), INVALID), (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID),
          (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
          (dict(rank=-1), INVALID), (dict(rank=65, down=F, up=F), INVALID),
          (dict(rank=8, up=F), INVALID), (dict(rank=8, down=F), INVALID), (dict(S=0), INVALID),
          (dict(S=-3), INVALID), (dict(len=None), INVALID), (dict(len=F + 2), INVALID)]


@pytest.mark.parametrize("kw,code", ATTEND, ids=[str(c[0]) for c in ATTEND])
def test_attention_refuses(lib, kw, code):
    for call in (prefill, decode, step):
        assert call(lib)(**kw) == code


def test_sizes_past_the_limits(lib):
    assert prefill(lib)(start=None) == INVALID
    assert prefill(lib)(N=-1) == INVALID
    assert prefill(lib)(N=0) == OK
    assert prefill(lib)(S=4097) == UNSUPPORTED
    assert prefill(lib)(N=1 << 25) == UNSUPPORTED
    assert prefill(lib)(N=(1 << 25) - 144 * 4096, S=4096) == UNSUPPORTED
    assert decode(lib)(S=65536) == UNSUPPORTED
    assert step(lib)(S=65536) == UNSUPPORTED
    assert step(lib)(k=None) == INVALID
    for name, args in (("hca_paged_prefill_workspace_size", (0, 4)),
                       ("hca_paged_prefill_workspace_size", (4, 0)),
                       ("hca_paged_decode_workspace_size", (0,))):
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = sz, [i32] * len(args)
        assert fn(*args) == 0


def table(**kw):
    t = CTable(F, 8, 5, 8, F, F, 32, 16)
    for k, v in kw.items():
        setattr(t, k, v)
    return ctypes.addressof(t), t


BAD_TABLE = [(dict(page_table=None), INVALID), (dict(n_pages=None), INVALID),
             (dict(ref=None), INVALID), (dict(ref=F + 2), INVALID), (dict(rows=0), INVALID),
             (dict(max_pages=0), INVALID), (dict(num_pages=0), INVALID),
             (dict(table_stride=7), INVALID), (dict(page_size=24), UNSUPPORTED)]


def page_calls(lib):
    one = (CArray * 9)(*[CArray(F, 4096)] * 9)
    resize = caller(lib, "hca_pages_resize", "cache entries ws bytes stream".split(),
                    [None, F, F, 1 << 30, None], [vp, vp, vp, sz, vp])
    fork = caller(lib, "hca_pages_fork",
                  "cache parents children entries n pools np rings nr ok ws bytes stream".split(),
                  [None, F, F, F, 3, one, 2, one, 1, F, F, 1 << 30, None],
                  [vp] * 4 + [i32, vp, i32, vp, i32, vp, vp, sz, vp])
    compact = caller(lib, "hca_pages_compact", "cache pools np live ws bytes stream".split(),
                     [None, one, 2, F, F, 1 << 30, None], [vp, vp, i32, vp, vp, sz, vp])
    return resize, fork, compact


@pytest.mark.parametrize("kw,code", BAD_TABLE, ids=[str(c[0]) for c in BAD_TABLE])
def test_page_calls_refuse_a_bad_table(lib, kw, code):
    for call in page_calls(lib):
        at, keep = table(**kw)
        assert call(cache=at) == code
        assert call(cache=None) == INVALID


def test_page_calls_refuse(lib):
    resize, fork, compact = page_calls(lib)
    at, keep = table()
    for kw in (dict(entries=None), dict(entries=F + 2), dict(ws=None), dict(ws=F + 8),
               dict(bytes=16)):
        assert resize(cache=at, **kw) == INVALID, kw
        assert fork(cache=at, **kw) == INVALID, kw
    for kw in (dict(parents=None), dict(children=F + 1), dict(ok=None), dict(n=-1), dict(np=-1),
               dict(pools=None), dict(rings=None),
               dict(pools=(CArray * 2)(CArray(F, 4096), CArray(F + 8, 4096))),
               dict(pools=(CArray * 2)(CArray(None, 4096), CArray(F, 4096))),
               dict(pools=(CArray * 2)(CArray(F, 8), CArray(F, 16))),
               dict(rings=(CArray * 1)(CArray(F, 24)))):
        assert fork(cache=at, **kw) == INVALID, kw
    assert fork(cache=at, n=8193) == UNSUPPORTED
    assert fork(cache=at, np=5, nr=4) == UNSUPPORTED
    assert fork(cache=at, n=0) == OK
    for kw in (dict(live=None), dict(live=F + 2), dict(pools=None), dict(ws=None),
               dict(bytes=16), dict(np=-1)):
        assert compact(cache=at, **kw) == INVALID, kw
    assert compact(cache=at, np=9) == UNSUPPORTED
    one = (CArray * 9)(*[CArray(F, 4096)] * 9)
    copy = caller(lib, "hca_pages_copy", "a na items src dst n ws bytes stream".split(),
                  [one, 1, 10, F, F, 4, F, 1 << 30, None],
                  [vp, i32, i32, vp, vp, i32, vp, sz, vp])
    for kw in (dict(a=None), dict(na=-1), dict(items=0), dict(src=None), dict(dst=F + 2),
               dict(n=-1), dict(n=1 << 30), dict(ws=None), dict(ws=F + 4), dict(bytes=16)):
        assert copy(**kw) == INVALID, kw
    assert copy(na=9) == UNSUPPORTED
    assert copy(n=0) == OK


@pytest.mark.parametrize("item_bytes,n", [(1 << 62, 1), (16384 << 31, 1), (16384 << 28, 4)])
def test_copies_past_the_units_of_a_call(lib, item_bytes, n):
    two = (CArray * 2)(CArray(F, item_bytes), CArray(F, item_bytes))
    st = lib.hca_pages_copy
    st.argtypes, st.restype = [vp, i32, i32, vp, vp, i32, vp, sz, vp], i32
    assert st(two, 2, 10, F, F, n, F, 1 << 40, None) == UNSUPPORTED


def test_page_workspace_size(lib):
    fn = lib.hca_pages_workspace_size
    fn.restype, fn.argtypes = sz, [i32] * 3
    assert fn(0, 1, 1) == fn(1, 0, 1) == fn(1, 1, -1) == 0
    for rows, pages, n in ((1, 1, 0), (5, 100, 3), (300, 7, 8192), (1, 1 << 20, 0)):
        # enough for the lists of each call: resize, fork, compact, copy
        need = max(pages + rows + 1, 4 * n, 2 * (pages // 2 + 1) + pages + 1, pages + 2 * n)
        assert fn(rows, pages, n) >= 4 * need


# ---------------------------------------------------------------- Python
def tensors(S=2, N=3, P=16):
    b = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    z = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    return dict(k=b(N, DIM), v=b(N, DIM), s=b(N), start=z(S + 1), len=z(S), wk=b(S, BLOCK, DIM),
                wv=b(S, BLOCK, DIM), ws=b(S, BLOCK), ck=b(4, P, DIM), cv=b(4, P, DIM),
                table=z(S, 3), q=b(N, HEADS, DIM), g=b(N, HEADS, DIM))


def test_functions_refuse_host_tensors_and_other_objects():
    t = tensors()
    chunk = [t[x] for x in ("k", "v", "s", "start", "len")]
    kept = [t[x] for x in ("wk", "wv", "ws", "ck", "cv", "table")]
    pages = [t["table"], t["len"], t["start"]]
    calls = [lambda: hca.paged_append(*chunk, *kept),
             lambda: hca.paged_prefill(t["q"], t["g"], *chunk, *kept),
             lambda: hca.paged_decode(t["q"], *kept[3:], *kept[:2], t["len"], t["g"]),
             lambda: hca.paged_decode_step(t["q"], t["g"], *chunk[:3], t["len"], *kept),
             lambda: hca.resize_pages(*pages, t["len"], 16),
             lambda: hca.fork_pages(*pages, t["len"], t["len"], t["len"], [t["ck"]], 16),
             lambda: hca.compact_pages(*pages, [t["ck"]]),
             lambda: hca.copy_pages([t["ck"]], t["len"], t["len"])]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    with pytest.raises(TypeError):
        hca.paged_append(*chunk, None, *kept[1:])
    with pytest.raises(TypeError):
        hca.resize_pages([[1]], t["len"], t["start"], t["len"], 16)
    with pytest.raises(TypeError):
        hca.copy_pages([np.zeros((2, 16))], t["len"], t["len"])
    hca.copy_pages([], t["len"], t["len"])        # no arrays: nothing to do


def test_checks_behind_the_compiled_module():
    """The checks that name what is wrong, on the CPU as the device of the call."""
    cpu = torch.device("cpu")
    t = tensors()
    with pytest.raises(ValueError, match="page_table"):
        hca._check_table(t["table"].long(), 2, cpu)
    with pytest.raises(ValueError, match="page_table"):
        hca._check_table(t["table"], 3, cpu)
    with pytest.raises(ValueError, match="overlap"):
        hca._check_table(t["table"].as_strided((2, 3), (1, 1)), 2, cpu)
    with pytest.raises(ValueError, match="contiguous"):
        hca._check_table(torch.zeros(3, 2, dtype=torch.int32).T, 2, cpu)
    wide = torch.zeros(2, 9, dtype=torch.int32)
    assert hca._check_table(wide[:, 2:5], 2, cpu) == (3, 9)
    assert hca._check_table(torch.zeros(1, 5, dtype=torch.int32)[:, :2], 1, cpu) == (2, 2)
    with pytest.raises(ValueError, match="dimension"):
        hca._rows(t["k"], "k", 1)
    with pytest.raises(TypeError):
        hca._rows([1], "k", 1)
    with pytest.raises(ValueError, match="16, 32, 64 or 128"):
        hca._page_table(t["table"], t["len"], t["start"], 24, cpu)
    with pytest.raises(ValueError, match="16, 32, 64 or 128"):
        hca._paged_cache(2, t["wk"], t["wv"], t["ws"], t["ck"][:, :8], t["cv"], t["table"], cpu)
    with pytest.raises(ValueError, match="multiple of 16"):
        hca._page_arrays([torch.zeros(4, 5, dtype=torch.int16)], 4, "pools", cpu)
    with pytest.raises(ValueError, match="contiguous"):
        hca._page_arrays([torch.zeros(4, 16).T], 16, "pools", cpu)
    with pytest.raises(ValueError, match=r"\[4, ...\]"):
        hca._page_arrays([torch.zeros(5, 16)], 4, "pools", cpu)
    packed = hca._page_arrays([t["ck"], t["cv"]], 4, "pools", cpu)
    assert len(packed) == 2 * ctypes.sizeof(CArray)
    c = CCache.from_buffer_copy(hca._paged_cache(2, t["wk"], t["wv"], t["ws"], t["ck"], t["cv"],
                                                 t["table"], cpu))
    assert (c.wk, c.cv, c.table_stride, c.max_pages, c.num_pages, c.page_size) == (
        t["wk"].data_ptr(), t["cv"].data_ptr(), 3, 3, 4, 16)
    p = CTable.from_buffer_copy(hca._page_table(t["table"], t["len"], t["start"], 64, cpu)[0])
    assert (p.page_table, p.rows, p.max_pages, p.ref, p.num_pages, p.page_size) == (
        t["table"].data_ptr(), 2, 3, t["start"].data_ptr(), 3, 64)


def test_compiled_module_leaves_what_it_cannot_take():
    calls = hca._calls()
    t = tensors()
    assert calls.paged_append(*[t[x] for x in "k v s start len wk wv ws ck cv table".split()]) is False
    assert calls.resize_pages(t["table"], t["len"], t["start"], t["len"], 16, None) is False
    assert calls.resize_pages(1, 2, 3, 4, 10 ** 30, None) is False
    with pytest.raises(TypeError):
        calls.paged_append(1, 2)


# ---------------------------------------------------------------- models
def test_attention_model_is_the_oracle():
    """The 64-bit model of one position against the oracle's prefill over unrounded entries."""
    gen = torch.Generator().manual_seed(5)
    T = 300
    s = Seq(T, gen, "cpu")
    q, g = (torch.randn((T, HEADS, DIM), generator=gen).bfloat16() for _ in range(2))
    to64 = lambda x: x.double().numpy()  # noqa: E731
    ref = O.prefill_forward(to64(q)[None], to64(s.k)[None], to64(s.v)[None], to64(s.s)[None],
                            to64(g)[None])
    ek, ev = entries64(s.k, s.v, s.s)
    for t in (0, 1, 126, 127, 128, 254, 255, 256, 299):
        out, bound = attend64(q[t], g[t], ek, ev, s.k, s.v, t)
        assert np.abs(out.numpy() - ref[0, t]).max() < 1e-12
        # one rounding of the output to bf16 lies well inside the bound
        assert ((out.bfloat16().double() - out).abs() <= bound).all()
        # and a missing or an extra key does not
        if t >= 255:
            far, _ = attend64(q[t], g[t], ek, ev, s.k, s.v, t - 128)
            assert ((far - out).abs() > bound).any()


def test_ring_holds_the_newest_tokens():
    s = Seq(300, torch.Generator().manual_seed(1), "cpu")
    ring = s.ring(s.k, 200, 0.0)
    assert all(torch.equal(ring[p % 128], s.k[p]) for p in range(72, 200))
    assert (s.ring(s.s, 5, 9.0)[5:] == 9.0).all()


@pytest.mark.parametrize("seed", range(4))
def test_page_model_keeps_its_counts(seed):
    """Random histories: ref counts name the table's uses, no row holds a free page, compaction
    leaves the used pages in front and every row's contents as they were."""
    r = random.Random(seed)
    rows, width, num, P = 7, 9, 30, 16
    p = Pages([[-1] * width] * rows, [0] * rows, [0] * num, P)
    what = {}                                    # page -> its contents
    for _ in range(60):
        op = r.randrange(3)
        if op == 0:
            p.resize([r.choice([-1, 0, r.randrange(width * P)]) for _ in range(rows)])
        elif op == 1:
            a, b = r.randrange(rows), r.randrange(rows)
            ok, pages, _ = p.fork([a], [b], [r.randrange(width * P)])
            for x, y in pages:
                what[y] = what.get(x)
        else:
            for row in p.rows:
                for x in row:
                    what.setdefault(x, object())
            before = [[what[x] for x in row] for row in p.rows]
            for x, y in p.compact():
                what[y] = what.pop(x)
            assert [[what[x] for x in row] for row in p.rows] == before
            live = sum(c > 0 for c in p.ref)
            assert all(c > 0 for c in p.ref[:live])
        uses = [0] * num
        for row in p.rows:
            assert len(set(row)) == len(row) <= width
            for x in row:
                uses[x] += 1
        assert uses == p.ref
        what = {x: c for x, c in what.items() if p.ref[x] > 0}
