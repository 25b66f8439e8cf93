"""A packed batch served in several calls: each call takes some of the sequences by its own part
of the offsets, rings and table, over the same packed inputs and outputs."""
import pytest
import torch

import compressed_sliding_window_b200 as hca
from tests.gpu_util import need_gpu
from tests.paged_ref import HEADS, Seq
from tests.test_gpu_paged import Cache, _gen, _no_error, _qg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rank", [0, 6])
@pytest.mark.parametrize("n,cut", [([5, 3, 7, 2], 2), ([1, 0, 0, 4], 3), ([40, 30, 90, 20], 1),
                                   ([1] * 100, 60)], ids=["17", "5", "180", "100"])
def test_offsets_that_start_inside(n, cut, rank):
    """Rows of sequences that a call does not name stay as they were, whatever its form."""
    need_gpu()
    gen = _gen(sum(n) + rank)
    L0 = [(700 * i + 300 * (i % 3)) % 9001 for i in range(len(n))]
    base = Seq(max(L0) + max(n), gen, "cuda")
    c = Cache([base] * len(n), L0, 16, room=max(n))
    k, v, s, start, ctx = c.chunk(n)
    N = sum(n)
    q, g = _qg(N, gen)
    vha = tuple((torch.randn((HEADS, rank), generator=gen, device="cuda") / 8).bfloat16()
                for _ in range(2)) if rank else None
    out = torch.full_like(q, 7.0)
    split = int(start[cut])
    for part, mine in ((slice(cut, None), slice(split, N)), (slice(0, cut), slice(0, split))):
        before = out.clone()
        hca.paged_prefill(q, g, k, v, s, start[part.start or 0:][:len(ctx[part]) + 1].clone(),
                          ctx[part].clone(), c.wk[part], c.wv[part], c.ws[part], c.ck, c.cv,
                          c.table[part], out=out, vha=vha)
        _no_error()
        rest = torch.ones(N, dtype=torch.bool, device="cuda")
        rest[mine] = False
        assert torch.equal(out[rest], before[rest])
    c.check_state()
    c.check_out(out, q, g, n, vha)
