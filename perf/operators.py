"""Cases of the paged HCA cache: appending ragged chunks of tokens to it, the
attention of a chunk over it, single-token decode steps from it, and forking,
resizing and compacting its pages.

A paged cache keeps the compressed entries (one per 128 tokens, K and V rows of
512 bf16) of all sequences in pages of `page` entries.  `page_table[i, c]` names
the page that holds entries c * page .. of sequence i.  The newest 128 raw
tokens of a sequence stay in its ring (slot = position mod 128).

`own` false: plain torch operations in 32 bits (64 nowhere needed: the weights
are softmaxes over at most a few thousand keys).  `own` true: the package's
paged operators.
"""
import random

import torch

own = False

HEADS, DIM, BLOCK = 64, 512, 128
ROW = DIM * 2                # bytes of one bf16 row
SCALE = DIM ** -0.5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a scheduler step that only feeds the cache: 32 prompts, a ragged piece of each
        {"name": "append, 32 ragged pieces", "op": "append", "seqs": 32, "n_min": 1, "n_max": 256,
         "ctx_min": 300, "ctx_max": 65536, "page": 32, "mix": 1},
        # a prompt of 32768 tokens that was prefilled elsewhere enters the cache
        {"name": "append, one 32K prompt", "op": "append", "seqs": 1, "n_min": 32768,
         "n_max": 32768, "ctx_min": 32768, "ctx_max": 32768, "page": 64, "mix": 2},
        # drafts of 4 tokens checked against 8 long conversations
        {"name": "chunk, 8 x 4 drafts at 128K", "op": "chunk", "seqs": 8, "n_min": 4, "n_max": 4,
         "ctx_min": 131072, "ctx_max": 131072, "page": 64, "mix": 3},
        # continuous batching: some sequences prefill, most take a token, one rests
        {"name": "chunk, 16 ragged to 128K", "op": "chunk", "seqs": 16, "n_min": 0, "n_max": 300,
         "ctx_min": 77, "ctx_max": 131072, "page": 32, "mix": 4},
        # a chunked prefill near the end of a 1M-token context
        {"name": "chunk, 2048 at 1M", "op": "chunk", "seqs": 1, "n_min": 2048, "n_max": 2048,
         "ctx_min": 1000003, "ctx_max": 1000003, "page": 128, "mix": 5},
        # the first answers to a short question: latency alone
        {"name": "decode, 1 at 300", "op": "decode", "seqs": 1, "ctx_min": 300, "ctx_max": 300,
         "page": 16, "mix": 6},
        # a batch of equal conversations; every sequence completes a block in this step
        {"name": "decode, 64 x 128K", "op": "decode", "seqs": 64, "ctx_min": 131072,
         "ctx_max": 131072, "page": 64, "mix": 7},
        # few long contexts of unequal length, small pages
        {"name": "decode, 16 x 64K to 1M", "op": "decode", "seqs": 16, "ctx_min": 65536,
         "ctx_max": 1048576, "page": 16, "mix": 8},
        # one conversation answered twice
        {"name": "fork, 1 into 2", "op": "fork", "seqs": 4, "forks": 1, "ctx_min": 20000,
         "ctx_max": 20000, "page": 16, "spare": 64, "mix": 9},
        # parallel sampling: 48 branches from a dozen long prompts
        {"name": "fork, 48 branches", "op": "fork", "seqs": 64, "forks": 48, "ctx_min": 30000,
         "ctx_max": 400000, "page": 64, "spare": 256, "mix": 10},
        # a few answers end, a few grow, the pool closes up
        {"name": "compact, 96 small pages", "op": "compact", "seqs": 8, "ctx_min": 9000,
         "ctx_max": 40000, "page": 16, "spare": 30, "mix": 11},
        # a busy pool after many answers ended
        {"name": "compact, 1500 pages", "op": "compact", "seqs": 96, "ctx_min": 30000,
         "ctx_max": 250000, "page": 64, "spare": 300, "mix": 12},
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(lo * (hi / lo) ** rng.random()))

    op = rng.choice(["append", "chunk", "decode", "fork", "compact"])
    page = rng.choice([16, 32, 64, 128])
    mix = rng.randrange(1 << 20)
    if op == "append":
        seqs = log(1, 64)
        n_max = log(1, 32768 // seqs)
        return {"op": op, "seqs": seqs, "n_min": rng.randrange(0, n_max + 1), "n_max": n_max,
                "ctx_min": n_max, "ctx_max": log(n_max, 131072), "page": page, "mix": mix}
    if op == "chunk":
        seqs = log(1, 24)
        n_max = log(1, 1024 // seqs + 1)
        ctx = log(max(n_max, 200), 1000000 // seqs)
        return {"op": op, "seqs": seqs, "n_min": rng.randrange(0, n_max + 1), "n_max": n_max,
                "ctx_min": rng.randrange(n_max, ctx + 1), "ctx_max": ctx, "page": page, "mix": mix}
    if op == "decode":
        seqs = log(1, 200)
        ctx = log(40, 8000000 // max(8, seqs))
        return {"op": op, "seqs": seqs, "ctx_min": rng.randrange(1, ctx + 1), "ctx_max": ctx,
                "page": page, "mix": mix}
    seqs = log(4, 64)
    ctx = log(4000, 250000)
    c = {"op": op, "seqs": seqs, "ctx_min": rng.randrange(1000, ctx + 1), "ctx_max": ctx,
         "page": page, "spare": log(seqs + 16, 200 + seqs), "mix": mix}
    if op == "fork":
        c["forks"] = rng.randrange(1, seqs // 2 + 1)
    return c


def lengths(case):
    """(new tokens, context length with them) of every sequence, as a scheduler has them."""
    r = random.Random(case["mix"])
    ctx = [r.randint(case["ctx_min"], case["ctx_max"]) for _ in range(case["seqs"])]
    if case["op"] in ("append", "chunk"):
        n = [r.randint(case["n_min"], case["n_max"]) for _ in range(case["seqs"])]
        if sum(n) == 0:
            n[0] = case["n_max"]
    else:
        n = [1] * case["seqs"]
    return n, [max(c, m, 1) for c, m in zip(ctx, n)]


def visible(L):
    """Compressed entries that the last of L tokens sees."""
    return max(0, (L - 128) // 128)


def work(case):
    n, ctx = lengths(case)
    page = case["page"]
    if case["op"] in ("append", "chunk", "decode"):
        N = sum(n)
        done = sum(L // BLOCK - (L - m) // BLOCK for m, L in zip(n, ctx))
        # new tokens in, their ring slots and completed entries out
        b = N * (2 * ROW + 2) + sum(min(m, 128) for m in n) * (2 * ROW + 2) + done * 2 * ROW
        # old ring tokens that a completing block needs
        b += sum((L - m) % BLOCK for m, L in zip(n, ctx)
                 if L // BLOCK > (L - m) // BLOCK) * (2 * ROW + 2)
        if case["op"] == "append":
            return {"bytes": b, "flops": 4 * DIM * BLOCK * done}
        pairs = 0
        for m, L in zip(n, ctx):
            for t in range(L - m, L):
                pairs += visible(t + 1) + min(t + 1, 128)
        b += N * 3 * HEADS * ROW                                  # q, g, out
        b += sum(visible(L) * 2 * ROW for m, L in zip(n, ctx) if m)
        b += sum(min(127, L - m) * 2 * ROW for m, L in zip(n, ctx) if m)
        return {"bytes": b, "flops": 4 * HEADS * DIM * pairs}
    table_ints = 4 * 3 * sum(-(-(L // BLOCK) // page) for L in ctx)
    if case["op"] == "fork":
        pairs = fork_pairs(case)
        part = sum(1 for a, _ in pairs if (ctx[a] // BLOCK) % page)
        ring = 2 * BLOCK * ROW + 2 * BLOCK
        return {"bytes": 2 * part * page * 2 * ROW + 2 * len(pairs) * ring + table_ints, "flops": 0}
    moves = compact_moves(case)
    return {"bytes": 2 * moves * page * 2 * ROW + table_ints, "flops": 0}


# ---------------------------------------------------------------------------
# page plans of the fork and compact cases, on the host
# ---------------------------------------------------------------------------
def fork_pairs(case):
    """The last `forks` rows are free; each becomes a branch of one of the others."""
    r = random.Random(case["mix"] + 1)
    live = case["seqs"] - case["forks"]
    few = max(1, min(live, case["forks"] // 4 + 1))
    return [(r.randrange(few), live + i) for i in range(case["forks"])]


def pool_plan(case):
    """(pages of each row, number of pages of the pool): rows own scattered pages."""
    r = random.Random(case["mix"] + 2)
    _, ctx = lengths(case)
    live = case["seqs"] - case.get("forks", 0)
    counts = [-(-(L // BLOCK) // case["page"]) if i < live else 0 for i, L in enumerate(ctx)]
    total = sum(counts) + case["spare"]
    ids = list(range(total))
    r.shuffle(ids)
    rows, at = [], 0
    for c in counts:
        rows.append(ids[at:at + c])
        at += c
    return rows, total


def new_sizes(case):
    """Entries that each row is to hold next (-1: as it is): some end, some are cut, some grow."""
    r = random.Random(case["mix"] + 3)
    _, ctx = lengths(case)
    out = []
    for L in ctx:
        e, x = L // BLOCK, r.random()
        out.append(0 if x < 0.3 else e // 2 if x < 0.4 else e + r.randint(0, case["page"])
                   if x < 0.6 else -1)
    return out


def resized(case):
    """The rows of the pool after new_sizes: the definition, page by page."""
    rows, total = pool_plan(case)
    rows = [list(x) for x in rows]
    want = [len(x) if e < 0 else -(-e // case["page"]) for x, e in zip(rows, new_sizes(case))]
    for x, w in zip(rows, want):
        del x[w:]
    free = sorted(set(range(total)) - {p for x in rows for p in x}, reverse=True)
    for x, w in zip(rows, want):
        while len(x) < w and free:
            x.append(free.pop())
    return rows, total


def compact_moves(case):
    rows, total = resized(case)
    used = {p for x in rows for p in x}
    return sum(1 for p in used if p >= len(used))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 13)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev, dtype=torch.float32).bfloat16()

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    n, ctx = lengths(case)
    S, page, op = case["seqs"], case["page"], case["op"]
    s = {"op": op, "page": page}
    # the rings in one allocation, [wk | wv | ws], so that a pass copies them at once
    s["rings"] = normal(S * BLOCK * (2 * DIM + 1))
    if op in ("fork", "compact"):
        rows, total = pool_plan(case)
        width = max(len(x) for x in rows) + 2
        s["table"] = ints([x + [-1] * (width - len(x)) for x in rows])
        s["n_pages"] = ints([len(x) for x in rows])
        ref = [0] * total
        for x in rows:
            for p in x:
                ref[p] += 1
        s["ref"] = ints(ref)
        s["ck"], s["cv"] = normal(total, page, DIM), normal(total, page, DIM)
        if op == "fork":
            pairs = fork_pairs(case)
            s["parents"], s["children"] = ints([a for a, _ in pairs]), ints([b for _, b in pairs])
            s["entries"] = ints([ctx[a] // BLOCK for a, _ in pairs])
        else:
            s["entries"] = ints(new_sizes(case))
        return s
    N = sum(n)
    counts = [-(-(L // BLOCK) // page) for L in ctx]
    total = sum(counts) + 3
    perm = torch.randperm(total, generator=gen, device=dev).to(torch.int32)
    width = max(counts) + 1
    at, rows = 0, []
    for c in counts:
        rows.append(list(range(at, at + c)) + [-1] * (width - c))
        at += c
    slots = torch.tensor(rows, device=dev)
    s["table"] = torch.where(slots >= 0, perm[slots.clamp(min=0)], -1).to(torch.int32)
    s["ck"], s["cv"] = normal(total, page, DIM), normal(total, page, DIM)
    starts = [0]
    for m in n:
        starts.append(starts[-1] + m)
    s["starts"], s["ctx"] = ints(starts), ints(ctx)
    s["k"], s["v"], s["s"] = normal(N, DIM), normal(N, DIM), normal(N)
    if op != "append":
        s["q"], s["g"] = normal(N, HEADS, DIM), normal(N, HEADS, DIM)
    # what the scheduler knows of this step on the host
    s["n_max"] = max(n)
    s["e_max"] = max(visible(L) for L in ctx)
    return s


def rings(flat, S):
    a = S * BLOCK * DIM
    return (flat[:a].view(S, BLOCK, DIM), flat[a:2 * a].view(S, BLOCK, DIM),
            flat[2 * a:].view(S, BLOCK))


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["op"]
    if op == "fork":
        return _fork(s)
    if op == "compact":
        return _compact(s)
    S = s["ctx"].shape[0]
    # a chunk replaces the ring's tokens, so each pass starts from the same ring; a
    # single token may be written again over itself
    wk, wv, ws = rings(s["rings"] if op == "decode" else s["rings"].clone(), S)
    if own:
        import compressed_sliding_window_b200 as hca
        cache = (wk, wv, ws, s["ck"], s["cv"], s["table"])
        if op == "append":
            hca.paged_append(s["k"], s["v"], s["s"], s["starts"], s["ctx"], *cache)
            out = None
        elif op == "chunk":
            if "ws" not in s:
                s["ws"] = hca.paged_prefill_workspace(S, s["k"].shape[0], s["k"].device)
            out = hca.paged_prefill(s["q"], s["g"], s["k"], s["v"], s["s"], s["starts"], s["ctx"],
                                    *cache, workspace=s["ws"])
        else:
            if "ws" not in s:
                s["ws"] = hca.paged_decode_workspace(S, s["k"].device)
            out = hca.paged_decode_step(s["q"], s["g"], s["k"], s["v"], s["s"], s["ctx"], *cache,
                                        workspace=s["ws"])
    else:
        ext = _extended(s, wk, wv, ws)
        _write_entries(s, ext)
        out = None if op == "append" else _attend(s, wk, wv)
        _write_rings(s, wk, wv, ws)
    res = {"ck": s["ck"], "cv": s["cv"], "wk": wk, "wv": wv, "ws": ws}
    if out is not None:
        res["out"] = out
    return res


def _lens(s):
    st = s["starts"].long()
    n = st[1:] - st[:-1]
    L1 = s["ctx"].long()
    return st[:-1], n, L1 - n, L1


def _tokens(s, wk, wv, ws, pos):
    """K, V (fp32) and scores of positions pos [S, W] of each sequence; zeros outside of it."""
    st, n, L0, L1 = _lens(s)
    slot = pos % BLOCK
    seq = torch.arange(pos.shape[0], device=pos.device)[:, None]
    row = (st[:, None] + pos - L0[:, None]).clamp(0, s["k"].shape[0] - 1)
    new = pos >= L0[:, None]
    ok = (pos >= 0) & (pos < L1[:, None])
    out = []
    for ring, fresh in ((wk, s["k"]), (wv, s["v"]), (ws, s["s"])):
        x = ring[seq, slot].float()
        y = fresh[row].float()
        m, o = (new[..., None], ok[..., None]) if x.dim() == 3 else (new, ok)
        out.append(torch.where(o, torch.where(m, y, x), 0.0))
    return out[0], out[1], out[2], ok


def _extended(s, wk, wv, ws):
    """The blocks that this step may complete: [S, blocks, 128, ...] from the block of the first
    new token on."""
    _, _, L0, L1 = _lens(s)
    nb = (s["n_max"] + 127 + BLOCK - 1) // BLOCK
    pos = (L0 - L0 % BLOCK)[:, None] + torch.arange(nb * BLOCK, device=L0.device)
    return _tokens(s, wk, wv, ws, pos), pos, nb


def _write_entries(s, ext):
    (k, v, sc, _), pos, nb = ext
    _, n, L0, L1 = _lens(s)
    S, P = pos.shape[0], s["page"]
    w = sc.view(S, nb, BLOCK)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    w = (w / w.sum(-1, keepdim=True))[:, :, None, :]
    j = (L0 // BLOCK)[:, None] + torch.arange(nb, device=pos.device)
    done = ((j + 1) * BLOCK <= L1[:, None]) & (n[:, None] > 0)
    page = s["table"].long().gather(1, (j // P).clamp(max=s["table"].shape[1] - 1))
    target = (page * P + j % P).flatten()
    done = done.flatten()
    # a block that does not complete repeats the first that does: equal values at one place
    some = done.any()
    pick = torch.where(done, torch.arange(done.numel(), device=done.device), done.int().argmax())
    target = torch.where(some, target[pick], 0)
    for pool, x in ((s["ck"], k), (s["cv"], v)):
        e = torch.matmul(w, x.view(S, nb, BLOCK, DIM)).view(S * nb, DIM)[pick].bfloat16()
        flat = pool.view(-1, DIM)
        flat[target] = torch.where(some, e, flat[target])


def _attend(s, wk, wv):
    st, n, L0, L1 = _lens(s)
    S, P, R, E = n.numel(), s["page"], s["n_max"], s["e_max"]
    N, dev = s["q"].shape[0], s["q"].device
    r = torch.arange(R, device=dev)
    t = L0[:, None] + r                                            # [S, R]
    rows = (st[:, None] + r).clamp(max=N - 1)
    q = s["q"][rows].float().view(S, R * HEADS, DIM)
    j = torch.arange(E, device=dev)
    page = s["table"].long()[:, j // P].clamp(min=0)               # [S, E]
    raw = (L0 - 127)[:, None] + torch.arange(127 + R, device=dev)
    rk, rv, _, _ = _tokens(s, wk, wv, wk[..., 0], raw)
    keys = torch.cat([s["ck"][page, j % P].float(), rk], 1)
    values = torch.cat([s["cv"][page, j % P].float(), rv], 1)
    seen = torch.cat([j < ((t - 127) // 128).clamp(min=0)[..., None],
                      (raw[:, None] <= t[..., None]) & (raw[:, None] > t[..., None] - 128)
                      & (raw[:, None] >= 0)], -1)                   # [S, R, E + 127 + R]
    x = torch.matmul(q, keys.transpose(1, 2)).view(S, R, HEADS, -1) * SCALE
    x.masked_fill_(~seen[:, :, None], float("-inf"))
    x = torch.exp(x - x.amax(-1, keepdim=True))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(S, R * HEADS, -1), values).view(S, R, HEADS, DIM) / total
    i = torch.arange(N, device=dev)
    seq = (i[:, None] >= (st + n)[None]).sum(1)
    o = o[seq, i - st[seq]]
    return (o / (1 + torch.exp(-s["g"].float()))).bfloat16()


def _write_rings(s, wk, wv, ws):
    st, n, L0, L1 = _lens(s)
    x = torch.arange(BLOCK, device=n.device)
    p = (L1 - 1)[:, None] - ((L1 - 1)[:, None] - x) % BLOCK        # newest position of slot x
    new = (p >= L0[:, None]) & (n > 0)[:, None]
    row = (st[:, None] + p - L0[:, None]).clamp(0, s["k"].shape[0] - 1)
    wk.copy_(torch.where(new[..., None], s["k"][row], wk))
    wv.copy_(torch.where(new[..., None], s["v"][row], wv))
    ws.copy_(torch.where(new, s["s"][row], ws))


def _free_list(ref):
    """Free pages in ascending order, then -1, and how many there are."""
    free = ref <= 0
    at = torch.where(free, free.cumsum(0) - 1, ref.numel())
    out = torch.full((ref.numel() + 1,), -1, dtype=torch.int32, device=ref.device)
    out[at] = torch.where(free, torch.arange(ref.numel(), device=ref.device), -1).to(torch.int32)
    return out[:-1], free.sum()


def _fork(s):
    table, n_pages, ref = s["table"].clone(), s["n_pages"].clone(), s["ref"].clone()
    S = table.shape[0]
    wk, wv, ws = rings(s["rings"], S)
    if own:
        import compressed_sliding_window_b200 as hca
        ok = hca.fork_pages(table, n_pages, ref, s["parents"], s["children"], s["entries"],
                            (s["ck"], s["cv"]), s["page"], rings=(wk, wv, ws))
        return {"table": table, "n_pages": n_pages, "ref": ref, "ok": ok, "ck": s["ck"],
                "cv": s["cv"], "rings": s["rings"]}
    a, b, e, P = s["parents"].long(), s["children"].long(), s["entries"].long(), s["page"]
    full, part = e // P, (e % P) > 0
    col = torch.arange(table.shape[1], device=table.device)
    shared = col < full[:, None]
    rows = torch.where(shared, table[a], -1)
    ref.index_add_(0, rows.clamp(min=0).flatten().long(), shared.flatten().int())
    free, count = _free_list(ref)
    rank = torch.where(part, part.cumsum(0) - 1, 0)
    fresh = free[rank]                                  # the pool has room for all of them
    old = table[a].gather(1, full[:, None].clamp(max=table.shape[1] - 1))[:, 0]
    rows = torch.where((col == full[:, None]) & part[:, None], fresh[:, None], rows)
    table[b] = rows
    n_pages[b] = (full + part).int()
    ref.index_add_(0, fresh.long(), part.int())
    # pages that a branch fills further are its own; without one it copies a page onto itself
    src = torch.where(part, old, table[0, 0]).long()
    dst = torch.where(part, fresh, table[0, 0]).long()
    for pool in (s["ck"], s["cv"]):
        pool[dst] = pool[src]
    for ring in (wk, wv, ws):
        ring[b] = ring[a]
    return {"table": table, "n_pages": n_pages, "ref": ref, "ok": torch.ones_like(s["parents"]),
            "ck": s["ck"], "cv": s["cv"], "rings": s["rings"]}


def _compact(s):
    table, n_pages, ref = s["table"].clone(), s["n_pages"].clone(), s["ref"].clone()
    if own:
        import compressed_sliding_window_b200 as hca
        hca.resize_pages(table, n_pages, ref, s["entries"], s["page"])
        live = hca.compact_pages(table, n_pages, ref, (s["ck"], s["cv"]))
        return {"table": table, "n_pages": n_pages, "ref": ref, "live": live, "ck": s["ck"],
                "cv": s["cv"]}
    P, total = s["page"], ref.numel()
    e = s["entries"].long()
    have = n_pages.long()
    want = torch.where(e < 0, have, (e + P - 1) // P).clamp(max=table.shape[1])
    col = torch.arange(table.shape[1], device=table.device)
    gone = (col >= want[:, None]) & (col < have[:, None])
    ref.index_add_(0, table.clamp(min=0).flatten().long(), -gone.flatten().int())
    table[:] = torch.where(gone, -1, table)
    grow = (col >= have[:, None]) & (col < want[:, None])
    rank = (grow.flatten().cumsum(0) - 1).view(grow.shape)
    free, count = _free_list(ref)
    got = grow & (rank < count)
    fresh = free[rank.clamp(0, total - 1)]
    table[:] = torch.where(got, fresh, table)
    ref.index_add_(0, torch.where(got, fresh, 0).flatten().long(), got.flatten().int())
    n_pages[:] = torch.minimum(have, want).int() + got.sum(1).int()
    # compact: live pages behind the live count move into the holes before it
    idx = torch.arange(total, device=ref.device)
    used = ref > 0
    live = used.sum()
    move, hole = used & (idx >= live), ~used & (idx < live)
    lists = []
    for m in (move, hole):
        x = torch.zeros(total + 1, dtype=torch.long, device=ref.device)
        x[torch.where(m, m.cumsum(0) - 1, total)] = idx
        lists.append(x[:-1])
    moves = move.sum()
    k = (total + 1) // 2                                 # never more moves than this
    real = torch.arange(k, device=ref.device) < moves
    # list places behind the last move copy a page onto itself (the last one, which no move fills)
    src = torch.where(real, lists[0][:k], total - 1)
    dst = torch.where(real, lists[1][:k], total - 1)
    for pool in (s["ck"], s["cv"]):
        pool[dst] = pool[src]
    to = torch.arange(total + 1, device=ref.device)
    to[torch.where(real, src, total)] = torch.where(real, dst, total)
    to = to[:-1]
    table[:] = torch.where(table >= 0, to[table.clamp(min=0).long()].int(), table)
    new_ref = torch.zeros_like(ref)
    new_ref.index_add_(0, to, torch.where(used, ref, 0))
    ref[:] = new_ref
    return {"table": table, "n_pages": n_pages, "ref": ref, "live": live.int()[None],
            "ck": s["ck"], "cv": s["cv"]}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    n, ctx = lengths(case)
    S, P = case["seqs"], case["page"]
    wk, wv, ws = (x.double() for x in rings(s["rings"], S))
    ck, cv = s["ck"].double(), s["cv"].double()
    if case["op"] == "fork":
        rows, total = pool_plan(case)
        free = sorted(set(range(total)) - {p for x in rows for p in x}, reverse=True)
        for a, b in fork_pairs(case):
            if (ctx[a] // BLOCK) % P:
                p, q = rows[a][ctx[a] // BLOCK // P], free.pop()
                ck[q], cv[q] = ck[p], cv[p]
            wk[b], wv[b], ws[b] = wk[a], wv[a], ws[a]
        flat = torch.cat([wk.flatten(), wv.flatten(), ws.flatten()])
        return {"table": None, "n_pages": None, "ref": None, "ok": None, "ck": ck, "cv": cv,
                "rings": flat}
    if case["op"] == "compact":
        rows, total = resized(case)
        used = sorted({p for x in rows for p in x})
        holes = sorted(set(range(len(used))) - set(used))
        for p, q in zip([p for p in used if p >= len(used)], holes):
            ck[q], cv[q] = ck[p], cv[p]
        return {"table": None, "n_pages": None, "ref": None, "live": None, "ck": ck, "cv": cv}
    k, v, sc = s["k"].double(), s["v"].double(), s["s"].double()
    table = s["table"].cpu().tolist()
    out = None if case["op"] == "append" else torch.empty_like(s["q"], dtype=torch.float64)
    at = 0
    for i, (m, L) in enumerate(zip(n, ctx)):
        if m == 0:
            continue
        L0 = L - m
        lo = max(0, L0 - 127)
        old = torch.arange(lo, L0, device=k.device) % BLOCK
        rk = torch.cat([wk[i, old], k[at:at + m]])      # raw tokens of positions lo .. L - 1
        rv = torch.cat([wv[i, old], v[at:at + m]])
        rs = torch.cat([ws[i, old], sc[at:at + m]])
        for j in range(L0 // BLOCK, L // BLOCK):
            a = j * BLOCK - lo
            w = torch.softmax(rs[a:a + BLOCK], 0)
            p, c = table[i][j // P], j % P
            ck[p, c], cv[p, c] = w @ rk[a:a + BLOCK], w @ rv[a:a + BLOCK]
        if out is not None:
            e = visible(L)
            pages = torch.tensor(table[i], device=k.device).clamp(min=0)
            ek, ev = ck[pages].view(-1, DIM)[:e], cv[pages].view(-1, DIM)[:e]
            # attention reads the entries as they are stored
            ek, ev = ek.bfloat16().double(), ev.bfloat16().double()
            for r0 in range(0, m, 64):
                r1 = min(m, r0 + 64)
                t0, t1 = L0 + r0, L0 + r1 - 1
                f0, f1 = max(0, t0 - 127), t1 + 1
                keys = torch.cat([ek[:visible(t1 + 1)], rk[f0 - lo:f1 - lo]])
                vals = torch.cat([ev[:visible(t1 + 1)], rv[f0 - lo:f1 - lo]])
                x = torch.einsum("rhd,kd->rhk", s["q"][at + r0:at + r1].double(), keys) * SCALE
                t = torch.arange(t0, t1 + 1, device=k.device)[:, None]
                seen = torch.cat([
                    torch.arange(visible(t1 + 1), device=k.device) < ((t - 127) // 128),
                    (torch.arange(f0, f1, device=k.device) <= t)
                    & (torch.arange(f0, f1, device=k.device) >= t - 127)], 1)
                x = torch.softmax(x.masked_fill(~seen[:, None], float("-inf")), -1)
                o = torch.einsum("rhk,kd->rhd", x, vals)
                out[at + r0:at + r1] = o * torch.sigmoid(s["g"][at + r0:at + r1].double())
        first = max(0, m - 128)
        p = torch.arange(L0 + first, L, device=k.device) % BLOCK
        wk[i, p], wv[i, p], ws[i, p] = k[at + first:at + m], v[at + first:at + m], \
            sc[at + first:at + m]
        at += m
    res = {"ck": ck, "cv": cv, "wk": wk, "wv": wv, "ws": ws}
    if out is not None:
        res["out"] = out
    return res
