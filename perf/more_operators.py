"""Workloads of the paged cache's block operators (copying blocks in every
layer, forking table rows with copy-on-write and room for new tokens, giving
blocks back, compacting the pool) and of causal attention over the cache whose
scores are capped by a tanh, lowered with the distance, or limited to a span of
positions per token (documents, prefixes).

A table row is a request's list of cache blocks; refcount[b] is the number of
table entries that hold block b, 0 for a free block.  A free block is taken
from the lowest number on.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits), or through the library where ``own`` is set; ``exact`` computes the
attention in 64 bits, request by request.
"""
import random

import torch

own = False

D_V = 512
BF16, E4M3, GROUP128, DS_MLA, GROUP4_KPE, BLOCK = 0, 1, 2, 3, 4, 5
TENSOR_SCALE = 0.015625


# ---------------------------------------------------------------- cases --

def _pages(name, op, **kw):
    c = dict(name=name, op=op, fmt=BF16, d=576, block=64, layers=24, reqs=1, ctx=1000, n=1,
             spare=8, shape=1)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", fmt=BF16, reqs=1, new=1, ragged=0, ctx=1024, h=128, d=576,
             block=64, window=0, sinks=0, cap=0.0, slopes=False, doc=0, prefix=0, gain=4.0, pad=0,
             shape=1)
    c.update(kw)
    return c


def listed():
    return [
        # One block of one request, in all 60 layers: what a scheduler issues
        # when a shared block is about to be written.  Bound by latency.
        _pages("copy_one_block", "copy", layers=60, reqs=4, ctx=600, n=1, shape=11),
        # A pool's worth of blocks to other places, whole layers of bf16 rows.
        _pages("copy_many_blocks", "copy", layers=24, reqs=40, ctx=900, n=280, shape=12),
        # Eight samples of one prompt begin: seven rows share its blocks, and
        # each gets its own last block and room for the next token.
        _pages("fork_samples", "fork", layers=24, reqs=12, ctx=4000, n=8, room=1, kind="samples",
               shape=21),
        # A step of beam search: 64 requests of four beams, every row the
        # child of some row of its request, 8-bit rows with block scales.
        _pages("fork_beams", "fork", fmt=BLOCK, layers=32, reqs=256, ctx=3000, n=256, room=1,
               kind="beams", shape=22),
        # 16 requests of 64 are done.
        _pages("free_finished", "free", reqs=64, ctx=8000, n=16, kind="whole", shape=31),
        # Every one of 1024 long requests gives back what left its window.
        _pages("free_window", "free", reqs=1024, ctx=60000, n=1024, kind="window", shape=32),
        # A small pool of three quarters live blocks, 8-bit rows with scales
        # per group, ten layers.
        _pages("compact_small", "compact", fmt=GROUP128, layers=10, reqs=12, ctx=2000, spare=90,
               shape=41),
        # A large pool, half of it free, before its upper half is given away.
        _pages("compact_half", "compact", layers=6, reqs=64, ctx=2600, spare=1900, shape=42),
        # One user's next token with a distance bias, 16 heads on this GPU.
        _attend("bias_one_token", reqs=1, ctx=20000, h=16, slopes=True, shape=51),
        # A decode step of 64 requests under a cap, all 128 heads.
        _attend("cap_decode", reqs=64, ctx=8192, h=128, cap=30.0, gain=8.0, shape=52),
        # A packed prompt of documents that see themselves alone, each with a
        # prefix whose tokens see each other, under a cap.
        _attend("documents_prefill", reqs=2, new=4096, ctx=0, h=64, cap=50.0, gain=8.0, doc=1500,
                prefix=200, shape=53),
        # A mixed batch on 8-bit rows: chunks beside single tokens, with a
        # cap, a distance bias and a window, and padding rows at the end.
        _attend("mixed_block8", fmt=BLOCK, reqs=20, new=600, ragged=2, ctx=5000, h=32, cap=30.0,
                slopes=True, window=2048, sinks=4, gain=6.0, pad=9, shape=54),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    d = rng.choice([512, 576, 576])
    block = rng.choice([1, 7, 16, 24, 32, 64, 64, 100, 128])
    shape = rng.randint(1, 1 << 30)
    if rng.random() < 0.5:
        op = rng.choice(["copy", "fork", "fork", "free", "compact"])
        fmt = rng.choice([BF16, BF16, E4M3, GROUP128, BLOCK] +
                         ([DS_MLA, GROUP4_KPE] if d == 576 else []))
        reqs, ctx = _log_int(rng, 1, 500), _log_int(rng, 1, 20000)
        while reqs * (-(-ctx // block)) > 2_000_000 // block and reqs * ctx > 1:
            reqs, ctx = max(1, reqs // 2), max(1, ctx // 2)
        layers = _log_int(rng, 1, 60)
        per = reqs * (ctx + block) * 2
        while layers > 1 and per * layers * _row_bytes(fmt, d) > 1 << 30:
            layers //= 2
        c = dict(op=op, fmt=fmt, d=d, block=block, layers=layers, reqs=reqs, ctx=ctx,
                 n=_log_int(rng, 1, reqs), spare=_log_int(rng, 1, reqs * (ctx // block + 1) + 4),
                 shape=shape)
        if op == "copy":
            c["n"] = _log_int(rng, 1, max(1, reqs * (ctx // block) // 2))
        if op == "fork":
            c.update(room=rng.choice([0, 1, 1, _log_int(rng, 1, 300)]),
                     kind=rng.choice(["samples", "beams", "mixed"]))
        if op == "free":
            c["kind"] = rng.choice(["whole", "window", "tail"])
        return c
    fmt = rng.choice([BF16, BF16, E4M3, BLOCK, BLOCK])
    h = rng.choice([1, 5, 8, 16, 24, 32, 64, 96, 128])
    window = rng.choice([0, 0, _log_int(rng, 1, 4096)])
    sinks = rng.choice([0, 4, rng.randint(1, 200)])
    reqs = _log_int(rng, 1, 64)
    new = rng.choice([1, _log_int(rng, 1, 2048)])
    ctx = _log_int(rng, 1, 32768)
    while reqs * new * h * (new + ctx) > 8e8:
        if new > 64:
            new //= 2
        elif reqs > 4:
            reqs //= 2
        else:
            ctx //= 2
    ctx = max(1, min(ctx, 400000 // reqs))
    return dict(op="attend", fmt=fmt, reqs=reqs, new=new, ragged=rng.randint(0, 2), ctx=ctx, h=h,
                d=d, block=block, window=window, sinks=sinks, cap=rng.choice([0.0, 20.0, 50.0]),
                slopes=rng.random() < 0.5, doc=rng.choice([0, 0, _log_int(rng, 3, 3000)]),
                prefix=rng.choice([0, _log_int(rng, 1, 500)]), gain=rng.choice([2.0, 4.0, 8.0]),
                pad=rng.choice([0, 0, rng.randint(1, 40)]), shape=shape)


def _row_bytes(fmt, d):
    return {BF16: 2 * d, DS_MLA: 656}.get(fmt, d)


def _scale_groups(fmt, d):
    """fp32 scales of one row."""
    return {GROUP128: -(-d // 128), GROUP4_KPE: 4}.get(fmt, 0)


def _copied(case, rows):
    """Bytes of `rows` rows of the cache in every layer."""
    return rows * case["layers"] * (_row_bytes(case["fmt"], case["d"]) +
                                    4 * _scale_groups(case["fmt"], case["d"]))


def _lengths(case):
    rng = random.Random(case["shape"])
    return [rng.randint(case["ctx"] // 2, case["ctx"]) for _ in range(case["reqs"])]


def _width(case):
    """Columns of the block table: the longest request and room to grow."""
    return -(-(case["ctx"] + case.get("room", 0)) // case["block"]) + 2


def _family(case):
    """(children, parents, room) of a fork."""
    rng = random.Random(case["shape"] + 1)
    R, n, kind, room = case["reqs"], case["n"], case["kind"], case["room"]
    children = rng.sample(range(R), n)
    if kind == "samples":                       # all of one request, which goes on itself
        parents = [children[0]] * n
    elif kind == "beams":                       # of one of four rows next to it
        parents = [min(R - 1, c // 4 * 4 + rng.randrange(4)) for c in children]
    else:                                       # forks, new requests, rows that go on
        parents = [rng.choice([-1, c, rng.randrange(R)]) for c in children]
    rooms = [rng.randint(0, room) if kind == "mixed" else room for _ in children]
    return children, parents, rooms


def _copies(case):
    """Rows of cache that a fork has to copy."""
    lens, B = _lengths(case), case["block"]
    children, parents, rooms = _family(case)
    kept = set(range(case["reqs"])) - set(children)
    rows = 0
    for p in set(parents):
        if p < 0 or lens[p] % B == 0:
            continue
        mine = [i for i, q in enumerate(parents) if q == p]
        writers = sum(rooms[i] > 0 for i in mine)
        alone = writers == len(mine) and p not in kept
        rows += max(0, writers - (1 if alone else 0)) * (lens[p] % B)
    return rows


def _batch(case):
    """[(new tokens, positions after them)] of the case's requests."""
    rng = random.Random(case["shape"])
    rows = []
    for _ in range(case["reqs"]):
        n = case["new"]
        if case["ragged"] and n > 1:
            n = rng.randint(max(1, n // 4), n)
        if case["ragged"] == 2 and rng.random() < 0.5:
            n = 1
        rows.append((n, n + rng.randint(case["ctx"] // 2, case["ctx"])))
    return rows


def _spans(case):
    """(first, last) position that each token sees by its document and its
    document's prefix, per request."""
    rng = random.Random(case["shape"] + 2)
    doc, prefix = case["doc"], case["prefix"]
    out = []
    for n, L in _batch(case):
        ends = []
        while doc and (not ends or ends[-1] < L):
            ends.append((ends[-1] if ends else 0) + rng.randint(max(1, doc // 2), 2 * doc))
        ends = [e for e in ends if e < L] + [L]
        first, last, at, begin = [], [], 0, 0
        for p in range(L - n, L):
            while p >= ends[at]:
                begin, at = ends[at], at + 1
            first.append(begin)
            last.append(min(max(p, begin + prefix - 1), ends[at] - 1))
        out.append((first, last))
    return out


def work(case):
    op = case["op"]
    if op != "attend":
        R, B = case["reqs"], case["block"]
        need = sum(-(-L // B) for L in _lengths(case))
        pool = need + case["spare"]
        table = 4 * R * _width(case)
        if op == "copy":
            return {"bytes": 8 * case["n"] + 2 * _copied(case, case["n"] * B), "flops": 0}
        meta = 2 * table + 2 * 4 * pool
        if op == "fork":
            return {"bytes": meta + 8 * R + 12 * case["n"] + 2 * _copied(case, _copies(case)),
                    "flops": 0}
        if op == "free":
            return {"bytes": meta + 12 * case["n"], "flops": 0}
        moved = need * case["spare"] // pool              # the expected number of moves
        return {"bytes": meta + 4 * pool + 2 * _copied(case, moved * B), "flops": 0}
    rows, h, d = _batch(case), case["h"], case["d"]
    N = sum(n for n, _ in rows)
    window, sinks = case["window"], case["sinks"]
    keys = pairs = 0
    for (n, L), (first, last) in zip(rows, _spans(case)):
        at = top = 0                                       # keys of the request that some token sees
        for p, f, l in zip(range(L - n, L), first, last):
            lo = max(f, p - window + 1) if window else f
            pairs += max(0, l + 1 - lo) + min(sinks, lo)
            keys += max(0, l + 1 - max(lo, at))
            at, top = max(at, l + 1), max(top, min(sinks, lo))
        keys += top
    pages = 4 * sum(-(-L // case["block"]) for _, L in rows)
    scales = pages if case["fmt"] == BLOCK else 0
    spans = 4 * N * (bool(case["doc"]) + bool(case["doc"] or case["prefix"]))
    return {"bytes": keys * _row_bytes(case["fmt"], d) + N * h * (2 * d + 2 * D_V + 4) + pages +
            scales + spans + (4 * h if case["slopes"] else 0),
            "flops": 2 * pairs * h * (d + D_V)}


# --------------------------------------------------------------- inputs --

def _fill(shape, fmt, d, gen):
    """Cache rows [*shape, row] as earlier steps left them."""
    if fmt == BF16:
        return torch.empty((*shape, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    c = torch.randint(0, 127, (*shape, _row_bytes(fmt, d)), dtype=torch.uint8, generator=gen,
                      device="cuda")                       # codes that are numbers
    if fmt == DS_MLA:
        c[..., 512:528] = torch.full((*shape, 4), 2.0 ** -6, device="cuda").view(torch.uint8)
        c[..., 528:] = torch.empty((*shape, 64), dtype=torch.bfloat16, device="cuda").normal_(
            generator=gen).view(torch.uint8)
    return c


def _prepare_pages(case, gen):
    B, R, L, fmt, d = (case[k] for k in ("block", "reqs", "layers", "fmt", "d"))
    W = _width(case)
    lens = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
    need = (lens.long() + B - 1) // B
    pool = int(need.sum()) + case["spare"]
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    at = (need.cumsum(0) - need)[:, None]
    col = torch.arange(W, device="cuda")[None, :]
    have = col < need[:, None]
    table = torch.where(have, order[(at + col).clamp(max=pool - 1)], -1).to(torch.int32)
    ref = torch.zeros(pool, dtype=torch.int32, device="cuda")
    ref[table[have].long()] = 1
    s = dict(case=case, table=table, lens=lens, ref=ref, pool=pool)
    if case["op"] != "free":
        s["cache"] = _fill((L, pool * B), fmt, d, gen)
        G = _scale_groups(fmt, d)
        s["scale"] = None
        if G:
            s["scale"] = torch.rand((L, pool * B, G), generator=gen, device="cuda")
        elif fmt == BLOCK:
            s["scale"] = torch.exp2(torch.randint(-9, -4, (L, pool), generator=gen,
                                                  device="cuda").float())
        elif fmt == E4M3:
            s["scale"] = torch.full((L, 1), TENSOR_SCALE, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    if case["op"] == "copy":
        both = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
        n = min(case["n"], pool // 2)
        s["src"], s["dst"] = both[:n].clone(), both[n:2 * n].clone()
    elif case["op"] == "fork":
        s["children"], s["parents"], s["room"] = (torch.tensor(x, **i32) for x in _family(case))
    elif case["op"] == "free":
        rng = random.Random(case["shape"] + 1)
        rows = rng.sample(range(R), case["n"])
        s["rows"] = torch.tensor(rows, **i32)
        s["begin"] = s["end"] = None
        lengths = _lengths(case)
        if case["kind"] == "window":                       # all but the sinks and the window
            s["begin"] = torch.full((len(rows),), 4, **i32)
            s["end"] = torch.tensor([max(0, lengths[r] - 1024) for r in rows], **i32)
        elif case["kind"] == "tail":                       # what was drafted and not accepted
            s["begin"] = torch.tensor([rng.randint(0, lengths[r]) for r in rows], **i32)
    return s


def _prepare_attend(case, gen):
    rows, block, h, d, fmt = _batch(case), case["block"], case["h"], case["d"], case["fmt"]
    need = [-(-L // block) for _, L in rows]
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    at = torch.cumsum(torch.tensor([0] + need[:-1], device="cuda"), 0)[:, None]
    col = torch.arange(max(need), device="cuda")[None, :]
    have = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(have, order[(at + col).clamp(max=pool - 1)], -1).to(torch.int32)
    N = sum(n for n, _ in rows) + case["pad"]
    s = dict(case=case, table=table.contiguous(), N=N,
             start=torch.tensor([0] + [n for n, _ in rows], device="cuda").cumsum(0).to(torch.int32),
             lens=torch.tensor([L for _, L in rows], dtype=torch.int32, device="cuda"),
             max_new=max(n for n, _ in rows), max_len=max(L for _, L in rows))
    x = torch.empty((pool * block, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    s["scale"] = None
    if fmt == BF16:
        s["cache"] = x
    else:
        s["cache"] = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        s["scale"] = torch.full((1,), TENSOR_SCALE, device="cuda") if fmt == E4M3 else \
            torch.exp2(torch.randint(-8, -4, (pool,), generator=gen, device="cuda").float())
    s["q"] = torch.empty((N, h, d), dtype=torch.bfloat16, device="cuda").normal_(
        generator=gen) * case["gain"]
    s["slopes"] = None
    if case["slopes"]:                                     # a geometric row of slopes
        s["slopes"] = torch.exp2(-8.0 * torch.arange(1, h + 1, device="cuda") / h).float()
    first, last = zip(*_spans(case))
    pack = [torch.tensor(sum(v, []) + [0] * case["pad"], dtype=torch.int32, device="cuda")
            for v in (first, last)]
    s["first"] = pack[0] if case["doc"] else None
    s["last"] = pack[1] if case["doc"] or case["prefix"] else None
    s["out"] = torch.zeros((N, h, D_V), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((N, h), dtype=torch.float32, device="cuda")
    s["sm_scale"] = d ** -0.5
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return _prepare_attend(case, gen) if case["op"] == "attend" else _prepare_pages(case, gen)


# ----------------------------------------------------------- plain forms --

def _values(s):
    """The cache as the values that it holds."""
    c, fmt = s["cache"], s["case"]["fmt"]
    if fmt == BF16:
        return {"cache": c}
    if fmt == DS_MLA:
        return {"codes": c[..., :512].view(torch.float8_e4m3fn),
                "scale": c[..., 512:528].view(torch.float32),
                "rope": c[..., 528:].view(torch.bfloat16)}
    return {"codes": c.view(torch.float8_e4m3fn), "scale": s["scale"]}


def _copy_rows(s, src, dst, rows):
    """Rows [0, rows) of blocks src to blocks dst in every layer, with their
    scales."""
    B, fmt, d = s["case"]["block"], s["case"]["fmt"], s["case"]["d"]
    j = torch.arange(B, device="cuda")
    keep = j[None, :] < rows[:, None]
    a = (src.long()[:, None] * B + j)[keep]
    b = (dst.long()[:, None] * B + j)[keep]
    s["cache"][:, b] = s["cache"][:, a]
    if _scale_groups(fmt, d):
        s["scale"][:, b] = s["scale"][:, a]
    elif fmt == BLOCK:
        s["scale"][:, dst.long()] = s["scale"][:, src.long()]


def _plain_copy(s):
    _copy_rows(s, s["src"], s["dst"], torch.full_like(s["src"], s["case"]["block"]))
    return _values(s)


def _plain_fork(s):
    B, table, ref = s["case"]["block"], s["table"], s["ref"].clone()
    c, p, room = s["children"].long(), s["parents"].long(), s["room"].long()
    length = torch.where(p >= 0, s["lens"].long()[p.clamp(min=0)], 0)
    col = torch.arange(table.shape[1], device="cuda")[None, :]
    have = (length + B - 1) // B
    row = torch.where(col < have[:, None], table[p.clamp(min=0)], -1)
    old = table[c]
    one = torch.ones((), dtype=torch.int32, device="cuda")
    ref.index_add_(0, old[old >= 0].long(), -one.expand(int((old >= 0).sum())))
    ref.index_add_(0, row[row >= 0].long(), one.expand(int((row >= 0).sum())))
    # a row that will be written and whose last block others hold too gets a
    # copy of it; where only such rows hold it, the first of them keeps it
    at = (length // B).clamp(max=table.shape[1] - 1)
    last = torch.gather(row, 1, at[:, None])[:, 0].long()
    writes = (room > 0) & (length % B > 0) & (last >= 0)
    same = (last[:, None] == last[None, :]) & writes[:, None] & writes[None, :]
    copy = writes & ((same.tril(-1).sum(1) > 0) | (ref[last.clamp(min=0)] > same.sum(1)))
    ref.index_add_(0, last[copy], -one.expand(int(copy.sum())))
    end = (length + room + B - 1) // B
    take = ((col >= have[:, None]) & (col < end[:, None])) | (copy[:, None] & (col == at[:, None]))
    free = torch.nonzero(ref == 0).flatten()
    k = take.flatten().cumsum(0)[take.flatten()] - 1
    got = torch.where(k < free.numel(), free[k.clamp(max=max(0, free.numel() - 1))], -1) \
        if free.numel() else torch.full_like(k, -1)
    row[take] = got.to(torch.int32)
    ref[got[got >= 0]] = 1
    dst = torch.gather(row, 1, at[:, None])[:, 0]
    do = copy & (dst >= 0)
    _copy_rows(s, last[do], dst[do], (length % B)[do])
    table, lens = table.clone(), s["lens"].clone()
    table[c] = row
    lens[c] = length.to(torch.int32)
    return {"table": table, "lens": lens, "ref": ref,
            "missing": (k.numel() - (got >= 0).sum()).to(torch.int32)[None], **_values(s)}


def _plain_free(s):
    B, table, ref = s["case"]["block"], s["table"].clone(), s["ref"].clone()
    r, W = s["rows"].long(), s["table"].shape[1]
    col = torch.arange(W, device="cuda")[None, :]
    lo = torch.zeros_like(r) if s["begin"] is None else (s["begin"].long() + B - 1) // B
    hi = torch.full_like(r, W) if s["end"] is None else s["end"].long() // B
    row = table[r]
    give = (col >= lo[:, None]) & (col < hi[:, None]) & (row >= 0)
    blocks = row[give].long()
    ref.index_add_(0, blocks, torch.full_like(blocks, -1).to(torch.int32))
    table[r] = torch.where(give, -1, row)
    return {"table": table, "ref": ref}


def _plain_compact(s):
    ref, table, B = s["ref"], s["table"], s["case"]["block"]
    live = torch.nonzero(ref > 0).flatten()
    count = live.numel()
    src = live[live >= count].flip(0)                      # the highest live blocks first
    dst = torch.nonzero(ref[:count] == 0).flatten()        # to the lowest free places
    where = torch.where(ref > 0, torch.arange(ref.numel(), device="cuda"), -1)
    where[src] = dst
    new = ref.clone()
    new[dst] = ref[src]
    new[src] = 0
    table = torch.where(table >= 0, where[table.long().clamp(min=0)], -1).to(torch.int32)
    _copy_rows(s, src, dst, torch.full_like(src, B))
    return {"table": table, "ref": new, "map": where.to(torch.int32),
            "live": torch.full((1,), count, dtype=torch.int32, device="cuda"), **_values(s)}


def _plain_attend(s):
    case, block = s["case"], s["case"]["block"]
    h, window, fmt = case["h"], case["window"], case["fmt"]
    start, lens = s["start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    i = torch.arange(s["max_new"], device="cuda")
    tok = (start[:-1, None] + i).clamp(max=s["N"] - 1)             # [R, new]
    live = i < n[:, None]
    qpos = (lens - n)[:, None] + i
    kpos = torch.arange(s["max_len"], device="cuda").expand(len(lens), -1)
    page = torch.gather(s["table"].long(), 1, (kpos // block).clamp(max=s["table"].shape[1] - 1))
    real = (kpos < lens[:, None]) & (page >= 0)
    slot = torch.where(real, page * block + kpos % block, 0)
    if fmt == BF16:
        k = s["cache"][slot].float()
    else:
        k = s["cache"][slot].view(torch.float8_e4m3fn).float()
        k *= s["scale"][page.clamp(min=0)][:, :, None] if fmt == BLOCK else s["scale"]
    lo = torch.zeros_like(qpos) if s["first"] is None else s["first"].long()[tok]
    if window:
        lo = torch.maximum(lo, qpos - window + 1)
    hi = qpos if s["last"] is None else s["last"].long()[tok]
    sees = (kpos[:, None, :] >= lo[:, :, None]) | (kpos < case["sinks"])[:, None, :]
    sees &= real[:, None, :] & (kpos[:, None, :] <= hi[:, :, None])
    q = s["q"][tok].float().flatten(1, 2)                          # [R, new * h, d]
    w = torch.matmul(q, k.transpose(1, 2)).mul_(s["sm_scale"])
    if case["cap"]:
        w = w.div_(case["cap"]).tanh_().mul_(case["cap"])
    w = w.view(len(lens), s["max_new"], h, -1)
    if s["slopes"] is not None:
        far = (kpos[:, None, :] - qpos[:, :, None]).abs().float()
        w -= s["slopes"][None, None, :, None] * far[:, :, None, :]
    w.masked_fill_(~sees[:, :, None, :], float("-inf"))
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0, top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.flatten(1, 2), k[:, :, :D_V]).view(*w.shape[:3], D_V)
    o = torch.where(total > 0, o / total, 0)
    s["out"][tok[live]] = o[live].to(torch.bfloat16)
    s["lse"][tok[live]] = (top + total.log())[..., 0][live]
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        import sparse_mla_attention_02_gb300 as smla
        if op == "attend":
            out, lse = smla.smla_fwd_scored(
                s["q"], s["cache"], case["fmt"], s["scale"], s["start"], s["lens"], s["table"],
                case["block"], s["sm_scale"], softcap=case["cap"], slopes=s["slopes"],
                first_pos=s["first"], last_pos=s["last"], window=case["window"],
                sinks=case["sinks"], max_seq_len=s["max_len"], out=s["out"], lse=s["lse"])
            return {"out": out, "lse": lse}
        if op == "copy":
            smla.smla_cache_copy(s["cache"], case["fmt"], s["scale"], s["src"], s["dst"],
                                 case["block"])
            return _values(s)
        # (new tables beside the ones that a step in flight still reads)
        table, ref = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
        if op == "fork":
            lens = torch.empty_like(s["lens"])
            missing = smla.smla_cache_fork(
                s["parents"], s["children"], s["room"], s["lens"], s["table"], s["ref"],
                case["block"], s["cache"], case["fmt"], s["scale"], out_seq_lens=lens,
                out_block_table=table, out_refcount=ref)
            return {"table": table, "lens": lens, "ref": ref, "missing": missing, **_values(s)}
        if op == "free":
            smla.smla_cache_free(s["rows"], s["begin"], s["end"], s["table"], s["ref"],
                                 case["block"], out_block_table=table, out_refcount=ref)
            return {"table": table, "ref": ref}
        where, live = smla.smla_cache_compact(
            s["table"], s["ref"], case["block"], s["cache"], case["fmt"], s["scale"],
            out_block_table=table, out_refcount=ref)
        return {"table": table, "ref": ref, "map": where, "live": live, **_values(s)}
    return {"copy": _plain_copy, "fork": _plain_fork, "free": _plain_free,
            "compact": _plain_compact, "attend": _plain_attend}[op](s)


# ------------------------------------------------------------- 64 bits --

def exact(case, seed):
    if case["op"] != "attend":                             # nothing that is rounded
        return None
    s = prepare(case, seed)
    block, h, window, sinks, fmt = (case[k] for k in ("block", "h", "window", "sinks", "fmt"))
    start, lens = s["start"].tolist(), s["lens"].tolist()
    out, lse = s["out"].double(), s["lse"].double()
    spans = _spans(case)
    for r, L in enumerate(lens):
        e = torch.arange(L, device="cuda")
        page = s["table"][r].long()[e // block]
        rows = s["cache"][page * block + e % block]
        if fmt == BF16:
            k = rows.double()
        else:
            k = rows.view(torch.float8_e4m3fn).double()
            k *= s["scale"].double()[page][:, None] if fmt == BLOCK else s["scale"].double()
        n = start[r + 1] - start[r]
        for c in range(0, n, 64):
            m = min(64, n - c)
            p = torch.arange(L - n + c, L - n + c + m, device="cuda")
            f = torch.tensor(spans[r][0][c:c + m], device="cuda") if case["doc"] else p * 0
            if window:
                f = torch.maximum(f, p - window + 1)
            f = f.clamp(min=0)
            t = torch.tensor(spans[r][1][c:c + m], device="cuda") \
                if case["doc"] or case["prefix"] else p
            lo, hi = int(f.min()), int(t.max())
            at = torch.cat([e[:min(sinks, lo)], e[lo:hi + 1]])
            x = (s["q"][start[r] + c:start[r] + c + m].double().flatten(0, 1) @ k[at].T)
            x = x.view(m, h, -1) * s["sm_scale"]
            if case["cap"]:
                x = torch.tanh(x / case["cap"]) * case["cap"]
            if case["slopes"]:
                x = x - s["slopes"].double()[None, :, None] * (at - p[:, None]).abs()[:, None, :]
            hide = (at > t[:, None]) | ((at < f[:, None]) & (at >= sinks))
            x = x.masked_fill(hide[:, None, :], float("-inf"))
            g = slice(start[r] + c, start[r] + c + m)
            lse[g] = torch.logsumexp(x, -1)
            out[g] = (torch.softmax(x, -1).flatten(0, 1) @ k[at, :D_V]).view(m, h, D_V)
    return {"out": out, "lse": lse}
