"""smla_cache_copy, smla_cache_fork, smla_cache_free and smla_cache_compact against
references that go block by block: every cache format, tables and counts equal entry
for entry, pools bit for bit (the rows that no block has among them), in place and
into other arrays, captured, on another stream."""
import random

import pytest
import torch

from tests import _blocks as K
from tests import _paged as P

pytestmark = pytest.mark.gpu


def i32(x):
    return None if x is None else torch.tensor(list(x), dtype=torch.int32, device="cuda")


def guarded(t):
    """A copy of `t` between words that must stay."""
    buf = torch.full((t.numel() + 16,), 0x5A5A5A5A, dtype=torch.int32, device="cuda")
    view = buf[8:8 + t.numel()].view(t.shape)
    return buf, view


def untouched(buf):
    assert bool((buf[:8] == 0x5A5A5A5A).all()) and bool((buf[-8:] == 0x5A5A5A5A).all())


def forked(smla, pool, lens, table, ref, parents, children, room, place, status=0, layers=None,
           **kw):
    """Run the fork and compare it with the reference."""
    smla.smla_get_device_status(clear=True)
    cache, scale = pool.dev()
    block = pool.block
    d_table, d_lens, d_ref = table.cuda(), lens.cuda(), ref.cuda()
    was = d_table.clone(), d_lens.clone(), d_ref.clone()
    out, bufs = {}, []
    if place == "apart":
        for k, t in (("out_block_table", table), ("out_seq_lens", lens), ("out_refcount", ref)):
            buf, out[k] = guarded(t)
            bufs.append(buf)
    nbytes = smla.smla_cache_fork_workspace_size(len(children), table.shape[1], len(ref))
    ws = torch.full((nbytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    missing = smla.smla_cache_fork(
        i32(parents), i32(children), i32(room), d_lens, d_table, d_ref, block,
        cache if layers is None else [c for c in cache],
        pool.fmt, scale if layers is None or scale is None else [s for s in scale],
        block_stride_rows=pool.stride_rows, workspace=ws[:nbytes], **out, **kw)
    want = K.fork(pool, table, lens, ref, parents, children, room, block)
    torch.cuda.synchronize()
    assert bool((ws[nbytes:] == 0x5A).all())
    for b in bufs:
        untouched(b)
    got = [out.get(k, v) for k, v in (("out_block_table", d_table), ("out_seq_lens", d_lens),
                                      ("out_refcount", d_ref))]
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)
    assert int(missing) == want[3]
    if place == "apart":
        assert all(torch.equal(a, b) for a, b in zip(was, (d_table, d_lens, d_ref)))
    pool.same(cache, scale)
    assert smla.smla_get_device_status(clear=True) == status
    return want


@pytest.mark.parametrize("place", ["inplace", "apart"])
@pytest.mark.parametrize("fmt,d", K.FORMATS)
def test_fork_formats(cuda_lib, fmt, d, place):
    lens = [130, 64, 1, 0, 63, 200, 129, 40]
    table, lens, ref = K.tables(lens, 64, 6, 40, seed=fmt, shared=1)
    pool = K.Pool(fmt, d, 3, 40, 64, seed=d)
    forked(cuda_lib, pool, lens, table, ref, [0, 0, 0, 2, -1, 5], [0, 3, 7, 2, 6, 4],
           [1, 70, 0, 5, 100, 64], place)


@pytest.mark.parametrize("place", ["inplace", "apart"])
@pytest.mark.parametrize("block,stride", [(1, 0), (2, 5), (7, 0), (24, 24), (100, 0), (128, 130)])
def test_fork_block_sizes(cuda_lib, block, stride, place):
    rng = random.Random(block)
    lens = [rng.randint(0, 5 * block) for _ in range(30)]
    table, lens, ref = K.tables(lens, block, 9, 400, seed=block, shared=2, holes=20,
                                extra_refs=50)
    pool = K.Pool(P.BLOCK, 576, 2, 400, block, stride, extra=3, seed=1)
    children = rng.sample(range(30), 25)
    parents = [rng.randint(-1, 29) for _ in children]
    forked(cuda_lib, pool, lens, table, ref, parents, children,
           [rng.randint(0, 3 * block) for _ in children], place)


@pytest.mark.parametrize("seed", range(12))
def test_fork_random(cuda_lib, seed):
    """Small to wide tables, few to many pairs, scarce blocks."""
    rng = random.Random(seed)
    block = rng.choice([1, 3, 16, 64])
    R, W = rng.choice([1, 5, 70, 300]), rng.choice([1, 3, 40, 700])
    lens = [rng.randint(0, min(W, 12) * block) for _ in range(R)]
    need = sum(-(-n // block) for n in lens)
    NB = need + rng.choice([0, 1, 10, need, 5000])
    table, lens, ref = K.tables(lens, block, W, max(NB, 1), seed=seed, shared=rng.randint(0, 3))
    pool = K.Pool(P.E4M3, 512, 1, max(NB, 1), block, seed=seed)
    n = rng.randint(1, R)
    children = rng.sample(range(R), n)
    kind = rng.choice(["self", "one", "any"])
    parents = None if kind == "self" else \
        [children[0] if kind == "one" else rng.randint(-1, R - 1) for _ in children]
    room = rng.choice([None, [1] * n, [rng.randint(0, 4 * block) for _ in children]])
    W_over = any(-(-(max(0, int(lens[c if parents is None else p]) if (parents is None or p >= 0)
                          else 0) + r) // block) > W
                 for c, p, r in zip(children, parents or children, room or [0] * n))
    forked(cuda_lib, pool, lens, table, ref, parents, children, room,
           rng.choice(["inplace", "apart"]), status=5 if W_over else 0)


def test_fork_many_pairs(cuda_lib):
    """More pairs than a scan's step, beams that permute whole groups."""
    R = 2600
    rng = random.Random(3)
    lens = [rng.randint(1, 100) for _ in range(R)]
    table, lens, ref = K.tables(lens, 16, 8, 12000, seed=3)
    pool = K.Pool(P.BF16, 512, 1, 12000, 16, seed=3)
    children = list(range(R))
    rng.shuffle(children)
    parents = [c // 4 * 4 + rng.randrange(4) for c in children]
    forked(cuda_lib, pool, lens, table, ref, [min(p, R - 1) for p in parents], children,
           [1] * R, "inplace")


def test_fork_same_child_twice_and_numbers_out_of_range(cuda_lib):
    table, lens, ref = K.tables([100, 30, 70, 5], 16, 10, 60, seed=4)
    pool = K.Pool(P.GROUP128, 576, 2, 60, 16, seed=4)
    forked(cuda_lib, pool, lens, table, ref, [0, 1, 2, 2], [3, 3, -1, 3], [5, 6, 7, 8], "apart")
    pool = K.Pool(P.GROUP128, 576, 2, 60, 16, seed=4)
    forked(cuda_lib, pool, lens, table, ref, [0, 9, 2], [4, 1, 3], [5, 6, 7], "inplace", status=5)
    # entries and lengths that say more than there is
    table[0, 1], lens[2] = 60, 1 << 30
    pool = K.Pool(P.GROUP128, 576, 2, 60, 16, seed=4)
    forked(cuda_lib, pool, lens, table, ref, [0, 2], [1, 3], [1, 1], "apart", status=5)


def test_fork_without_pairs_or_room(cuda_lib):
    smla = cuda_lib
    table, lens, ref = K.tables([100, 30], 16, 10, 60, seed=5)
    pool = K.Pool(P.BF16, 576, 1, 60, 16)
    forked(smla, pool, lens, table, ref, [], [], [], "apart")
    forked(smla, pool, lens, table, ref, [1], [0], None, "apart")
    forked(smla, pool, lens, table, ref, None, [0, 1], None, "inplace", layers="list")


def test_fork_more_layers_than_a_launch_takes(cuda_lib):
    table, lens, ref = K.tables([33, 7], 16, 4, 12, seed=6)
    pool = K.Pool(P.BLOCK, 512, 300, 12, 16, seed=6)
    forked(cuda_lib, pool, lens, table, ref, [0, 0], [0, 1], [1, 20], "inplace")
    pool = K.Pool(P.DS_MLA, 576, 129, 12, 16, seed=6)
    forked(cuda_lib, pool, lens, table, ref, [0, 0], [0, 1], [1, 20], "apart", layers="list")


# ------------------------------------------------------------------ copy --

@pytest.mark.parametrize("fmt,d", K.FORMATS)
@pytest.mark.parametrize("block,stride", [(1, 0), (16, 0), (50, 64), (700, 0)])
def test_copy(cuda_lib, fmt, d, block, stride):
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    pool = K.Pool(fmt, d, 3, 12, block, stride, extra=2, seed=block)
    cache, scale = pool.dev()
    src, dst = [3, 7, -1, 3, 5, 11], [0, 1, 2, 4, 5, -1]
    smla.smla_cache_copy(cache, fmt, scale, i32(src), i32(dst), block, block_stride_rows=stride)
    for a, b in zip(src, dst):
        if a >= 0 and b >= 0:
            pool.copy(a, b, block)
    pool.same(cache, scale)
    assert smla.smla_get_device_status(clear=True) == 0
    end = (cache.shape[1] - block) // pool.step + 1       # the first number that is no block
    smla.smla_cache_copy(cache, fmt, scale, i32([end, 1 << 30, 1]), i32([6, 7, end]), block,
                         block_stride_rows=stride)
    pool.same(cache, scale)
    assert smla.smla_get_device_status(clear=True) == 5
    smla.smla_cache_copy(cache, fmt, scale, i32([]), i32([]), block, block_stride_rows=stride)


def test_copy_blocks_behind_2_to_32_bytes(cuda_lib):
    """A cache of 4.9 GB: its last block to its first, and back to one in the middle."""
    smla = cuda_lib
    blocks, block = 66000, 64
    cache = torch.zeros((blocks * block, 576), dtype=torch.bfloat16, device="cuda")
    last = torch.randn((block, 576), device="cuda").bfloat16()
    cache[-block:] = last
    smla.smla_cache_copy(cache, P.BF16, None, i32([blocks - 1]), i32([0]), block)
    smla.smla_cache_copy(cache, P.BF16, None, i32([0]), i32([60001]), block)
    assert torch.equal(cache[:block], last)
    assert torch.equal(cache[60001 * block:60002 * block], last)
    assert float(cache[block:2 * block].float().abs().sum()) == 0


# ------------------------------------------------------------------ free --

@pytest.mark.parametrize("place", ["inplace", "apart"])
@pytest.mark.parametrize("seed", range(8))
def test_free(cuda_lib, seed, place):
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    rng = random.Random(seed)
    block = rng.choice([1, 7, 64])
    R, W = rng.choice([1, 9, 200]), rng.choice([1, 20, 600])
    lens = [rng.randint(0, min(W, 30) * block) for _ in range(R)]
    NB = sum(-(-n // block) for n in lens) + 3
    table, _, ref = K.tables(lens, block, W, NB, seed=seed, shared=4, holes=R)
    rows = [rng.randint(-1, R - 1) for _ in range(rng.randint(1, 2 * R))]
    begin = None if seed % 3 == 0 else [rng.randint(-3, W * block) for _ in rows]
    end = None if seed % 2 == 0 else [rng.randint(-3, W * block + 9) for _ in rows]
    d_table, d_ref = table.cuda(), ref.cuda()
    out, bufs = {}, []
    if place == "apart":
        for k, t in (("out_block_table", table), ("out_refcount", ref)):
            buf, out[k] = guarded(t)
            bufs.append(buf)
    got = smla.smla_cache_free(i32(rows), i32(begin), i32(end), d_table, d_ref, block, **out)
    want = K.free(table, ref, rows, begin, end, block)
    for g, w in zip(got, want):
        assert torch.equal(g.cpu(), w)
    for b in bufs:
        untouched(b)
    assert smla.smla_get_device_status(clear=True) == 0
    smla.smla_cache_free(i32([R]), None, None, d_table, d_ref, block)
    assert smla.smla_get_device_status(clear=True) == 5


def test_free_positions_at_the_ends_of_int32(cuda_lib):
    table, _, ref = K.tables([100], 16, 8, 20, seed=1)
    for begin, end in ((0, 2**31 - 1), (2**31 - 1, 2**31 - 1), (-2**31, -2**31), (17, 2**31 - 1)):
        d_table, d_ref = table.cuda(), ref.cuda()
        cuda_lib.smla_cache_free(i32([0]), i32([begin]), i32([end]), d_table, d_ref, 16)
        want = K.free(table, ref, [0], [begin], [end], 16)
        assert torch.equal(d_table.cpu(), want[0]) and torch.equal(d_ref.cpu(), want[1])


# --------------------------------------------------------------- compact --

def compacted(smla, pool, table, ref, place, status=0):
    smla.smla_get_device_status(clear=True)
    cache, scale = pool.dev()
    d_table, d_ref = table.cuda(), ref.cuda()
    out, bufs = {}, []
    if place == "apart":
        for k, t in (("out_block_table", table), ("out_refcount", ref)):
            buf, out[k] = guarded(t)
            bufs.append(buf)
    nbytes = smla.smla_cache_compact_workspace_size(len(ref))
    ws = torch.full((nbytes + 256,), 0x5A, dtype=torch.uint8, device="cuda")
    mbuf, where = guarded(ref)
    got_map, live = smla.smla_cache_compact(d_table, d_ref, pool.block, cache, pool.fmt, scale,
                                            block_stride_rows=pool.stride_rows, block_map=where,
                                            workspace=ws[:nbytes], **out)
    want = K.compact(pool, table, ref, pool.block)
    torch.cuda.synchronize()
    for b in bufs + [mbuf]:
        untouched(b)
    assert bool((ws[nbytes:] == 0x5A).all())
    assert torch.equal(out.get("out_block_table", d_table).cpu(), want[0])
    assert torch.equal(out.get("out_refcount", d_ref).cpu(), want[1])
    assert torch.equal(got_map.cpu(), want[2]) and int(live) == want[3]
    pool.same(cache, scale)
    assert smla.smla_get_device_status(clear=True) == status


@pytest.mark.parametrize("place", ["inplace", "apart"])
@pytest.mark.parametrize("fmt,d", K.FORMATS)
def test_compact_formats(cuda_lib, fmt, d, place):
    table, _, ref = K.tables([130, 64, 1, 0, 63, 200], 16, 14, 90, seed=fmt + d, shared=2,
                             extra_refs=7)
    compacted(cuda_lib, K.Pool(fmt, d, 2, 90, 16, 18, extra=5, seed=2), table, ref, place)


@pytest.mark.parametrize("seed", range(10))
def test_compact_random(cuda_lib, seed):
    rng = random.Random(seed)
    block = rng.choice([1, 5, 32])
    R, W = rng.choice([1, 8, 300]), rng.choice([1, 30, 400])
    lens = [rng.randint(0, min(W, 20) * block) for _ in range(R)]
    need = sum(-(-n // block) for n in lens)
    NB = max(1, need + rng.choice([0, 1, need // 2, 4 * need, 30000]))
    table, _, ref = K.tables(lens, block, W, NB, seed=seed, shared=1)
    compacted(cuda_lib, K.Pool(P.BLOCK, 512, 1, NB, block, seed=seed), table, ref,
              ["inplace", "apart"][seed % 2])


def test_compact_full_empty_and_bad_entries(cuda_lib):
    smla = cuda_lib
    table = torch.arange(12, dtype=torch.int32).view(2, 6)
    pool = K.Pool(P.BF16, 512, 1, 12, 4)
    compacted(smla, pool, table, torch.ones(12, dtype=torch.int32), "inplace")
    compacted(smla, pool, torch.full((2, 6), -1, dtype=torch.int32),
              torch.zeros(12, dtype=torch.int32), "inplace")
    ref = torch.tensor([0, 1] * 6, dtype=torch.int32)     # entries that name free blocks, too
    compacted(smla, pool, table, ref, "apart")
    table[1, 2] = 12
    compacted(smla, pool, table, ref, "apart", status=5)


# ---------------------------------------------------- graphs and streams --

def test_captured_and_replayed(cuda_lib):
    """Fork, free and compact captured in place; each replay goes on from the last."""
    smla = cuda_lib
    block, NB = 16, 80
    table, lens, ref = K.tables([50, 20, 33, 0], block, 6, NB, seed=8)
    pool = K.Pool(P.BLOCK, 576, 2, NB, block, seed=8)
    cache, scale = pool.dev()
    t, l, r = table.cuda(), lens.cuda(), ref.cuda()
    parents, children, room = [1, 1, 0, -1], [0, 1, 3, 2], [20, 1, 3, 40]
    dp, dc, dr = i32(parents), i32(children), i32(room)
    rows, begin = i32([2]), i32([17])
    ws = torch.empty(smla.smla_cache_fork_workspace_size(4, 6, NB), dtype=torch.uint8,
                     device="cuda")
    ws2 = torch.empty(smla.smla_cache_compact_workspace_size(NB), dtype=torch.uint8, device="cuda")
    where, live, missing = (torch.empty(n, dtype=torch.int32, device="cuda") for n in (NB, 1, 1))

    def step():
        smla.smla_cache_fork(dp, dc, dr, l, t, r, block, cache, P.BLOCK, scale, workspace=ws,
                             missing=missing)
        smla.smla_cache_free(rows, begin, None, t, r, block)
        smla.smla_cache_compact(t, r, block, cache, P.BLOCK, scale, workspace=ws2,
                                block_map=where, num_live=live)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for _ in range(5):
        graph.replay()
        table, lens, ref, miss = K.fork(pool, table, lens, ref, parents, children, room, block)
        table, ref = K.free(table, ref, [2], [17], None, block)
        table, ref, _, n = K.compact(pool, table, ref, block)
        assert torch.equal(t.cpu(), table) and torch.equal(l.cpu(), lens)
        assert torch.equal(r.cpu(), ref) and int(live) == n and int(missing) == miss
        pool.same(cache, scale)


def test_another_stream(cuda_lib):
    smla = cuda_lib
    table, lens, ref = K.tables([500] * 40, 16, 40, 3000, seed=9)
    pool = K.Pool(P.BF16, 576, 2, 3000, 16, seed=9)
    cache, scale = pool.dev()
    t, l, r = table.cuda(), lens.cuda(), ref.cuda()
    children = list(range(40))
    parents = [c // 8 * 8 for c in children]
    args = i32(parents), i32(children), i32([1] * 40)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    missing = smla.smla_cache_fork(*args, l, t, r, 16, cache, P.BF16, stream=side)
    where, live = smla.smla_cache_compact(t, r, 16, cache, P.BF16, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    table, lens, ref, miss = K.fork(pool, table, lens, ref, parents, children, [1] * 40, 16)
    table, ref, want, n = K.compact(pool, table, ref, 16)
    assert torch.equal(t.cpu(), table) and torch.equal(r.cpu(), ref)
    assert torch.equal(where.cpu(), want) and int(live) == n and int(missing) == miss
    pool.same(cache, scale)


def test_binding_refusals(cuda_lib):
    smla = cuda_lib
    table, lens, ref = (x.cuda() for x in K.tables([50, 20], 16, 6, 20, seed=1))
    pool = K.Pool(P.BLOCK, 576, 2, 20, 16)
    cache, scale = pool.dev()
    one = i32([0])
    good = dict(parents=one, children=one, room=one, seq_lens=lens, block_table=table,
                refcount=ref, block_size=16, kv_caches=cache, kv_dtype=P.BLOCK, k_scales=scale)
    smla.smla_cache_fork(**good)
    for bad in (dict(parents=i32([0, 1])), dict(room=one.long()), dict(children=one.cpu()),
                dict(seq_lens=lens[:1]), dict(block_table=table.t()), dict(refcount=ref[:, None]),
                dict(k_scales=None), dict(k_scales=scale[:1]), dict(kv_caches=cache[:, :, :512]),
                dict(kv_caches=cache.cpu()), dict(kv_caches=[]), dict(kv_caches=cache.view(-1)),
                dict(kv_caches=[cache[0], cache[1][:16]]), dict(block_size=0),
                dict(block_stride_rows=8), dict(num_slots=321), dict(out_refcount=ref[:5]),
                dict(kv_dtype=9), dict(k_scales=scale.double())):
        with pytest.raises(ValueError):
            smla.smla_cache_fork(**{**good, **bad})
    with pytest.raises(smla.SmlaError):                   # more counted blocks than rows
        smla.smla_cache_fork(**{**good, "num_slots": 319})
    with pytest.raises(smla.SmlaError):
        smla.smla_cache_fork(**good, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        smla.smla_cache_copy(cache, P.BLOCK, scale, one, i32([1, 2]), 16)
    with pytest.raises(ValueError):
        smla.smla_cache_free(one, i32([1, 2]), None, table, ref, 16)
    with pytest.raises(ValueError):
        smla.smla_cache_compact(table, ref, 16, cache, P.BLOCK, scale, block_map=ref[:3])


def test_fork_and_free_of_most_rows(cuda_lib):
    """65536 rows at once (the most that a call names), each its own."""
    smla = cuda_lib
    R = 65536
    table = torch.arange(R, dtype=torch.int32, device="cuda")[:, None].repeat(1, 2)
    table[:, 1] = -1
    lens = torch.ones(R, dtype=torch.int32, device="cuda")
    ref = torch.zeros(2 * R, dtype=torch.int32, device="cuda")
    ref[:R] = 1
    cache = torch.zeros((2 * R * 2, 512), dtype=torch.uint8, device="cuda")
    names = torch.randperm(R, device="cuda").to(torch.int32)
    parents = names ^ 1                                   # pairs of rows trade places
    room = torch.full_like(names, 2)
    missing = smla.smla_cache_fork(parents, names, room, lens, table, ref, 2, cache, P.E4M3)
    assert int(missing) == 0
    # a row keeps its parent's only block and gets one free block, in the order of the pairs
    assert torch.equal(table[names.long(), 0], parents)
    assert torch.equal(table[names.long(), 1], torch.arange(R, 2 * R, dtype=torch.int32,
                                                            device="cuda"))
    assert bool((ref == 1).all())
    smla.smla_cache_free(names, None, None, table, ref, 2)
    assert bool((ref == 0).all()) and bool((table == -1).all())
