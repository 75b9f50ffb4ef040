"""Forks that run out of free blocks: what a row has written stays, the shared block with
its holders where no block was left to copy it into, and a later call makes the copy."""
import random

import pytest
import torch

from tests import _blocks as K
from tests import _paged as P
from tests.test_blocks_gpu import guarded, i32, untouched

pytestmark = pytest.mark.gpu


def short_fork(pool, table, lens, ref, parents, children, room, block):
    """(table, lens, ref, missing); the pool is changed.  The same fork on a pool that is
    large enough, blocks behind the real ones standing for those that could not be had:
    a row's last block stays the shared one, its columns stay empty."""
    NB, W = len(ref), table.shape[1]
    more = len(children) * (W + 1)
    pad = torch.zeros((pool.cache.shape[0], more * pool.step, pool.cache.shape[2]),
                      dtype=pool.cache.dtype)
    big = K.Pool.__new__(K.Pool)
    big.__dict__.update(pool.__dict__, cache=torch.cat([pool.cache, pad], 1))
    if pool.scale is not None:
        n = more if pool.fmt == P.BLOCK else more * pool.step
        shape = (pool.scale.shape[0], n, *pool.scale.shape[2:])
        big.scale = torch.cat([pool.scale, torch.zeros(shape)], 1)
    t, l, r, _ = K.fork(big, table, lens, torch.cat([ref, torch.zeros(more, dtype=ref.dtype)]),
                        parents, children, room, block)
    pool.cache = big.cache[:, :pool.cache.shape[1]].clone()
    if pool.scale is not None:
        pool.scale = big.scale[:, :pool.scale.shape[1]].clone()
    missing = int((t >= NB).sum())
    r = r[:NB].clone()
    for i in K.last_only(list(children), len(table)):
        c, p = children[i], children[i] if parents is None else parents[i]
        have = -(-int(l[c]) // block)
        for col in range(W):
            if t[c, col] >= NB:
                if col < have:
                    t[c, col] = table[p, col]
                    r[t[c, col]] += 1
                else:
                    t[c, col] = -1
    return t, l, r, missing


class State:
    def __init__(self, smla, pool, table, lens, ref):
        self.smla, self.pool, self.host = smla, pool, (table, lens, ref)
        self.dev = table.cuda(), lens.cuda(), ref.cuda()
        self.cache, self.scale = pool.dev()
        smla.smla_get_device_status(clear=True)

    def fork(self, parents, children, room, place="inplace"):
        block, out, bufs = self.pool.block, {}, []
        t, l, r = self.dev
        if place == "apart":
            for k, x in (("out_block_table", t), ("out_seq_lens", l), ("out_refcount", r)):
                buf, out[k] = guarded(x)
                bufs.append(buf)
        missing = self.smla.smla_cache_fork(
            i32(parents), i32(children), i32(room), l, t, r, block, self.cache, self.pool.fmt,
            self.scale, block_stride_rows=self.pool.stride_rows, **out)
        *self.host, want = short_fork(self.pool, *self.host, parents, children, room, block)
        if place == "apart":
            for x, was in zip(self.dev, (t, l, r)):
                assert torch.equal(x, was)
            self.dev = out["out_block_table"], out["out_seq_lens"], out["out_refcount"]
        for g, w in zip(self.dev, self.host):
            assert torch.equal(g.cpu(), w)
        for b in bufs:
            untouched(b)
        assert int(missing) == want
        self.pool.same(self.cache, self.scale)
        assert self.smla.smla_get_device_status(clear=True) == 0
        return want


@pytest.mark.parametrize("place", ["inplace", "apart"])
@pytest.mark.parametrize("fmt,d", K.FORMATS)
def test_the_shared_block_stays_and_a_later_call_copies_it(cuda_lib, fmt, d, place):
    """Three samples of a row of ten positions, one free block for two copies."""
    table = torch.full((3, 3), -1, dtype=torch.int32)
    table[0, 0] = 1
    s = State(cuda_lib, K.Pool(fmt, d, 2, 2, 16, seed=fmt), table,
              torch.tensor([10, 0, 0], dtype=torch.int32),
              torch.tensor([0, 1], dtype=torch.int32))
    assert s.fork([0, 0, 0], [0, 1, 2], [1, 1, 1], place) == 1
    table, lens, ref = s.host
    assert table[:, 0].tolist() == [1, 0, 1] and ref.tolist() == [1, 2]
    assert lens.tolist() == [10, 10, 10]
    # the row that shares still does, and says so again
    assert s.fork(None, [2], [1], place) == 1
    # the second row is done: its block becomes the third's own
    free = torch.tensor([1], dtype=torch.int32, device="cuda")
    cuda_lib.smla_cache_free(free, None, None, s.dev[0], s.dev[2], 16)
    s.host[0][1, 0], s.host[2][0] = -1, 0
    assert s.fork(None, [2], [1], place) == 0
    assert s.host[0][:, 0].tolist() == [1, -1, 0] and s.host[2].tolist() == [1, 1]


@pytest.mark.parametrize("seed", range(24))
def test_short_at_random(cuda_lib, seed):
    """Few to many pairs on small and large tables, next to no free blocks, then again
    after some came back."""
    rng = random.Random(seed)
    block = rng.choice([3, 16, 64])
    R = [5, 40, 300, 1500][seed % 4]
    W = rng.choice([5, 9, 200 if R == 300 else 9])
    # odd rows are empty and become samples of even ones, which go on
    lens = [0 if r % 2 else rng.randint(1, 4 * block) for r in range(R)]
    NB = sum(-(-n // block) for n in lens) + rng.choice([1, R // 8, R // 4])
    table, lens, ref = K.tables(lens, block, W, NB, seed=seed)
    s = State(cuda_lib, K.Pool(P.BLOCK, 512, 1, NB, block, seed=seed), table, lens, ref)
    children = rng.sample(range(R), rng.randint(R // 2 + 1, R))
    parents = [rng.randrange(0, R, 2) if c % 2 else c for c in children]
    room = [rng.randint(0, block) for _ in children]
    place = rng.choice(["inplace", "apart"])
    first = s.fork(parents, children, room, place)
    rows = rng.sample(range(R), max(1, R // 8))
    s.host[0], s.host[2] = K.free(s.host[0], s.host[2], rows, None, None, block)
    t, l, r = s.dev
    s.smla.smla_cache_free(i32(rows), None, None, t, r, block)
    l[i32(rows).long()] = 0
    s.host[1] = l.cpu()
    s.fork(None, children, [1] * len(children), place)
    assert first > 0 or R == 5


def test_short_in_a_graph(cuda_lib):
    """Captured: replays ask again until a block is free."""
    smla = cuda_lib
    table = torch.tensor([[0, -1], [0, -1]], dtype=torch.int32)
    pool = K.Pool(P.BF16, 512, 3, 3, 16, seed=1)
    ref = torch.tensor([2, 1, 1], dtype=torch.int32)          # (block 1 and 2: held elsewhere)
    s = State(smla, pool, table, torch.tensor([7, 9], dtype=torch.int32), ref)
    t, l, r = s.dev
    both, room = i32([0, 1]), i32([1, 1])
    missing = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = torch.empty(smla.smla_cache_fork_workspace_size(2, 2, 3), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.smla_cache_fork(None, both, room, l, t, r, 16, s.cache, P.BF16, workspace=ws,
                             missing=missing)
    for _ in range(2):
        graph.replay()
        assert int(missing) == 1 and t[:, 0].tolist() == [0, 0] and r.tolist() == [2, 1, 1]
        pool.same(s.cache, None)
    r[1] = 0
    graph.replay()
    pool.copy(0, 1, 9)
    assert int(missing) == 0 and t[:, 0].tolist() == [0, 1] and r.tolist() == [1, 1, 1]
    pool.same(s.cache, None)


def test_nothing_written_is_lost_to_the_attention(cuda_lib):
    """The rows that had no block for their copy attend to all they have written."""
    smla = cuda_lib
    g = torch.Generator().manual_seed(5)
    cache = torch.randn((4 * 16, 576), generator=g).bfloat16().cuda()
    table = torch.full((4, 2), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[0, 1] = 0, 1
    lens, ref = i32([27, 0, 0, 0]), i32([1, 1, 0, 1])
    q = (torch.randn((1, 16, 576), generator=g) * 2).bfloat16().cuda()
    missing = smla.smla_cache_fork(i32([0] * 4), i32([0, 1, 2, 3]), i32([1] * 4), lens, table, ref,
                                   16, cache, P.BF16)
    assert int(missing) == 2 and lens.tolist() == [27] * 4
    out, lse = smla.smla_fwd_window(q.repeat(4, 1, 1), cache, P.BF16, None, i32(range(5)), lens,
                                    table, 16, 0.04, max_seq_len=32)
    assert all(torch.equal(out[i], out[0]) and torch.equal(lse[i], lse[0]) for i in range(4))
    assert bool(torch.isfinite(lse).all())
