"""Block tables and pools for the tests of the block operators, with references that
go row by row and block by block on the CPU."""
from __future__ import annotations

import numpy as np
import torch

from tests._paged import BF16, BLOCK, DS_MLA, DS_MLA_ROW, E4M3, GROUP128, GROUP4_KPE

FORMATS = [(BF16, 576), (BF16, 512), (E4M3, 576), (GROUP128, 576), (GROUP128, 512),
           (DS_MLA, 576), (GROUP4_KPE, 576), (BLOCK, 576), (BLOCK, 512)]


def groups(fmt, d):
    return {GROUP128: -(-d // 128), GROUP4_KPE: 4}.get(fmt, 0)


class Pool:
    """Layers of one cache format: random bytes, and random bits as scales."""

    def __init__(self, fmt, d, layers, blocks, block, stride_rows=0, extra=0, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.d, self.block = fmt, d, block
        self.stride_rows = stride_rows
        step = self.step = stride_rows or block
        slots = blocks * step + extra
        row = DS_MLA_ROW if fmt == DS_MLA else 2 * d if fmt == BF16 else d
        raw = torch.randint(0, 256, (layers, slots, row), dtype=torch.uint8, generator=g)
        self.cache = raw.view(torch.bfloat16) if fmt == BF16 else raw
        n = groups(fmt, d)
        self.scale = None
        if n:
            self.scale = torch.rand((layers, slots, n), generator=g)
        elif fmt == BLOCK:
            self.scale = torch.rand((layers, -(-slots // step)), generator=g)

    def copy(self, src, dst, rows):
        a, b = src * self.step, dst * self.step
        self.cache[:, b:b + rows] = self.cache[:, a:a + rows].clone()
        if groups(self.fmt, self.d):
            self.scale[:, b:b + rows] = self.scale[:, a:a + rows].clone()
        elif self.fmt == BLOCK:
            self.scale[:, dst] = self.scale[:, src]

    def dev(self):
        return self.cache.cuda(), None if self.scale is None else self.scale.cuda()

    def same(self, cache, scale):
        assert torch.equal(cache.cpu().view(torch.uint8), self.cache.view(torch.uint8))
        if self.scale is not None:
            assert torch.equal(scale.cpu().view(torch.int32), self.scale.view(torch.int32))


def tables(lens, block, width, blocks, seed=0, shared=0, holes=0, extra_refs=0):
    """A table whose rows hold blocks at random places; the first `shared` blocks of
    neighbouring rows are the same; `extra_refs` blocks have holders elsewhere."""
    rng = np.random.default_rng(seed)
    order = list(rng.permutation(blocks))
    table = np.full((len(lens), width), -1, np.int32)
    for r, n in enumerate(lens):
        for c in range(min(width, -(-n // block))):
            if r % 2 and c < shared and table[r - 1, c] >= 0 and n >= (c + 1) * block:
                table[r, c] = table[r - 1, c]
            else:
                table[r, c] = order.pop()
    for _ in range(holes):
        r = rng.integers(len(lens))
        table[r, rng.integers(width)] = -1
    ref = np.zeros(blocks, np.int32)
    for b in table[table >= 0]:
        ref[b] += 1
    for b in rng.choice(blocks, extra_refs, replace=False):
        ref[b] += 1
    return (torch.from_numpy(table), torch.tensor(lens, dtype=torch.int32),
            torch.from_numpy(ref))


def last_only(names, rows):
    """Indexes of the pairs that count: in range, the last of their name."""
    return [i for i, c in enumerate(names) if 0 <= c < rows and c not in names[i + 1:]]


def fork(pool, table, lens, ref, parents, children, room, block):
    """(table, lens, ref, missing); the pool is changed."""
    R, W = table.shape
    NB = len(ref)
    new_table, new_lens, new_ref = table.clone(), lens.clone(), ref.clone()
    names = list(children)
    todo = last_only(names, R)
    rows, length = {}, {}
    for i in todo:
        p = children[i] if parents is None else parents[i]
        n = 0 if not 0 <= p < R else max(0, int(lens[p]))
        n = min(n, W * block)
        have = -(-n // block)
        row = [int(table[p, c]) if c < have else -1 for c in range(W)]
        rows[i] = [b if b < NB else -1 for b in row]
        length[i] = n
        for b in table[children[i]].tolist():
            if 0 <= b < NB:
                new_ref[b] -= 1
        for b in rows[i]:
            if b >= 0:
                new_ref[b] += 1
    writers = {}
    for i in todo:
        if room is not None and room[i] > 0 and length[i] % block:
            b = rows[i][length[i] // block]
            if b >= 0:
                writers.setdefault(b, []).append(i)
    own = set()
    for b, who in writers.items():
        own.update(who if new_ref[b] > len(who) else who[1:])
    free = [b for b in range(NB) if new_ref[b] == 0]
    missing = 0
    for i in todo:
        n, grow = length[i], 0 if room is None else max(0, room[i])
        have, end = -(-n // block), min(W, -(-(n + grow) // block))
        cols = ([n // block] if i in own else []) + list(range(have, end))
        for c in cols:
            b = free.pop(0) if free else -1
            missing += b < 0
            if i in own and c == n // block:
                new_ref[rows[i][c]] -= 1
                if b >= 0:
                    pool.copy(rows[i][c], b, n % block)
            rows[i][c] = b
            if b >= 0:
                new_ref[b] = 1
        new_table[children[i]] = torch.tensor(rows[i], dtype=torch.int32)
        new_lens[children[i]] = n
    return new_table, new_lens, new_ref, missing


def free(table, ref, rows, begin, end, block):
    table, ref = table.clone(), ref.clone()
    R, W = table.shape
    for i in last_only(list(rows), R):
        for c in range(W):
            lo, hi = c * block, (c + 1) * block
            b = int(table[rows[i], c])
            if b < 0 or (begin is not None and lo < begin[i]) or \
                    (end is not None and hi > end[i]):
                continue
            table[rows[i], c] = -1
            if b < len(ref):
                ref[b] -= 1
    return table, ref


def compact(pool, table, ref, block):
    """(table, ref, map, live); the pool is changed."""
    NB = len(ref)
    live = int((ref > 0).sum())
    where = [b if ref[b] > 0 else -1 for b in range(NB)]
    new = ref.clone()
    low = [b for b in range(live) if ref[b] <= 0]
    for b in reversed(range(live, NB)):
        if ref[b] > 0:
            to = low.pop(0)
            pool.copy(b, to, block)
            where[b], new[to], new[b] = to, ref[b], 0
    out = table.clone()
    for r in range(table.shape[0]):
        for c in range(table.shape[1]):
            b = int(table[r, c])
            if b < NB:
                out[r, c] = -1 if b < 0 else where[b]
    return out, new, torch.tensor(where, dtype=torch.int32), live
