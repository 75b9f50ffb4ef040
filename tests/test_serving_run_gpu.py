"""The paged operators together, as a serving loop uses them: rooms for prompts, appends,
attention, samples forked from a prompt, a beam step, blocks given back behind a window,
the pool compacted, attention again.  The tables' contents are followed by a plain model
of the requests (a list of rows each); the attention is checked against it in fp64."""
import random

import pytest
import torch

from tests import _paged as P
from tests import _scored as R

pytestmark = pytest.mark.gpu

H, D, BLOCK, LAYERS, ROWS, WIDTH, NB = 8, 576, 16, 2, 9, 12, 60


class Loop:
    def __init__(self, smla, fmt, seed):
        self.smla, self.fmt = smla, fmt
        self.gen = torch.Generator().manual_seed(seed)
        self.rng = random.Random(seed)
        slots = NB * BLOCK
        self.table = torch.full((ROWS, WIDTH), -1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(ROWS, dtype=torch.int32, device="cuda")
        self.ref = torch.zeros(NB, dtype=torch.int32, device="cuda")
        if fmt == P.BF16:
            self.cache = torch.zeros((LAYERS, slots, D), dtype=torch.bfloat16, device="cuda")
            self.scale = None
        else:
            self.cache = torch.zeros((LAYERS, slots, D), dtype=torch.uint8, device="cuda")
            self.scale = torch.zeros((LAYERS, NB), device="cuda")
        # each row: per layer the rows that it holds, position by position (None: given back)
        self.rows = {r: [] for r in range(ROWS)}
        self.cos_sin = torch.cat([torch.ones(WIDTH * BLOCK, 32), torch.zeros(WIDTH * BLOCK, 32)],
                                 1).cuda()                # no turn: rows stay what they are

    def fork(self, parents, children, room):
        t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
        missing = self.smla.smla_cache_fork(
            t(parents), t(children), t(room), self.lens, self.table, self.ref, BLOCK, self.cache,
            self.fmt, self.scale)
        assert int(missing) == 0
        old = dict(self.rows)
        for i, c in enumerate(children):
            p = c if parents is None else parents[i]
            self.rows[c] = list(old[p]) if p >= 0 else []

    def append(self, new):
        """new: {row: tokens}; the packed batch has every row, in order."""
        n = [new.get(r, 0) for r in range(ROWS)]
        start = torch.tensor([0] + n, device="cuda").cumsum(0).to(torch.int32)
        self.lens += torch.tensor(n, dtype=torch.int32, device="cuda")
        N = sum(n)
        x = torch.randn((LAYERS, N, D), generator=self.gen).bfloat16()
        for l in range(LAYERS):
            kv = x[l].cuda()
            self.smla.smla_cache_append(kv[:, :512], kv[:, 512:], self.cos_sin, start, self.lens,
                                        self.table, BLOCK, self.cache[l], self.fmt,
                                        None if self.scale is None else self.scale[l])
        at = 0
        for r in range(ROWS):
            self.rows[r] = self.rows[r] + [x[:, at + i] for i in range(n[r])]
            at += n[r]
        return start

    def attend(self, start, cap, slopes, window=0, sinks=0, first=None, last=None):
        N = int(start[-1])
        q = (torch.randn((N, H, D), generator=self.gen) * 2).bfloat16()
        dev = lambda t: None if t is None else t.cuda()
        lens, starts = self.lens.cpu(), start.cpu()
        for l in range(LAYERS):
            scale = None if self.scale is None else self.scale[l]
            out, lse = self.smla.smla_fwd_scored(
                q.cuda(), self.cache[l], self.fmt, scale, start, self.lens, self.table, BLOCK,
                D ** -0.5, softcap=cap, slopes=dev(slopes), window=window, sinks=sinks,
                first_pos=dev(first), last_pos=dev(last))
            # the model's rows laid out one request behind the other
            batch = P.Batch([(int(starts[r + 1] - starts[r]), int(lens[r])) for r in range(ROWS)],
                            BLOCK, seed=1)
            want = torch.zeros((batch.num_slots, D), dtype=torch.float64)
            held = torch.ones(batch.num_slots, dtype=torch.float64)
            for r in range(ROWS):
                for e, row in enumerate(self.rows[r]):
                    if row is not None:
                        want[batch.slot(r, e)] = row[l].double()
                for c in range(batch.table.shape[1]):
                    span = self.rows[r][c * BLOCK:(c + 1) * BLOCK]
                    if span and span[0] is None:
                        batch.table[r, c] = -1
            if self.fmt != P.BF16:                        # what the cache holds of it
                got = self.cache[l].cpu().view(torch.float8_e4m3fn).double()
                unit = self.scale[l].cpu().double()
                table = self.table.cpu()
                for r in range(ROWS):
                    for e, row in enumerate(self.rows[r]):
                        b = int(table[r, e // BLOCK])
                        if row is None:
                            assert b == -1
                            continue
                        x = got[b * BLOCK + e % BLOCK] * unit[b]
                        # (a grown scale rounds older codes twice)
                        worst = 2 * (2.0 ** -4 * row[l].double().abs() + unit[b] * 2.0 ** -10)
                        assert bool(((x - row[l].double()).abs() <= worst).all())
                        want[batch.slot(r, e)] = x
                        held[batch.slot(r, e)] = unit[b]
            batch.row_scale, batch.fp8 = held, self.fmt != P.BF16
            ref = R.attend(q, want, batch, D ** -0.5, window, sinks, cap, slopes, first, last)
            R.check(out, lse, ref, batch, self.fmt)

    def free(self, rows, begin=None, end=None):
        t = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
        self.smla.smla_cache_free(t(rows), t(begin), t(end), self.table, self.ref, BLOCK)
        for i, r in enumerate(rows):
            lo = 0 if begin is None else begin[i]
            hi = WIDTH * BLOCK if end is None else end[i]
            for c in range(WIDTH):
                if c * BLOCK >= lo and (c + 1) * BLOCK <= hi:
                    for e in range(c * BLOCK, min((c + 1) * BLOCK, len(self.rows[r]))):
                        self.rows[r][e] = None

    def drop(self, rows):
        self.free(rows)
        for r in rows:
            self.rows[r] = []
            self.lens[r] = 0

    def compact(self):
        _, live = self.smla.smla_cache_compact(self.table, self.ref, BLOCK, self.cache, self.fmt,
                                               self.scale)
        live = int(live)
        assert bool((self.ref[:live] > 0).all()) and not bool(self.ref[live:].any())
        self.check_counts()
        return live

    def check_counts(self):
        held = self.table[self.table >= 0].long()
        assert torch.equal(torch.bincount(held, minlength=NB).int(), self.ref)


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
@pytest.mark.parametrize("seed", [1, 2])
def test_serving_loop(cuda_lib, fmt, seed):
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    g = Loop(smla, fmt, seed)
    slopes = torch.exp2(-torch.arange(1, H + 1).float())
    # three prompts
    prompt = {0: 37, 4: 64, 7: 5}
    g.fork([-1] * 3, list(prompt), list(prompt.values()))
    start = g.append(prompt)
    pos = torch.cat([torch.arange(n) for _, n in sorted(prompt.items())]).int()
    g.attend(start, 20.0, None, last=torch.maximum(pos, torch.full_like(pos, 3)))
    # four samples of the first, two of the second, the third goes on
    g.fork([0, 0, 0, 0, 4, 4, 7], [0, 1, 2, 3, 4, 5, 7], [1] * 7)
    g.check_counts()
    live = [0, 1, 2, 3, 4, 5, 7]
    for step in range(3):
        start = g.append({r: 1 for r in live})
        g.attend(start, 15.0, slopes)
        # a beam step: rows of a family continue each other
        parents = [g.rng.choice([0, 1, 2, 3]) for _ in range(4)] + \
            [g.rng.choice([4, 5]) for _ in range(2)] + [7]
        g.fork(parents, live, [1] * 7)
        g.check_counts()
    # a draft of 20 tokens on one row, 4 of them kept
    g.fork(None, [2], [20])
    start = g.append({2: 20})
    g.attend(start, 0.0, slopes)
    keep = len(g.rows[2]) - 16
    g.rows[2] = g.rows[2][:keep]
    g.lens[2] = keep
    g.free([2], begin=[keep])
    # one request is done, another leaves its first blocks behind its window
    g.drop([1, 4])
    g.free([5], begin=[4], end=[len(g.rows[5]) - 20])
    g.check_counts()
    before = g.compact()
    live = [r for r in live if r not in (1, 4)]
    g.fork(None, live, [2] * len(live))
    start = g.append({r: 2 for r in live})
    g.attend(start, 12.0, slopes, window=19, sinks=4)
    assert before < int((g.ref > 0).sum()) + 6
    assert smla.smla_get_device_status(clear=True) == 0
