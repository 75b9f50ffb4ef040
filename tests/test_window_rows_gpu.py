"""The attention over cache blocks of few rows (bf16: copied row by row): the same
positions with the same rows give the same bits whatever the blocks are, rows that were
never written do not show, and a wait that runs out leaves the next call right."""
import pytest
import torch

from tests import _paged as P
from tests import _scored as R
from tests.test_scored_gpu import slopes_of

pytestmark = pytest.mark.gpu

ROWS = [(1, 700), (70, 333), (0, 5), (3, 2), (200, 200), (1, 1), (5, 129)]


def laid_out(rows, block, logical, stride_rows=0, fill=0.0, seed=1):
    """A batch in blocks of `block`, its cache with the requests' rows; what no position
    has is `fill`."""
    b = P.Batch(rows, block, seed=seed, pad=2, stride_rows=stride_rows)
    cache = torch.full((b.num_slots, logical.shape[-1]), fill, dtype=torch.bfloat16)
    at = 0
    for r, (_, L) in enumerate(rows):
        for e in range(max(L, 0)):
            cache[b.slot(r, e)] = logical[at + e]
        at += max(L, 0)
    return b, cache


def calls(smla, b, cache, q, **kw):
    start, lens, tab = b.dev()
    first, last = R.spans(b, docs=[64, 150], prefix=9)
    args = (q.cuda(), cache.cuda(), P.BF16, None, start, lens, tab, b.block, 0.05)
    out = smla.smla_fwd_window(*args, block_stride_rows=b.stride_rows, **kw)
    out += smla.smla_fwd_scored(*args, block_stride_rows=b.stride_rows, softcap=9.0,
                                slopes=slopes_of(q.shape[1]).cuda(), first_pos=first.cuda(),
                                last_pos=last.cuda(), **kw)
    n = int(b.start[-1])
    return [t[:n].clone() for t in out]


@pytest.mark.parametrize("h,d", [(16, 576), (128, 576), (5, 512)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_blocks_of_any_size_give_the_same_bits(cuda_lib, h, d, window, sinks):
    smla = cuda_lib
    g = torch.Generator().manual_seed(h + d)
    logical = torch.randn((sum(max(L, 0) for _, L in ROWS), d), generator=g).bfloat16()
    q = torch.randn((sum(n for n, _ in ROWS) + 2, h, d), generator=g).bfloat16()
    smla.smla_get_device_status(clear=True)
    kw = dict(window=window, sinks=sinks, max_seq_len=700)
    want = None
    for block, stride in ((64, 0), (1, 0), (2, 0), (3, 0), (4, 0), (8, 0), (16, 24), (24, 0),
                          (32, 0), (100, 0), (1, 3)):
        # (rows that were never written: NaN)
        b, cache = laid_out(ROWS, block, logical, stride, fill=float("nan"), seed=block)
        got = calls(smla, b, cache, q, **kw)
        if want is None:
            want = got
            assert all(bool(torch.isfinite(t.float()).all()) for t in (got[0], got[2]))
        for x, y in zip(got, want):
            assert torch.equal(x, y), f"blocks of {block} rows"
    assert smla.smla_get_device_status(clear=True) == 0


@pytest.mark.parametrize("block", [1, 4, 7])
def test_a_wait_that_runs_out(cuda_lib, block):
    smla = cuda_lib
    g = torch.Generator().manual_seed(3)
    logical = torch.randn((sum(max(L, 0) for _, L in ROWS), 576), generator=g).bfloat16()
    q = torch.randn((sum(n for n, _ in ROWS) + 2, 16, 576), generator=g).bfloat16()
    b, cache = laid_out(ROWS, block, logical)
    smla.smla_get_device_status(clear=True)
    want = calls(smla, b, cache, q)
    for _ in range(2):
        smla.smla_test_set_stall(True, 2000)
        try:
            calls(smla, b, cache, q)
            torch.cuda.synchronize()
        finally:
            smla.smla_test_set_stall(False)
        assert smla.smla_get_device_status(clear=True) == 4
        got = calls(smla, b, cache, q)
        for x, y in zip(got, want):
            assert torch.equal(x, y)
        assert smla.smla_get_device_status(clear=True) == 0


def test_rows_past_the_cache_and_the_table(cuda_lib):
    """Table entries behind the cache and lengths behind the table: not seen, and said."""
    smla = cuda_lib
    g = torch.Generator().manual_seed(4)
    for block in (1, 4, 6):
        b = P.Batch([(4, 90), (1, 40)], block, seed=2)
        cache = torch.randn((b.num_slots, 576), generator=g).bfloat16()
        q = torch.randn((b.N, 8, 576), generator=g).bfloat16()
        b.table[0, 3] = b.pool
        b.table[1, 0] = 2**31 - 1
        b.lens[1] = 2**31 - 1
        smla.smla_get_device_status(clear=True)
        start, lens, tab = b.dev()
        out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), P.BF16, None, start, lens, tab,
                                        block, 0.05)
        assert smla.smla_get_device_status(clear=True) == 5
        assert bool(torch.isfinite(out.float()).all())
        b.table[0, 3] = -1
        ref = P.attend(q[:4], P.dequant(cache, P.BF16, None, b),
                       P_first(b), 0.05, 0, 0)
        assert bool(((lse[:4].double().cpu() - ref[1]).abs() < 1e-3).all())


def P_first(b):
    """The first request of the batch alone."""
    one = P.Batch([(4, 90)], b.block, seed=2)
    one.table, one.num_slots = b.table[:1], b.num_slots
    one.start, one.lens, one.N = b.start[:2], b.lens[:1], 4
    return one
