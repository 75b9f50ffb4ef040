"""The attention over cache blocks of few rows (bf16: copied row by row): the same
positions with the same rows give the same bits whatever the blocks are, rows that were
never written do not show, and a wait that runs out leaves the next call right."""
import pytest
import torch

from tests import _paged as P
from tests import _scored as R
from tests.test_scored_gpu import run as run_scored
from tests.test_scored_gpu import slopes_of
from tests.test_window_gpu import make
from tests.test_window_gpu import run as run_window

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
def test_a_wait_that_runs_out_8_bit(cuda_lib, block):
    smla = cuda_lib
    b = P.Batch(ROWS, block, seed=5)
    q, cache, scale = make(b, P.BLOCK, 16, 576, 4)
    start, lens, tab = b.dev()
    args = (q.cuda(), cache.cuda(), P.BLOCK, scale.cuda(), start, lens, tab, block, 0.05)
    n = int(b.start[-1])
    smla.smla_get_device_status(clear=True)
    want = smla.smla_fwd_window(*args)
    smla.smla_test_set_stall(True, 2000)
    try:
        smla.smla_fwd_window(*args)
        torch.cuda.synchronize()
    finally:
        smla.smla_test_set_stall(False)
    assert smla.smla_get_device_status(clear=True) == 4
    got = smla.smla_fwd_window(*args)
    assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:n], want[1][:n])
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


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
@pytest.mark.parametrize("block", [1, 3, 4, 6, 16])
def test_rows_past_the_cache_and_the_table(cuda_lib, fmt, block):
    """Table entries behind the cache and lengths behind the table: not seen, and said."""
    smla = cuda_lib
    b = P.Batch([(4, 90), (1, 40)], block, seed=2)
    q, cache, scale = make(b, fmt, 8, 576, 4)
    b.table[0, 3] = b.pool
    b.table[1, 0] = 2**31 - 1
    b.lens[1] = 2**31 - 1
    smla.smla_get_device_status(clear=True)
    start, lens, tab = b.dev()
    out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), fmt,
                                    None if scale is None else scale.cuda(), start, lens, tab,
                                    block, 0.05)
    assert smla.smla_get_device_status(clear=True) == 5
    one = P.Batch([(4, 90)], block, seed=2)
    one.table, one.num_slots = b.table[:1].clone(), b.num_slots
    one.table[0, 3] = -1
    rows = P.dequant(cache, fmt, scale, one)
    ref = P.attend(q[:4], rows, one, 0.05, 0, 0)
    P.check_attention(out[:4], lse[:4], ref, q[:4], fmt, 0.05, one)


@pytest.mark.parametrize("fmt", [P.E4M3, P.BLOCK])
@pytest.mark.parametrize("h", [5, 16, 64, 128])
def test_8_bit_blocks_of_few_rows(cuda_lib, fmt, h):
    """Against the fp64 formula: blocks of every small size, scales of their own, units of
    one block and of many, one request after the other on a pair."""
    rows = [(1, 900), (70, 333), (3, 2), (130, 260), (1, 1), (5, 129), (2, 64)]
    for block in (1, 2, 5, 8, 12, 16, 20, 24):
        b = P.Batch(rows, block, seed=block + h, pad=3, holes=4)
        first, last = R.spans(b, docs=[65, 151], prefix=9)
        run_window(cuda_lib, b, fmt, h, d=576 if block % 2 == 0 else 512, pow2=False)
        run_scored(cuda_lib, b, fmt, h, d=512 if block % 2 == 0 else 576, cap=9.0,
                   slopes=slopes_of(h), first=first, last=last)


@pytest.mark.parametrize("fmt", [P.E4M3, P.BLOCK])
def test_8_bit_prompts_of_many_units(cuda_lib, fmt):
    """More tiles than pairs: each pair goes from unit to unit."""
    smla = cuda_lib
    rows = [(400, 400), (300, 700)]
    b = P.Batch(rows, 7, seed=3)
    q, cache, scale = make(b, fmt, 96, 576, 4)
    start, lens, tab = b.dev()
    args = (fmt, None if scale is None else scale.cuda(), start, lens, tab, 7, 0.04)
    out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), *args, window=130, sinks=3)
    pick = list(range(0, 700, 41)) + [399, 400, 699]
    ref = P.attend(q, P.dequant(cache, fmt, scale, b), Some(b, pick), 0.04, 130, 3)
    keep = torch.zeros(b.N, dtype=torch.bool)
    keep[pick] = True
    for x in (out, lse):
        x[~keep.cuda()] = 0
    for x in ref[:2]:
        x[~keep] = 0
    P.check_attention(out, lse, ref, q, fmt, 0.04, b)


class Some:
    """Some tokens of a batch."""

    def __init__(self, b, pick):
        self.b, self.pick = b, set(pick)

    def __getattr__(self, name):
        return getattr(self.b, name)

    def tokens(self):
        return (t for t in self.b.tokens() if t[0] in self.pick)
