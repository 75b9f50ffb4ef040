"""smla_fwd_scored against the fp64 formula: caps, distance biases, documents and
prefixes, alone and together with windows and sinks, on bf16 and E4M3 rows, in every
plan; what a token does not see, rows without a key, spans that say more than there is."""
import pytest
import torch

from tests import _paged as P
from tests import _scored as R
from tests._helpers import Guarded
from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu

FMTS = [P.BF16, P.E4M3, P.BLOCK]
RAGGED = [(1, 1), (3, 150), (0, 40), (70, 70), (1, 257), (33, 400), (2, 2)]


def call(smla, batch, fmt, q, cache, scale, sm, cap=0.0, slopes=None, first=None, last=None, **kw):
    start, lens, tab = batch.dev()
    dev = lambda t: None if t is None else t.cuda()
    return smla.smla_fwd_scored(q.cuda(), cache.cuda(), fmt, dev(scale), start, lens, tab,
                                batch.block, sm, softcap=cap, slopes=dev(slopes),
                                first_pos=dev(first), last_pos=dev(last),
                                block_stride_rows=batch.stride_rows, **kw)


def slopes_of(h, lo=-8.0):
    return torch.exp2(lo * torch.arange(1, h + 1) / h).float()


def run(smla, batch, fmt, h, d=576, seed=1, pow2=True, q_gain=2.0, window=0, sinks=0, cap=0.0,
        slopes=None, first=None, last=None, status=0, **kw):
    smla.smla_get_device_status(clear=True)
    q, cache, scale = make(batch, fmt, h, d, seed, q_gain, pow2)
    sm = d ** -0.5
    out, lse = Guarded((batch.N, h, 512), torch.bfloat16), Guarded((batch.N, h), torch.float32)
    n = int(batch.start[-1])
    was = out.t[n:].clone().view(torch.int16)
    call(smla, batch, fmt, q, cache, scale, sm, cap, slopes, first, last, window=window,
         sinks=sinks, out=out.t, lse=lse.t, **kw)
    torch.cuda.synchronize()
    out.check("O")
    lse.check("LSE")
    assert torch.equal(out.t[n:].view(torch.int16), was)
    rows = P.dequant(cache, fmt, scale, batch)
    batch.fp8 = fmt != P.BF16
    ref = R.attend(q, rows, batch, sm, window, sinks, cap, slopes, first, last)
    R.check(out.t, lse.t, ref, batch, fmt, pow2)
    assert smla.smla_get_device_status(clear=True) == status
    return out.t.clone(), lse.t.clone()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cap,gain", [(30.0, 8.0), (50.0, 2.0), (1.0, 30.0), (1e-3, 4.0),
                                      (300.0, 200.0), (1e4, 3000.0), (1e6, 4.0), (1e30, 30.0)])
def test_caps(cuda_lib, fmt, cap, gain):
    run(cuda_lib, P.Batch(RAGGED, 64, seed=3, pad=2), fmt, 16, cap=cap, q_gain=gain)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("h", [1, 5, 16, 64, 96, 128])
def test_heads(cuda_lib, fmt, h):
    b = P.Batch(RAGGED, 64, seed=h, pad=3)
    first, last = R.spans(b, docs=[60, 64, 130, 301], prefix=20)
    run(cuda_lib, b, fmt, h, seed=h, cap=20.0, slopes=slopes_of(h), first=first, last=last,
        q_gain=6.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("lo", [-8.0, 0.0, -40.0, 7.0])
def test_distance_bias(cuda_lib, fmt, lo):
    b = P.Batch([(1, 900), (40, 300), (130, 130), (2, 1)], 64, seed=5)
    run(cuda_lib, b, fmt, 24, slopes=slopes_of(24, lo))
    run(cuda_lib, b, fmt, 24, slopes=-slopes_of(24, lo), window=100, sinks=3)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block", [1, 2, 7, 12, 16, 32, 64, 100, 128])
def test_block_sizes(cuda_lib, fmt, block):
    b = P.Batch(RAGGED, block, seed=block)
    first, last = R.spans(b, docs=[50, 200], prefix=30)
    run(cuda_lib, b, fmt, 8, d=512 if block % 2 else 576, window=90, sinks=3, first=first,
        last=last, slopes=slopes_of(8))
    run(cuda_lib, b, fmt, 24, d=576 if block % 2 else 512, cap=15.0, last=last, q_gain=8.0)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("docs,prefix,window,sinks", [
    ([1], 1, 0, 0), ([128, 256], 0, 0, 0), ([127, 129, 400], 300, 0, 5), ([], 700, 0, 0),
    ([300], 64, 50, 0), ([300], 64, 50, 200), (list(range(10, 800, 10)), 3, 0, 1)])
def test_documents_and_prefixes(cuda_lib, fmt, docs, prefix, window, sinks):
    b = P.Batch([(140, 640), (1, 130), (9, 129), (4, 4), (640, 640), (1, 500)], 64, seed=9)
    first, last = R.spans(b, docs, prefix)
    run(cuda_lib, b, fmt, 16, window=window, sinks=sinks, first=first, last=last)
    run(cuda_lib, b, fmt, 5, window=window, sinks=sinks, first=first if docs else None, last=last,
        cap=9.0)


@pytest.mark.parametrize("fmt", FMTS)
def test_spans_that_say_more_than_there_is(cuda_lib, fmt):
    """Spans that are empty, begin behind the request, end before or behind it; tokens at
    negative positions, requests of no length, unallocated blocks."""
    b = P.Batch([(6, 4), (3, 0), (1, 0), (40, 500), (2, 64), (5, 90)], 16, seed=3, holes=12)
    n = torch.arange(b.N, dtype=torch.int32)
    big = torch.full_like(n, 2**31 - 1)
    for first, last in ((n * 0, big), (big, big), (n * 0 + 40, n * 0 + 20), (n * 0, n * 0 - 1),
                        (n * 0 - 2**31, n * 0 - 2**31), (n * 0 - 7, n * 9), (n * 5, None),
                        (None, n * 3)):
        run(cuda_lib, b, fmt, 32, first=first, last=last, window=20, sinks=2)
        run(cuda_lib, b, fmt, 128, first=first, last=last, cap=5.0)
    b.table[:] = -1
    run(cuda_lib, b, fmt, 16, cap=5.0, slopes=slopes_of(16))


@pytest.mark.parametrize("fmt", FMTS)
def test_falling_spans_stay_in_bounds(cuda_lib, fmt):
    """Spans out of order leave keys out; nothing else is touched."""
    smla = cuda_lib
    b = P.Batch([(100, 300), (1, 200), (30, 600)], 64, seed=6, pad=4)
    q, cache, scale = make(b, fmt, 16, 576, 3)
    g = torch.Generator().manual_seed(1)
    first = torch.randint(-50, 700, (b.N,), generator=g, dtype=torch.int32)
    last = torch.randint(-50, 700, (b.N,), generator=g, dtype=torch.int32)
    out = Guarded((b.N, 16, 512), torch.bfloat16)
    lse = Guarded((b.N, 16), torch.float32)
    call(smla, b, fmt, q, cache, scale, 0.04, 9.0, slopes_of(16), first, last, out=out.t,
         lse=lse.t)
    torch.cuda.synchronize()
    out.check("O")
    lse.check("LSE")
    assert bool(torch.isfinite(out.t[:131].float()).all())
    assert smla.smla_get_device_status(clear=True) == 0


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_shared_keys(cuda_lib, fmt):
    """Ranges of the keys of few and of many tiles, other scales, a stride of blocks."""
    smla = cuda_lib
    b = P.Batch([(1, 6000), (1, 300), (2, 1), (1, 4097)], 64, seed=6)
    assert smla.smla_fwd_window_workspace_size(4, b.N, 16, 576, fmt, b.table.shape[1], 64) > 0
    first, last = R.spans(b, docs=[2000, 4000])
    run(smla, b, fmt, 16, cap=10.0, slopes=slopes_of(16), q_gain=5.0)
    run(smla, b, fmt, 128, window=3000, sinks=300, slopes=slopes_of(128))
    run(smla, b, fmt, 16, first=first, last=last)
    rows = [(1, 1 + 97 * r % 1500) for r in range(76)] + [(0, 40), (3, 2), (0, 0), (1, 0)]
    b = P.Batch(rows, 16, seed=21, pad=3, stride_rows=24)
    first, last = R.spans(b, docs=[700], prefix=900)
    run(smla, b, fmt, 16, pow2=False, cap=10.0, slopes=slopes_of(16), first=first, last=last)
    b = P.Batch([(300, 300), (260, 900)], 64, seed=22)
    first, last = R.spans(b, docs=[100, 290, 700], prefix=90)
    run(smla, b, fmt, 8, cap=10.0, slopes=slopes_of(8), first=first, last=last)


@pytest.mark.parametrize("fmt", FMTS)
def test_nothing_set_is_the_windowed_call(cuda_lib, fmt):
    smla = cuda_lib
    b = P.Batch(RAGGED, 64, seed=7)
    q, cache, scale = make(b, fmt, 16, 576, 2)
    start, lens, tab = b.dev()
    want = smla.smla_fwd_window(q.cuda(), cache.cuda(), fmt,
                                None if scale is None else scale.cuda(), start, lens, tab, 64,
                                0.04, window=77, sinks=2)
    got = call(smla, b, fmt, q, cache, scale, 0.04, window=77, sinks=2)
    n = int(b.start[-1])
    assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:n], want[1][:n])


@pytest.mark.parametrize("docs,cap", [([30, 200, 410], 8.0), ([31, 207, 401], 8.0),
                                      ([31, 207, 401], 1e6), ([31, 207, 401], 1e30)])
@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_unseen_positions_may_hold_anything(cuda_lib, fmt, bad, docs, cap):
    """Rows of other documents, of the window's past and of other requests' ends that are
    not finite: the tokens that do not see them are as without them."""
    smla = cuda_lib
    b = P.Batch([(20, 420), (1, 301), (61, 61)], 64, seed=11)
    first, last = R.spans(b, docs=docs, prefix=7)
    q, cache, scale = make(b, fmt, 16, 576, 4)
    seen = torch.zeros(b.num_slots, dtype=torch.bool)
    for n, r, pos in b.tokens():
        for e in range(int(first[n]), int(last[n]) + 1):
            seen[b.slot(r, e)] = True
    kw = dict(cap=cap, slopes=slopes_of(16), first=first, last=last)
    want = call(smla, b, fmt, q, cache, scale, 0.04, **kw)
    dirty = cache.clone()
    if fmt == P.BF16:
        dirty[~seen] = bad
    else:
        dirty[~seen] = 0x7F                               # E4M3's NaN
    got = call(smla, b, fmt, q, dirty, scale, 0.04, **kw)
    rows = P.dequant(cache, fmt, scale, b)
    b.fp8 = fmt != P.BF16
    ref = R.attend(q, rows, b, 0.04, cap=cap, slopes=kw["slopes"], first=first, last=last)
    R.check(want[0], want[1], ref, b, fmt)
    R.check(got[0], got[1], ref, b, fmt)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_unseen_positions_in_whole_tiles(cuda_lib, fmt, bad):
    """The same where every tile is one unit: its rows are computed again and written
    over what the tile stored."""
    smla = cuda_lib
    b = P.Batch([(199, 300), (3, 40)], 64, seed=13, pad=2)
    h = 64
    first, last = R.spans(b, docs=[131, 207], prefix=7)
    q, cache, scale = make(b, fmt, h, 576, 9)
    assert smla.smla_fwd_window_workspace_size(2, b.N, h, 576, fmt, b.table.shape[1], 64) == 0
    seen = torch.zeros(b.num_slots, dtype=torch.bool)
    for n, r, pos in b.tokens():
        for e in range(int(first[n]), int(last[n]) + 1):
            seen[b.slot(r, e)] = True
    dirty = cache.clone()
    dirty[~seen] = bad if fmt == P.BF16 else 0x7F          # E4M3's NaN
    # (and a position that only the second document's tokens see)
    dirty[b.slot(0, 135)] = bad if fmt == P.BF16 else 0x7F
    kw = dict(cap=8.0, slopes=slopes_of(h), first=first, last=last)
    out, lse = call(smla, b, fmt, q, dirty, scale, 0.04, **kw)
    rows = P.dequant(cache, fmt, scale, b)
    b.fp8 = fmt != P.BF16
    ref = R.attend(q, rows, b, 0.04, cap=8.0, slopes=kw["slopes"], first=first, last=last)
    sees = torch.zeros(b.N, dtype=torch.bool)
    for n, r, pos in b.tokens():
        sees[n] = r == 0 and int(first[n]) <= 135 <= int(last[n])
    assert bool(sees.any()) and not bool(sees.all())
    assert not bool(torch.isfinite(out[sees].float()).all(-1).any())
    out[sees] = ref[0][sees].to(out)                       # (the others are checked)
    lse[sees] = ref[1][sees].to(lse)
    R.check(out, lse, ref, b, fmt)


def test_seen_positions_that_are_not_finite(cuda_lib):
    """A key with an infinite channel, seen: its score is capped, and O has its V; a NaN
    makes the rows that see it NaN and no others."""
    smla = cuda_lib
    b = P.Batch([(70, 200)], 64, seed=12)
    q, cache, _ = make(b, P.BF16, 16, 576, 4)
    at = 150
    first, last = R.spans(b, docs=[160])
    for bad in (float("inf"), float("nan")):
        dirty = cache.clone()
        dirty[b.slot(0, at), 3] = bad
        out, lse = call(smla, b, P.BF16, q, dirty, None, 0.04, cap=8.0, first=first, last=last)
        for n, _, pos in b.tokens():
            sees = int(first[n]) <= at <= pos
            assert bool(torch.isfinite(out[n].float()).all()) != sees
            assert bool(torch.isfinite(lse[n]).all()) != (sees and bad != bad)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("toward_start", [True, False])
@pytest.mark.parametrize("step", [3.0, 9.0, 15.5, 16.5, 40.0, 150.0])
@pytest.mark.parametrize("cap", [0.0, 1e4])
def test_scores_that_grow_block_by_block(cuda_lib, fmt, toward_start, step, cap):
    """Every 128 keys' scores lie 2^step above or below the next ones': the running
    maximum rises by less and by more than O is rescaled for."""
    smla = cuda_lib
    b = P.Batch([(130, 700), (1, 513), (40, 40)], 64, seed=21)
    h, sm = 16, 0.0625
    q, cache, scale = make(b, fmt, h, 576, 5)
    q[:] *= 0.03125 if fmt == P.BF16 else 0.00390625
    q[:, :, 575] = step                                   # (bf16 has all of the steps)
    level = lambda e: float(8 * (e // 128) if not toward_start else 8 * (5 - e // 128))
    codes = torch.tensor([8 * level(128 * i) for i in range(6)]).to(torch.float8_e4m3fn)
    for r, (_, length) in enumerate(b.rows):
        for e in range(length):
            s = b.slot(r, e)
            if s >= 0:
                cache[s, 575] = level(e) if fmt == P.BF16 else codes.view(torch.uint8)[e // 128]
    if scale is not None:
        scale[:] = 0.125
    # a score's difference from one 128 keys to the next: step * 8 * sm nats / ln 2
    sm_scale = sm * 2 * 0.6931471805599453
    rows = P.dequant(cache, fmt, scale, b)
    b.fp8 = fmt != P.BF16
    slopes = slopes_of(h)
    out, lse = call(smla, b, fmt, q, cache, scale, sm_scale, cap=cap, slopes=slopes)
    R.check(out, lse, R.attend(q, rows, b, sm_scale, cap=cap, slopes=slopes), b, fmt)
    # and no cap or bias, but a span: documents that begin inside of a block
    first, last = R.spans(b, docs=[127, 300], prefix=9)
    out, lse = call(smla, b, fmt, q, cache, scale, sm_scale, first=first, last=last)
    R.check(out, lse, R.attend(q, rows, b, sm_scale, first=first, last=last), b, fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("h", [16, 40, 64])
@pytest.mark.parametrize("at", [0, 8, 16, 24])
def test_output_alignments(cuda_lib, fmt, h, at):
    """O on any 16-byte boundary, with whole tiles and partial ones."""
    smla = cuda_lib
    b = P.Batch([(1200, 1200), (7, 90), (150, 300)] if at < 16 else [(5, 90), (33, 300)], 64,
                seed=31)
    q, cache, scale = make(b, fmt, h, 576, 6)
    slopes = slopes_of(h)
    kw = dict(cap=20.0, slopes=slopes, max_seq_len=1200)
    want, _ = call(smla, b, fmt, q, cache, scale, 0.04, **kw)
    flat = torch.full((b.N * h * 512 + 32,), 7.0, dtype=torch.bfloat16, device="cuda")
    out = flat[at:at + b.N * h * 512].view(b.N, h, 512)
    call(smla, b, fmt, q, cache, scale, 0.04, out=out, **kw)
    assert torch.equal(out, want)
    assert bool((flat[:at] == 7).all()) and bool((flat[at + b.N * h * 512:] == 7).all())


def test_captured_and_on_another_stream(cuda_lib):
    smla = cuda_lib
    b = P.Batch([(1, 3000), (5, 700), (1, 64)], 64, seed=13)
    first, last = R.spans(b, docs=[500], prefix=40)
    q, cache, _ = make(b, P.BF16, 16, 576, 4)
    args = dict(cap=12.0, slopes=slopes_of(16), first=first, last=last, max_seq_len=3000)
    want = call(smla, b, P.BF16, q, cache, None, 0.04, **args)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    start, lens, tab = b.dev()
    gq, gc, gs, gf, gl = q.cuda(), cache.cuda(), slopes_of(16).cuda(), first.cuda(), last.cuda()
    torch.cuda.synchronize()
    kw = dict(softcap=12.0, slopes=gs, first_pos=gf, last_pos=gl, max_seq_len=3000)
    got = smla.smla_fwd_scored(gq, gc, P.BF16, None, start, lens, tab, 64, 0.04, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
    ws = torch.empty(smla.smla_fwd_window_workspace_size(3, b.N, 16, 576, P.BF16, tab.shape[1], 64,
                                                         max_seq_len=3000), dtype=torch.uint8,
                     device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        smla.smla_fwd_scored(gq, gc, P.BF16, None, start, lens, tab, 64, 0.04, out=out, lse=lse,
                             workspace=ws, **kw)
    for _ in range(3):
        out.zero_()
        graph.replay()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
    gf.copy_(first + 20)                                   # (the graph reads them again)
    graph.replay()
    rows = P.dequant(cache, P.BF16, None, b)
    ref = R.attend(q, rows, b, 0.04, cap=12.0, slopes=slopes_of(16), first=first + 20, last=last)
    R.check(out, lse, ref, b, P.BF16)


def test_binding_refusals(cuda_lib):
    smla = cuda_lib
    b = P.Batch([(2, 90)], 64, seed=14)
    q, cache, _ = make(b, P.BF16, 16, 576, 4)
    start, lens, tab = b.dev()
    good = dict(q=q.cuda(), kv_cache=cache.cuda(), kv_dtype=P.BF16, k_scale=None,
                query_start=start, seq_lens=lens, block_table=tab, block_size=64, sm_scale=0.04,
                softcap=5.0, slopes=slopes_of(16).cuda(),
                first_pos=torch.zeros(2, dtype=torch.int32, device="cuda"),
                last_pos=torch.zeros(2, dtype=torch.int32, device="cuda"))
    smla.smla_fwd_scored(**good)
    for bad in (dict(slopes=good["slopes"][:8]), dict(slopes=good["slopes"].double()),
                dict(slopes=slopes_of(16)), dict(first_pos=good["first_pos"][:1]),
                dict(last_pos=good["last_pos"].long()), dict(q=good["q"][:, :, :512])):
        with pytest.raises(ValueError):
            smla.smla_fwd_scored(**{**good, **bad})
    for cap in (-1.0, float("nan"), float("inf")):
        with pytest.raises(smla.SmlaError):
            smla.smla_fwd_scored(**{**good, "softcap": cap})
