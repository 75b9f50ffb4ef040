"""smla_fwd_window against the fp64 formula: ragged batches of every shape,
windows and sinks, bf16 and E4M3 rows, values that are not finite where a token
does not look, split keys, captured graphs and the refusals' device side."""
import pytest
import torch

from tests import _paged as P
from tests._helpers import Guarded

pytestmark = pytest.mark.gpu

FMTS = [P.BF16, P.E4M3, P.BLOCK]


def make(batch, fmt, h, d, seed, q_gain=2.0, pow2=True):
    g = torch.Generator().manual_seed(seed)
    q = (torch.randn((batch.N, h, d), generator=g) * q_gain).bfloat16()
    x = torch.randn((batch.num_slots, d), generator=g)
    step = batch.stride_rows or batch.block
    if fmt == P.BF16:
        return q, x.bfloat16(), None
    cache = (x * 64).to(torch.float8_e4m3fn).view(torch.uint8)
    if fmt == P.E4M3:
        return q, cache, torch.tensor([2.0 ** -6 if pow2 else 0.0171])
    n = -(-batch.num_slots // step)
    scale = torch.exp2(torch.randint(-8, -4, (n,), generator=g).float())
    return q, cache, scale if pow2 else scale * (1 + torch.rand(n, generator=g))


def launch(smla, batch, fmt, q, cache, scale, sm_scale, window, sinks, **kw):
    start, lens, tab = batch.dev()
    return smla.smla_fwd_window(q.cuda(), cache.cuda(), fmt,
                                None if scale is None else scale.cuda(), start, lens, tab,
                                batch.block, sm_scale, window=window, sinks=sinks,
                                block_stride_rows=batch.stride_rows, **kw)


def run(smla, batch, fmt, h, d=576, window=0, sinks=0, seed=1, pow2=True, q_gain=2.0, status=0,
        **kw):
    smla.smla_get_device_status(clear=True)
    q, cache, scale = make(batch, fmt, h, d, seed, q_gain, pow2)
    sm = d ** -0.5
    out, lse = Guarded((batch.N, h, 512), torch.bfloat16), Guarded((batch.N, h), torch.float32)
    was = out.t[int(batch.start[-1]):].clone().view(torch.int16)
    launch(smla, batch, fmt, q, cache, scale, sm, window, sinks, out=out.t, lse=lse.t, **kw)
    torch.cuda.synchronize()
    out.check("O")
    lse.check("LSE")
    # padding rows behind the last request are as they were
    assert torch.equal(out.t[int(batch.start[-1]):].view(torch.int16), was)
    ref = P.attend(q, P.dequant(cache, fmt, scale, batch), batch, sm, window, sinks)
    P.check_attention(out.t, lse.t, ref, q, fmt, sm, batch, pow2)
    assert smla.smla_get_device_status(clear=True) == status
    return out.t.clone(), lse.t.clone()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("length", [1, 2, 63, 64, 65, 128, 129, 300])
def test_one_token(cuda_lib, fmt, length):
    run(cuda_lib, P.Batch([(1, length)], 64, seed=length), fmt, 16)


RAGGED = [(1, 1), (3, 150), (0, 40), (70, 70), (1, 257), (33, 400), (2, 2)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("h", [1, 5, 16, 64, 96, 128])
def test_ragged_heads(cuda_lib, fmt, h):
    run(cuda_lib, P.Batch(RAGGED, 64, seed=h, pad=3), fmt, h, seed=h)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("block", [1, 2, 7, 12, 16, 32, 64, 100, 128])
def test_block_sizes(cuda_lib, fmt, block):
    run(cuda_lib, P.Batch(RAGGED, block, seed=block), fmt, 8, d=512 if block % 2 else 576,
        window=90, sinks=3)
    run(cuda_lib, P.Batch(RAGGED, block, seed=block), fmt, 24, d=576 if block % 2 else 512)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (2, 200), (64, 4), (128, 128), (129, 5),
                                          (200, 0), (700, 130), (5000, 4)])
def test_windows(cuda_lib, fmt, window, sinks):
    b = P.Batch([(1, 900), (140, 640), (1, 130), (9, 129), (4, 4)], 64, seed=window)
    run(cuda_lib, b, fmt, 16, window=window, sinks=sinks)


@pytest.mark.parametrize("fmt", FMTS)
def test_rows_that_see_nothing(cuda_lib, fmt):
    """Tokens at negative positions, requests of length 0, unallocated blocks."""
    b = P.Batch([(6, 4), (3, 0), (1, 0), (40, 500), (2, 64)], 16, seed=3, holes=12)
    run(cuda_lib, b, fmt, 32, window=20, sinks=2)
    run(cuda_lib, b, fmt, 128)
    b = P.Batch([(2, 100)], 64, seed=4)
    b.table[:] = -1
    run(cuda_lib, b, fmt, 16)


@pytest.mark.parametrize("fmt", FMTS)
def test_stride_of_blocks_and_other_scales(cuda_lib, fmt):
    b = P.Batch(RAGGED, 16, seed=8, stride_rows=24)
    run(cuda_lib, b, fmt, 16, pow2=False)
    run(cuda_lib, b, fmt, 40, window=50, sinks=1, pow2=False)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gain", [1e-3, 30.0])
def test_flat_and_peaked_rows(cuda_lib, fmt, gain):
    run(cuda_lib, P.Batch([(3, 1500), (100, 300)], 64, seed=5), fmt, 16, q_gain=gain)


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_split_keys(cuda_lib, fmt):
    smla = cuda_lib
    b = P.Batch([(1, 6000), (1, 300), (2, 1), (1, 4097)], 64, seed=6)
    assert smla.smla_fwd_window_workspace_size(4, b.N, 16, 576, fmt, b.table.shape[1], 64) > 0
    run(smla, b, fmt, 16)
    run(smla, b, fmt, 128, window=3000, sinks=300)


def shared_out(smla, b, h, **kw):
    """Whether the plan cuts the keys of all tiles into ranges."""
    return smla.smla_fwd_window_workspace_size(len(b.rows), b.N, h, 576, P.BF16, b.table.shape[1],
                                               b.block, **kw) > 0


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_ranges_over_many_requests(cuda_lib, fmt):
    """Ranges that hold several tiles: 80 requests (more than a warp), some of no
    token, some with more tokens than positions."""
    rows = [(1, 1 + 97 * r % 1500) for r in range(76)] + [(0, 40), (3, 2), (0, 0), (1, 0)]
    b = P.Batch(rows, 64, seed=21, pad=3)
    assert shared_out(cuda_lib, b, 16)
    run(cuda_lib, b, fmt, 16, pow2=False)
    b = P.Batch(rows[40:], 16, seed=22)
    run(cuda_lib, b, fmt, 24, window=200, sinks=33)


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_ranges_over_tiles_of_a_request(cuda_lib, fmt):
    b = P.Batch([(46, 3300), (0, 5), (34, 1700)], 64, seed=23)
    assert shared_out(cuda_lib, b, 128)
    run(cuda_lib, b, fmt, 128)


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_fewer_blocks_than_ranges(cuda_lib, fmt):
    """A wide table lets the plan expect long requests; these are short or empty."""
    for rows in ([(1, 3), (1, 1), (0, 0), (2, 1)], [(1, 0), (2, 0)], [(1, 129), (1, 300)]):
        b = P.Batch(rows, 64, seed=24)
        b.table = torch.cat([b.table, torch.full((len(rows), 200), -1, dtype=torch.int32)], 1)
        assert shared_out(cuda_lib, b, 16)
        run(cuda_lib, b, fmt, 16)
        run(cuda_lib, b, fmt, 16, window=100, sinks=2)


@pytest.mark.parametrize("fmt", FMTS)
def test_long_tiles_and_a_wrong_bound(cuda_lib, fmt):
    """54 key blocks in one piece (the bound says one) and in ranges."""
    b = P.Batch([(1, 6900), (3, 6500)], 64, seed=25)
    assert shared_out(cuda_lib, b, 40) and not shared_out(cuda_lib, b, 40, max_seq_len=1)
    run(cuda_lib, b, fmt, 40, max_seq_len=1)
    run(cuda_lib, b, fmt, 40)
    run(cuda_lib, b, fmt, 40, max_seq_len=1, window=5000, sinks=700)


def test_a_workspace_used_again(cuda_lib):
    """Calls of different shapes, one after the other in one workspace: what the
    last one left does not show."""
    smla = cuda_lib
    ws = torch.full((64 << 20,), 0x7F, dtype=torch.uint8, device="cuda")
    for rows, h, window in (([(1, 5000), (1, 90)], 128, 0), ([(2, 700), (1, 3000), (0, 3)], 16, 0),
                            ([(1, 40)], 1, 0), ([(1, 5000), (1, 90)], 128, 900)):
        b = P.Batch(rows, 64, seed=26, pad=2)
        q, cache, scale = make(b, P.BLOCK, h, 576, 5)
        want = launch(smla, b, P.BLOCK, q, cache, scale, 0.04, window, 1)
        got = launch(smla, b, P.BLOCK, q, cache, scale, 0.04, window, 1, workspace=ws)
        torch.cuda.synchronize()
        n = int(b.start[-1])
        assert torch.equal(got[0][:n], want[0][:n]) and torch.equal(got[1][:n], want[1][:n])


@pytest.mark.parametrize("window", [0, 80])
def test_lengths_that_no_table_holds(cuda_lib, window):
    """Not followed past the table, however long: the call ends and says so."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    b = P.Batch([(1, 100), (2, 300), (1, 70)], 64, seed=27)
    for fmt in (P.BF16, P.BLOCK):
        q, cache, scale = make(b, fmt, 16, 576, 5)
        ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, 0.04, window, 2)
        b.lens[1] = 2 ** 31 - 1
        out, lse = launch(smla, b, fmt, q, cache, scale, 0.04, window, 2)
        torch.cuda.synchronize()
        b.lens[1] = 300
        assert smla.smla_get_device_status(clear=True) == 5
        for n in (0, 3):                               # the other requests' tokens
            one = tuple(x[n:n + 1] for x in ref)
            alone = P.Batch([(1, 1)], 64)
            P.check_attention(out[n:n + 1], lse[n:n + 1], one, q[n:n + 1], fmt, 0.04, alone)


@pytest.mark.parametrize("h", [16, 40])
def test_same_as_the_sparse_forward(cuda_lib, h):
    """The visible positions' rows listed for smla_fwd: two answers, each within
    its bound of the formula's."""
    smla = cuda_lib
    b = P.Batch([(1, 700), (1, 333), (2, 90)], 64, seed=28)
    q, cache, scale = make(b, P.BF16, h, 576, 6)
    sm, window, sinks = 576 ** -0.5, 400, 3
    out, lse = launch(smla, b, P.BF16, q, cache, scale, sm, window, sinks)
    idx = torch.full((b.N, 512), -1, dtype=torch.int32)
    for n, r, p in b.tokens():
        seen = [b.slot(r, e) for e in range(p + 1) if e > p - window or e < sinks]
        idx[n, :len(seen)] = torch.tensor(seen, dtype=torch.int32)
    other, lse2 = smla.smla_fwd(q.cuda(), cache.cuda(), P.BF16, None, idx.cuda(), None,
                                sm)
    torch.cuda.synchronize()
    ref = P.attend(q, P.dequant(cache, P.BF16, scale, b), b, sm, window, sinks)
    P.check_attention(out, lse, ref, q, P.BF16, sm, b)
    P.check_attention(other, lse2, ref, q, P.BF16, sm, b)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_values_that_a_token_does_not_see(cuda_lib, fmt, bad):
    """Not-a-number rows past the end, before the window, in unallocated
    blocks, and in a later token's row: earlier rows come out as without."""
    smla = cuda_lib
    b = P.Batch([(90, 200), (1, 130), (1, 3000)], 64, seed=12)
    window, sinks, h, d = 70, 5, 16, 576
    q, cache, scale = make(b, fmt, h, d, 3)
    used = {b.slot(r, e) for r, (_, L) in enumerate(b.rows) for e in range(L)}
    rows = [s for s in range(b.num_slots) if s not in used]          # never written
    rows += [b.slot(0, e) for e in range(5, 30)]                     # before every window
    code = 0x7F if fmt != P.BF16 else bad
    poisoned = cache.clone()
    poisoned[rows] = code
    later = b.slot(0, 180)                                           # seen from position 180 on
    poisoned[later, 7] = code
    sm = d ** -0.5
    ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, sm, window, sinks)
    for splits_by in (None, 3000):                                   # also with split keys
        out, lse = launch(smla, b, fmt, q, poisoned, scale, sm, window if splits_by is None else 0,
                          sinks, max_seq_len=splits_by)
        torch.cuda.synchronize()
        if splits_by:
            ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, sm, 0, 0)
            # (without a window the rows before it are seen: nothing to compare there)
            clean = torch.arange(b.N) >= 90
        else:
            pos = torch.tensor([p for _, _, p in b.tokens()])
            clean = ~((torch.arange(b.N) < 90) & (pos >= 180))
        assert bool(torch.isnan(out[:90].float().cpu()[~clean[:90]]).any())
        keep = clean.nonzero().flatten()
        O = out.double().cpu()
        assert bool(torch.isfinite(O[keep]).all()) and bool(torch.isfinite(lse.cpu()[keep]).all())
        tol = 2.0 ** -8 * ref[0].abs() + (2.0 ** -7 + 2.0 ** -9) * ref[2] + 2.0 ** -23 * ref[5]
        assert bool(((O - ref[0]).abs() <= tol)[keep].all())


def test_offsets_past_32_bits(cuda_lib):
    """A cache of more than 2^32 bytes, in both widths."""
    smla = cuda_lib
    for fmt, S in ((P.BF16, 4_000_000), (P.BLOCK, 8_000_000)):
        bs = 64
        b = P.Batch([(1, 200)], bs, seed=2)
        q, cache, scale = make(b, fmt, 16, 576, 4)
        big = torch.zeros((S, 576), dtype=cache.dtype, device="cuda")
        top = S // bs - 1
        sc = None if scale is None else torch.ones(S // bs, device="cuda")
        tab = b.table.clone()
        for k in range(tab.shape[1]):
            blk = int(b.table[0, k])
            big[(top - k) * bs:(top - k + 1) * bs] = cache[blk * bs:(blk + 1) * bs].cuda()
            if sc is not None:
                sc[top - k] = scale[blk]
            tab[0, k] = top - k
        start, lens, _ = b.dev()
        out, lse = smla.smla_fwd_window(q.cuda(), big, fmt, sc, start, lens, tab.cuda(), bs,
                                        576 ** -0.5)
        torch.cuda.synchronize()
        ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, 576 ** -0.5, 0, 0)
        P.check_attention(out, lse, ref, q, fmt, 576 ** -0.5, b)
        del big


def test_past_the_table_and_the_cache(cuda_lib):
    """Positions past the block table and rows past the cache are not seen."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    b = P.Batch([(2, 128), (1, 64)], 64, seed=9, spare=0)
    q, cache, _ = make(b, P.BF16, 16, 576, 4)
    start, lens, tab = b.dev()
    ref = P.attend(q, cache.double(), b, 0.04, 0, 0)
    longer = lens.clone()
    tab2 = torch.cat([tab, torch.full((2, 1), 99, dtype=torch.int32, device="cuda")], 1)
    longer[1] = 64
    for table, ln in ((tab, lens), (tab2, lens)):
        out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), P.BF16, None, start, ln, table, 64,
                                        0.04)
        P.check_attention(out, lse, ref, q, P.BF16, 0.04, b)
    assert smla.smla_get_device_status(clear=True) == 0
    lens2 = lens.clone()
    lens2[0] = 500                                   # its last columns are missing
    out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), P.BF16, None, start, lens2, tab2, 64,
                                    0.04)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out.float()).all())
    assert smla.smla_get_device_status(clear=True) == 5


def test_no_lse_zero_tokens_and_workspace(cuda_lib):
    smla = cuda_lib
    b = P.Batch([(1, 5000)], 64, seed=10)
    q, cache, _ = make(b, P.BF16, 16, 576, 4)
    start, lens, tab = b.dev()
    args = (q.cuda(), cache.cuda(), P.BF16, None, start, lens, tab, 64, 0.04)
    O, L = smla.smla_fwd_window(*args)
    n = smla.smla_fwd_window_workspace_size(1, 1, 16, 576, P.BF16, tab.shape[1], 64)
    ws = Guarded((n,), torch.uint8)
    pad = (-ws.t.data_ptr()) % 256
    assert pad == 0
    O2, L2 = smla.smla_fwd_window(*args, want_lse=False, workspace=ws.t)
    ws.check("workspace")
    assert L2 is None and torch.equal(O, O2)
    with pytest.raises(smla.SmlaError) as e:
        smla.smla_fwd_window(*args, workspace=ws.t[:n - 256])
    assert e.value.code == 6
    out, lse = smla.smla_fwd_window(q.cuda()[:0], *args[1:4], torch.zeros(2, dtype=torch.int32).cuda(),
                                    lens, tab, 64, 0.04)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16)


def test_captured_and_two_streams(cuda_lib):
    """A captured call replayed on new contents, and two calls at once on two
    streams with a workspace each."""
    smla = cuda_lib
    b = P.Batch([(1, 3000), (2, 500)], 64, seed=11)
    q, cache, scale = make(b, P.BLOCK, 16, 576, 4)
    start, lens, tab = b.dev()
    gq, gc, gs = q.cuda(), cache.cuda(), scale.cuda()
    call = lambda: smla.smla_fwd_window(gq, gc, P.BLOCK, gs, start, lens, tab, 64, 0.04,  # noqa: E731
                                        window=2500, sinks=4)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = call()
    for seed in (20, 21):
        q2, c2, s2 = make(b, P.BLOCK, 16, 576, seed)
        gq.copy_(q2), gc.copy_(c2), gs.copy_(s2)
        graph.replay()
        torch.cuda.synchronize()
        ref = P.attend(q2, P.dequant(c2, P.BLOCK, s2, b), b, 0.04, 2500, 4)
        P.check_attention(out, lse, ref, q2, P.BLOCK, 0.04, b)
    want = call()
    torch.cuda.synchronize()
    got = []
    streams = [torch.cuda.Stream() for _ in range(2)]
    for k in range(6):
        got.append(smla.smla_fwd_window(gq, gc, P.BLOCK, gs, start, lens, tab, 64, 0.04,
                                        window=2500, sinks=4, stream=streams[k % 2]))
    torch.cuda.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_append_then_attend(cuda_lib):
    """A prompt in two chunks and three decode steps through the append and
    the attention, against the formula on the cache's contents."""
    smla = cuda_lib
    h, bs, d = 16, 16, 576
    g = torch.Generator().manual_seed(1)
    steps = [[(40, 40), (7, 7)], [(35, 75), (20, 27)]] + [[(1, 76 + k), (1, 28 + k)] for k in range(3)]
    full = P.Batch(steps[-1], bs, seed=3)
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    ang = torch.arange(100, dtype=torch.float64)[:, None] * inv
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    for fmt in FMTS:
        cache = torch.zeros((full.num_slots, d), dtype=torch.bfloat16 if fmt == P.BF16 else
                            torch.uint8, device="cuda")
        scale = {P.BF16: None, P.E4M3: torch.full((1,), 0.0625, device="cuda"),
                 P.BLOCK: torch.zeros(full.pool, device="cuda")}[fmt]
        rows = torch.zeros((full.num_slots, d), dtype=torch.float64)
        for step in steps:
            b = P.Batch(step, bs, seed=3)
            b.table, b.num_slots = full.table, full.num_slots
            x = torch.randn((b.N, d), generator=g).bfloat16()
            q = torch.randn((b.N, h, d), generator=g).bfloat16()
            start, lens, tab = b.dev()
            gx, gq = x.cuda(), q.cuda()
            smla.smla_cache_append(gx[:, :512], gx[:, 512:], cs.cuda(), start, lens, tab, bs,
                                   cache, fmt, scale, q_pe=gq[:, :, 512:])
            out, lse = smla.smla_fwd_window(gq, cache, fmt, scale, start, lens, tab, bs, d ** -0.5,
                                            window=30, sinks=2)
            torch.cuda.synchronize()
            for n, r, pos in b.tokens():
                rows[b.slot(r, pos)] = torch.cat(
                    [x[n, :512], P.rotate(x[n, 512:].float(), cs[pos], True)]).double()
            held = P.dequant(cache.cpu(), fmt, None if scale is None else scale.cpu(), full)
            used = [full.slot(r, e) for r, (_, L) in enumerate(step) for e in range(L)]
            # e4m3's half step, 2^-4, twice where a growing scale rounds again;
            # 2^-9 scales (its smallest value) below that
            amax = rows[used].abs().max()
            off = (held - rows)[used].abs()
            lim = 2.0 ** -8 * rows[used].abs() if fmt == P.BF16 else \
                2.0 ** -4 * rows[used].abs() * 1.07 + 2.0 ** -9 * amax / 224
            if fmt != P.E4M3:
                assert bool((off <= lim).all())
            ref = P.attend(gq.cpu(), held, b, d ** -0.5, 30, 2)
            P.check_attention(out, lse, ref, gq.cpu(), fmt, d ** -0.5, b)


def test_binding_refusals(cuda_lib):
    """Tensors of another device, type or layout never reach a launch."""
    smla = cuda_lib
    b = P.Batch([(1, 700), (2, 90)], 64, seed=14)
    q, cache, scale = make(b, P.BLOCK, 16, 576, 4)
    start, lens, tab = b.dev()
    good = dict(q=q.cuda(), kv_cache=cache.cuda(), kv_dtype=P.BLOCK, k_scale=scale.cuda(),
                query_start=start, seq_lens=lens, block_table=tab, block_size=64, sm_scale=0.04)
    smla.smla_fwd_window(**good)
    wide = torch.zeros((b.N, 16, 600), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(q=q), dict(q=wide[:, :, :576]), dict(q=good["q"].float()),
                dict(kv_cache=cache), dict(kv_cache=good["kv_cache"].view(torch.int8)),
                dict(k_scale=None), dict(k_scale=scale), dict(k_scale=good["k_scale"][:1]),
                dict(query_start=b.start), dict(seq_lens=b.lens), dict(block_table=b.table),
                dict(query_start=start.long()), dict(seq_lens=lens[:1]), dict(block_table=tab[0]),
                dict(block_table=tab.t()), dict(num_slots=b.num_slots + 1),
                dict(out=torch.zeros((b.N, 16, 512), dtype=torch.bfloat16)),
                dict(lse=torch.zeros((b.N, 16))), dict(lse=torch.zeros((b.N, 8), device="cuda")),
                dict(workspace=torch.zeros(1 << 26, dtype=torch.uint8)), dict(kv_dtype=6)):
        with pytest.raises(ValueError):
            smla.smla_fwd_window(**{**good, **bad})
    assert smla.smla_get_device_status(clear=True) == 0


def test_back_to_back_calls(cuda_lib):
    """Calls that share their buffers and one workspace on a stream, read between
    them without a wait of the host: the merge of one is done before the next."""
    smla = cuda_lib
    b = P.Batch([(1, 4000), (2, 2500)], 64, seed=16)
    assert shared_out(smla, b, 32)
    start, lens, tab = b.dev()
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    out = torch.empty((b.N, 32, 512), dtype=torch.bfloat16, device="cuda")
    lse = torch.empty((b.N, 32), device="cuda")
    qs, want, got = [], [], []
    for seed in (1, 2):
        q, cache, _ = make(b, P.BF16, 32, 576, seed)
        qs.append((q.cuda(), cache.cuda()))
        want.append(smla.smla_fwd_window(*qs[-1], P.BF16, None, start, lens, tab, 64, 0.04))
        torch.cuda.synchronize()
    for k in range(12):
        smla.smla_fwd_window(*qs[k % 2], P.BF16, None, start, lens, tab, 64, 0.04, out=out, lse=lse,
                             workspace=ws)
        got.append((out.clone(), lse.clone()))
    torch.cuda.synchronize()
    for k, (o, l) in enumerate(got):
        assert torch.equal(o, want[k % 2][0]) and torch.equal(l, want[k % 2][1])


def test_a_wait_that_runs_out(cuda_lib):
    """A stalled launch reports the timeout, and the next one is right: a tile in
    one piece, and in ranges."""
    smla = cuda_lib
    whole = P.Batch([(1, 300), (20, 90)], 64, seed=13)
    parts = P.Batch([(1, 6000), (1, 90)], 64, seed=13)
    assert not shared_out(smla, whole, 16) and shared_out(smla, parts, 16)
    smla.smla_get_device_status(clear=True)
    for b in (whole, parts):
        for fmt in (P.BF16, P.BLOCK):
            q, cache, scale = make(b, fmt, 16, 576, 4)
            smla.smla_test_set_stall(True, 2000)
            try:
                launch(smla, b, fmt, q, cache, scale, 0.04, 0, 0)
                assert smla.smla_get_device_status(clear=True) == 4
            finally:
                smla.smla_test_set_stall(False)
            run(smla, b, fmt, 16)
