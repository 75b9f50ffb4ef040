"""smla_cache_append against its own arithmetic on the CPU, bit for bit: every
format, both rope forms, strided inputs, blocks that already hold rows, tokens
that are skipped, and the rows, scales and queries that must stay as they were."""
import pytest
import torch

from tests import _paged as P

pytestmark = pytest.mark.gpu


def table(length):
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64) / 64)
    a = torch.arange(length, dtype=torch.float64)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def make(batch, fmt, d, h, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    N, S = batch.N, batch.num_slots
    x = torch.randn((N, 704), generator=g).mul_(spread).bfloat16()
    kv_c, k_pe = x[:, :512], x[:, 640:] if d == 576 else None
    q_pe = torch.randn((N, h, 192), generator=g).bfloat16()[:, :, 128:] if d == 576 and h else None
    width = P.DS_MLA_ROW if fmt == P.DS_MLA else d
    if fmt == P.BF16:
        cache = torch.randn((S, d), generator=g).bfloat16()
    else:
        cache = torch.randint(0, 120, (S, width), generator=g).to(torch.uint8)
    step = batch.stride_rows or batch.block
    scale = {P.BF16: None, P.DS_MLA: None, P.E4M3: torch.tensor([0.013]),
             P.GROUP128: torch.rand((S, -(-d // 128)), generator=g),
             P.GROUP4_KPE: torch.rand((S, 4), generator=g),
             P.BLOCK: torch.exp2(torch.randint(-12, 4, (S // step,), generator=g).float())}[fmt]
    return kv_c, k_pe, q_pe, cache, scale


def on_gpu(t):
    """A copy on the GPU with the same strides."""
    if t is None:
        return None
    base = torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda")
    return base.copy_(t)


def run(smla, batch, fmt, d, h=3, interleaved=True, seed=1, in_place=False, spread=1.0,
        positions=None, edit=None):
    smla.smla_get_device_status(clear=True)
    kv_c, k_pe, q_pe, cache, scale = make(batch, fmt, d, h, seed, spread)
    if edit:
        edit(kv_c, k_pe, cache, scale)
    cs = table(positions or max(1, int(batch.lens.max()))) if d == 576 else None
    q_out = None if q_pe is None else (q_pe.clone() if in_place else
                                       torch.full(q_pe.shape, 7.0).bfloat16())
    start, lens, tab = batch.dev()
    gc, gs = cache.cuda(), on_gpu(scale)
    gq = on_gpu(q_pe)
    go = gq if in_place else on_gpu(q_out)
    smla.smla_cache_append(on_gpu(kv_c), on_gpu(k_pe), on_gpu(cs), start, lens, tab, batch.block,
                           gc, fmt, gs, kpe_scale=0.07, interleaved=interleaved, q_pe=gq,
                           q_out=go, block_stride_rows=batch.stride_rows)
    torch.cuda.synchronize()
    P.append(batch, kv_c, k_pe, cs, cache, fmt, scale, 0.07, interleaved, q_pe, q_out)
    got = gc.cpu()
    if fmt == P.BF16:
        assert torch.equal(got.view(torch.int16), cache.view(torch.int16))
    else:
        assert torch.equal(got, cache)
    if scale is not None:
        assert torch.equal(gs.cpu(), scale)
    if q_pe is not None:
        assert torch.equal(go.cpu(), q_out)
    return smla.smla_get_device_status(clear=True)


RAGGED = [(1, 1), (5, 70), (0, 9), (130, 130), (1, 64), (1, 65), (3, 129), (64, 191)]


@pytest.mark.parametrize("d", [512, 576])
@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.GROUP128, P.DS_MLA, P.GROUP4_KPE, P.BLOCK])
def test_formats(cuda_lib, fmt, d):
    if d == 512 and fmt in (P.DS_MLA, P.GROUP4_KPE):
        pytest.skip("the format has 576 channels")
    for block, interleaved in ((64, True), (16, False), (7, True)):
        b = P.Batch(RAGGED, block, seed=block, pad=3)
        assert run(cuda_lib, b, fmt, d, interleaved=interleaved, seed=block) == 0


@pytest.mark.parametrize("h", [1, 4, 16, 37, 128])
def test_query_heads_and_in_place(cuda_lib, h):
    b = P.Batch([(2, 40), (9, 300), (1, 5)], 32, seed=3, pad=2)
    assert run(cuda_lib, b, P.BF16, 576, h=h) == 0
    assert run(cuda_lib, b, P.BF16, 576, h=h, interleaved=False, in_place=True) == 0


def test_decode_of_many_requests(cuda_lib):
    b = P.Batch([(1, 1 + 37 * r % 500) for r in range(300)], 16, seed=5)
    for fmt in (P.BF16, P.BLOCK):
        assert run(cuda_lib, b, fmt, 576, h=2) == 0


@pytest.mark.parametrize("block", [1, 3, 64, 100, 256])
def test_block_scale_grows_and_keeps(cuda_lib, block):
    """Blocks with older rows: larger, smaller and equal new rows."""
    for spread in (1e-4, 1.0, 300.0):
        b = P.Batch([(1, 10), (2, 64), (3, 200), (block, 2 * block), (300, 301)], block, seed=block)
        assert run(cuda_lib, b, P.BLOCK, 576, spread=spread, seed=block + 9) == 0


def test_block_scale_of_zeros_and_non_finite_values(cuda_lib):
    def edit(kv_c, k_pe, cache, scale):
        kv_c.zero_()
        k_pe.zero_()
        kv_c[1, 5], kv_c[1, 6], kv_c[2, 0] = float("inf"), float("-inf"), 3.0
    b = P.Batch([(1, 1), (2, 2), (2, 30)], 16, seed=4)
    assert run(cuda_lib, b, P.BLOCK, 576, edit=edit) == 0


def test_rows_that_are_skipped(cuda_lib):
    smla = cuda_lib
    # negative positions, unallocated blocks, a stride larger than the block
    for fmt in (P.BF16, P.BLOCK, P.DS_MLA):
        b = P.Batch([(5, 3), (4, 0), (20, 50), (1, 33)], 8, seed=6, pad=5, stride_rows=11, holes=4)
        assert run(smla, b, fmt, 576) == 0
    # positions without a rope row: skipped, and the status says so
    b = P.Batch([(4, 40), (10, 25)], 8, seed=7)
    for fmt in (P.BF16, P.BLOCK):
        assert run(smla, b, fmt, 576, positions=38) == 5


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_past_the_table_and_the_cache(cuda_lib, fmt):
    """A position past the block table and a block past the cache write
    nothing and set the status."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    N, bs, S = 6, 4, 16
    start = torch.tensor([0, 3, 6], dtype=torch.int32).cuda()
    lens = torch.tensor([12, 4], dtype=torch.int32).cuda()       # positions 9..11 and 1..3
    tab = torch.tensor([[0, 1], [9, 2]], dtype=torch.int32).cuda()
    cache = torch.full((S, 512), 3, dtype=torch.uint8, device="cuda") if fmt else \
        torch.full((S, 512), 3.0, device="cuda").bfloat16()
    scale = torch.ones(4, device="cuda") if fmt else None
    before = cache.clone()
    kv = torch.randn((N, 512), device="cuda").bfloat16()
    smla.smla_cache_append(kv, None, None, start, lens, tab, bs, cache, fmt, scale)
    torch.cuda.synchronize()
    assert torch.equal(cache, before)
    assert smla.smla_get_device_status(clear=True) == 5


def test_offsets_past_32_bits(cuda_lib):
    """Rows behind 2^32 bytes of the cache."""
    smla = cuda_lib
    S, bs = 4_000_000, 64
    cache = torch.zeros((S, 576), dtype=torch.bfloat16, device="cuda")
    blk = S // bs - 1
    tab = torch.tensor([[blk]], dtype=torch.int32).cuda()
    start = torch.tensor([0, 2], dtype=torch.int32).cuda()
    lens = torch.tensor([2], dtype=torch.int32).cuda()
    kv = torch.randn((2, 512), device="cuda").bfloat16()
    pe = torch.randn((2, 64), device="cuda").bfloat16()
    smla.smla_cache_append(kv, pe, table(2).cuda(), start, lens, tab, bs, cache, P.BF16)
    assert torch.equal(cache[blk * bs:blk * bs + 2, :512], kv)
    assert int((cache.view(torch.int16) != 0).any(1).sum()) == 2


def test_captured_and_on_another_stream(cuda_lib):
    smla = cuda_lib
    b = P.Batch([(1, 65), (1, 30)], 64, seed=9)
    kv_c, k_pe, q_pe, cache, scale = make(b, P.BLOCK, 576, 4, 3)
    cs = table(65)
    start, lens, tab = b.dev()
    kc, kp, q, gs = on_gpu(kv_c), on_gpu(k_pe), on_gpu(q_pe), scale.cuda()
    gcs, gc, go = cs.cuda(), cache.cuda(), torch.zeros((b.N, 4, 64)).bfloat16().cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        smla.smla_cache_append(kc, kp, gcs, start, lens, tab, 64, gc, P.BLOCK, gs, q_pe=q, q_out=go)
    for seed in (5, 6):
        kv2, pe2, q2, cache2, scale2 = make(b, P.BLOCK, 576, 4, seed)
        for t, s in ((kc, kv2), (kp, pe2), (q, q2), (gc, cache2), (gs, scale2)):
            t.copy_(s)
        graph.replay()
        torch.cuda.synchronize()
        out = torch.zeros((b.N, 4, 64)).bfloat16()
        P.append(b, kv2, pe2, cs, cache2, P.BLOCK, scale2, 1.0, True, q2, out)
        assert torch.equal(gc.cpu(), cache2) and torch.equal(gs.cpu(), scale2)
        assert torch.equal(go.cpu(), out)


def test_group_rows_equal_the_slot_mapped_write(cuda_lib):
    """Without rope the group format's rows are smla_cache_write_e4m3_group's."""
    smla = cuda_lib
    b = P.Batch([(40, 100), (7, 7)], 16, seed=11)
    kv = torch.randn((b.N, 512), device="cuda").bfloat16()
    start, lens, tab = b.dev()
    one = torch.zeros((b.num_slots, 512), dtype=torch.uint8, device="cuda")
    two, s1 = one.clone(), torch.zeros((b.num_slots, 4), device="cuda")
    s2 = s1.clone()
    smla.smla_cache_append(kv, None, None, start, lens, tab, 16, one, P.GROUP128, s1)
    slots = torch.tensor([b.slot(r, p) for _, r, p in b.tokens()], dtype=torch.int32).cuda()
    smla.smla_cache_write_e4m3_group(kv, None, slots, two, s2)
    assert torch.equal(one, two) and torch.equal(s1, s2)


def test_binding_refusals(cuda_lib):
    """Tensors of another device, type or layout never reach a launch."""
    smla = cuda_lib
    b = P.Batch([(2, 70), (3, 20)], 64, seed=15)
    kv_c, k_pe, q_pe, cache, scale = make(b, P.BLOCK, 576, 4, 5)
    start, lens, tab = b.dev()
    good = dict(kv_c=on_gpu(kv_c), k_pe=on_gpu(k_pe), cos_sin=table(80).cuda(), query_start=start,
                seq_lens=lens, block_table=tab, block_size=64, kv_cache=cache.cuda(),
                kv_dtype=P.BLOCK, k_scale=scale.cuda(), q_pe=on_gpu(q_pe))
    smla.smla_cache_append(**good)
    for bad in (dict(kv_c=kv_c), dict(kv_c=good["kv_c"].half()), dict(kv_c=good["kv_c"][:, :500]),
                dict(k_pe=k_pe), dict(k_pe=good["k_pe"][:2]), dict(cos_sin=None),
                dict(cos_sin=table(80)), dict(cos_sin=good["cos_sin"].double()),
                dict(cos_sin=good["cos_sin"].t().contiguous()), dict(query_start=b.start),
                dict(seq_lens=lens.long()), dict(block_table=b.table), dict(block_size=0),
                dict(block_stride_rows=32), dict(kv_cache=cache), dict(k_scale=scale),
                dict(k_scale=None), dict(q_pe=q_pe), dict(q_pe=good["q_pe"][:2]),
                dict(q_out=q_pe), dict(q_out=good["q_pe"].transpose(1, 2)), dict(kv_dtype=-1)):
        with pytest.raises(ValueError):
            smla.smla_cache_append(**{**good, **bad})
    assert smla.smla_get_device_status(clear=True) == 0
