"""smla_fwd_window where its arithmetic has to hold over a wide range: block scales
that differ by many powers of two, scales of zero, and scores of any size."""
import math

import pytest
import torch

from tests import _paged as P
from tests.test_window_gpu import launch, make, shared_out

pytestmark = pytest.mark.gpu


def compare(smla, batch, fmt, q, cache, scale, sm, window=0, sinks=0, slack=0.0, **kw):
    """Against the fp64 formula, within P.check_attention's bounds (``slack``: added
    to O's)."""
    smla.smla_get_device_status(clear=True)
    out, lse = launch(smla, batch, fmt, q, cache, scale, sm, window, sinks, **kw)
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    rows = P.dequant(cache, fmt, scale, batch)
    if fmt == P.BLOCK:
        batch.row_scale = batch.row_scale.clamp(min=2.0 ** -64)
    O, L, A, D, K, G = P.attend(q, rows, batch, sm, window, sinks)
    P.check_attention(out, lse, (O, L, A + slack, D, K, G), q, fmt, sm, batch, pow2=False)
    return out, lse


# (rows, bound on the lengths: 1 takes every tile in one piece, None cuts the keys of
# all tiles into ranges)
WHOLE = ([(1, 900), (30, 400), (1, 130)], 1)
RANGES = ([(1, 5000), (2, 700), (1, 130)], None)


def mixed_scales(b, seed, low, share):
    """Scales 2^-6 with a share of 2^low ones among them; codes of normal values."""
    g = torch.Generator().manual_seed(seed)
    n = -(-b.num_slots // (b.stride_rows or b.block))
    return torch.where(torch.rand(n, generator=g) < share, 2.0 ** low, 2.0 ** -6).float()


@pytest.mark.parametrize("rows,limit", [WHOLE, RANGES], ids=["whole", "ranges"])
@pytest.mark.parametrize("block", [7, 16, 32, 64, 128])
@pytest.mark.parametrize("low", [-24, -30, -40, -64])
def test_block_scales_far_apart(cuda_lib, rows, limit, block, low):
    """Rows whose scores are near each other: the blocks of a tiny scale hold their
    share of the softmax, although their values are next to nothing."""
    for share, h in ((0.5, 16), (0.93, 128)):
        b = P.Batch(rows, block, seed=31)
        q, cache, _ = make(b, P.BLOCK, h, 576, 5, q_gain=0.2)
        scale = mixed_scales(b, 7, low, share)
        assert limit or shared_out(cuda_lib, b, h)
        compare(cuda_lib, b, P.BLOCK, q, cache, scale, 576 ** -0.5, max_seq_len=limit)
    compare(cuda_lib, b, P.BLOCK, q, cache, scale, 576 ** -0.5, 200, 5, max_seq_len=limit)


@pytest.mark.parametrize("rows,limit", [WHOLE, RANGES], ids=["whole", "ranges"])
@pytest.mark.parametrize("high", [40, 90, 120])
@pytest.mark.parametrize("block", [16, 64])
def test_block_scales_of_any_size(cuda_lib, rows, limit, high, block):
    """Scales 2^high and 2^-64 in one row, to the ends of what the append writes.  Keys of
    a large scale have only channel 0 (2^-6), to which the queries are blind, the others
    have all but it: every score is 0 (2^-50 at most), so LSE = ln n and O's channel 0 is
    a count, to bf16's rounding, 2^-9 of a 9-bit weight and the exponentials' 2^-16; the
    other channels hold 448 * 2^-64 at most.  LSE: the reference is `high` log2 units, so
    its sum with log2 l is off by 2^-17 at most, and ln 2 of that."""
    b = P.Batch(rows, block, seed=32)
    q, cache, scale = make(b, P.BLOCK, 16, 576, 6)
    g = torch.Generator().manual_seed(9)
    top = torch.rand(scale.shape, generator=g) < 0.3
    codes = cache.view(b.pool, block, 576)
    codes[top, :, 1:] = 0
    codes[top, :, 0] = 0x08                            # 2^-6
    codes[~top, :, 0] = 0
    q[:, :, 0] = 0
    scale = torch.where(top, 2.0 ** high, 2.0 ** -64).float()
    out, lse = launch(cuda_lib, b, P.BLOCK, q, cache, scale, 576 ** -0.5, 0, 0,
                      max_seq_len=limit)
    out, lse = out.double().cpu(), lse.double().cpu()
    assert bool(top[b.table[0].long()].any())
    for n, r, pos in b.tokens():
        large = sum(bool(top[b.table[r, e // block]]) for e in range(pos + 1))
        assert bool(((lse[n] - math.log(pos + 1)).abs() <= 2.0 ** -16).all())
        want = large / (pos + 1) * 2.0 ** (high - 6)
        assert bool(((out[n, :, 0] - want).abs() <= (2.0 ** -8 + 2.0 ** -8) * want).all())
        assert bool((out[n, :, 1:].abs() <= 450 * 2.0 ** -64).all())


@pytest.mark.parametrize("rows,limit", [WHOLE, RANGES], ids=["whole", "ranges"])
@pytest.mark.parametrize("fill", [0.0, 2.0 ** -40])
def test_appended_rows_of_zeros_beside_normal_ones(cuda_lib, rows, limit, fill):
    """The append gives a block of zero rows (dummy tokens) the scale 2^-64."""
    smla = cuda_lib
    h, block = 16, 64
    b = P.Batch(rows, block, seed=33)
    g = torch.Generator().manual_seed(2)
    full = P.Batch([(L, L) for _, L in rows], block, seed=33)
    assert torch.equal(full.table, b.table)
    x = torch.randn((full.N, 512), generator=g)
    at = torch.tensor([p for _, _, p in full.tokens()])
    x[(at // block) % 3 == 1] = fill
    cache = torch.zeros((b.num_slots, 512), dtype=torch.uint8, device="cuda")
    scale = torch.ones(b.pool, device="cuda")
    smla.smla_cache_append(x.bfloat16().cuda(), None, None, *full.dev(), block, cache, P.BLOCK,
                           scale)
    assert float(scale.min()) <= 2.0 ** -48
    q = (torch.randn((b.N, h, 512), generator=g) * 0.3).bfloat16()
    compare(smla, b, P.BLOCK, q, cache.cpu(), scale.cpu(), 512 ** -0.5, max_seq_len=limit)


@pytest.mark.parametrize("rows,limit", [WHOLE, RANGES], ids=["whole", "ranges"])
@pytest.mark.parametrize("block", [16, 64])
def test_scales_of_zero(cuda_lib, rows, limit, block):
    """A zero scale makes keys and values zero: score 0, weight 1 of the softmax.  First,
    among, last and alone; the other scores far below them and far above.  (A scale
    below 2^-64 counts as 2^-64: values of at most 448 * 2^-64.)"""
    tiny = 448 * 2.0 ** -64 * 2 ** 7
    for where in ("first", "last", "mixed", "all"):
        for shift in (0.0, -60.0, 60.0):
            b = P.Batch(rows, block, seed=34)
            q, cache, scale = make(b, P.BLOCK, 16, 576, 8, q_gain=0.2)
            for r, (_, L) in enumerate(rows):
                pages = -(-L // block)
                for k in range(pages):
                    zero = {"first": k < pages // 2, "last": k >= pages // 2, "mixed": k % 3 == 1,
                            "all": True}[where]
                    if zero:
                        scale[b.table[r, k]] = 0.0
            # every other key's score moves by `shift` nats (through one channel of its own)
            cache[:, 575] = 0x7E                       # 448, by 2^-6: 7
            q[:, :, 575] = shift * 24 / 7
            scale[(scale > 0)] = 2.0 ** -6
            compare(cuda_lib, b, P.BLOCK, q, cache, scale, 576 ** -0.5, slack=tiny,
                    max_seq_len=limit)


def test_scales_that_are_no_numbers(cuda_lib):
    """A scale that is negative or not finite makes the rows that see its block NaN, and
    no other's."""
    for bad in (float("nan"), float("inf"), -1.0):
        for block in (16, 64):
            b = P.Batch([(100, 300), (1, 500)], block, seed=35)
            q, cache, scale = make(b, P.BLOCK, 16, 576, 9)
            cache[(cache & 0x7F) == 0] = 1             # (no infinity times zero)
            ref = P.attend(q, P.dequant(cache, P.BLOCK, scale, b), b, 576 ** -0.5, 0, 0)
            page = 256 // block                        # positions from 256 on
            changed = scale.clone()
            changed[b.table[0, page]] = bad
            out, lse = launch(cuda_lib, b, P.BLOCK, q, cache, changed, 576 ** -0.5, 0, 0)
            O = out.float().cpu()
            sees = torch.tensor([r == 0 and p >= page * block for _, r, p in b.tokens()])
            assert bool(torch.isnan(O[sees]).all())
            clean = (~sees).nonzero().flatten()
            assert bool(torch.isfinite(O[clean]).all())
            tol = 2.0 ** -8 * ref[0].abs() + (2.0 ** -7 + 2.0 ** -9) * ref[2] + 2.0 ** -23 * ref[5]
            assert bool(((O - ref[0]).abs() <= tol)[clean].all())


@pytest.mark.parametrize("rows,limit", [WHOLE, RANGES], ids=["whole", "ranges"])
@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
def test_large_scores(cuda_lib, rows, limit, fmt):
    """Scores up to 1.3e5 of either sign.  Queries have one channel, which no value has,
    and it takes two values over the keys: a row's scores are S, or S less a thousandth
    and more.  Products of one bf16 (or E4M3) pair are exact in fp32; S, as a product of
    three fp32 factors, is off by 2^-22 |S|, the same for all keys of equal value.  So O
    is the mean of the keys of the larger score (the others' weights underflow, or S is
    below 100 and their error is 2^-22 * 100)."""
    sm, h = 1 / 24, 32
    b = P.Batch(rows, 64, seed=36)
    q, cache, scale = make(b, fmt, h, 576, 10)
    g = torch.Generator().manual_seed(3)
    q.zero_()
    mag = torch.exp2(torch.rand((b.N, h), generator=g) * 14 - 1)
    q[:, :, 570] = (mag * torch.where(torch.rand((b.N, h), generator=g) < 0.5, -1.0, 1.0)).bfloat16()
    q[:, 0, 570], q[:, 1, 570] = 8000.0, -8000.0
    pick = torch.rand(b.num_slots, generator=g) < 0.4
    if fmt == P.BF16:
        cache[:, 570] = torch.where(pick, 384.0, 192.0).bfloat16()
    else:
        scale = torch.ones_like(scale)
        cache[:, 570] = torch.where(pick, 0x7C, 0x74).to(torch.uint8)      # 384 and 192
    out, lse = launch(cuda_lib, b, fmt, q, cache, scale, sm, 0, 0, max_seq_len=limit)
    O, L, A, _, _, G = P.attend(q, P.dequant(cache, fmt, scale, b), b, sm, 0, 0)
    assert float(L.max()) > 1e5 and float(L.min()) < -5e4
    out, lse = out.double().cpu(), lse.double().cpu()
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
    assert bool(((lse - L).abs() <= 2.0 ** -21 * L.abs() + 2.0 ** -16).all())
    tol = 2.0 ** -8 * O.abs() + (2.0 ** -7 + 2.0 ** -9) * A + 2.0 ** -23 * G
    assert bool(((out - O).abs() <= tol).all())


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("size", [3e4, 1e5])
def test_scores_around_a_large_value(cuda_lib, sign, size):
    """Normal scores moved by a large common value through one channel."""
    for rows, limit in (WHOLE, RANGES):
        b = P.Batch(rows, 64, seed=37)
        q, cache, _ = make(b, P.BF16, 16, 576, 11)
        cache[:, 570] = 384.0
        q[:, :, 570] = sign * size * 24 / 384
        compare(cuda_lib, b, P.BF16, q, cache, None, 1 / 24, max_seq_len=limit)


def test_equal_scores_of_every_size(cuda_lib):
    """All scores of a row equal: O is the mean of V and LSE = S + ln n, for S over
    bf16's steps between 2^13 and 2^17 (log2 units)."""
    n, h = 129, 128
    b = P.Batch([(1, n)] * 40, 64, seed=38)
    q, cache, _ = make(b, P.BF16, h, 576, 12)
    q.zero_()
    cache[:, 575] = 256.0
    exact = torch.linspace(2.0 ** 13, 2.0 ** 17, b.N * h).view(b.N, h) * math.log(2) * 24 / 256
    q[:, :, 575] = exact.bfloat16()
    out, lse = launch(cuda_lib, b, P.BF16, q, cache, None, 1 / 24, 0, 0)
    S = q[:, :, 575].double() * 256 / 24
    assert bool(((lse.double().cpu() - S - math.log(n)).abs() <= 2.0 ** -21 * S).all())
    V = cache.double()
    for t in range(b.N):
        rows = V[[b.slot(t, e) for e in range(n)], :512]
        tol = 2.0 ** -8 * rows.mean(0).abs() + (2.0 ** -7 + 2.0 ** -9) * rows.abs().mean(0)
        assert bool(((out[t].double().cpu() - rows.mean(0)).abs() <= tol).all())


@pytest.mark.parametrize("fmt", [P.E4M3, P.BLOCK])
@pytest.mark.parametrize("nats", [2.0, 11.0, 13.0, 14.5, 16.0, 17.5])
@pytest.mark.parametrize("first", [True, False])
def test_many_small_weights_behind_a_large_one(cuda_lib, fmt, nats, first):
    """E4M3 rows: 16,384 keys of equal score `nats` below that of one key, whose value is
    zero.  Their weights are 2^-b, b = nats / ln 2, of the row's reference, held to 9
    bits (2^-9 of each) on a grid of 2^-27 (half of it: 2^(b - 28) of each); the large
    one's is exact; 2^-8 for O's rounding, 2^-12 for exponentials and sums."""
    n = 16385
    b = P.Batch([(1, n), (1, 40)], 64, seed=39)
    q, cache, scale = make(b, fmt, 16, 576, 13)
    scale = torch.full_like(scale, 2.0 ** -6)
    cache &= 0x7F                                      # (values of one sign)
    cache[:, 575] = 0
    large = b.slot(0, 0 if first else n - 1)
    cache[large, :512] = 0
    cache[large, 575] = 0x7E                           # 448 * 2^-6 = 7
    q.zero_()
    q[:, :, 575] = nats * 24 / 7
    exact = float(q[0, 0, 575]) * 7 / 24               # (q's rounding)
    out, lse = launch(cuda_lib, b, fmt, q, cache, scale, 1 / 24, 0, 0, max_seq_len=1)
    rows = P.dequant(cache, fmt, scale, b)
    total = sum(rows[b.slot(0, e), :512] for e in range(n))
    want = total / (n - 1 + math.exp(exact))
    rel = 2.0 ** -8 + 2.0 ** -9 + 2.0 ** (exact / math.log(2) - 28) + 2.0 ** -12
    assert bool(((out[0].double().cpu() - want).abs() <= rel * want).all())
    assert abs(float(lse[0, 0]) - math.log(n - 1 + math.exp(exact))) <= 2.0 ** -16
