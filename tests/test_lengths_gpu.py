"""The append and the windowed attention at the ends of what a length can be."""
import pytest
import torch

from tests import _paged as P
from tests.test_append_gpu import table
from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu

LOW, HIGH = -2 ** 31, 2 ** 31 - 1


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.GROUP128, P.DS_MLA, P.GROUP4_KPE, P.BLOCK])
@pytest.mark.parametrize("length", [LOW, LOW + 2, -1])
def test_append_of_a_negative_length(cuda_lib, fmt, length):
    """Its tokens are at negative positions: skipped, and no error."""
    smla = cuda_lib
    torch.manual_seed(1)
    smla.smla_get_device_status(clear=True)
    S, row = 128, P.DS_MLA_ROW if fmt == P.DS_MLA else 576
    cache = torch.full((S, row), 3, device="cuda",
                       dtype=torch.bfloat16 if fmt == P.BF16 else torch.uint8)
    scale = torch.full((S, 5), 0.5, device="cuda")
    if fmt == P.GROUP4_KPE:
        scale = scale[:, :4].contiguous()
    start = torch.tensor([0, 3, 5], dtype=torch.int32, device="cuda")
    lens = torch.tensor([length, 2], dtype=torch.int32, device="cuda")
    tab = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    x = torch.randn((5, 576), device="cuda").bfloat16()
    q = torch.randn((5, 2, 64), device="cuda").bfloat16()
    out = torch.full_like(q, 9.0)
    was, was_scale = cache.clone(), scale.clone()
    smla.smla_cache_append(x[:, :512], x[:, 512:], table(4).cuda(), start, lens, tab, 64, cache,
                           fmt, None if fmt in (P.BF16, P.DS_MLA) else scale, q_pe=q, q_out=out)
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    assert bool((out[:3] == 9.0).all()) and not bool((out[3:] == 9.0).all())
    rows = (cache != was).any(1).nonzero().flatten().tolist()
    assert rows == [64, 65]                            # the other request's
    if fmt == P.BLOCK:
        assert torch.equal(scale.flatten()[0], was_scale.flatten()[0])


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
@pytest.mark.parametrize("length", [LOW, LOW + 2, -1])
@pytest.mark.parametrize("limit", [None, 1])
def test_attention_of_a_negative_length(cuda_lib, fmt, length, limit):
    smla = cuda_lib
    torch.manual_seed(1)
    smla.smla_get_device_status(clear=True)
    b = P.Batch([(3, 500), (2, 700), (1, 300)], 64, seed=51)
    q, cache, scale = make(b, fmt, 16, 576, 4)
    ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, 0.04, 0, 0)
    b.lens[0] = length
    start, lens, tab = b.dev()
    out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), fmt,
                                    None if scale is None else scale.cuda(), start, lens, tab, 64,
                                    0.04, max_seq_len=limit)
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    assert bool((out[:3] == 0).all()) and bool(torch.isneginf(lse[:3]).all())
    rest = tuple(x[3:] for x in ref)
    alone = P.Batch([(1, 1)] * 3, 64)
    P.check_attention(out[3:], lse[3:], rest, q[3:], fmt, 0.04, alone)


@pytest.mark.parametrize("columns", [2 ** 25, 2 ** 25 + 2])
def test_append_at_the_last_position(cuda_lib, columns):
    """The last positions that an int holds, in a table that reaches them (its entries
    are all block 0 but the last two of the positions')."""
    smla = cuda_lib
    torch.manual_seed(1)
    smla.smla_get_device_status(clear=True)
    block, n = 64, 70
    tab = torch.zeros((1, columns), dtype=torch.int32, device="cuda")
    tab[0, 2 ** 25 - 2:2 ** 25] = torch.tensor([2, 1], dtype=torch.int32)
    x = torch.randn((n, 512), device="cuda").bfloat16()
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([HIGH], dtype=torch.int32, device="cuda")
    # positions 2^31 - 71 .. 2^31 - 2: the last 7 rows of block 2, the first 63 of block 1
    want = torch.zeros((4 * block, 512), dtype=torch.bfloat16, device="cuda")
    want[3 * block - 7:3 * block] = x[:7]
    want[block:block + 63] = x[7:]
    cache = torch.zeros_like(want)
    smla.smla_cache_append(x, None, None, start, lens, tab, block, cache, P.BF16)
    assert torch.equal(cache, want)
    codes = torch.zeros((4 * block, 512), dtype=torch.uint8, device="cuda")
    scale = torch.full((4,), 2.0 ** -64, device="cuda")
    smla.smla_cache_append(x, None, None, start, lens, tab, block, codes, P.BLOCK, scale)
    got = codes.view(torch.float8_e4m3fn).float().view(4, block, 512) * scale[:, None, None]
    err = (got.view(-1, 512) - want.float()).abs()
    assert bool((err <= 2.0 ** -4 * want.float().abs() + 2.0 ** -9 * scale.max()).all())
    assert smla.smla_get_device_status(clear=True) == 0
