"""What the binding of the append and the windowed attention refuses beside types and
devices: caches whose rows are another format's, arguments without their partner."""
import pytest
import torch

from tests import _paged as P
from tests.test_append_gpu import make as make_append
from tests.test_append_gpu import on_gpu, table
from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu


def test_append(cuda_lib):
    smla = cuda_lib
    b = P.Batch([(2, 70), (3, 20)], 64, seed=15)
    kv_c, k_pe, q_pe, cache, scale = make_append(b, P.BLOCK, 576, 4, 5)
    start, lens, tab = b.dev()
    gq = on_gpu(q_pe)
    good = dict(kv_c=on_gpu(kv_c), k_pe=on_gpu(k_pe), cos_sin=table(80).cuda(), query_start=start,
                seq_lens=lens, block_table=tab, block_size=64, kv_cache=cache.cuda(),
                kv_dtype=P.BLOCK, k_scale=scale.cuda(), q_pe=gq, q_out=torch.zeros_like(gq))
    smla.smla_cache_append(**good)
    flat = good["kv_cache"].view(-1)
    smla.smla_cache_append(**{**good, "kv_cache": flat})
    smla.smla_cache_append(**{**good, "kv_cache": good["kv_cache"].view(-1, 64, 576)})
    short = flat[:-(flat.numel() % 512) or None].view(-1, 512)
    bf16 = torch.zeros((b.num_slots, 576), dtype=torch.bfloat16, device="cuda")
    for bad in (dict(kv_cache=short), dict(kv_cache=bf16, kv_dtype=P.BF16, k_pe=None),
                dict(kv_dtype=P.DS_MLA), dict(k_pe=None, q_pe=None, q_out=None, kv_cache=short),
                dict(k_pe=None, cos_sin=None, q_out=None, kv_cache=short), dict(q_pe=None)):
        with pytest.raises(ValueError):
            smla.smla_cache_append(**{**good, **bad})
    over = torch.zeros((b.N, 1, 64), dtype=torch.bfloat16, device="cuda").expand(-1, 4, -1)
    with pytest.raises(smla.SmlaError):
        smla.smla_cache_append(**{**good, "q_out": over})
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0


def test_window(cuda_lib):
    smla = cuda_lib
    b = P.Batch([(1, 700), (2, 90)], 64, seed=14)
    q, cache, scale = make(b, P.BLOCK, 16, 576, 4)
    start, lens, tab = b.dev()
    good = dict(q=q.cuda(), kv_cache=cache.cuda(), kv_dtype=P.BLOCK, k_scale=scale.cuda(),
                query_start=start, seq_lens=lens, block_table=tab, block_size=64, sm_scale=0.04)
    want = smla.smla_fwd_window(**good)
    for shape in ((-1,), (-1, 64, 576)):
        got = smla.smla_fwd_window(**{**good, "kv_cache": good["kv_cache"].view(shape)})
        assert torch.equal(got[0], want[0])
    flat = good["kv_cache"].view(-1)
    short = flat[:-(flat.numel() % 512) or None].view(-1, 512)
    for bad in (dict(kv_cache=short), dict(q=good["q"][:, :, :512].contiguous()),
                dict(q=good["q"][:, :, :0].contiguous())):
        with pytest.raises(ValueError):
            smla.smla_fwd_window(**{**good, **bad})
    assert smla.smla_get_device_status(clear=True) == 0
