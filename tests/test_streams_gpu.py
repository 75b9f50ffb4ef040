"""Outputs that the binding allocates for a call on another stream than the current
one: their memory may have held a tensor that work still queued on the current stream
reads, and they may be let go before that stream has read them."""
import pytest
import torch

from sparse_mla_attention_02_gb300 import workloads as W
from tests import _paged as P
from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu


def calls(smla):
    b = P.Batch([(1, 300), (40, 90)], 64, seed=41)
    q, cache, _ = make(b, P.BF16, 16, 576, 4)
    window = (q.cuda(), cache.cuda(), P.BF16, None, *b.dev(), 64, 0.04)
    w = W.custom(name="streams", T=41, h=16, topk=256, num_slots=700, kv_dtype=0,
                 valid=[256] * 41, seed=5).to("cuda")
    fwd = (w.q, w.kv, w.kv_dtype, w.k_scale, w.indices, w.valid_len, w.sm_scale)
    parts = torch.randn((3, 41 * 16, 512), device="cuda")
    lses = torch.randn((3, 41 * 16), device="cuda")
    table = torch.arange(700 // 10, dtype=torch.int32, device="cuda").view(1, -1)
    req = torch.zeros(41, dtype=torch.int32, device="cuda")
    ws = torch.empty(smla.smla_workspace_size(41, 16, 576, 256, 0) + 256, dtype=torch.uint8,
                     device="cuda")
    return {
        "smla_fwd_window": lambda s: smla.smla_fwd_window(*window, stream=s),
        "smla_fwd": lambda s: smla.smla_fwd(*fwd, stream=s),
        "smla_fwd_ws": lambda s: smla.smla_fwd_ws(*fwd, ws, stream=s),
        "smla_fwd_split_q": lambda s: smla.smla_fwd_split_q(fwd[0], None, *fwd[1:], stream=s),
        "smla_fwd_partial": lambda s: smla.smla_fwd_partial(*fwd, stream=s),
        "smla_fwd_paged": lambda s: smla.smla_fwd_paged(
            *fwd[:5], req, table, 10, fwd[6], valid_len=fwd[5], stream=s),
        "smla_combine": lambda s: smla.smla_combine(parts, lses, stream=s),
    }


NAMES = ["smla_fwd_window", "smla_fwd", "smla_fwd_ws", "smla_fwd_split_q", "smla_fwd_partial",
         "smla_fwd_paged", "smla_combine"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_do_not_share_memory_with_queued_reads(cuda_lib, name):
    torch.manual_seed(1)
    call = calls(cuda_lib)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    marks = [torch.full_like(x, 7.0) for x in want]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                     # the reads below wait about 0.1 s
    copies = [m.clone() for m in marks]
    del marks                                          # free for a call on this stream
    got = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    for c in copies:
        assert bool((c == 7.0).all())
    for g, w in zip(got, want):
        assert torch.equal(g, w)


@pytest.mark.parametrize("name", NAMES)
def test_outputs_let_go_before_they_are_read(cuda_lib, name):
    """The current stream reads an output that the program has let go; a later call on
    the other stream must not be given its memory meanwhile."""
    torch.manual_seed(1)
    call = calls(cuda_lib)[name]
    want = [x.clone() for x in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    got = call(side)
    shapes = [(x.shape, x.dtype) for x in got]
    side.synchronize()
    torch.cuda._sleep(200_000_000)
    copies = [g.clone() for g in got]
    del got
    with torch.cuda.stream(side):
        over = [torch.full(s, 7.0, dtype=t, device="cuda") for s, t in shapes]
    torch.cuda.synchronize()
    assert all(bool((o == 7.0).all()) for o in over)
    for c, w in zip(copies, want):
        assert torch.equal(c, w)
