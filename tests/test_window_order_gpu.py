"""smla_fwd_window right behind the kernels that write what it reads, without a wait of
the host: descriptors, scales, queries and cache rows all change from call to call."""
import pytest
import torch

from tests import _paged as P
from tests.test_append_gpu import table
from tests.test_window_gpu import make, shared_out

pytestmark = pytest.mark.gpu

ROWS = [[(1, 3000), (2, 700), (1, 65)], [(2, 650), (0, 40), (2, 2900)], [(1, 1), (1, 64), (2, 3000)]]


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
def test_descriptors_written_just_before(cuda_lib, fmt):
    smla = cuda_lib
    h, block, sm = 16, 64, 576 ** -0.5
    batches = [P.Batch(r, block, seed=60 + i) for i, r in enumerate(ROWS)]
    width = max(b.table.shape[1] for b in batches)
    slots = max(b.num_slots for b in batches)
    N = max(b.N for b in batches)
    held = []
    for i, b in enumerate(batches):
        b.table = torch.cat([b.table, torch.full((3, width - b.table.shape[1]), -1,
                                                 dtype=torch.int32)], 1)
        b.num_slots, b.N = slots, N
        q, cache, scale = make(b, fmt, h, 576, 70 + i)
        held.append([x.cuda() for x in (q, cache, b.start, b.lens, b.table)] +
                    [None if scale is None else scale.cuda()])
    assert shared_out(smla, batches[0], h)
    for limit in (None, 1):                            # in ranges, and every tile in one piece
        want = []
        for q, cache, start, lens, tab, scale in held:
            out = [torch.zeros((N, h, 512), dtype=torch.bfloat16, device="cuda"),
                   torch.zeros((N, h), device="cuda")]
            smla.smla_fwd_window(q, cache, fmt, scale, start, lens, tab, block, sm,
                                 max_seq_len=limit, out=out[0], lse=out[1])
            torch.cuda.synchronize()
            want.append(out)
        live = [None if x is None else x.clone() for x in held[0]]
        got = []
        for k in range(30):
            for x, new in zip(live, held[k % 3]):
                if x is not None:
                    x.copy_(new)
            q, cache, start, lens, tab, scale = live
            out = [torch.zeros_like(want[0][0]), torch.zeros_like(want[0][1])]
            for x, new in ((lens, 2), (start, 1)) if k % 2 else ():
                x.copy_(held[k % 3][new + 1])          # (written last, right before the call)
            smla.smla_fwd_window(q, cache, fmt, scale, start, lens, tab, block, sm,
                                 max_seq_len=limit, out=out[0], lse=out[1])
            got.append(out)
        torch.cuda.synchronize()
        for k, (o, l) in enumerate(got):
            assert torch.equal(o, want[k % 3][0]) and torch.equal(l, want[k % 3][1]), (limit, k)


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
def test_append_just_before(cuda_lib, fmt):
    """Sixty decode steps, append and attention in turn with no wait, and again with
    one behind every call."""
    smla = cuda_lib
    h, block, steps, d = 16, 16, 60, 576
    first = [1, 40, 2000]
    full = P.Batch([(1, L + steps) for L in first], block, seed=80)
    cs = table(max(first) + steps).cuda()
    g = torch.Generator().manual_seed(4)
    x = torch.randn((steps, 3, d), generator=g).bfloat16().cuda()
    q = torch.randn((steps, 3, h, d), generator=g).bfloat16().cuda()
    start, _, tab = full.dev()
    _, before, scale0 = make(full, fmt, h, d, 5)
    res = []
    for wait in (True, False):
        cache = before.cuda()
        scale = None if scale0 is None else scale0.cuda()
        lens = torch.tensor(first, dtype=torch.int32, device="cuda")
        qs, got = q.clone(), []
        for k in range(steps):
            smla.smla_cache_append(x[k, :, :512], x[k, :, 512:], cs, start, lens, tab, block,
                                   cache, fmt, scale, q_pe=qs[k, :, :, 512:])
            if wait:
                torch.cuda.synchronize()
            got.append(smla.smla_fwd_window(qs[k], cache, fmt, scale, start, lens, tab, block,
                                            d ** -0.5, window=1500, sinks=4))
            if wait:
                torch.cuda.synchronize()
            lens += 1
        torch.cuda.synchronize()
        res.append(got)
    for a, b in zip(*res):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
