"""The append and the windowed attention in captured graphs, behind copies and fills and
on forked streams, on outputs of more than 2^32 elements, and under other bounds and
softmax scales than the usual ones."""
import pytest
import torch

from tests import _paged as P
from tests.test_append_gpu import table
from tests.test_window_gpu import make, shared_out

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_a_step_with_copies_and_two_streams(cuda_lib, fmt):
    """One graph: new lengths by a copy, outputs cleared by a fill, an append, the
    attention in ranges and in whole tiles on two streams, a second append behind both;
    replayed on changing inputs, against eager calls with a wait behind each."""
    smla = cuda_lib
    h, d, block, steps = 16, 576, 64, 12
    first = [70, 700, 2500]
    full = P.Batch([(1, L + steps + 1) for L in first], block, seed=95)
    start, _, tab = full.dev()
    cs = table(max(first) + steps + 2).cuda()
    g = torch.Generator().manual_seed(6)
    xs = torch.randn((steps, 3, d), generator=g).bfloat16().cuda()
    qs = torch.randn((steps, 3, h, d), generator=g).bfloat16().cuda()
    _, cache0, scale0 = make(full, fmt, h, d, 5)
    assert smla.smla_fwd_window_workspace_size(3, 3, h, d, fmt, tab.shape[1], block) > 0
    x, q = torch.zeros_like(xs[0]), torch.zeros_like(qs[0])
    at = torch.zeros(3, dtype=torch.int32, device="cuda")
    lens = torch.zeros_like(at)
    one = torch.empty((3, h, 512), dtype=torch.bfloat16, device="cuda")
    two, l1, l2 = torch.empty_like(one), *torch.empty((2, 3, h), device="cuda")
    side = torch.cuda.Stream()

    def step(cache, scale, wait):
        def done():
            if wait:
                torch.cuda.synchronize()
        lens.copy_(at)
        one.zero_(), two.zero_()
        done()
        smla.smla_cache_append(x[:, :512], x[:, 512:], cs, start, lens, tab, block, cache, fmt,
                               scale, q_pe=q[:, :, 512:])
        done()
        side.wait_stream(torch.cuda.current_stream())
        smla.smla_fwd_window(q, cache, fmt, scale, start, lens, tab, block, d ** -0.5, out=one,
                             lse=l1)
        done()
        with torch.cuda.stream(side):
            smla.smla_fwd_window(q, cache, fmt, scale, start, lens, tab, block, d ** -0.5, 300, 5,
                                 max_seq_len=1, out=two, lse=l2)
        done()
        torch.cuda.current_stream().wait_stream(side)
        lens.add_(1)
        smla.smla_cache_append(x[:, :512], x[:, 512:], cs, start, lens, tab, block, cache, fmt,
                               scale)
        done()

    def feed(k):
        x.copy_(xs[k]), q.copy_(qs[k])
        at.copy_(torch.tensor([L + k + 1 for L in first], dtype=torch.int32))

    results = []
    for captured in (False, True):
        cache = cache0.cuda()
        scale = None if scale0 is None else scale0.cuda()
        if captured:
            feed(0)
            spare = cache.clone(), None if scale is None else scale.clone()
            step(*spare, wait=True)                    # (first uses outside the capture)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step(cache, scale, wait=False)
        got = []
        for k in range(steps):
            feed(k)
            if captured:
                graph.replay()
            else:
                step(cache, scale, wait=True)
            got += [one.clone(), two.clone(), l1.clone(), l2.clone()]
        torch.cuda.synchronize()
        results.append(got + [cache] + ([] if scale is None else [scale]))
    for a, b in zip(*results):
        assert torch.equal(a, b)
    assert smla.smla_get_device_status(clear=True) == 0


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_outputs_past_32_bits(cuda_lib, fmt):
    """9 million rows of the output, 4.6e9 elements; tokens from all over it checked."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    h, d, n = 128, 576, 70000
    b = P.Batch([(n - 3, n + 50), (3, 20)], 64, seed=96)
    _, cache, scale = make(b, fmt, 1, d, 7)
    g = torch.Generator("cuda").manual_seed(1)
    q = torch.empty((n, h, d), dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    start, lens, tab = b.dev()
    out, lse = smla.smla_fwd_window(q, cache.cuda(), fmt, None if scale is None else scale.cuda(),
                                    start, lens, tab, 64, d ** -0.5, window=40, sinks=2)
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    rows = P.dequant(cache, fmt, scale, b)
    for i in (0, 1, n // 2, 65535, 65536, n - 4, n - 3, n - 1):
        r, pos = (0, 53 + i) if i < n - 3 else (1, 17 + i - (n - 3))
        e = [e for e in range(pos + 1) if e > pos - 40 or e < 2]
        k = rows[[b.slot(r, x) for x in e]]
        w = torch.softmax(q[i].double().cpu() @ k.T * d ** -0.5, -1)
        O, A = w @ k[:, :512], w @ k[:, :512].abs()
        tol = 2.0 ** -8 * O.abs() + (2.0 ** -7 + 2.0 ** -9) * A
        assert bool(((out[i].double().cpu() - O).abs() <= tol).all()), i


def test_queries_past_32_bits(cuda_lib):
    """The append's rotation of queries whose elements lie behind 2^32."""
    smla = cuda_lib
    h, n = 128, 180000
    b = P.Batch([(n, n)], 64, seed=97)
    q = torch.zeros((n, h, 192), dtype=torch.bfloat16, device="cuda")
    g = torch.Generator("cuda").manual_seed(2)
    q[-5:].normal_(generator=g)
    was = q[-5:, :, 128:].cpu()
    kv = torch.zeros((n, 576), dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros((b.num_slots, 576), dtype=torch.bfloat16, device="cuda")
    start, lens, tab = b.dev()
    cs = table(n)
    smla.smla_cache_append(kv[:, :512], kv[:, 512:], cs.cuda(), start, lens, tab, 64, cache,
                           P.BF16, q_pe=q[:, :, 128:])
    want = P.rotate(was.float(), cs[-5:, None], True).bfloat16()
    assert torch.equal(q[-5:, :, 128:].cpu(), want)
    assert not bool(q[:-5].any())


def test_ranges_by_another_bound_are_the_same_answer(cuda_lib):
    """Bounds on the lengths that are too small, right and too large."""
    b = P.Batch([(1, 2600), (3, 900), (1, 10)], 64, seed=98)
    q, cache, scale = make(b, P.BLOCK, 16, 576, 4)
    ref = P.attend(q, P.dequant(cache, P.BLOCK, scale, b), b, 0.04, 0, 0)
    assert shared_out(cuda_lib, b, 16)
    for limit in (1, 300, 2600, 1 << 20, 2 ** 31 - 1):
        out, lse = cuda_lib.smla_fwd_window(q.cuda(), cache.cuda(), P.BLOCK, scale.cuda(),
                                            *b.dev(), 64, 0.04, max_seq_len=limit)
        P.check_attention(out, lse, ref, q, P.BLOCK, 0.04, b)


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
@pytest.mark.parametrize("sm", [0.0, -0.05])
def test_softmax_scales_of_zero_and_below(cuda_lib, fmt, sm):
    for limit in (None, 1):
        b = P.Batch([(1, 2600), (30, 200)], 64, seed=99)
        q, cache, scale = make(b, fmt, 16, 576, 4)
        out, lse = cuda_lib.smla_fwd_window(q.cuda(), cache.cuda(), fmt,
                                            None if scale is None else scale.cuda(), *b.dev(), 64,
                                            sm, window=900, sinks=3, max_seq_len=limit)
        ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, sm, 900, 3)
        P.check_attention(out, lse, ref, q, fmt, sm, b)


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
@pytest.mark.parametrize("h", [3, 128])
def test_thousands_of_requests(cuda_lib, fmt, h):
    """A wide decode batch, a third of its requests without a token."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    rows = [((1, 1 + 7 * r % 90), (0, 30), (2, 5 + r % 60))[r % 3] for r in range(4000 if h < 9
                                                                                  else 1500)]
    b = P.Batch(rows, 16, seed=100, pad=7)
    q, cache, scale = make(b, fmt, h, 576, 4)
    out, lse = smla.smla_fwd_window(q.cuda(), cache.cuda(), fmt,
                                    None if scale is None else scale.cuda(), *b.dev(), 16, 0.04,
                                    window=50, sinks=2)
    torch.cuda.synchronize()
    ref = P.attend(q, P.dequant(cache, fmt, scale, b), b, 0.04, 50, 2)
    P.check_attention(out, lse, ref, q, fmt, 0.04, b)
    assert smla.smla_get_device_status(clear=True) == 0
