"""smla_fwd_scored where its mathematics is the windowed call's, right behind the kernels
that write what it reads, and with an output of more than 2^32 elements."""
import pytest
import torch

from tests import _paged as P
from tests import _scored as R
from tests.test_scored_gpu import FMTS, call, slopes_of
from tests.test_window_gpu import launch, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("h,rows", [
    (16, [(1, 1), (3, 150), (0, 40), (70, 70), (1, 257), (33, 400), (2, 2)]),   # ranges
    (128, [(1, 900), (1, 5), (2, 1100)]),
    (64, [(180, 300), (150, 150), (40, 700)])])                                # whole tiles
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_the_same_mathematics_as_the_windowed_call(cuda_lib, fmt, h, rows, window, sinks):
    """Slopes of 0, and spans from 0 to the token itself, take the scored form; the keys,
    scores and weights are the windowed form's.  Each may be off by what a result may be
    off by, so they by twice that from one another."""
    smla = cuda_lib
    b = P.Batch(rows, 64, seed=h, pad=3, holes=2)
    q, cache, scale = make(b, fmt, h, 576, 3, 4.0)
    sm = 576 ** -0.5
    n = int(b.start[-1])
    pos = torch.zeros(b.N, dtype=torch.int32)
    for i, _, p in b.tokens():
        pos[i] = p
    zero = torch.zeros(b.N, dtype=torch.int32)
    want = launch(smla, b, fmt, q, cache, scale, sm, window, sinks)
    held = P.dequant(cache, fmt, scale, b)
    b.fp8 = fmt != P.BF16
    O, L, A, S, E, G = (x[:n] for x in R.attend(q, held, b, sm, window, sinks))
    # tests._scored.check's bounds
    fin = ~torch.isneginf(L)
    most_l = 2 * S + 2.0 ** -19 * L.abs() + 2.0 ** -20
    most_o = 2.0 ** -8 * O.abs() + (2.0 ** -7 + 2.0 ** -16) * A + 2 * E + \
        (2.0 ** -23 * G if b.fp8 else 0)
    for kw in (dict(slopes=torch.zeros(h)), dict(first=zero), dict(last=pos),
               dict(slopes=torch.zeros(h), first=zero, last=pos)):
        out, lse = call(smla, b, fmt, q, cache, scale, sm, window=window, sinks=sinks, **kw)
        lse, other = lse.double().cpu()[:n], want[1].double().cpu()[:n]
        assert torch.equal(torch.isneginf(lse), ~fin) and torch.equal(torch.isneginf(other), ~fin)
        assert bool(((lse - other).abs() <= 2 * most_l)[fin].all())
        d = (out.double() - want[0].double()).abs().cpu()[:n]
        assert bool((d <= 2 * most_o).all()), float((d - 2 * most_o).max())


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
@pytest.mark.parametrize("limit", [None, 1])               # in ranges, every tile in one piece
def test_slopes_and_spans_written_just_before(cuda_lib, fmt, limit):
    smla = cuda_lib
    b = P.Batch([(1, 3000), (5, 700), (60, 64)], 64, seed=13)
    h = 16
    q, cache, scale = make(b, fmt, h, 576, 4)
    start, lens, tab = b.dev()
    q, cache = q.cuda(), cache.cuda()
    scale = None if scale is None else scale.cuda()
    sets = []
    for i in range(3):
        first, last = R.spans(b, docs=[40 + 90 * i, 600], prefix=30 * i)
        sets.append([x.cuda() for x in (slopes_of(h, -4.0 - i), first, last)])

    def attend(s):
        out, lse = smla.smla_fwd_scored(q, cache, fmt, scale, start, lens, tab, 64, 0.04,
                                        softcap=20.0, slopes=s[0], first_pos=s[1], last_pos=s[2],
                                        max_seq_len=limit)
        return out, lse

    want = []
    for s in sets:
        want.append(attend(s))
        torch.cuda.synchronize()
    live, got = [x.clone() for x in sets[0]], []
    for k in range(30):
        for x, new in zip(live, sets[k % 3]):
            torch.add(new, 0, out=x)                       # (a kernel, not a copy)
        got.append(attend(live))
    torch.cuda.synchronize()
    for k, (out, lse) in enumerate(got):
        assert torch.equal(out, want[k % 3][0]) and torch.equal(lse, want[k % 3][1]), k


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
@pytest.mark.parametrize("limit", [None, 1])
def test_forks_and_copies_just_before(cuda_lib, fmt, limit):
    """Tables, lengths, rows and block scales by the block operators, whose kernels let the
    next one in early; with no wait, and again with one behind every call."""
    smla = cuda_lib
    b = P.Batch([(1, 2000), (1, 700), (1, 70), (1, 1)], 16, seed=17, spare=40)
    h = 16
    q, cache0, scale0 = make(b, fmt, h, 576, 4)
    start, lens0, tab0 = b.dev()
    q, slopes = q.cuda(), slopes_of(h).cuda()
    ref0 = torch.zeros(b.pool, dtype=torch.int32)
    for x in b.table[b.table >= 0]:
        ref0[x] += 1
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    children = i32([0, 1, 2, 3])
    parents = [i32(p) for p in ([1, 0, 3, 2], [2, 2, 0, 1], [3, 1, 2, 0], [0, 0, 3, 1])]
    room = i32([3, 3, 3, 3])
    moves = [(i32([int(b.table[0, c]), int(b.table[1, c])]), i32([int(b.table[0, c + 9]),
                                                                 int(b.table[1, c + 9])]))
             for c in range(6)]
    res = []
    for wait in (True, False):
        cache, tab, lens, ref = cache0.cuda(), tab0.clone(), lens0.clone(), ref0.cuda()
        scale = None if scale0 is None else scale0.cuda()
        got = []
        for k in range(24):
            for op in range(2):
                if op == 0:
                    smla.smla_cache_fork(parents[k % 4], children, room, lens, tab, ref, 16, cache,
                                         fmt, scale)
                else:
                    smla.smla_cache_copy(cache, fmt, scale, *moves[k % 6], 16)
                if wait:
                    torch.cuda.synchronize()
                got.append(smla.smla_fwd_scored(q, cache, fmt, scale, start, lens, tab, 16, 0.04,
                                                softcap=15.0, slopes=slopes, max_seq_len=limit))
                if wait:
                    torch.cuda.synchronize()
        torch.cuda.synchronize()
        res.append(got)
    for (o0, l0), (o1, l1) in zip(*res):
        assert torch.equal(o0, o1) and torch.equal(l0, l1)


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
    pos = torch.cat([torch.arange(53, n + 50), torch.arange(17, 20)])
    first = (pos // 45 * 45).int()                         # documents of 45 tokens
    slopes = slopes_of(h)
    out, lse = smla.smla_fwd_scored(q, cache.cuda(), fmt, None if scale is None else scale.cuda(),
                                    start, lens, tab, 64, d ** -0.5, softcap=10.0,
                                    slopes=slopes.cuda(), first_pos=first.cuda())
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    held = P.dequant(cache, fmt, scale, b)
    some = torch.tensor([0, 1, 2, 3, n // 2, n // 2 + 1, 65535, 65536, n - 4, n - 3, n - 1])
    tokens = {int(i) for i in some}

    class Some:
        rows, fp8, row_scale, block, table = b.rows, fmt != P.BF16, b.row_scale, b.block, b.table
        start = torch.tensor([0, len(some)])

        def slot(self, r, e):
            return b.slot(r, e)

        def tokens(self):
            return [(k, r, p) for k, (i, r, p) in enumerate(
                t for t in b.tokens() if t[0] in tokens)]

    sub = Some()
    ref = R.attend(q[some.cuda()].cpu(), held, sub, d ** -0.5, cap=10.0, slopes=slopes,
                   first=first[some])
    R.check(out[some.cuda()], lse[some.cuda()], ref, sub, fmt)
    del out, q
    torch.cuda.empty_cache()
