"""Rows that smla_fwd_window computes again, because a position that they do not see
holds an infinity or NaN: long contexts, many such rows, other requests beside them."""
import pytest
import torch

from tests import _paged as P
from tests.test_window_gpu import launch, make

pytestmark = pytest.mark.gpu


def formula(q, rows, batch, sm, window=0, sinks=0, keep=None):
    """fp64 on the GPU: (O, LSE, sum softmax |V|, sum |V| / scale times the largest scale)
    of the tokens in ``keep``."""
    rows = rows.cuda()
    unit = batch.row_scale.cuda()
    res = {}
    for n, r, pos in batch.tokens():
        if keep is not None and n not in keep:
            continue
        e = torch.arange(pos + 1)
        if window:
            e = e[(e > pos - window) | (e < sinks)]
        at = (batch.table[r].long()[e // batch.block] * batch.block + e % batch.block).cuda()
        k = rows[at]
        s = q[n].double().cuda() @ k.T * sm
        w = torch.softmax(s, -1)
        v = k[:, :512]
        res[n] = (w @ v, torch.logsumexp(s, -1), w @ v.abs(),
                  (v.abs() / unit[at][:, None]).sum(0) * unit[at].max())
    return res


def check(out, lse, ref):
    for n, (O, L, A, G) in ref.items():
        tol = 2.0 ** -8 * O.abs() + (2.0 ** -7 + 2.0 ** -9) * A + 2.0 ** -23 * G
        assert bool(torch.isfinite(out[n].float()).all()), n
        assert bool(((out[n].double() - O).abs() <= tol).all()), n
        assert bool(((lse[n].double() - L).abs() <= 2.0 ** -10).all()), n


def poison(cache, fmt, slot, bad):
    cache[slot, 7] = 0x7F if fmt != P.BF16 else bad


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
@pytest.mark.parametrize("h,tokens", [(1, 128), (16, 8), (5, 40)])
@pytest.mark.parametrize("limit", [1, None], ids=["whole", "ranges"])
def test_longer_than_a_wait(cuda_lib, fmt, h, tokens, limit):
    """Waits limited to 2 ms, which the rows computed again take many times over: no
    wait of the others may run out, and the request beside is right."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    b = P.Batch([(tokens, 20000), (1, 900), (2, 70)], 64, seed=90)
    q, cache, scale = make(b, fmt, h, 576, 7)
    rows = P.dequant(cache, fmt, scale, b)
    poison(cache, fmt, b.slot(0, 19999), float("nan"))
    smla.smla_test_set_stall(False, 2000)
    try:
        out, lse = launch(smla, b, fmt, q, cache, scale, 576 ** -0.5, 0, 0, max_seq_len=limit)
        torch.cuda.synchronize()
    finally:
        smla.smla_test_set_stall(False)
    assert smla.smla_get_device_status(clear=True) == 0
    assert bool(torch.isnan(out[tokens - 1].float()).all())
    keep = {0, 1, tokens // 2, tokens - 2, tokens, tokens + 1, tokens + 2}
    check(out, lse, formula(q, rows, b, 576 ** -0.5, keep=keep))
    first = torch.arange(b.N) != tokens - 1
    assert bool(torch.isfinite(out.float().cpu()[first]).all())


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
def test_behind_131072_keys(cuda_lib, fmt):
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    tokens, h, L = 128, 1, 131072 + 128
    b = P.Batch([(tokens, L), (1, 3000)], 64, seed=91)
    q, cache, scale = make(b, fmt, h, 576, 8)
    rows = P.dequant(cache, fmt, scale, b)
    poison(cache, fmt, b.slot(0, L - 1), float("inf"))
    out, lse = launch(smla, b, fmt, q, cache, scale, 576 ** -0.5, 0, 0, max_seq_len=1)
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    check(out, lse, formula(q, rows, b, 576 ** -0.5, keep={0, 64, tokens - 2, tokens}))


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
@pytest.mark.parametrize("block", [16, 7])
def test_windows_over_poisoned_rows(cuda_lib, fmt, block):
    """Poison before the window, between the sinks and it, and in later tokens; several
    units one after the other in one cluster."""
    smla = cuda_lib
    smla.smla_get_device_status(clear=True)
    b = P.Batch([(60, 700)] * 30, block, seed=92)
    q, cache, scale = make(b, fmt, 16, 576, 9)
    rows = P.dequant(cache, fmt, scale, b)
    window, sinks = 90, 5
    for r in range(0, 30, 2):
        for e in (6, 300, 549, 660):                   # (640 is the first token's position)
            poison(cache, fmt, b.slot(r, e), float("inf") if r % 4 else float("nan"))
    out, lse = launch(smla, b, fmt, q, cache, scale, 576 ** -0.5, window, sinks)
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    keep = {60 * r + i for r in (0, 1, 2, 28, 29) for i in (0, 10, 19)}
    check(out, lse, formula(q, rows, b, 576 ** -0.5, window, sinks, keep))
