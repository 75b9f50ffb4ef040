"""Many tiles of one or two key blocks, some without a row in one CTA of the pair: E4M3
rows' Q is split for the next tile while the softmax still is at the one before, and no
wait runs out over it, call after call."""
import pytest
import torch

from tests import _paged as P
from tests import _scored as R
from tests.test_scored_gpu import call, run, slopes_of
from tests.test_window_gpu import launch, make
from tests.test_window_gpu import run as run_window

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [P.E4M3, P.BLOCK, P.BF16])
@pytest.mark.parametrize("h", [16, 33, 64, 96, 128])
@pytest.mark.parametrize("longest", [40, 130, 250])
def test_call_after_call(cuda_lib, fmt, h, longest):
    smla = cuda_lib
    rows = [((1, 2, 1, 0, 1)[r % 5], 1 + 37 * r % longest) for r in range(220)]
    b = P.Batch(rows, 64, seed=h, pad=2, holes=5)
    n = int(b.start[-1])
    first, last = R.spans(b, docs=[13, 70, 128], prefix=5)
    kw = dict(cap=5.0, slopes=slopes_of(h), first=first, last=last)
    want = run(smla, b, fmt, h, **kw), run_window(smla, b, fmt, h)
    q, cache, scale = make(b, fmt, h, 576, 1, 2.0, True)
    q, cache, scale = q.cuda(), cache.cuda(), None if scale is None else scale.cuda()
    got = []
    for _ in range(15):
        got.append((call(smla, b, fmt, q, cache, scale, 576 ** -0.5, **kw),
                    launch(smla, b, fmt, q, cache, scale, 576 ** -0.5, 0, 0)))
    torch.cuda.synchronize()
    assert smla.smla_get_device_status(clear=True) == 0
    for pair in got:
        for (o, l), (wo, wl) in zip(pair, want):
            assert torch.equal(o[:n], wo[:n]) and torch.equal(l[:n], wl[:n])
