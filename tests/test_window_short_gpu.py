"""Many requests of a few key blocks: right, and the same bits however their rows are copied
(by boxes, or row by row), which a looser bound on the lengths changes."""
import pytest
import torch

from tests import _paged as P
from tests.test_scored_gpu import run as run_scored
from tests.test_scored_gpu import slopes_of
from tests.test_window_gpu import run as run_window

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("block", [4, 16, 48])
@pytest.mark.parametrize("d", [512, 576])
@pytest.mark.parametrize("new", [1, 3])
def test_short_requests(cuda_lib, block, d, new):
    smla = cuda_lib
    rows = [(min(new, 1 + 7 * r % 300), 1 + 7 * r % 300) for r in range(200)]
    b = P.Batch(rows, block, seed=block, pad=3, holes=9)
    more = 700 // block                                    # (a table that bounds no length here)
    b.table = torch.nn.functional.pad(b.table, (0, more), value=-1)
    n, h = int(b.start[-1]), 24
    kw = dict(cap=9.0, slopes=slopes_of(h))
    want = want_scored = None
    for limit in (300, 384, 385, 600):
        # (units of whole tiles: ranges of tiles round otherwise)
        assert smla.smla_fwd_window_workspace_size(len(rows), b.N, h, d, P.BF16, b.table.shape[1],
                                                   block, max_seq_len=limit) == 0
        got = run_window(smla, b, P.BF16, h, d=d, max_seq_len=limit)
        scored = run_scored(smla, b, P.BF16, h, d=d, max_seq_len=limit, **kw)
        if want is None:
            want, want_scored = got, scored
        for x, y in zip((*got, *scored), (*want, *want_scored)):
            assert torch.equal(x[:n], y[:n])
