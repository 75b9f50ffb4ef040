"""Few tiles whose keys are shared by most of the GPU: the merge of many parts a row, with
few rows and with more than its narrow form takes, plain and scored."""
import pytest

from tests import _paged as P
from tests.test_scored_gpu import run, slopes_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [P.BF16, P.BLOCK])
@pytest.mark.parametrize("rows,h", [([(1, 5000)], 1), ([(1, 5000)], 64), ([(1, 5000)], 65),
                                    ([(1, 5000)], 96), ([(1, 5000)], 128),
                                    ([(1, 5000), (1, 3333)], 128),
                                    ([(1, 2600), (1, 2500), (1, 2700)], 64),
                                    ([(1, 2600), (1, 2500), (1, 2700), (1, 40)], 128)])
def test_many_parts(cuda_lib, fmt, rows, h):
    smla = cuda_lib
    b = P.Batch(rows, 64, seed=h, pad=2, holes=3)
    assert smla.smla_fwd_window_workspace_size(len(rows), b.N, h, 576, fmt, b.table.shape[1],
                                               64) > 0
    run(smla, b, fmt, h)
    run(smla, b, fmt, h, slopes=slopes_of(h), window=2000, sinks=70)
