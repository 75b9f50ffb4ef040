"""The distance bias key by key: every token sees one position, at a chosen distance, and
its score is 0, so LSE is the bias.

A bias is within 2^-22 of itself (include/smla.h), four half steps of fp32, and with a cap
the score within 2^-20 of the cap.  LSE adds ln 2 and its product, less than two half
steps.  A block's scale goes into the maximum by its logarithm, of at most 8 here, and comes
out again: two half steps more, all of them of the bias and that logarithm (8 ln 2 nats)
together; and log2f(ex2.approx(x)) stands for x there, off by 2^-22 of a weight and, as an
ulp of a logarithm of 4 to 8, by 2^-21 ln 2: 2^-20 at most.
"""
import math

import pytest
import torch

from tests import _paged as P
from tests.test_scored_gpu import call
from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu


def slopes(h):
    g = torch.Generator().manual_seed(h)
    return torch.exp2(torch.rand(h, generator=g) * 24 - 10).float()


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
@pytest.mark.parametrize("block", [16, 64])
@pytest.mark.parametrize("cap", [0.0, 1.0, 256.0, 1000.0])
def test_one_key_at_a_distance(cuda_lib, fmt, block, cap):
    b = P.Batch([(70, 300), (1, 200), (131, 131), (3, 90)], block, seed=3, pad=2)
    h = 16
    q, cache, scale = make(b, fmt, h, 576, 5, 1.0, True)
    q[:] = 0
    slope = slopes(h)
    pos = torch.full((b.N,), -1, dtype=torch.int32)
    length = torch.zeros(b.N, dtype=torch.int32)
    for n, r, p in b.tokens():
        pos[n], length[n] = p, b.rows[r][1]
    for far in (0, 1, 2, 3, 7, 8, 9, 30, 31, 32, 33, 63, 64, 65, 100, 129, -1, -2, -5, -31, -32,
                -60):
        at = pos - far
        out, lse = call(cuda_lib, b, fmt, q, cache, scale, 0.04, cap, slope, at, at)
        n = int(b.start[-1])
        seen = ((at >= 0) & (at < length))[:n]
        lse = lse.double().cpu()[:n]
        assert bool(torch.isneginf(lse[~seen]).all())
        bias = -slope.double() * abs(far)
        off, most = (lse[seen] - bias).abs(), 2.0 ** -20 * min(cap, 256.0)
        if fmt == P.BLOCK:
            off -= 8 * 2.0 ** -24 * (bias.abs() + 8 * math.log(2.0))
            most += 2.0 ** -20
        else:
            off -= 6 * 2.0 ** -24 * bias.abs()
        assert bool((off <= most).all()), (far, float(off.max()))


@pytest.mark.parametrize("fmt", [P.BF16, P.E4M3, P.BLOCK])
def test_the_token_itself(cuda_lib, fmt):
    """No distance, no bias, however steep the slope: LSE is the score, 0."""
    b = P.Batch([(300, 300), (7, 131)], 64, seed=4)
    q, cache, scale = make(b, fmt, 32, 576, 5, 1.0, True)
    q[:] = 0
    _, lse = call(cuda_lib, b, fmt, q, cache, scale, 0.04, slopes=slopes(32) * 1e3, window=1)
    assert not bool(lse.any())
