"""smla_fwd_scored at the ends of its arguments: the smallest caps under large scales, the
cap at which the form of tanh changes."""
import math

import pytest
import torch

from tests import _paged as P
from tests.test_scored_gpu import FMTS, RAGGED, call, run, slopes_of
from tests.test_window_gpu import make

pytestmark = pytest.mark.gpu


def means(batch, rows):
    """(LSE, O, sum |V| / n) of tokens that weigh all of their keys alike."""
    L = torch.full((batch.N,), -float("inf"), dtype=torch.float64)
    O, A = (torch.zeros((batch.N, 512), dtype=torch.float64) for _ in range(2))
    for n, r, pos in batch.tokens():
        slot = [s for s in (batch.slot(r, e) for e in range(pos + 1)) if s >= 0]
        if slot:
            v = rows[slot][:, :512]
            L[n], O[n], A[n] = math.log(len(slot)), v.mean(0), v.abs().mean(0)
    return L, O, A


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cap", [1e-30, 1e-20])
@pytest.mark.parametrize("gain,sm", [(0.0, 1e12), (1.0, 1e12), (1e30, 1.0), (1e18, -1e20),
                                     (2.0, 0.04)])
@pytest.mark.parametrize("block", [16, 64])
def test_smallest_caps(cuda_lib, fmt, cap, gain, sm, block):
    """Every score is within the cap, next to nothing, however large the products: a
    mean of V.  Some of the products are 0."""
    b = P.Batch(RAGGED, block, seed=3, pad=2)
    q, cache, scale = make(b, fmt, 16, 576, 7, 1.0, True)
    q = (q.float() * gain).bfloat16()
    q[:, ::3] = 0
    out, lse = call(cuda_lib, b, fmt, q, cache, scale, sm, cap)
    rows = P.dequant(cache, fmt, scale, b)
    L, O, A = means(b, rows)
    n = int(b.start[-1])
    out, lse = out.double().cpu()[:n], lse.double().cpu()[:n]
    L, O, A = L[:n, None], O[:n, None], A[:n, None]
    fin = torch.isfinite(L).expand(lse.shape)
    assert torch.equal(torch.isneginf(lse), ~fin)
    # as tests._scored.check, where the scores are off by nothing
    off = (lse - L).abs()[fin] - (2.0 ** -19 * L.abs() + 2.0 ** -20).expand(lse.shape)[fin]
    assert bool((off <= 0).all()), float(off.max())
    most = 2.0 ** -8 * O.abs() + (2.0 ** -7 + 2.0 ** -16) * A
    if fmt != P.BF16:
        most = most + 2.0 ** -23 * largest(b, rows)[:n, None]
    assert bool(((out - O).abs() <= most).all())


def largest(batch, rows):
    """tests._paged.attend's G: the largest scale times the sum of |V| / scale."""
    G = torch.zeros((batch.N, 512), dtype=torch.float64)
    for n, r, pos in batch.tokens():
        slot = [s for s in (batch.slot(r, e) for e in range(pos + 1)) if s >= 0]
        if slot:
            unit = batch.row_scale[slot]
            G[n] = (rows[slot][:, :512].abs() / unit[:, None]).sum(0) * unit.max()
    return G


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("gain", [1.0, 60.0, 400.0])
def test_where_the_form_of_tanh_changes(cuda_lib, fmt, gain):
    b = P.Batch(RAGGED, 64, seed=5, pad=2)
    for cap in (255.99998474121094, 256.0, 256.000030517578125):
        run(cuda_lib, b, fmt, 16, cap=cap, q_gain=gain)
        run(cuda_lib, b, fmt, 16, cap=cap, q_gain=gain, slopes=slopes_of(16))


@pytest.mark.parametrize("fmt", FMTS)
def test_the_ends_of_the_caps(cuda_lib, fmt):
    b = P.Batch(RAGGED, 64, seed=6, pad=2)
    for cap in (1e-30, 1e30):
        run(cuda_lib, b, fmt, 16, cap=cap, slopes=slopes_of(16), window=90, sinks=3)
