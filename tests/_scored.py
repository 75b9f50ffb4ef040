"""Attention with capped and distance-biased scores and a span of positions for every
token, in fp64 on the CPU, with the first-order bounds of a row's error."""
from __future__ import annotations

import torch

from tests import _paged as P


def spans(batch, docs=None, prefix=0):
    """(first, last) of every packed token: documents ending at positions `docs` (the
    same in every request), the first `prefix` tokens of each seeing each other."""
    first = torch.zeros(batch.N, dtype=torch.int32)
    last = torch.zeros(batch.N, dtype=torch.int32)
    for n, r, pos in batch.tokens():
        ends = [e for e in (docs or []) if e < batch.rows[r][1]] + [max(batch.rows[r][1], 1)]
        begin, end = 0, ends[0]
        for a, b in zip(ends, ends[1:]):
            if pos >= a:
                begin, end = a, b
        first[n] = begin
        last[n] = min(max(pos, begin + prefix - 1), end - 1)
    return first, last


def attend(q, rows, batch, sm_scale, window=0, sinks=0, cap=0.0, slopes=None, first=None,
           last=None):
    """(O, LSE, A, S, E, G): A = sum softmax |V|; S and E the first-order errors of LSE
    and O from the scores' (what the QK sum, the cap and the bias may be off by, weighted
    as the row weighs its keys); G as in tests._paged.attend."""
    T, h, d = q.shape
    O = torch.zeros((T, h, 512), dtype=torch.float64)
    L = torch.full((T, h), -float("inf"), dtype=torch.float64)
    A, E, G = torch.zeros_like(O), torch.zeros_like(O), torch.zeros_like(O)
    S = torch.zeros_like(L)
    fp8 = getattr(batch, "fp8", False)
    unit = batch.row_scale
    qd = q.double()
    for n, r, pos in batch.tokens():
        if pos < 0:
            continue
        length = batch.rows[r][1]
        lo = max(0, int(first[n])) if first is not None else 0
        hi = min(int(last[n]), length - 1) if last is not None else pos
        e = torch.arange(hi + 1) if hi >= 0 else torch.zeros(0, dtype=torch.long)
        seen = (e >= lo) & ((e > pos - window) if window else torch.ones_like(e, dtype=torch.bool))
        e = e[seen | (e < sinks)]
        slot = torch.tensor([batch.slot(r, int(x)) for x in e], dtype=torch.long)
        e, slot = e[slot >= 0], slot[slot >= 0]
        if not len(e):
            continue
        k = rows[slot]
        x = qd[n] @ k.T * sm_scale                                 # [h, keys]
        mag = qd[n].abs() @ k.abs().T * abs(sm_scale)
        # 36 (bf16) or 2 x 18 (E4M3) fp32 accumulations, 40 counted; Q's two E4M3 terms
        err = 40 * 2.0 ** -23 * mag
        if fp8:
            err = err + 2.0 ** -17.8 * qd[n].abs().amax(-1, keepdim=True) * \
                k.abs().sum(1) * abs(sm_scale)
        s = x
        if cap:
            s = cap * torch.tanh(x / cap)
            # tanh = 1 - 2 / (1 + u): 2 (2^-23 + 2^-24 + 2^-21.5 / 4) < 2^-20 of the cap, up
            # to a cap of 256; above only for scores of an eighth of the cap, whose tanh is
            # 0.124 at least: 2^-20 / 0.124 < 2^-16 of the score (others: 2^-22, products)
            err = err + (2.0 ** -20 * cap if cap <= 256 else 2.0 ** -16 * s.abs())
        if slopes is not None:
            bias = slopes.double()[:, None] * (e - pos).abs().double()
            s = s - bias
            err = err + 2.0 ** -22 * bias.abs()
        err = err + 2.0 ** -22 * s.abs()                           # s - max in fp32, exp2
        L[n] = torch.logsumexp(s, -1)
        w = torch.softmax(s, -1)
        v = k[:, :512]
        O[n] = w @ v
        A[n] = w @ v.abs()
        S[n] = (w * err).sum(-1)
        E[n] = (w * err) @ v.abs() + S[n][:, None] * A[n]
        G[n] = (v.abs() / unit[slot][:, None]).sum(0) * unit[slot].max()
    return O, L, A, S, E, G


def check(out, lse, ref, batch, fmt, pow2=True):
    """As tests._paged.check_attention: weights rounded to 2^-8 (numerator and divisor),
    once more where the key's scale is no power of two, O rounded to 2^-8, 2^-16 for
    exponentials and sums, E4M3 rows 2^-23 G; the scores' errors to first order, doubled
    for the higher ones."""
    O, L, A, S, E, G = ref
    wt = 2.0 ** -7 + (0 if pow2 else 2.0 ** -8) + 2.0 ** -16
    n = int(batch.start[-1])
    out, lse = out.double().cpu()[:n], lse.double().cpu()[:n]
    O, L, A, S, E, G = (x[:n] for x in (O, L, A, S, E, G))
    assert torch.equal(torch.isneginf(lse), torch.isneginf(L))
    fin = ~torch.isneginf(L)
    assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse[fin]).all())
    dl = (lse - L)[fin].abs() - (2 * S + 2.0 ** -19 * L.abs() + 2.0 ** -20)[fin]
    assert bool((dl <= 0).all()), f"LSE off by {float(dl.max())} over its bound"
    to = 2.0 ** -8 * O.abs() + wt * A + 2 * E + (2.0 ** -23 * G if fmt != P.BF16 else 0)
    do = (out - O).abs() - to
    assert bool((do <= 0).all()), f"O off by {float(do.max())} over its bound"
