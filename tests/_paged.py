"""Ragged batches over a paged cache for the tests of the append and the
windowed attention, with plain references on the CPU (fp64 for the attention,
the append's own fp32 arithmetic operation by operation)."""
from __future__ import annotations

import numpy as np
import torch

BF16, E4M3, GROUP128, DS_MLA, GROUP4_KPE, BLOCK = range(6)
DS_MLA_ROW = 656


class Batch:
    """rows: [(new tokens, length after them)]; the blocks of every request
    lie at random places of a pool, `holes` of them unallocated."""

    def __init__(self, rows, block, seed=0, pad=0, stride_rows=0, holes=0, spare=2):
        rng = np.random.default_rng(seed)
        self.rows, self.block, self.pad = rows, block, pad
        self.stride_rows = stride_rows
        step = stride_rows or block
        need = [max(0, -(-L // block)) for _, L in rows]
        pool = sum(need) + spare
        order = rng.permutation(pool).astype(np.int32)
        table = np.full((len(rows), max(max(need), 1)), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = order[at:at + n]
            at += n
        for _ in range(holes):
            r = rng.integers(len(rows))
            if need[r]:
                table[r, rng.integers(need[r])] = -1
        self.table = torch.from_numpy(table)
        self.pool, self.num_slots = pool, pool * step
        self.start = torch.tensor(np.cumsum([0] + [n for n, _ in rows]), dtype=torch.int32)
        self.lens = torch.tensor([L for _, L in rows], dtype=torch.int32)
        self.N = int(self.start[-1]) + pad

    def tokens(self):
        """(packed index, request, position) of every token of a request."""
        n = 0
        for r, (k, L) in enumerate(self.rows):
            for i in range(k):
                yield n, r, L - k + i
                n += 1

    def slot(self, r, pos):
        page = pos // self.block
        blk = int(self.table[r, page]) if page < self.table.shape[1] else -1
        if blk < 0:
            return -1
        return blk * (self.stride_rows or self.block) + pos % self.block

    def dev(self):
        return self.start.cuda(), self.lens.cuda(), self.table.cuda()


def dequant(cache, fmt, scale, batch):
    """fp64 rows [S, d] of a bf16, per-tensor or per-block cache (and each
    row's scale as batch.row_scale, for the tolerances)."""
    S = cache.shape[0]
    if fmt == BF16:
        batch.row_scale = torch.ones(S, dtype=torch.float64)
        return cache.double()
    x = cache.view(torch.float8_e4m3fn).double()
    if fmt == E4M3:
        batch.row_scale = scale.double().expand(S)
    else:
        batch.row_scale = scale.double().repeat_interleave(batch.stride_rows or batch.block)[:S]
    return x * batch.row_scale[:, None]


def attend(q, rows, batch, sm_scale, window, sinks):
    """fp64 reference: (O, LSE, A, D, K, G) with A = sum softmax |V|, D the largest
    sum |q k| and K the largest sum |k| of a visible key, G = the largest scale
    times the sum of the visible keys' |V| / scale, for the tolerances."""
    T, h, d = q.shape
    O = torch.zeros((T, h, 512), dtype=torch.float64)
    L = torch.full((T, h), -float("inf"), dtype=torch.float64)
    A, D, K, G = torch.zeros_like(O), torch.zeros_like(L), torch.zeros_like(L), torch.zeros_like(O)
    unit = getattr(batch, "row_scale", torch.ones(rows.shape[0], dtype=torch.float64))
    qd = q.double()
    slots = {}
    for n, r, pos in batch.tokens():
        seen = range(max(0, pos + 1)) if not window else \
            [e for e in range(max(0, pos + 1)) if e > pos - window or e < sinks]
        at = [s for s in (slots.setdefault((r, e), batch.slot(r, e)) for e in seen) if s >= 0]
        if not at:
            continue
        k = rows[at]
        s = qd[n] @ k.T * sm_scale
        L[n] = torch.logsumexp(s, -1)
        w = torch.softmax(s, -1)
        O[n] = w @ k[:, :512]
        A[n] = w @ k[:, :512].abs()
        D[n] = (qd[n].abs() @ k.abs().T).amax(-1)
        K[n] = k.abs().sum(1).max()
        G[n] = (k[:, :512].abs() / unit[at][:, None]).sum(0) * unit[at].max()
    return O, L, A, D, K, G


def check_attention(out, lse, ref, q, fmt, sm_scale, batch, pow2=True):
    """Tolerances.  Scores: a QK is 36 (bf16) or 2 x 18 (E4M3) accumulations in
    fp32, each off by at most 2^-23 of the sum of magnitudes (40 counted), and
    with E4M3 rows Q's two terms leave at most half of E4M3's smallest step,
    2^-10, where the row's largest value is 224 or more: 2^-17.8 of it per
    channel.  Weights: bf16 (2^-8 each, numerator and the sum that
    divides), a second rounding where the key's scale is no power of two; O is
    rounded to bf16 once (2^-8); 2^-16 for exponentials and sums.
    E4M3 rows: a weight is cut to a grid of 2^-23 of 2^(t - m), t = s + log2(scale)
    and m at most the row's largest t, so the row's sum of weight / scale is at
    least 1 / (that key's scale) and each key's share of O is off by at most
    2^-23 |V| / scale times that scale: together 2^-23 G."""
    O, L, A, D, K, G = ref
    ds = 40 * 2.0 ** -23 * D * abs(sm_scale)
    if fmt != BF16:
        ds = ds + 2.0 ** -17.8 * q.double().abs().amax(-1) * K * abs(sm_scale)
    wt = 2.0 ** -7 + (0 if pow2 else 2.0 ** -8) + 2.0 ** -16
    out, lse = out.double().cpu(), lse.double().cpu()
    n = int(batch.start[-1])
    assert torch.equal(torch.isneginf(lse[:n]), torch.isneginf(L[:n]))
    fin = ~torch.isneginf(L[:n])
    dl = (lse[:n] - L[:n])[fin].abs()
    tl = (ds[:n] + 2.0 ** -19 * L[:n].abs() + 2.0 ** -20)[fin]
    assert bool((dl <= tl).all()), f"LSE off by {float((dl - tl).max())} over its bound"
    do = (out[:n] - O[:n]).abs()
    to = 2.0 ** -8 * O[:n].abs() + (wt + 2 * ds[:n, :, None]) * A[:n]
    if fmt != BF16:
        to = to + 2.0 ** -23 * G[:n]
    assert bool(torch.isfinite(out[:n]).all())
    assert bool((do <= to).all()), f"O off by {float((do - to).max())} over its bound"


# ---------------------------------------------------------------- append --

def rotate(x, cs, interleaved):
    """fp32 rotation, each product and sum rounded on its own."""
    cos, sin = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    return torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)


def e4m3(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def block_scale(amax):
    s = np.float32(2.0 ** -64)
    while np.float64(amax) > 448 * np.float64(s):
        s = np.float32(s * 2)
    return float(s)


def append(batch, kv_c, k_pe, cos_sin, cache, fmt, scale, kpe_scale, interleaved, q_pe, q_out):
    """The append on CPU tensors, in place on cache, scale and q_out."""
    d = 512 if k_pe is None else 576
    written = {}
    limit = cos_sin.shape[0] if cos_sin is not None else 1 << 31
    for n, r, pos in batch.tokens():
        if pos < 0 or pos >= limit:
            continue
        x = kv_c[n].float()
        if d == 576:
            x = torch.cat([x, rotate(k_pe[n].float(), cos_sin[pos], interleaved)])
            if q_pe is not None:
                q_out[n] = rotate(q_pe[n].float(), cos_sin[pos], interleaved).bfloat16()
        slot = batch.slot(r, pos)
        if slot < 0:
            continue
        if fmt == BF16:
            cache[slot] = x.bfloat16()
        elif fmt == E4M3:
            cache[slot] = e4m3(x / scale[0])
        elif fmt == BLOCK:
            written.setdefault((r, pos // batch.block), []).append((pos, slot, x))
        else:
            G = 5 if fmt == GROUP128 and d == 576 else 4
            for g in range(G):
                c = slice(128 * g, min(128 * g + 128, d))
                top = x[c].abs().max()
                s = top / 448 if top > 0 else torch.ones(())
                cache[slot, c] = e4m3(x[c] / s)
                if fmt == DS_MLA:
                    cache[slot, 512 + 4 * g:516 + 4 * g] = s.view(1).view(torch.uint8)
                else:
                    scale[slot, g] = s
            if fmt == DS_MLA:
                cache[slot, 528:] = x[512:].bfloat16().view(torch.uint8)
            elif fmt == GROUP4_KPE:
                cache[slot, 512:] = e4m3(x[512:] / torch.tensor(kpe_scale))
    for (r, page), items in written.items():
        blk = int(batch.table[r, page])
        k, L = batch.rows[r]
        old_rows = max(0, (L - k) - page * batch.block)
        x = torch.stack([i[2] for i in items])
        fin = x[torch.isfinite(x)].abs()
        s = block_scale(float(fin.max()) if fin.numel() else 0.0)
        if old_rows:
            s0 = float(scale[blk])
            if s > s0 > 0:
                at = blk * (batch.stride_rows or batch.block)
                old = cache[at:at + old_rows].view(torch.float8_e4m3fn).float()
                cache[at:at + old_rows] = e4m3(old * (torch.tensor(s0) / torch.tensor(s)))
            s = max(s, s0)
        scale[blk] = s
        for (_, slot, _), row in zip(items, x):
            cache[slot] = e4m3(row * (1 / torch.tensor(s)))
