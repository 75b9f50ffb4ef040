"""Workloads of the paged latent-cache operators: appending tokens to the
cache (with the rotary embedding applied on the way) and causal attention over
it, whole or through a sliding window with first tokens that stay visible, on
bf16 rows and on E4M3 rows with one scale per cache block.

Every batch is ragged: request r owns the tokens [query_start[r],
query_start[r + 1]) of the packed inputs and, after they are appended,
seq_lens[r] positions, so its token i sits at position seq_lens[r] - n_r + i;
position e lives in cache row block_table[r, e // block] * block + e % block.

``run`` computes an operator in its plain form (elementary torch operations in
32 bits), or through the library where ``own`` is set; ``exact`` computes it in
64 bits, request by request.
"""
import random

import torch

own = False

D_V = 512
ROPE = 64
BF16, E4M3, GROUP128, DS_MLA, GROUP4_KPE, BLOCK = 0, 1, 2, 3, 4, 5
KPE_SCALE = 0.03125
TENSOR_SCALE = 0.015625
MIN_SCALE_EXP = -64            # the smallest block scale is 2^-64


# ---------------------------------------------------------------- cases --

def _append(name, **kw):
    c = dict(name=name, op="append", fmt=BF16, reqs=1, new=1, ragged=0, ctx=0, h=128, d=576,
             block=64, interleaved=True, pad=0, shape=1)
    c.update(kw)
    return c


def _attend(name, **kw):
    c = dict(name=name, op="attend", fmt=BF16, reqs=1, new=1, ragged=0, ctx=1024, h=128, d=576,
             block=64, window=0, sinks=0, pad=0, shape=1)
    c.update(kw)
    return c


def listed():
    return [
        # One decode step of 64 requests with all 128 heads on this GPU: the
        # smallest append that a serving loop makes, bound by latency.
        _append("append_decode_bf16", reqs=64, ctx=8192, shape=11),
        # A prefill of 8192 tokens in four requests: the queries' rotation
        # is most of the traffic.
        _append("append_prefill_bf16", reqs=4, new=2048, h=128, shape=12),
        # The decode step on the 8-bit cache: most tokens land in a block
        # that holds older rows, whose codes follow a growing scale.
        _append("append_decode_block8", fmt=BLOCK, reqs=128, ctx=4096, h=64, shape=13),
        # A long ragged prefill into the 8-bit cache with 16 heads a GPU.
        _append("append_prefill_block8", fmt=BLOCK, reqs=24, new=1024, ragged=1, ctx=500, h=16,
                shape=14),
        # One user's next token: a window of 1024 and four sinks, 16 heads.
        _attend("window_one_token", reqs=1, ctx=20000, h=16, window=1024, sinks=4, shape=21),
        # A decode step of 64 requests, 128 heads, window 2048.
        _attend("window_decode", reqs=64, ctx=8192, h=128, window=2048, sinks=4, shape=22),
        # A prompt of 4096 tokens through the same window.
        _attend("window_prefill", reqs=1, new=4096, ctx=0, h=128, window=2048, sinks=4, shape=23),
        # A mixed batch without a window, 16 heads: prompts' chunks beside
        # single tokens, with padding rows behind the last request.
        _attend("causal_mixed", reqs=24, new=500, ragged=2, ctx=4000, h=16, pad=13, shape=24),
        # Decode over 8-bit rows, 128 heads, whole contexts of 8 to 16 thousand.
        _attend("block8_decode", fmt=BLOCK, reqs=32, ctx=16384, h=128, shape=31),
        # Few requests with long contexts and 16 heads: split over the keys.
        _attend("block8_decode_long", fmt=BLOCK, reqs=6, ctx=65536, h=16, shape=32),
        # A prefill chunk of 2048 tokens behind 6000 cached ones, 64 heads.
        _attend("block8_prefill", fmt=BLOCK, reqs=1, new=2048, ctx=6000, h=64, shape=33),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    d = rng.choice([512, 576, 576])
    block = rng.choice([1, 7, 16, 24, 32, 64, 64, 100, 128])
    h = rng.choice([1, 5, 8, 16, 24, 32, 64, 96, 128])
    pad = rng.choice([0, 0, rng.randint(1, 40)])
    shape = rng.randint(1, 1 << 30)
    if rng.random() < 0.4:
        fmt = rng.choice([BF16, E4M3, GROUP128, BLOCK, BLOCK] +
                         ([DS_MLA, GROUP4_KPE] if d == 576 else []))
        reqs = _log_int(rng, 1, 200)
        new = _log_int(rng, 1, 8192 // reqs)
        return dict(op="append", fmt=fmt, reqs=reqs, new=new, ragged=rng.randint(0, 2),
                    ctx=_log_int(rng, 1, 4000), h=h, d=d, block=block,
                    interleaved=rng.random() < 0.6, pad=pad, shape=shape)
    fmt = rng.choice([BF16, BF16, E4M3, BLOCK, BLOCK, BLOCK])
    window = rng.choice([0, _log_int(rng, 1, 4096)])
    sinks = rng.choice([0, 1, 4, rng.randint(1, 200)])
    reqs = _log_int(rng, 1, 64)
    new = rng.choice([1, _log_int(rng, 1, 2048)])
    ctx = _log_int(rng, 1, 32768)
    while reqs * new * h * (new + (min(ctx, window + sinks) if window else ctx)) > 8e8:
        if new > 64:
            new //= 2
        elif reqs > 4:
            reqs //= 2
        else:
            ctx //= 2
    ctx = min(ctx, 400000 // reqs)
    return dict(op="attend", fmt=fmt, reqs=reqs, new=new, ragged=rng.randint(0, 2), ctx=max(ctx, 1),
                h=h, d=d, block=block, window=window, sinks=sinks, pad=pad, shape=shape)


def _batch(case):
    """[(new tokens, positions after them)] of the case's requests."""
    rng = random.Random(case["shape"])
    rows = []
    for _ in range(case["reqs"]):
        n = case["new"]
        if case["ragged"] and n > 1:
            n = rng.randint(max(1, n // 4), n)
        if case["ragged"] == 2 and rng.random() < 0.5:
            n = 1
        rows.append((n, n + rng.randint(case["ctx"] // 2, case["ctx"])))
    return rows


def _lo(case, first):
    """The first position, past the sinks, that the token at `first` sees."""
    return max(0, first - case["window"] + 1) if case["window"] else 0


def _row_bytes(case):
    return {BF16: 2 * case["d"], DS_MLA: 656}.get(case["fmt"], case["d"])


def work(case):
    rows = _batch(case)
    N, h, d = sum(n for n, _ in rows), case["h"], case["d"]
    pages = 4 * sum(-(-L // case["block"]) for _, L in rows)
    if case["op"] == "append":
        rope = ROPE if d == 576 else 0
        scales = {E4M3: 0, GROUP128: 4 * N * -(-d // 128), GROUP4_KPE: 16 * N,
                  BLOCK: 4 * sum(-(-n // case["block"]) for n, _ in rows)}.get(case["fmt"], 0)
        return {"bytes": N * (2 * d + _row_bytes(case) + 2 * 2 * rope * h + 4 * rope) + scales,
                "flops": 3 * N * rope * (h + 1) + 2 * N * d}
    keys = pairs = 0
    for n, L in rows:
        first = L - n
        sinks, window = case["sinks"], case["window"]
        lo = _lo(case, first)
        keys += L - lo + min(sinks, lo)
        for p in range(first, L):
            plo = _lo(case, p)
            pairs += p + 1 - plo + min(sinks, plo)
    scales = pages if case["fmt"] == BLOCK else 0
    return {"bytes": keys * _row_bytes(case) + N * h * (2 * d + 2 * D_V + 4) + pages + scales,
            "flops": 2 * pairs * h * (d + D_V)}


# --------------------------------------------------------------- inputs --

def _tables(case, gen):
    """The batch's descriptors: starts, lengths and a block table whose
    blocks lie in random order in the pool."""
    rows, block = _batch(case), case["block"]
    need = [-(-L // block) for _, L in rows]
    pool = sum(need) + 2
    order = torch.randperm(pool, generator=gen, device="cuda").to(torch.int32)
    width = max(need)
    at = torch.cumsum(torch.tensor([0] + need[:-1], device="cuda"), 0)[:, None]
    col = torch.arange(width, device="cuda")[None, :]
    have = col < torch.tensor(need, device="cuda")[:, None]
    table = torch.where(have, order[torch.clamp(at + col, max=pool - 1)], -1).to(torch.int32)
    start = torch.tensor([0] + [n for n, _ in rows], device="cuda").cumsum(0).to(torch.int32)
    lens = torch.tensor([L for _, L in rows], dtype=torch.int32, device="cuda")
    return rows, pool, table.contiguous(), start, lens


def _pool_rows(case, pool, gen):
    """A cache pool as earlier steps left it, and its scales."""
    S, d, fmt, block = pool * case["block"], case["d"], case["fmt"], case["block"]
    x = torch.empty((S, d), dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    if fmt == BF16:
        return x, None
    if fmt == DS_MLA:
        raw = torch.zeros((S, 656), dtype=torch.uint8, device="cuda")
        raw[:, :512] = (x[:, :512].float() * 64).to(torch.float8_e4m3fn).view(torch.uint8)
        raw[:, 512:528] = torch.full((S, 4), 2.0 ** -6, device="cuda").view(torch.uint8)
        raw[:, 528:] = x[:, 512:].contiguous().view(torch.uint8)
        return raw, None
    if fmt == BLOCK:
        # codes of normal values reach 64 * 5; the blocks differ in magnitude
        scale = torch.exp2(torch.randint(-9, -4, (pool,), generator=gen, device="cuda").float())
        return (x * 64).to(torch.float8_e4m3fn).view(torch.uint8), scale
    G = {E4M3: 0, GROUP128: -(-d // 128), GROUP4_KPE: 4}[fmt]
    scale = (torch.full((1,), TENSOR_SCALE, device="cuda") if fmt == E4M3 else
             torch.empty((S, G), device="cuda").uniform_(0.01, 0.02, generator=gen))
    return (x * 64).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _cos_sin(length):
    """fp32 [length, 64]: 32 cosines, then 32 sines of each position."""
    inv = 10000.0 ** (-torch.arange(0, ROPE, 2, dtype=torch.float64, device="cuda") / ROPE)
    a = torch.arange(length, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, pool, table, start, lens = _tables(case, gen)
    N = sum(n for n, _ in rows) + case["pad"]
    h, d = case["h"], case["d"]
    cache, scale = _pool_rows(case, pool, gen)
    s = dict(case=case, table=table, start=start, lens=lens, cache=cache, scale=scale, N=N,
             max_new=max(n for n, _ in rows), max_len=max(L for _, L in rows))

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)

    if case["op"] == "append":
        # k_pe as a slice of the layer's joint projection, the queries' rope
        # part as a slice of [nope 128 | rope 64] heads; the rotated part
        # goes behind the 512 latent channels of the attention's query.
        s["kv_c"] = normal(N, 512)
        rope = d == 576
        s["k_pe"] = normal(N, 576)[:, 512:] * 4 if rope else None
        if rope:
            s["k_pe"] = torch.cat([s["kv_c"], s["k_pe"]], 1)[:, 512:]
        s["cos_sin"] = _cos_sin(s["max_len"]) if rope else None
        s["q_pe"] = normal(N, h, 192)[:, :, 128:] if rope else None
        s["q"] = torch.zeros((N, h, 576), dtype=torch.bfloat16, device="cuda") if rope else None
        return s
    s["q"] = normal(N, h, d) * 2
    s["out"] = torch.zeros((N, h, D_V), dtype=torch.bfloat16, device="cuda")
    s["lse"] = torch.zeros((N, h), dtype=torch.float32, device="cuda")
    first = [L - n for n, L in rows]
    s["max_keys"] = max(L - _lo(case, f) for (_, L), f in zip(rows, first))
    s["max_sinks"] = max(min(case["sinks"], _lo(case, f)) for f in first)
    s["sm_scale"] = d ** -0.5
    return s


# ----------------------------------------------------------- plain forms --

def _tokens(s, count):
    """Request, position and validity of the first `count` packed tokens."""
    n = torch.arange(count, device="cuda")
    req = torch.searchsorted(s["start"].long(), n, right=True) - 1
    live = req < s["lens"].numel()
    req = req.clamp(max=s["lens"].numel() - 1)
    pos = s["lens"].long()[req] - s["start"].long()[req + 1] + n
    live = live & (pos >= 0)
    return req, torch.where(live, pos, 0), live


def _rotate(x, cs, interleaved):
    """x fp32 [..., 64] rotated by cs fp32 [..., 64] = [cos | sin]."""
    cos, sin = cs[..., :32], cs[..., 32:]
    a, b = (x[..., 0::2], x[..., 1::2]) if interleaved else (x[..., :32], x[..., 32:])
    ra, rb = a * cos - b * sin, b * cos + a * sin
    return torch.stack([ra, rb], -1).flatten(-2) if interleaved else torch.cat([ra, rb], -1)


def _block_scale(amax):
    """The smallest power of two s >= 2^-64 with amax <= 448 s."""
    m, e = torch.frexp(amax)
    k = torch.where(amax > 0, e - 9 + (m > 0.875).int(), torch.full_like(e, MIN_SCALE_EXP))
    return torch.ldexp(torch.ones_like(amax), k.clamp(min=MIN_SCALE_EXP))


def _codes(x):
    return x.clamp(-448, 448).to(torch.float8_e4m3fn)


def _cache_view(s):
    """The cache as the values that it holds."""
    c, fmt = s["cache"], s["case"]["fmt"]
    if fmt == BF16:
        return {"cache": c}
    if fmt == DS_MLA:
        return {"codes": c[:, :512].view(torch.float8_e4m3fn),
                "scale": c[:, 512:528].view(torch.float32),
                "rope": c[:, 528:].view(torch.bfloat16)}
    return {"codes": c.view(torch.float8_e4m3fn), "scale": s["scale"]}


def _plain_append(s):
    case, block = s["case"], s["case"]["block"]
    d, fmt, cache, scale = case["d"], case["fmt"], s["cache"], s["scale"]
    req, pos, live = _tokens(s, s["N"])
    x = s["kv_c"].float()
    if d == 576:
        cs = s["cos_sin"][pos]
        rq = _rotate(s["q_pe"].float(), cs[:, None], case["interleaved"]).to(torch.bfloat16)
        s["q"][:, :, 512:] = torch.where(live[:, None, None], rq, s["q"][:, :, 512:])
        x = torch.cat([x, _rotate(s["k_pe"].float(), cs, case["interleaved"])], 1)
    page = s["table"].long()[req, pos // block]
    live = live & (page >= 0)
    x, req, pos, page = x[live], req[live], pos[live], page[live]
    slot = page * block + pos % block
    if fmt == BF16:
        cache[slot] = x.to(torch.bfloat16)
    elif fmt == E4M3:
        cache[slot] = _codes(x / scale).view(torch.uint8)
    elif fmt == BLOCK:
        amax = torch.zeros_like(scale).scatter_reduce_(0, page, x.abs().amax(1), "amax")
        first = (s["lens"] - (s["start"][1:] - s["start"][:-1])).long()[req]
        kept = (pos // block * block < first)          # the block holds older rows
        old = torch.zeros_like(scale)
        old[page] = torch.where(kept, scale[page], 0)
        new = torch.maximum(_block_scale(amax), old)
        # older rows follow a growing scale: rows below `first` of its block
        older = torch.zeros_like(scale, dtype=torch.long)
        older[page] = torch.where(kept, first - pos // block * block, 0).clamp(max=block)
        grown = torch.nonzero((old > 0) & (new > old)).flatten()
        rows = grown[:, None] * block + torch.arange(block, device="cuda")
        keep = rows - grown[:, None] * block < older[grown][:, None]
        rows, ratio = rows[keep], (old / new)[grown][:, None].expand_as(keep)[keep]
        cache[rows] = _codes(cache[rows].view(torch.float8_e4m3fn).float() *
                             ratio[:, None]).view(torch.uint8)
        scale[page] = new[page]
        cache[slot] = _codes(x * (1 / scale[page])[:, None]).view(torch.uint8)
    else:
        xg = torch.nn.functional.pad(x, (0, -d % 128)).view(len(x), -1, 128)
        if fmt != GROUP128:
            xg = xg[:, :4]
        amax = xg.abs().amax(2)
        sc = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        codes = _codes(xg / sc[:, :, None]).view(torch.uint8).flatten(1)
        if fmt == DS_MLA:
            cache[slot, :512] = codes
            cache[slot, 512:528] = sc.view(torch.uint8)
            cache[slot, 528:] = x[:, 512:].to(torch.bfloat16).view(torch.uint8)
        else:
            scale[slot] = sc
            cache[slot, :min(d, codes.shape[1])] = codes[:, :d]
            if fmt == GROUP4_KPE:
                cache[slot, 512:] = _codes(x[:, 512:] / KPE_SCALE).view(torch.uint8)
    return {**_cache_view(s), **({"q": s["q"]} if d == 576 else {})}


def _plain_attend(s):
    case, block = s["case"], s["case"]["block"]
    h, d, window = case["h"], case["d"], case["window"]
    start, lens = s["start"].long(), s["lens"].long()
    n = start[1:] - start[:-1]
    first = lens - n
    i = torch.arange(s["max_new"], device="cuda")
    tok = (start[:-1, None] + i).clamp(max=s["N"] - 1)             # [R, new]
    live = i < n[:, None]
    qpos = first[:, None] + i
    lo = (first - window + 1).clamp(min=0) if window else torch.zeros_like(first)
    # a request's key positions: its sinks below `lo`, then [lo, len)
    j = torch.arange(s["max_sinks"], device="cuda").expand(len(lens), -1)
    kpos = torch.cat([j, lo[:, None] + torch.arange(s["max_keys"], device="cuda")], 1)
    real = torch.cat([(j < lo[:, None]) & (j < case["sinks"]),
                      kpos[:, s["max_sinks"]:] < lens[:, None]], 1)
    page = torch.gather(s["table"].long(), 1, (kpos // block).clamp(max=s["table"].shape[1] - 1))
    real = real & (page >= 0)
    slot = torch.where(real, page * block + kpos % block, 0)
    if case["fmt"] == BF16:
        k = s["cache"][slot].float()
    else:
        k = s["cache"][slot].view(torch.float8_e4m3fn).float()
        k *= s["scale"][page.clamp(min=0)][:, :, None] if case["fmt"] == BLOCK else s["scale"]
    sees = real[:, None, :] & (kpos[:, None, :] <= qpos[:, :, None])
    if window:
        sees &= (kpos[:, None, :] > qpos[:, :, None] - window) | (kpos < case["sinks"])[:, None, :]
    q = s["q"][tok].float().flatten(1, 2)                          # [R, new * h, d]
    w = torch.matmul(q, k.transpose(1, 2)).mul_(s["sm_scale"])
    w = w.view(len(lens), s["max_new"], h, -1)
    w.masked_fill_(~sees[:, :, None, :], float("-inf"))
    top = w.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), 0, top)
    w = w.sub_(top).exp_()
    total = w.sum(-1, keepdim=True)
    o = torch.matmul(w.flatten(1, 2), k[:, :, :D_V]).view(*w.shape[:3], D_V)
    o = torch.where(total > 0, o / total, 0)
    s["out"][tok[live]] = o[live].to(torch.bfloat16)
    s["lse"][tok[live]] = (top + total.log())[..., 0][live]
    return {"out": s["out"], "lse": s["lse"]}


def run(s):
    if own:
        import sparse_mla_attention_02_gb300 as smla
        c = s["case"]
        if c["op"] == "append":
            smla.smla_cache_append(
                s["kv_c"], s["k_pe"], s["cos_sin"], s["start"], s["lens"], s["table"], c["block"],
                s["cache"], c["fmt"], s["scale"], kpe_scale=KPE_SCALE, interleaved=c["interleaved"],
                q_pe=s["q_pe"], q_out=None if s["q"] is None else s["q"][:, :, 512:])
            return {**_cache_view(s), **({} if s["q"] is None else {"q": s["q"]})}
        out, lse = smla.smla_fwd_window(
            s["q"], s["cache"], c["fmt"], s["scale"], s["start"], s["lens"], s["table"], c["block"],
            s["sm_scale"], window=c["window"], sinks=c["sinks"], max_seq_len=s["max_len"],
            out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    return _plain_append(s) if s["case"]["op"] == "append" else _plain_attend(s)


# ------------------------------------------------------------- 64 bits --

def _exact_append(s):
    case, block, d, fmt = s["case"], s["case"]["block"], s["case"]["d"], s["case"]["fmt"]
    table, start, lens = s["table"].tolist(), s["start"].tolist(), s["lens"].tolist()
    res = {k: v.double() for k, v in _cache_view(s).items()}
    if d == 576:
        res["q"] = s["q"].double()
    for r, L in enumerate(lens):
        a, b = start[r], start[r + 1]
        if a == b:
            continue
        p = torch.arange(L - (b - a), L, device="cuda")
        x = s["kv_c"][a:b].double()
        if d == 576:
            z = torch.complex(*s["cos_sin"].double()[p].view(-1, 2, 32).unbind(1))

            def turn(v, z):
                v = v.double()
                v = v.unflatten(-1, (32, 2)) if case["interleaved"] else \
                    v.unflatten(-1, (2, 32)).transpose(-1, -2)
                w = torch.view_as_real(torch.view_as_complex(v.contiguous()) * z)
                return (w if case["interleaved"] else w.transpose(-1, -2)).flatten(-2)
            res["q"][a:b, :, 512:] = turn(s["q_pe"][a:b], z[:, None])
            x = torch.cat([x, turn(s["k_pe"][a:b], z)], 1)
        pages = torch.tensor(table[r], device="cuda")[p // block]
        slot = pages * block + p % block
        if fmt == BF16:
            res["cache"][slot] = x
        elif fmt == E4M3:
            res["codes"][slot] = (x / s["scale"].double()).clamp(-448, 448)
        elif fmt == BLOCK:
            for g in pages.unique().tolist():
                here = pages == g
                low = int(p[here][0]) // block * block
                amax = float(x[here].abs().amax())
                new = 2.0 ** MIN_SCALE_EXP
                while amax > 448 * new:
                    new *= 2
                kept = max(0, int(p[0]) - low)
                if kept:
                    old = float(s["scale"][g])
                    new = max(new, old)
                    res["codes"][g * block:g * block + kept] *= old / new
                res["scale"][g] = new
                res["codes"][slot[here]] = x[here] / new
        else:
            for g in range(5 if fmt == GROUP128 and d == 576 else 4):
                xg = x[:, 128 * g:128 * g + 128]
                top = xg.abs().amax(1)
                sc = torch.where(top > 0, top / 448, 1.0)
                res["codes"][slot, 128 * g:128 * g + xg.shape[1]] = xg / sc[:, None]
                res["scale"][slot, g] = sc
            if fmt == DS_MLA:
                res["rope"][slot] = x[:, 512:]
            elif fmt == GROUP4_KPE:
                res["codes"][slot, 512:] = (x[:, 512:] / KPE_SCALE).clamp(-448, 448)
    return res


def _exact_attend(s):
    case, block = s["case"], s["case"]["block"]
    h, window, sinks = case["h"], case["window"], case["sinks"]
    start, lens = s["start"].tolist(), s["lens"].tolist()
    out, lse = s["out"].double(), s["lse"].double()
    for r, L in enumerate(lens):
        e = torch.arange(L, device="cuda")
        page = s["table"][r].long()[e // block]
        rows = s["cache"][page * block + e % block]
        if case["fmt"] != BF16:
            rows = rows.view(torch.float8_e4m3fn)
        k = rows.double()
        if case["fmt"] != BF16:
            k = k * (s["scale"].double()[page][:, None] if case["fmt"] == BLOCK
                     else s["scale"].double())
        n = start[r + 1] - start[r]
        for c in range(0, n, 64):
            m = min(64, n - c)
            p = torch.arange(L - n + c, L - n + c + m, device="cuda")
            lo = max(0, int(p[0]) - window + 1) if window else 0
            at = torch.cat([e[:min(sinks, lo)], e[lo:int(p[-1]) + 1]])
            hide = at[None, :] > p[:, None]
            if window:
                hide |= (at[None, :] <= p[:, None] - window) & (at[None, :] >= sinks)
            t = slice(start[r] + c, start[r] + c + m)
            x = s["q"][t].double().flatten(0, 1) @ k[at].T * s["sm_scale"]
            x = x.view(m, h, -1).masked_fill(hide[:, None, :], float("-inf"))
            lse[t] = torch.logsumexp(x, -1)
            out[t] = (torch.softmax(x, -1).flatten(0, 1) @ k[at, :D_V]).view(m, h, D_V)
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_append(s) if case["op"] == "append" else _exact_attend(s)
