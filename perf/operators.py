"""Cases and plain forms of the rotary and 4-bit cache operators.

    rope      pa.rope_and_cache: queries and keys rotated by position, K and V rows written to the paged pools
    rope_q4   pa.rope_and_cache_q4, then pa.dequantize_blocks_q4 of the blocks it wrote (what a prefill over a
              4-bit prefix does next), so that the pass returns the values which the 4-bit rows stand for
    decode_q4 pa.decode_q4: one query row per sequence over a 4-bit paged cache
    convert   pa.quantize_blocks_q4, then pa.dequantize_blocks_q4 of the same blocks

The 4-bit pool is uint8 [num_blocks, num_kv_heads, slab]: per block and kv-head block_size * D / 2 code bytes, then
block_size * D / 32 bf16 scales.  A group is 32 consecutive dims of one token row; a nibble n stands for
(n - 8) * scale.  Inside a token row of D / 2 bytes a K pool holds 4 x (D/32) words of 8 dims (word q, g: dims
32 g + 8 q ...), a V pool 8 x (D/32) units of 4 dims (unit r, g: dims 32 g + 4 r ...), low nibble first.
"""
import math

import numpy as np
import torch

own = False  # True: run() calls the library; False: it computes the plain forms

GROUP = 32
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one decode step of 256 running requests: one token each, rows of a fused QKV projection
        dict(name="rope_decode", op="rope", dtype="bf16", seqs=256, tokens=256, heads=32, kv_heads=8, dim=128, rot=128,
             block=16, interleaved=False, max_pos=4096, pad=0),
        # eight prompts of 1024 tokens prefilled together
        dict(name="rope_prefill", op="rope", dtype="bf16", seqs=8, tokens=8192, heads=32, kv_heads=8, dim=128, rot=128,
             block=16, interleaved=False, max_pos=4096, pad=0),
        # a ragged batch with padding rows, half of each head rotated in neighbouring pairs, fp32
        dict(name="rope_f32_partial", op="rope", dtype="f32", seqs=7, tokens=1031, heads=12, kv_heads=4, dim=64, rot=32,
             block=8, interleaved=True, max_pos=2048, pad=5),
        # the decode step of 256 requests whose cache is held in 4 bits
        dict(name="append_q4_decode", op="rope_q4", dtype="bf16", seqs=256, tokens=256, heads=32, kv_heads=8, dim=128,
             rot=128, block=16, interleaved=False, max_pos=4096, pad=0),
        # prompts prefilled into the 4-bit cache and read back for their attention
        dict(name="append_q4_prefill", op="rope_q4", dtype="bf16", seqs=8, tokens=8191, heads=32, kv_heads=8, dim=128,
             rot=128, block=16, interleaved=False, max_pos=4096, pad=1),
        # a single short chat request: the latency of one call
        dict(name="decode_q4_one", op="decode_q4", dtype="bf16", seqs=1, lo=50, hi=50, law="uniform", heads=32, kv_heads=8,
             dim=128, block=16),
        # 256 running requests, power-law contexts, grouped heads
        dict(name="decode_q4_gqa256", op="decode_q4", dtype="bf16", seqs=256, lo=16, hi=4096, law="power", heads=32,
             kv_heads=8, dim=128, block=16),
        # 64 requests of a model without grouped heads
        dict(name="decode_q4_mha64", op="decode_q4", dtype="bf16", seqs=64, lo=128, hi=384, law="uniform", heads=32,
             kv_heads=32, dim=128, block=16),
        # sixteen long documents
        dict(name="decode_q4_long", op="decode_q4", dtype="bf16", seqs=16, lo=32768, hi=32768, law="uniform", heads=32,
             kv_heads=8, dim=128, block=16),
        # fp32 queries, small heads, blocks of 32
        dict(name="decode_q4_f32", op="decode_q4", dtype="f32", seqs=12, lo=1, hi=777, law="uniform", heads=14, kv_heads=2,
             dim=64, block=32),
        # the blocks of finished prefills turned to 4 bits
        dict(name="convert_bf16", op="convert", dtype="bf16", pairs=2048, kv_heads=8, dim=128, block=16),
        # a few fp32 blocks, some pairs skipped
        dict(name="convert_f32_small", op="convert", dtype="f32", pairs=37, kv_heads=5, dim=64, block=8),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "rope_q4", "decode_q4", "decode_q4", "convert"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), dim=rng.choice([64, 128]), block=rng.choice([8, 16, 32]))
    if op == "convert":
        c.update(pairs=_log(rng, 1, 2000), kv_heads=rng.randint(1, 8))
        if c["block"] == 32 or c["dtype"] == "f32":
            c["pairs"] = min(c["pairs"], 1000 if c["block"] < 32 or c["dtype"] == "bf16" else 500)
        return c
    group = rng.choice([1, 2, 4, 4, 7, 8, 16])
    c["kv_heads"] = max(1, min(8, 32 // group) if op != "decode_q4" or group > 1 else rng.choice([5, 32]))
    c["heads"] = group * c["kv_heads"]
    if op == "decode_q4":
        c["seqs"] = _log(rng, 1, 300)
        most = max(1, min(65536, 400_000 * 8 // (c["seqs"] * max(8, c["kv_heads"], c["heads"] // 4))))
        c["hi"] = _log(rng, 1, most) if rng.random() < 0.3 else _log(rng, max(1, most // 16), most)
        c["lo"] = _log(rng, 1, c["hi"])
        c["law"] = rng.choice(["uniform", "power"])
        if c["dtype"] == "f32":
            c["hi"] = min(c["hi"], 4000)
            c["lo"] = min(c["lo"], c["hi"])
        return c
    half = c["dim"] // 2
    c["rot"] = rng.choice([c["dim"], c["dim"], half, half + 8 * rng.randint(0, 4), 2 * rng.randint(1, half)])
    c["interleaved"] = rng.random() < 0.4
    c["pad"] = rng.choice([0, 0, 1, 9])
    c["tokens"] = _log(rng, 1, 8000 if c["dtype"] == "bf16" else 3900)
    c["seqs"] = max(1, min(c["tokens"], _log(rng, 1, 300)))
    c["max_pos"] = max(_log(rng, 512, 65536), 2 * (c["tokens"] // c["seqs"] + 2 + c["block"]))
    return c


def _lengths(case):
    """The multiset of context lengths: quantiles of the law (the seed only orders them)."""
    n, lo, hi = case["seqs"], case["lo"], case["hi"]
    u = (np.arange(n) + 0.5) / n
    if case["law"] == "power":
        x = (lo ** -0.2 + u * (hi ** -0.2 - lo ** -0.2)) ** -5.0
    else:
        x = lo + u * (hi + 1 - lo)
    return np.clip(np.floor(x), lo, hi).astype(np.int64)


def _seq_tokens(case):
    n, s = case["tokens"], case["seqs"]
    return np.array([n // s + (1 if i < n % s else 0) for i in range(s)], dtype=np.int64)


def work(case):
    e, d = ESIZE[case["dtype"]], case["dim"]
    q4 = d * 9 / 16
    if case["op"] == "convert":
        n = 2 * case["pairs"] * case["block"] * case["kv_heads"]
        return {"bytes": n * (2 * d * e + 2 * q4), "flops": 4.0 * n * d}
    h, hk = case["heads"], case["kv_heads"]
    if case["op"] == "decode_q4":
        toks = float(_lengths(case).sum())
        return {"bytes": toks * 2 * hk * q4 + 2 * case["seqs"] * h * d * e + 4 * toks / case["block"],
                "flops": 4 * toks * h * d}
    n = case["tokens"]
    table = min(n, case["max_pos"]) * case["rot"] * 4 + 12 * n
    if case["op"] == "rope":
        return {"bytes": 2.0 * n * (h + 2 * hk) * d * e + table, "flops": 3.0 * n * (h + hk) * case["rot"]}
    blocks = _blocks_written(case)
    return {"bytes": n * (2.0 * h + 2 * hk) * d * e + 2 * n * hk * q4 + table
            + 2.0 * blocks * case["block"] * hk * (q4 + d * e), "flops": 3.0 * n * (h + hk) * case["rot"] + 4.0 * n * hk * d}


def _blocks_written(case):
    b = case["block"]
    return int(sum(-(-(int(n) + 7 * i % b) // b) for i, n in enumerate(_seq_tokens(case))))


# ------------------------------------------------------------------ the 4-bit format, in torch

def _dims(kind, d, device):
    """The dim that nibble p of a token row stands for."""
    p = torch.arange(d, device=device)
    per = 8 if kind == "k" else 4
    ng = d // GROUP
    unit, n = p // per, p % per
    return GROUP * (unit % ng) + per * (unit // ng) + n


def _encode(rows, kind):
    """rows [..., D] (f32 or bf16) -> code bytes [..., D/2] and scales [..., D/32] (bf16)."""
    d = rows.shape[-1]
    x = rows.float().reshape(*rows.shape[:-1], d // GROUP, GROUP)
    amax = x.abs().amax(-1)
    s = (amax / 7).to(torch.bfloat16)
    bad = ~torch.isfinite(x).all(-1)
    s = torch.where(bad, torch.full_like(s, float("nan")), s)
    sf = s.float()[..., None]
    n = torch.where((sf > 0) & ~bad[..., None], torch.round(x / sf).clamp(-7, 7), torch.zeros_like(x)) + 8
    n = n.reshape(*rows.shape)[..., _dims(kind, d, rows.device)].to(torch.uint8)
    return n[..., 0::2] | (n[..., 1::2] << 4), s


def _decode(codes, scales, kind):
    """The values in 32 bits, dims in their order: codes [..., D/2], scales [..., D/32]."""
    d = codes.shape[-1] * 2
    n = torch.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], d)
    back = torch.argsort(_dims(kind, d, codes.device))
    v = (n[..., back].float() - 8).reshape(*codes.shape[:-1], d // GROUP, GROUP)
    return (v * scales.float()[..., None]).reshape(*codes.shape[:-1], d)


def _split(pool, block, d):
    """(codes [n, heads, block, D/2], scales [n, heads, block, D/32]) as views of a 4-bit pool."""
    n, h, _ = pool.shape
    cb = block * d // 2
    return (pool[:, :, :cb].unflatten(2, (block, d // 2)),
            pool[:, :, cb:].view(torch.bfloat16).unflatten(2, (block, d // GROUP)))


def _random_pool(n, case, kind, gen):
    """A 4-bit pool of n blocks of N(0, 1) rows."""
    b, h, d = case["block"], case["kv_heads"], case["dim"]
    pool = torch.empty(n, h, b * d * 9 // 16, dtype=torch.uint8, device="cuda")
    codes, scales = _split(pool, b, d)
    step = max(1, (1 << 26) // (b * h * d))
    for i in range(0, n, step):
        m = min(step, n - i)
        rows = torch.randn(m, h, b, d, generator=gen, device="cuda").to(torch.bfloat16)
        if kind == "k":  # a few channels of the keys are large, as those of real models are
            rows[..., 5::37] *= 4
        c, s = _encode(rows, kind)
        codes[i:i + m], scales[i:i + m] = c, s
    return pool


# ------------------------------------------------------------------ inputs

def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    b, hk, d = case["block"], case["kv_heads"], case["dim"]
    if case["op"] == "convert":
        n = case["pairs"]
        total = n + n // 4 + 2
        s["src_k"], s["src_v"] = (torch.randn(total, b, hk, d, generator=gen, device="cuda").to(dt) for _ in "kv")
        s["src_k"][..., 5::37] *= 4
        s["q4_k"], s["q4_v"] = _random_pool(total, case, "k", gen), _random_pool(total, case, "v", gen)
        s["dst_k"], s["dst_v"] = (torch.zeros(n, b, hk, d, dtype=dt, device="cuda") for _ in "kv")
        src, mid = rng.permutation(total)[:n], rng.permutation(total)[:n]
        there, back = np.stack([src, mid], 1), np.stack([mid, np.arange(n)], 1)
        there[5::11, 0] = -1  # skipped pairs leave their destinations as they were
        back[7::13, 1] = -1
        s["there"] = torch.from_numpy(there.astype(np.int32)).cuda()
        s["back"] = torch.from_numpy(back.astype(np.int32)).cuda()
        return s
    h = case["heads"]
    if case["op"] == "decode_q4":
        ctx = rng.permutation(_lengths(case))
        nb = -(-ctx // b)
        total = int(nb.sum()) + 3
        ids, bt = rng.permutation(total).astype(np.int32), np.full((ctx.size, int(nb.max())), -1, dtype=np.int32)
        bt[np.arange(bt.shape[1])[None, :] < nb[:, None]] = ids[:int(nb.sum())]
        s["bt"], s["ctx"] = torch.from_numpy(bt).cuda(), torch.from_numpy(ctx.astype(np.int32)).cuda()
        s["q"] = torch.randn(ctx.size, h, d, generator=gen, device="cuda").to(dt)
        s["k4"], s["v4"] = _random_pool(total, case, "k", gen), _random_pool(total, case, "v", gen)
        s["out"] = torch.empty_like(s["q"])
        s["scale"] = float(np.float32(1 / math.sqrt(d)))
        return s
    # a batch of `seqs` sequences with their new tokens at consecutive positions, padding rows behind them
    lens, pad = _seq_tokens(case), case["pad"]
    n = case["tokens"] + pad
    phase = 7 * np.arange(lens.size) % b  # where in a block each sequence goes on: by the case, not by the seed
    start = b * rng.integers(0, (case["max_pos"] - lens - phase) // b + 1) + phase
    within = np.concatenate([np.arange(m) for m in lens]) if lens.size else np.zeros(0, dtype=np.int64)
    pos = np.repeat(start, lens) + within
    first = start // b
    nb = (start + lens - 1) // b - first + 1
    base = np.concatenate([[0], np.cumsum(nb)])
    total = int(base[-1]) + 5
    ids = rng.permutation(total)
    block = ids[np.repeat(base[:-1], lens) + pos // b - np.repeat(first, lens)]
    slot = block * b + pos % b
    s["pos"] = torch.from_numpy(np.concatenate([pos, np.full(pad, -1)]).astype(np.int32)).cuda()
    s["slot"] = torch.from_numpy(np.concatenate([slot, np.full(pad, -1)]).astype(np.int64)).cuda()
    r = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(r, device="cuda", dtype=torch.float64) / r)
    angle = torch.arange(case["max_pos"], device="cuda", dtype=torch.float64)[:, None] * freq
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    qkv = torch.randn(n, (h + 2 * hk) * d, generator=gen, device="cuda").to(dt)
    s["q"] = qkv[:, :h * d].unflatten(1, (h, d))
    s["key"] = qkv[:, h * d:(h + hk) * d].unflatten(1, (hk, d))
    s["value"] = qkv[:, (h + hk) * d:].unflatten(1, (hk, d))
    s["q_out"] = torch.zeros(n, h, d, dtype=dt, device="cuda")
    if case["op"] == "rope":
        s["k"], s["v"] = (torch.zeros(total, b, hk, d, dtype=dt, device="cuda") for _ in "kv")
        return s
    s["k4"], s["v4"] = _random_pool(total, case, "k", gen), _random_pool(total, case, "v", gen)
    touched = ids[:int(base[-1])]
    s["back"] = torch.from_numpy(np.stack([touched, np.arange(touched.size)], 1).astype(np.int32)).cuda()
    s["dst_k"], s["dst_v"] = (torch.zeros(touched.size, b, hk, d, dtype=dt, device="cuda") for _ in "kv")
    return s


# ------------------------------------------------------------------ plain forms

def _rotated(x, table, pos, rot, interleaved):
    """x [tokens, heads, D] rotated, in 64 bits, rounded once to its type."""
    r = rot // 2
    c, s = table[pos].double()[:, None].split(r, -1)
    y = x.double()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if interleaved else (y[..., :r], y[..., r:rot])
    a, b = a * c - b * s, b * c + a * s
    front = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([front, y[..., rot:]], -1).float().to(x.dtype)


def _plain_rope(s):
    live = torch.nonzero(s["slot"] >= 0).flatten()
    pos, slot = s["pos"][live].long(), s["slot"][live]
    s["q_out"][live] = _rotated(s["q"][live], s["table"], pos, s["rot"], s["interleaved"])
    return slot, _rotated(s["key"][live], s["table"], pos, s["rot"], s["interleaved"]), s["value"][live]


def _plain_back(s):
    """Blocks of the 4-bit pools written out in the wider type, along the pairs."""
    b, d = s["block"], s["dim"]
    pairs = s["back"].long()
    pairs = pairs[(pairs >= 0).all(1)]
    for pool, dst, kind in ((s["k4"], s["dst_k"], "k"), (s["v4"], s["dst_v"], "v")):
        codes, scales = _split(pool, b, d)
        v = _decode(codes[pairs[:, 0]], scales[pairs[:, 0]], kind)
        dst[pairs[:, 1]] = v.transpose(1, 2).to(dst.dtype)


def _plain_decode(s):
    b, d, hk = s["block"], s["dim"], s["kv_heads"]
    bt, ctx, q = s["bt"].clamp(min=0).long(), s["ctx"].long(), s["q"].float()
    n = q.shape[0]
    q = q.unflatten(1, (hk, -1))
    kc, ks = _split(s["k4"], b, d)
    vc, vs = _split(s["v4"], b, d)
    k = _decode(kc[bt], ks[bt], "k").transpose(1, 2).reshape(n, hk, -1, d)
    x = torch.matmul(q, k.transpose(2, 3)) * s["scale"]
    del k
    seen = torch.arange(x.shape[-1], device=x.device) < ctx[:, None]
    x = torch.where(seen[:, None, None, :], x, torch.full_like(x, -math.inf))
    p = torch.exp(x - x.amax(-1, keepdim=True))
    v = _decode(vc[bt], vs[bt], "v").transpose(1, 2).reshape(n, hk, -1, d)
    v = torch.where(seen[:, None, :, None], v, torch.zeros((), device=v.device))
    o = torch.matmul(p, v) / p.sum(-1, keepdim=True)
    return o.flatten(1, 2).to(s["q"].dtype)


def run(state):
    s, op = state, state["op"]
    if own:
        from pagedattention_kv_cache_reshape_gb300 import pa
        if op == "rope":
            pa.rope_and_cache(s["q"], s["key"], s["value"], s["table"], s["pos"], s["k"], s["v"], s["slot"],
                              interleaved=s["interleaved"], q_out=s["q_out"])
            return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
        if op == "rope_q4":
            pa.rope_and_cache_q4(s["q"], s["key"], s["value"], s["table"], s["pos"], s["k4"], s["v4"], s["slot"],
                                 interleaved=s["interleaved"], q_out=s["q_out"])
            pa.dequantize_blocks_q4(s["k4"], s["v4"], s["dst_k"], s["dst_v"], s["back"])
            return {"q": s["q_out"], "k": s["dst_k"], "v": s["dst_v"]}
        if op == "decode_q4":
            if "ws" not in s:  # a serving loop keeps its workspace
                need = pa.decode_q4_workspace_size(s["q"].shape[0], s["heads"], s["kv_heads"], s["dim"], s["block"],
                                                   s["bt"].shape[1])
                s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
            pa.decode_q4(s["q"], s["k4"], s["v4"], s["bt"], s["ctx"], s["scale"], out=s["out"], workspace=s["ws"])
            return s["out"]
        pa.quantize_blocks_q4(s["src_k"], s["src_v"], s["q4_k"], s["q4_v"], s["there"])
        pa.dequantize_blocks_q4(s["q4_k"], s["q4_v"], s["dst_k"], s["dst_v"], s["back"])
        return {"k": s["dst_k"], "v": s["dst_v"]}
    if op == "decode_q4":
        return _plain_decode(s)
    if op == "convert":
        pairs = s["there"].long()
        pairs = pairs[(pairs >= 0).all(1)]
        for src, pool, kind in ((s["src_k"], s["q4_k"], "k"), (s["src_v"], s["q4_v"], "v")):
            codes, scales = _split(pool, s["block"], s["dim"])
            codes[pairs[:, 1]], scales[pairs[:, 1]] = _encode(src[pairs[:, 0]].transpose(1, 2), kind)
        _plain_back({**s, "k4": s["q4_k"], "v4": s["q4_v"]})
        return {"k": s["dst_k"], "v": s["dst_v"]}
    slot, key, value = _plain_rope(s)
    if op == "rope":
        s["k"].flatten(0, 1)[slot] = key
        s["v"].flatten(0, 1)[slot] = value
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    blk, off = slot // s["block"], slot % s["block"]
    for rows, pool, kind in ((key, s["k4"], "k"), (value, s["v4"], "v")):
        codes, scales = _split(pool, s["block"], s["dim"])
        codes[blk, :, off], scales[blk, :, off] = _encode(rows, kind)
    _plain_back(s)
    return {"q": s["q_out"], "k": s["dst_k"], "v": s["dst_v"]}


# ------------------------------------------------------------------ the definition in 64 bits

def _nearest(x, bits):
    """float64 values rounded to `bits` significant bits, ties to even (normal numbers)."""
    m, e = np.frexp(x)
    return np.ldexp(np.rint(np.ldexp(m, bits)), e - bits)


def _exact_values(rows):
    """What float64 rows [..., D] stand for after the 4-bit form."""
    g = rows.reshape(*rows.shape[:-1], -1, GROUP)
    s = _nearest(np.abs(g).max(-1, keepdims=True) / 7, 8)
    v = np.zeros_like(g)
    np.divide(g, s, out=v, where=s > 0)
    return (np.clip(np.rint(v), -7, 7) * s).reshape(rows.shape)


def _exact_pool(pool, case, kind):
    """Every value of a 4-bit pool in 64 bits, [n, block, heads, D], by index arithmetic on the bytes."""
    b, d, raw = case["block"], case["dim"], pool.cpu().numpy()
    ng = d // GROUP
    dim = np.arange(d)
    g, w = dim // GROUP, dim % GROUP
    nib = ((w // 8) * ng + g) * 8 + w % 8 if kind == "k" else ((w // 4) * ng + g) * 4 + w % 4
    tok = np.arange(b)[:, None]
    byte = raw[:, :, tok * (d // 2) + nib // 2]
    n = (byte >> (4 * (nib % 2)).astype(np.uint8)) & 15
    at = b * d // 2 + 2 * (tok * ng + g)
    bits = (raw[:, :, at].astype(np.uint32) << 16) | (raw[:, :, at + 1].astype(np.uint32) << 24)
    return np.ascontiguousarray(((n.astype(np.float64) - 8) * bits.view(np.float32)).transpose(0, 2, 1, 3))


def exact(case, seed):
    s = prepare(case, seed)
    b, d, hk = case["block"], case["dim"], case["kv_heads"]
    if case["op"] == "decode_q4":
        ctx, bt = s["ctx"].tolist(), s["bt"].long()
        q, out = s["q"].double().unflatten(1, (hk, -1)), []
        order = {k: torch.from_numpy(np.argsort(_dims(k, d, "cpu").numpy())).cuda() for k in "kv"}

        def rows(pool, ids, kind):  # [heads, tokens, D]
            cb = b * d // 2
            p = pool[ids]
            lo, hi = (p[:, :, :cb].long() % 16).double() - 8, (p[:, :, :cb].long() // 16).double() - 8
            v = torch.stack([lo, hi], -1).reshape(ids.numel(), hk, b, d)[..., order[kind]]
            sc = p[:, :, cb:].contiguous().view(torch.bfloat16).double().reshape(ids.numel(), hk, b, -1)
            return (v * sc.repeat_interleave(GROUP, -1)).transpose(0, 1).reshape(hk, -1, d)

        for i, n in enumerate(ctx):
            ids = bt[i, :-(-n // b)]
            w = torch.softmax((q[i] @ rows(s["k4"], ids, "k")[:, :n].transpose(1, 2)) * s["scale"], -1)
            out.append((w @ rows(s["v4"], ids, "v")[:, :n]).flatten(0, 1))
        return torch.stack(out)
    if case["op"] == "convert":
        there, back = s["there"].cpu().numpy(), s["back"].cpu().numpy()
        got = {}
        for name, kind in (("k", "k"), ("v", "v")):
            mid = _exact_pool(s["q4_" + name], case, kind)
            ok = (there >= 0).all(1)
            mid[there[ok, 1]] = _exact_values(s["src_" + name].double().cpu().numpy()[there[ok, 0]])
            dst = np.zeros(tuple(s["dst_" + name].shape))
            ok = (back >= 0).all(1)
            dst[back[ok, 1]] = mid[back[ok, 0]]
            got[name] = dst
        return got
    slot = s["slot"].cpu().numpy()
    live = slot >= 0
    pos, slot = s["pos"].cpu().numpy()[live], slot[live]
    table, r = s["table"].cpu().numpy().astype(np.float64)[pos], case["rot"] // 2
    i = np.arange(r)
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r)

    def turned(x):
        y = x.copy()
        c, t = table[:, None, :r], table[:, None, r:]
        y[..., one] = x[..., one] * c - x[..., two] * t
        y[..., two] = x[..., two] * c + x[..., one] * t
        return y

    q, key, value = (s[n].double().cpu().numpy()[live] for n in ("q", "key", "value"))
    out = np.zeros(tuple(s["q_out"].shape))
    out[live] = turned(q)
    key = turned(key)
    got = {"q": out}
    for name, rows in (("k", key), ("v", value)):
        if case["op"] == "rope":
            pool = np.zeros(tuple(s[name].shape))
            pool.reshape(-1, hk, d)[slot] = rows
        else:
            mid = _exact_pool(s[name + "4"], case, name)
            stored = _nearest(rows, 8 if case["dtype"] == "bf16" else 24)  # the row as the model's type holds it
            mid.reshape(-1, hk, d)[slot] = _exact_values(stored)
            back = s["back"].cpu().numpy()
            pool = np.zeros(tuple(s["dst_" + name].shape))
            pool[back[:, 1]] = mid[back[:, 0]]
        got[name] = pool
    return got
