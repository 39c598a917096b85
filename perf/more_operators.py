"""Cases and plain forms of the shared-prefix decode and of the rotary cache writes with several position axes.

    shared    pa.decode_shared_prefix: one query row per sequence; neighbours in the batch form groups whose
              sequences begin with the same blocks, and what all of a group see is computed once for them
    mrope     pa.mrope_and_cache: queries and keys rotated by positions of several axes (time, height, width), K and
              V rows written to the paged pools
    mrope_q4  pa.mrope_and_cache_q4, then pa.dequantize_blocks_q4 of the blocks it wrote, so that the pass returns
              the values which the 4-bit rows stand for

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
        # four samples of one short chat request: the latency of one call
        dict(name="shared_small", op="shared", dtype="bf16", seqs=4, groups=1, alone=0, uneven=False, prefix_lo=512,
             prefix_hi=512, own_lo=1, own_hi=40, law="uniform", heads=32, kv_heads=8, dim=128, block=16),
        # 256 running requests, 64 of them behind one system prompt, power-law contexts
        dict(name="shared_gqa256", op="shared", dtype="bf16", seqs=256, groups=1, alone=192, uneven=False,
             prefix_lo=1024, prefix_hi=1024, own_lo=16, own_hi=4096, law="power", heads=32, kv_heads=8, dim=128,
             block=16),
        # 256 questions about one long document
        dict(name="shared_document", op="shared", dtype="bf16", seqs=256, groups=1, alone=0, uneven=False,
             prefix_lo=32768, prefix_hi=32768, own_lo=32, own_hi=512, law="uniform", heads=32, kv_heads=8, dim=128,
             block=16),
        # 16 requests about one video of 128k tokens
        dict(name="shared_video", op="shared", dtype="bf16", seqs=16, groups=1, alone=0, uneven=False,
             prefix_lo=131072, prefix_hi=131072, own_lo=16, own_hi=300, law="uniform", heads=32, kv_heads=8, dim=128,
             block=16),
        # eight samples of each of 24 prompts, prompts of all lengths, a model without grouped heads
        dict(name="shared_samples", op="shared", dtype="bf16", seqs=192, groups=24, alone=0, uneven=False,
             prefix_lo=256, prefix_hi=4096, own_lo=1, own_hi=256, law="uniform", heads=32, kv_heads=32, dim=128,
             block=16),
        # fp32, small heads in odd groups, blocks of 32, groups of all sizes
        dict(name="shared_f32", op="shared", dtype="f32", seqs=53, groups=4, alone=3, uneven=True, prefix_lo=64,
             prefix_hi=2016, own_lo=1, own_hi=333, law="uniform", heads=14, kv_heads=2, dim=64, block=32),
        # one decode step of 256 running requests: rows of a fused QKV projection, three axes in sections
        dict(name="mrope_decode", op="mrope", dtype="bf16", seqs=256, tokens=256, heads=32, kv_heads=8, dim=128, rot=128,
             axes=3, cycled=False, block=16, interleaved=False, max_pos=4096, pad=0),
        # eight prompts of 1024 tokens, pictures and text, the axes taking turns over the frequencies
        dict(name="mrope_prefill", op="mrope", dtype="bf16", seqs=8, tokens=8192, heads=32, kv_heads=8, dim=128, rot=128,
             axes=3, cycled=True, block=16, interleaved=False, max_pos=4096, pad=0),
        # a ragged fp32 batch with padding rows, half of each head rotated in neighbouring pairs by two axes
        dict(name="mrope_f32_partial", op="mrope", dtype="f32", seqs=7, tokens=1031, heads=12, kv_heads=4, dim=64,
             rot=32, axes=2, cycled=False, block=8, interleaved=True, max_pos=2048, pad=5),
        # the decode step of 256 requests whose cache is held in 4 bits
        dict(name="mrope_q4_decode", op="mrope_q4", dtype="bf16", seqs=256, tokens=256, heads=32, kv_heads=8, dim=128,
             rot=128, axes=3, cycled=False, block=16, interleaved=False, max_pos=4096, pad=0),
        # prompts with pictures prefilled into the 4-bit cache and read back for their attention
        dict(name="mrope_q4_prefill", op="mrope_q4", dtype="bf16", seqs=8, tokens=8191, heads=32, kv_heads=8, dim=128,
             rot=128, axes=3, cycled=False, block=16, interleaved=False, max_pos=4096, pad=1),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["shared", "shared", "shared", "mrope", "mrope_q4"])
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), dim=rng.choice([64, 128]), block=rng.choice([8, 16, 32]))
    if op == "shared":
        g = rng.choice([1, 1, 2, 3, 4, 4, 5, 7, 8, 16, 32])
        c["kv_heads"] = rng.choice([k for k in (1, 2, 4, 5, 8, 16, 32) if g * k <= 32])
        c["heads"] = g * c["kv_heads"]
        c["seqs"] = _log(rng, 1, 256)
        c["groups"] = _log(rng, 1, max(1, c["seqs"] // 2))
        c["alone"] = rng.randint(0, c["seqs"] - c["groups"]) if rng.random() < 0.4 else 0
        c["uneven"] = rng.random() < 0.4
        # bounds: visible (query, key) pairs of all q-heads, and half the cache bytes for prefixes, half for own tokens
        pairs = 100_000_000 if c["dtype"] == "bf16" else 20_000_000
        kept = 550_000_000 // (2 * c["kv_heads"] * c["dim"] * ESIZE[c["dtype"]])
        most = min(100_000, pairs // (c["heads"] * c["seqs"]), kept // c["groups"])
        most = max(c["block"], most // c["block"] * c["block"])
        c["prefix_hi"] = max(1, _log(rng, c["block"], most) // c["block"]) * c["block"]
        c["prefix_lo"] = max(1, _log(rng, c["block"], c["prefix_hi"]) // c["block"]) * c["block"]
        c["own_hi"] = _log(rng, 1, max(1, min(4096, kept // c["seqs"], pairs // (2 * c["heads"] * c["seqs"]))))
        c["own_lo"] = _log(rng, 1, c["own_hi"])
        c["law"] = rng.choice(["uniform", "power"])
        return c
    g = rng.choice([1, 2, 4, 4, 7, 8])
    c["kv_heads"] = max(1, min(8, 32 // g))
    c["heads"] = g * c["kv_heads"]
    half = c["dim"] // 2
    c["rot"] = rng.choice([c["dim"], c["dim"], half, half + 8 * rng.randint(0, 4), 2 * rng.randint(4, half)])
    c["axes"] = rng.choice([1, 2, 3, 3, 4])
    c["cycled"] = rng.random() < 0.5
    c["interleaved"] = rng.random() < 0.4
    c["pad"] = rng.choice([0, 0, 1, 9])
    c["tokens"] = _log(rng, 1, 8000 if c["dtype"] == "bf16" else 3900)
    c["seqs"] = max(1, min(c["tokens"], _log(rng, 1, 300)))
    c["max_pos"] = max(_log(rng, 512, 65536), 2 * (c["tokens"] // c["seqs"] + 2 + c["block"]))
    return c


def _quantiles(n, lo, hi, law):
    u = (np.arange(n) + 0.5) / max(n, 1)
    x = (lo ** -0.2 + u * (hi ** -0.2 - lo ** -0.2)) ** -5.0 if law == "power" else lo + u * (hi + 1 - lo)
    return np.clip(np.floor(x), lo, hi).astype(np.int64)


def _groups(case):
    """(sequences, prefix tokens) of every group, the ones that share nothing as a last group without a prefix."""
    n, m = case["groups"], case["seqs"] - case["alone"]
    w = 1.0 / np.arange(1, n + 1) if case["uneven"] else np.ones(n)
    size = 1 + np.floor((m - n) * w / w.sum()).astype(np.int64)
    size[:m - int(size.sum())] += 1
    prefix = _quantiles(n, case["prefix_lo"], case["prefix_hi"], "uniform") // case["block"] * case["block"]
    out = list(zip(size.tolist(), prefix.tolist()))
    return out + ([(case["alone"], 0)] if case["alone"] else [])


def _own(case):
    """The multiset of the sequences' own tokens (the seed only orders them)."""
    return _quantiles(case["seqs"], case["own_lo"], case["own_hi"], case["law"])


def _seq_tokens(case):
    n, s = case["tokens"], case["seqs"]
    return np.array([n // s + (1 if i < n % s else 0) for i in range(s)], dtype=np.int64)


def _blocks_written(case):
    b = case["block"]
    return int(sum(-(-(int(n) + 7 * i % b) // b) for i, n in enumerate(_seq_tokens(case))))


def work(case):
    e, d, h, hk = ESIZE[case["dtype"]], case["dim"], case["heads"], case["kv_heads"]
    if case["op"] == "shared":
        kept = float(sum(p for _, p in _groups(case)) + _own(case).sum())
        seen = float(sum(n * p for n, p in _groups(case)) + _own(case).sum())
        return {"bytes": kept * 2 * hk * d * e + 2.0 * case["seqs"] * h * d * e + 4 * kept / case["block"],
                "flops": 4 * seen * h * d}
    n = case["tokens"]
    table = min(n * case["axes"], case["max_pos"]) * case["rot"] * 4 + (8 + 4 * case["axes"]) * n
    if case["op"] == "mrope":
        return {"bytes": 2.0 * n * (h + 2 * hk) * d * e + table, "flops": 3.0 * n * (h + hk) * case["rot"]}
    q4 = d * 9 / 16
    return {"bytes": n * (2.0 * h + 2 * hk) * d * e + 2 * n * hk * q4 + table
            + 2.0 * _blocks_written(case) * case["block"] * hk * (q4 + d * e),
            "flops": 3.0 * n * (h + hk) * case["rot"] + 4.0 * n * hk * d}


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
    s = (x.abs().amax(-1) * torch.tensor(1 / 7, dtype=torch.float32, device=x.device)).to(torch.bfloat16)
    sf = s.float()[..., None]
    n = torch.where(sf > 0, torch.round(x / sf).clamp(-7, 7), torch.zeros_like(x)) + 8
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
    codes[:], scales[:] = _encode(torch.randn(n, h, b, d, generator=gen, device="cuda"), kind)
    return pool


# ------------------------------------------------------------------ inputs

def _prepare_shared(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    dt, b, hk, d = DTYPES[case["dtype"]], case["block"], case["kv_heads"], case["dim"]
    groups, own = _groups(case), rng.permutation(_own(case))
    size = np.array([n for n, _ in groups])
    prefix = np.array([p for _, p in groups])
    seq_prefix = np.repeat(prefix, size)
    ctx = seq_prefix + own
    nb_own = -(-own // b)
    total = int(prefix.sum() // b + nb_own.sum()) + 3
    ids = rng.permutation(total).astype(np.int32)
    bt = np.full((ctx.size, int((seq_prefix // b + nb_own).max())), -1, dtype=np.int32)
    at, i = 0, 0
    for n, p in groups:  # a group's blocks, then each of its sequences' own
        for j in range(i, i + n):
            bt[j, :p // b] = ids[at:at + p // b]
        at, first, i = at + p // b, i, i + n
        for j in range(first, i):
            bt[j, p // b:p // b + nb_own[j]] = ids[at:at + nb_own[j]]
            at += int(nb_own[j])
    s = dict(case)
    s["bt"], s["ctx"] = torch.from_numpy(bt).cuda(), torch.from_numpy(ctx.astype(np.int32)).cuda()
    s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(size)]).astype(np.int32)).cuda()
    s["prefix"] = torch.from_numpy(prefix.astype(np.int32)).cuda()
    s["plan"] = [(int(n), int(p)) for n, p in groups]  # the same on the host, for the plain form's loop
    s["longest"] = int(own.max())
    s["q"] = torch.randn(ctx.size, case["heads"], d, generator=gen, device="cuda").to(dt)
    s["k"], s["v"] = (torch.empty(total, b, hk, d, dtype=dt, device="cuda") for _ in "kv")
    step = max(1, (1 << 27) // (b * hk * d))
    for i in range(0, total, step):
        m = min(step, total - i)
        key = torch.randn(m, b, hk, d, generator=gen, device="cuda")
        key[..., 5::37] *= 4  # a few channels of the keys are large, as those of real models are
        s["k"][i:i + m] = key.to(dt)
        s["v"][i:i + m] = torch.randn(m, b, hk, d, generator=gen, device="cuda").to(dt)
    s["out"] = torch.empty_like(s["q"])
    s["scale"] = float(np.float32(1 / math.sqrt(d)))
    return s


def _pair_axis(case):
    """The axis whose position turns each pair: in sections (the first shorter), or taking turns."""
    r, a = case["rot"] // 2, case["axes"]
    i = np.arange(r)
    if case["cycled"]:
        return np.where(i < r // a * a, i % a, 0)
    first = r if a == 1 else max(1, r // (a + 1))
    rest = max(1, -(-(r - first) // max(1, a - 1)))
    return np.where(i < first, 0, np.minimum(a - 1, 1 + (i - first) // rest)) if a > 1 else np.zeros(r, dtype=np.int64)


def _axis_positions(start, n, axes, rng):
    """Positions [axes, n] of n tokens from `start` on: runs of text (all axes alike) and pictures, whose tokens share
    a time and lie on a grid; what follows a picture goes on behind its largest position."""
    pos, at, p = np.zeros((axes, n), dtype=np.int64), 0, start
    while at < n:
        m = min(n - at, int(rng.integers(1, 65)))
        pos[:, at:at + m] = p + np.arange(m)
        at, p = at + m, p + m
        if at == n:
            break
        h, w = int(rng.integers(2, 17)), int(rng.integers(2, 17))
        m = min(n - at, h * w)
        i = np.arange(m)
        grid = [np.zeros(m, dtype=np.int64), i // w, i % w, i % 2]
        for a in range(axes):
            pos[a, at:at + m] = p + grid[a]
        at, p = at + m, p + int(max(pos[:, at:at + m].max() - p + 1, 1))
    return pos


def prepare(case, seed):
    if case["op"] == "shared":
        return _prepare_shared(case, seed)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    rng = np.random.default_rng(int(seed))
    dt = DTYPES[case["dtype"]]
    s = dict(case)
    b, h, hk, d = case["block"], case["heads"], case["kv_heads"], case["dim"]
    # a batch of `seqs` sequences with their new tokens in consecutive slots, padding rows behind them
    lens, pad = _seq_tokens(case), case["pad"]
    n = case["tokens"] + pad
    phase = 7 * np.arange(lens.size) % b  # where in a block each sequence goes on: by the case, not by the seed
    start = b * rng.integers(0, (case["max_pos"] - lens - phase) // b + 1) + phase
    where = np.repeat(phase, lens) + np.concatenate([np.arange(m) for m in lens])
    nb = (phase + lens - 1) // b + 1
    base = np.concatenate([[0], np.cumsum(nb)])
    total = int(base[-1]) + 5
    ids = rng.permutation(total)
    slot = ids[np.repeat(base[:-1], lens) + where // b] * b + where % b
    pos = np.concatenate([_axis_positions(int(p), int(m), case["axes"], rng) for p, m in zip(start, lens)]
                         + [np.full((case["axes"], pad), -1)], 1)
    s["pos"] = torch.from_numpy(pos.astype(np.int32)).cuda()
    s["axis"] = torch.from_numpy(_pair_axis(case).astype(np.int32)).cuda()
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
    if case["op"] == "mrope":
        s["k"], s["v"] = (torch.zeros(total, b, hk, d, dtype=dt, device="cuda") for _ in "kv")
        return s
    s["k4"], s["v4"] = _random_pool(total, case, "k", gen), _random_pool(total, case, "v", gen)
    touched = ids[:int(base[-1])]
    s["back"] = torch.from_numpy(np.stack([touched, np.arange(touched.size)], 1).astype(np.int32)).cuda()
    s["dst_k"], s["dst_v"] = (torch.zeros(touched.size, b, hk, d, dtype=dt, device="cuda") for _ in "kv")
    return s


# ------------------------------------------------------------------ plain forms

def _plain_shared(s):
    """Group by group: the prefix's logits for all rows at once, every sequence's own behind them."""
    b, d, hk, scale = s["block"], s["dim"], s["kv_heads"], s["scale"]
    q = s["q"].float().unflatten(1, (hk, -1))  # [seqs, kv-heads, q-heads of one, D]
    g = q.shape[2]
    out = torch.empty_like(q)
    rows = max(1, (1 << 28) // (s["longest"] * hk * max(d, g)))
    i = 0
    for n, p in s["plan"]:
        ids = s["bt"][i, :p // b].long()
        pk, pv = (s[x][ids].flatten(0, 1).float().transpose(0, 1) for x in "kv")  # [kv-heads, p, D]
        for j in range(i, i + n, rows):
            m = min(rows, i + n - j)
            qq = q[j:j + m]
            shared = torch.matmul(qq.transpose(0, 1).flatten(1, 2), pk.transpose(1, 2)) * scale
            shared = shared.unflatten(1, (m, g)).transpose(0, 1)  # [m, kv-heads, q-heads of one, p]
            ids = s["bt"][j:j + m, p // b:].clamp(min=0).long()[:, :-(-s["longest"] // b)]
            k, v = (s[x][ids].flatten(1, 2).float().transpose(1, 2) for x in "kv")
            seen = p + torch.arange(k.shape[2], device=k.device) < s["ctx"][j:j + m, None]
            x = torch.matmul(qq, k.transpose(2, 3)) * scale
            x = torch.where(seen[:, None, None, :], x, torch.full_like(x, -math.inf))
            v = torch.where(seen[:, None, :, None], v, torch.zeros((), device=v.device))
            top = x.amax(-1, keepdim=True)
            if p:
                top = torch.maximum(top, shared.amax(-1, keepdim=True))
            w, ws = torch.exp(x - top), torch.exp(shared - top)
            o = torch.matmul(w, v)
            o = o + torch.matmul(ws.transpose(0, 1).flatten(1, 2), pv).unflatten(1, (m, g)).transpose(0, 1)
            out[j:j + m] = o / (w.sum(-1, keepdim=True) + ws.sum(-1, keepdim=True))
        i += n
    return out.flatten(1, 2).to(s["q"].dtype)


def _rotated(x, s, pos):
    """x [tokens, heads, D] rotated by positions [axes, tokens], in 64 bits, rounded once to its type."""
    rot, r = s["rot"], s["rot"] // 2
    pair = torch.arange(r, device=x.device)
    p = pos[s["axis"].long()].T  # [tokens, pairs]
    c, t = s["table"][p, pair].double()[:, None], s["table"][p, r + pair].double()[:, None]
    y = x.double()
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if s["interleaved"] else (y[..., :r], y[..., r:rot])
    a, b = a * c - b * t, b * c + a * t
    front = torch.stack([a, b], -1).flatten(-2) if s["interleaved"] else torch.cat([a, b], -1)
    return torch.cat([front, y[..., rot:]], -1).float().to(x.dtype)


def _plain_mrope(s):
    live = torch.nonzero(s["slot"] >= 0).flatten()
    pos, slot = s["pos"][:, live].long(), s["slot"][live]
    s["q_out"][live] = _rotated(s["q"][live], s, pos)
    key, value = _rotated(s["key"][live], s, pos), s["value"][live]
    if s["op"] == "mrope":
        s["k"].flatten(0, 1)[slot] = key
        s["v"].flatten(0, 1)[slot] = value
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    b, d = s["block"], s["dim"]
    blk, off = slot // b, slot % b
    pairs = s["back"].long()
    for rows, pool, dst, kind in ((key, s["k4"], s["dst_k"], "k"), (value, s["v4"], s["dst_v"], "v")):
        codes, scales = _split(pool, b, d)
        codes[blk, :, off], scales[blk, :, off] = _encode(rows, kind)
        wide = _decode(codes[pairs[:, 0]], scales[pairs[:, 0]], kind)
        dst[pairs[:, 1]] = wide.transpose(1, 2).to(dst.dtype)
    return {"q": s["q_out"], "k": s["dst_k"], "v": s["dst_v"]}


def run(state):
    s, op = state, state["op"]
    if not own:
        return _plain_shared(s) if op == "shared" else _plain_mrope(s)
    from pagedattention_kv_cache_reshape_gb300 import pa
    if op == "shared":
        if "ws" not in s:  # a serving loop keeps its workspace
            need = pa.decode_shared_prefix_workspace_size(s["q"].shape[0], s["prefix"].shape[0], s["heads"],
                                                          s["kv_heads"], s["dim"], s["block"], s["bt"].shape[1])
            s["ws"] = torch.empty(need, dtype=torch.uint8, device="cuda")
        pa.decode_shared_prefix(s["q"], s["k"], s["v"], s["bt"], s["ctx"], s["starts"], s["prefix"], s["scale"],
                                out=s["out"], workspace=s["ws"])
        return s["out"]
    if op == "mrope":
        pa.mrope_and_cache(s["q"], s["key"], s["value"], s["table"], s["pos"], s["axis"], s["k"], s["v"], s["slot"],
                           interleaved=s["interleaved"], q_out=s["q_out"])
        return {"q": s["q_out"], "k": s["k"], "v": s["v"]}
    pa.mrope_and_cache_q4(s["q"], s["key"], s["value"], s["table"], s["pos"], s["axis"], s["k4"], s["v4"], s["slot"],
                          interleaved=s["interleaved"], q_out=s["q_out"])
    pa.dequantize_blocks_q4(s["k4"], s["v4"], s["dst_k"], s["dst_v"], s["back"])
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
    if case["op"] == "shared":
        # sequence by sequence over its own table, whatever it shares
        out = []
        for i, n in enumerate(s["ctx"].tolist()):
            ids = s["bt"][i, :-(-n // b)].long()
            k, v = (s[x][ids].reshape(-1, hk, d)[:n].double().transpose(0, 1) for x in "kv")
            q = s["q"][i].double().unflatten(0, (hk, -1))
            w = torch.softmax((q @ k.transpose(1, 2)) * s["scale"], -1)
            out.append((w @ v).flatten(0, 1))
        return torch.stack(out)
    slot = s["slot"].cpu().numpy()
    live = slot >= 0
    pos, slot = s["pos"].cpu().numpy()[:, live], slot[live]
    r, i = case["rot"] // 2, np.arange(case["rot"] // 2)
    table, axis = s["table"].cpu().numpy().astype(np.float64), s["axis"].cpu().numpy()
    one, two = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r)
    c, t = np.zeros((slot.size, 1, r)), np.zeros((slot.size, 1, r))
    for j in range(r):
        c[:, 0, j], t[:, 0, j] = table[pos[axis[j]], j], table[pos[axis[j]], r + j]

    def turned(x):
        y = x.copy()
        y[..., one] = x[..., one] * c - x[..., two] * t
        y[..., two] = x[..., two] * c + x[..., one] * t
        return y

    q, key, value = (s[n].double().cpu().numpy()[live] for n in ("q", "key", "value"))
    out = np.zeros(tuple(s["q_out"].shape))
    out[live] = turned(q)
    got = {"q": out}
    for name, rows in (("k", turned(key)), ("v", value)):
        if case["op"] == "mrope":
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
