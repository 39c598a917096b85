"""Reference of the position rotation and the 4-bit cache rows, in numpy (64 bits; the code of a value by the
format's own fp32 division), sharing nothing with the library."""
import numpy as np
import torch

GROUP = 32


def f64(t):
    return t.detach().cpu().double().numpy()


def slab_bytes(B, D):
    return B * (D // 2 + D // 16)


def new_pool(n, B, H, D, device, fill=None, seed=0):
    """A 4-bit pool: random bytes (every scale an arbitrary bf16, NaN and infinities among them) or one byte."""
    if fill is not None:
        return torch.full((n, H, slab_bytes(B, D)), fill, dtype=torch.uint8, device=device)
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, 256, (n, H, slab_bytes(B, D)), generator=g, dtype=torch.uint8).to(device)


def table(max_pos, rot, base=10000.0):
    r = rot // 2
    ang = np.arange(max_pos)[:, None] * base ** (-np.arange(r) / max(r, 1))
    return torch.from_numpy(np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32))


def rotate(x, cos_sin, pos, rot, interleaved):
    """(rotated rows in 64 bits, sum of the products' magnitudes) of x [n, heads, D]."""
    x = f64(x)
    y, mag = x.copy(), np.abs(x)
    r = rot // 2
    cs = f64(cos_sin)[np.asarray(pos)]
    for i in range(r):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + r)
        c, s = cs[:, None, i], cs[:, None, r + i]
        y[..., a], y[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
        mag[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        mag[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y, mag


def bf16_bits(x32):
    return torch.from_numpy(np.ascontiguousarray(x32)).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)


def quantize(rows):
    """rows [..., D] float32 values -> (nibbles [..., D] of the dims in order, scale bits [..., D/32])."""
    x = np.ascontiguousarray(rows, dtype=np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        amax = np.abs(g).max(-1)
        bits = bf16_bits(amax * (np.float32(1) / np.float32(7)))
        bad = ~np.isfinite(g).all(-1)
        bits = np.where(bad, np.uint16(0x7fc0), bits)
        s = (bits.astype(np.uint32) << 16).view(np.float32)[..., None]
        n = np.clip(np.rint(g / s), -7, 7)
        n = np.where((s > 0) & ~bad[..., None], n, 0)
    return (n + 8).astype(np.uint8).reshape(x.shape), bits


def _nibble(kind, D):
    """Nibble index inside a row of every dim."""
    ng, out = D // GROUP, np.empty(D, dtype=np.int64)
    per = 8 if kind == "k" else 4
    for d in range(D):
        g, w = d // GROUP, d % GROUP
        out[d] = ((w // per) * ng + g) * per + w % per
    return out


def store(pool, kind, blk, head, tok, nib, bits, B, D):
    """Writes one row (nibbles of the dims in order, scale bits) into a uint8 numpy pool."""
    row = np.zeros(D, dtype=np.uint8)
    row[_nibble(kind, D)] = nib
    slab = pool[blk, head]
    slab[tok * D // 2:(tok + 1) * D // 2] = row[0::2] | (row[1::2] << 4)
    at = B * D // 2 + tok * (D // 16)
    slab[at:at + D // 16] = bits.astype("<u2").view(np.uint8)


def values(pool, kind, B, D):
    """All values of a pool [n, heads, slab] as float64 [n, B, heads, D]."""
    raw = pool.cpu().numpy() if torch.is_tensor(pool) else pool
    n, H, _ = raw.shape
    codes = raw[:, :, :B * D // 2].reshape(n, H, B, D // 2)
    nib = np.stack([codes & 15, codes >> 4], -1).reshape(n, H, B, D)[..., _nibble(kind, D)]
    bits = np.ascontiguousarray(raw[:, :, B * D // 2:]).view("<u2").reshape(n, H, B, D // GROUP)
    with np.errstate(all="ignore"):
        s = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
        v = (nib.astype(np.float64) - 8).reshape(n, H, B, D // GROUP, GROUP) * s[..., None]
    return v.reshape(n, H, B, D).transpose(0, 2, 1, 3)


def scales(pool, B, D):
    """The scale of every value of a pool, float64 [n, B, heads, D]."""
    raw = pool.cpu().numpy()
    n, H, _ = raw.shape
    bits = np.ascontiguousarray(raw[:, :, B * D // 2:]).view("<u2").reshape(n, H, B, D // GROUP)
    s = (bits.astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    return np.repeat(s, GROUP, -1).transpose(0, 2, 1, 3)


def attention(q, k, v, scale):
    """q [H, D], k / v [n, Hkv, D] float64 -> (out, sum p |v|, largest sum |scale| |q||k|)."""
    H, D = q.shape
    G = H // k.shape[1]
    kk, vv = np.repeat(k, G, axis=1), np.repeat(v, G, axis=1)
    x = scale * np.einsum("hd,nhd->hn", q, kk)
    mag = abs(scale) * np.einsum("hd,nhd->hn", np.abs(q), np.abs(kk)).max(-1)
    p = np.exp(x - x.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    return np.einsum("hn,nhd->hd", p, vv), np.einsum("hn,nhd->hd", p, np.abs(vv)), mag
