"""The bound of one 4-bit decode call against 64 bits, by groups of 32 dims, shared by the range tests."""
import numpy as np
import torch

import q4_reference as R


def check(c, out, what="", exact_q=False):
    """`c` is a test_gpu_decode_q4.Case.  The bound is that of Case.check, with a weight's fp16 step taken against the
    largest scale of V in the dims' own group (exact_q: the queries are given without rounding in the call), and the
    relative 2-norm is taken by group."""
    k, v = R.values(c.k4, "k", c.B, c.D), R.values(c.v4, "v", c.B, c.D)
    z = R.scales(c.v4, c.B, c.D)
    bt, q, o, G, bf16 = c.bt.cpu().numpy(), R.f64(c.q), R.f64(out), c.H // c.Hkv, c.dtype == torch.bfloat16
    for s in range(len(c.ctx)):
        n = int(c.ctx[s])
        ids = bt[s, :-(-n // c.B)]

        def rows(x):
            return x[ids].reshape(-1, c.Hkv, c.D)[:n]
        kr, vr, zr = rows(k), rows(v), np.repeat(rows(z), G, 1)
        ref, mean, mag = R.attention(q[s], kr, vr, c.scale)
        # logits: 16 fp32 steps of a sum of up to 5 times the values' own (codes enter as n), exponent 2^-22
        dx = mag * ((5 if bf16 else 1) * 16 * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -21
        if bf16 and not exact_q:   # what lies under fp16's smallest step of the scaled query
            dx = dx + 2.0 ** -35 * np.abs(q[s]).max(-1) * abs(c.scale) * np.repeat(np.abs(kr).sum(-1).max(0), G)
        rel = 2 * dx[:, None] + (2.0 ** -11 if bf16 else 2.0 ** -24) + 2 * (n / 16 + 16) * 2.0 ** -23
        half = 2.0 ** -8 if bf16 else 2.0 ** -24
        tol = half * np.abs(ref) * (1 + rel) + rel * mean * (1 + half)
        if bf16:
            x = c.scale * np.einsum("hd,nhd->hn", q[s], np.repeat(kr, G, 1))
            w = np.exp(x - x.max(-1, keepdims=True))
            # the surplus of the codes, cut at 2^-24 of sums of 15 w s; and half of fp16's step 2^-24, times |n - 8|,
            # a token, under a largest scale at 2^6 or more
            tol = tol + 2 * 17 * 15 * 2.0 ** -24 * np.einsum("hn,nhd->hd", w / w.sum(-1, keepdims=True), zr)
            tol = tol + n * 8 * 2.0 ** -25 / 2.0 ** 6 * zr.max(0)
        err = np.abs(o[s] - ref)
        assert np.all(np.isfinite(o[s])), f"{what} seq {s}: non-finite"
        assert np.all(err <= tol + 1e-300), f"{what} seq {s} (ctx {n}): {float((err / (tol + 1e-300)).max()):.2f} of the bound"
        if bf16 and n > 1:
            for g in range(c.D // 32):
                d = slice(32 * g, 32 * g + 32)
                e, r = np.linalg.norm(err[:, d]), np.linalg.norm(ref[:, d])
                assert e <= 1e-2 * r, f"{what} seq {s} group {g}: relative RMS {e / max(r, 1e-300):.2e}"
