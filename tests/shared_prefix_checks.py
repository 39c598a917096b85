"""Inputs and the 64-bit check of the shared-prefix decode, used by its GPU tests."""
import numpy as np
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

DEV = "cuda"
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}   # half a step, relative


class Case:
    """A batch in groups: `groups` is [(sequences, shared tokens)], `own` the tokens each sequence has beside them.
    Blocks of the shared tokens are the group's; where they end inside a block, each sequence holds a copy of that
    block's shared part.  Whatever no sequence may read is NaN.  anchor: one more group of 64 sequences over so many
    tokens that the call shares what it can (it shares nothing where all groups together would gain little)."""

    def __init__(self, groups, own, H, Hkv, D, B, dtype, seed=0, prefix=None, spare=3, nan=True, anchor=False):
        self.rows = None
        if anchor:
            first = sum(n for n, _ in groups)
            groups = list(groups) + [(64, -(-max(1300 // Hkv, 320) // B) * B)]
            own = np.concatenate([np.resize(np.asarray(own), first), np.arange(64) % 19 + 1])
            self.rows = list(range(first)) + [first, first + 31, first + 63]
        g = torch.Generator().manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.H, self.Hkv, self.D, self.B, self.dtype, self.groups = H, Hkv, D, B, dtype, groups
        size = np.array([n for n, _ in groups], dtype=np.int64)
        shared = np.repeat([p for _, p in groups], size).astype(np.int64)
        S = int(size.sum())
        own = np.resize(np.asarray(own, dtype=np.int64), S)
        self.S, self.lens = S, (shared + own).tolist()
        nb = -(-(shared + own) // B)
        self.mb = max(1, int(nb.max()) if S else 1)
        total = int(sum(p // B for _, p in groups) + (nb - shared // B).sum()) + spare
        self.nb = total
        ids = rng.permutation(total).astype(np.int32)
        k = torch.randn(total, B, Hkv, D, generator=g)
        v = torch.randn(total, B, Hkv, D, generator=g)
        bt = np.full((S, self.mb), -1, dtype=np.int32)
        used = np.zeros((total, B), dtype=bool)
        at, s = 0, 0
        for n, p in groups:
            whole, rest = p // B, p % B
            mine = ids[at:at + whole]
            at += whole
            used[mine] = True
            first = None
            for _ in range(n):
                bt[s, :whole] = mine
                m = int(nb[s]) - whole
                blocks = ids[at:at + m]
                bt[s, whole:whole + m] = blocks
                at += m
                for i, b in enumerate(blocks):
                    used[b, :min(B, self.lens[s] - (whole + i) * B)] = True
                if rest:
                    if first is None:
                        first = blocks[0]
                    k[blocks[0], :rest], v[blocks[0], :rest] = k[first, :rest], v[first, :rest]
                s += 1
        if nan:
            hole = torch.from_numpy(~used)
            k[hole], v[hole] = float("nan"), float("nan")
        self.k, self.v = k.to(dtype).to(DEV), v.to(dtype).to(DEV)
        self.q = torch.randn(S, H, D, generator=g).to(dtype).to(DEV)
        self.bt = torch.from_numpy(bt).to(DEV)
        self.ctx = torch.tensor(self.lens, dtype=torch.int32, device=DEV)
        self.starts = torch.from_numpy(np.concatenate([[0], np.cumsum(size)]).astype(np.int32)).to(DEV)
        self.prefix = torch.tensor([p for _, p in groups] if prefix is None else prefix, dtype=torch.int32, device=DEV)
        self.scale = float(np.float32(1 / np.sqrt(D)))

    def run(self, **kw):
        a = dict(q=self.q, k_cache=self.k, v_cache=self.v, block_tables=self.bt, context_lens=self.ctx,
                 group_starts=self.starts, prefix_lens=self.prefix, scale=self.scale)
        return pa.decode_shared_prefix(**{**a, **kw})

    def run_checked(self, **kw):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = self.run(dev_status=st, **kw)
        assert pa.get_device_status(st) == pa.OK
        self.check(out, self.rows)
        return out

    def workspace(self, fill=0xFF):
        n = pa.decode_shared_prefix_workspace_size(self.S, self.prefix.numel(), self.H, self.Hkv, self.D, self.B, self.mb)
        return torch.full((n,), fill, dtype=torch.uint8, device=DEV)

    def check(self, out, rows=None):
        """out against the definition in 64 bits.

        Element by element: a logit is a sum of D products in fp32, scaled, its exponential taken by an instruction of
        2^-22, so a weight is off by at most e_w = 2 (D + 8) 2^-24 mag + 2^-21 relative, mag the largest sum of
        |scale q k|; sums of n weights and of n products add n 2^-24; joining pieces adds a few roundings each (at most
        600 pieces).  With bf16 a weight is rounded to bf16 once more, and the result is rounded to its type.
        And the root mean square of all errors: the roundings to bf16 are independent, half a step at most each."""
        half = HALF[self.dtype]
        bf = self.dtype == torch.bfloat16
        sq_err = sq_tol = count = 0.0
        for s in range(self.S) if rows is None else rows:
            n = self.lens[s]
            ids = self.bt[s, :-(-n // self.B)].long()
            G = self.H // self.Hkv
            k, v = (t[ids].reshape(-1, self.Hkv, self.D)[:n].double().transpose(0, 1) for t in (self.k, self.v))
            q = self.q[s].double().view(self.Hkv, G, self.D)
            x = q @ k.transpose(1, 2) * self.scale
            mag = (q.abs() @ k.abs().transpose(1, 2) * abs(self.scale)).amax(-1, keepdim=True)
            w = torch.softmax(x, -1)
            ref, spread, var = w @ v, w @ v.abs(), w.square() @ v.square()
            got = out[s].double().view(self.Hkv, G, self.D)
            e_w = 2 * (self.D + 8) * 2.0 ** -24 * mag + 2.0 ** -21 + (2 * n + 600) * 2.0 ** -24
            tol = 2 * e_w * spread + half * ref.abs() + (half * spread if bf else 0.0) + 1e-30
            err = (got - ref).abs()
            assert bool((err <= tol).all()), f"row {s} ({n} tokens): {float((err / tol).max()):.3g} of the bound"
            sq_err += float(err.square().sum())
            sq_tol += float(((2 * e_w * spread).square() + half ** 2 * (ref.square() + (var if bf else 0))).sum())
            count += err.numel()
        assert sq_err <= sq_tol, f"rms {np.sqrt(sq_err / count):.3g} over {np.sqrt(sq_tol / count):.3g}"
