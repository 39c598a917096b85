"""Calls of different sizes made by several host threads at once, each on a stream and a workspace of its own: none is
refused, and every result is that of the call made alone."""
import threading

import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

from shared_prefix_checks import DEV, Case
from test_gpu_rope_q4 import _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
ROUNDS = 3000


def shared(groups, own, H, Hkv, D, B, dtype=torch.bfloat16):
    c = Case(groups, own, H, Hkv, D, B, dtype, seed=H)
    return c, lambda out, ws, stream: c.run(out=out, workspace=ws, stream=stream), c.workspace()


def plain(S, tokens, H, Hkv, D, B, dtype=torch.bfloat16):
    c = Case([(S, 0)], [tokens], H, Hkv, D, B, dtype, seed=H)
    ws = torch.empty(pa.decode_workspace_size(S, H, Hkv, D, B, c.mb), dtype=torch.uint8, device=DEV)
    return c, lambda out, ws, stream: pa.decode(c.q, c.k, c.v, c.bt, c.ctx, c.scale, out=out, workspace=ws, stream=stream), ws


# each pair shares kernels whose shared memory follows the call's sizes: many sequences and groups or few, many heads or one
PAIRS = {
    "shared": lambda: [shared([(4, 64)] * 2000, [3], 4, 2, 64, 8), shared([(3, 64)], [9], 2, 1, 64, 8)],
    "shared_heads": lambda: [shared([(6, 320)], [40], 32, 8, 128, 16), shared([(6, 320)], [40], 1, 1, 128, 16)],
    "decode": lambda: [plain(15000, 9, 2, 1, 64, 16), plain(3, 40, 2, 1, 64, 16)],
    "decode_heads": lambda: [plain(5, 333, 32, 8, 128, 32), plain(5, 333, 1, 1, 128, 32)],
    "generic": lambda: [plain(5, 33, 32, 1, 128, 16, torch.float32), plain(5, 33, 1, 1, 128, 16, torch.float32)],
}


@pytest.mark.parametrize("name", PAIRS)
def test_two_host_threads(name):
    calls = PAIRS[name]()
    want = []
    for c, call, ws in calls:
        out = torch.zeros_like(c.q)
        call(out, ws, None)
        want.append(out)
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2 * len(calls)), []

    def work(i):
        c, call, ws = calls[i % 2]
        ws, out, stream = ws.clone(), torch.zeros_like(c.q), torch.cuda.Stream()
        torch.cuda.synchronize()
        start.wait()
        try:
            for _ in range(ROUNDS):
                call(out, ws, stream)
        except Exception as e:
            wrong.append(f"{name} {i % 2}: {e}")
        stream.synchronize()
        if not torch.equal(out, want[i % 2]):
            wrong.append(f"{name} {i % 2}: another result")
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2 * len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong, wrong
