"""The shared-prefix decode by where its buffers begin, at head sizes and q-heads that the CUDA-core kernels serve in
forms of their own."""
import pytest
import torch

from shared_prefix_checks import DEV, Case
from test_gpu_rope_q4 import _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu


def off(t, elements):
    """A copy of t that begins `elements` elements behind an aligned address."""
    return torch.empty(t.numel() + elements, dtype=t.dtype, device=DEV)[elements:].copy_(t.flatten()).view(t.shape)


# H, Hkv, D, B: up to 8 q-heads a kv-head, and more
HEADS = [(8, 2, 128, 16), (16, 2, 64, 8), (32, 1, 128, 32), (22, 2, 128, 16), (3, 3, 64, 16)]


@pytest.mark.parametrize("elements", [2, 4, 6])
@pytest.mark.parametrize("H,Hkv,D,B", HEADS)
def test_an_output_on_4_bytes_takes_the_same_kernels(H, Hkv, D, B, elements):
    """Bit for bit the result of an output on 16 bytes; the CUDA-core kernels, which round no weight, give another."""
    c = Case([(6, 192), (70, 640), (2, 64), (3, 0)], [5, 40, 20], H, Hkv, D, B, torch.bfloat16, seed=H, anchor=True)
    want, out = c.run(), off(torch.zeros_like(c.q), elements)
    assert torch.equal(c.run(out=out), want)
    c.check(out, [0, 5, 6, 75, 76, 78])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,Hkv,D,B", HEADS)
@pytest.mark.parametrize("what", ["q", "k_cache", "v_cache", "out", "scale -0.3", "scale 0"])
def test_the_other_kernels_at_every_head_size(what, H, Hkv, D, B, dtype):
    """Rows one element off the grid and scales that are not positive: in bf16 they leave the tensor cores."""
    c = Case([(6, 192), (70, 640), (2, 64), (3, 0)], [5, 40, 20, 300], H, Hkv, D, B, dtype, seed=H, anchor=True)
    rows = [0, 3, 5, 6, 75, 76, 78]
    if what.startswith("scale"):
        c.scale = float(what.split()[1])
        c.check(c.run(), rows)
    elif what == "out":
        c.check(c.run(out=off(torch.zeros_like(c.q), 1)), rows)
    else:
        t = {"q": c.q, "k_cache": c.k, "v_cache": c.v}[what]
        c.check(c.run(**{what: off(t, 1)}), rows)
