"""What a shared-prefix decode takes as shared, read from the plan in its workspace: results alone do not show it, as a
batch that shares nothing gives the same.  So that the tests of lengths, group sizes, teams and values are about the
shared kernels, their cases are planned here once more."""
import pytest
import torch

from shared_prefix_checks import Case
from test_gpu_rope_q4 import _lib  # noqa: F401  (builds and loads the library)
from test_gpu_shared_prefix import HEADS

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
ids = dict(ids=lambda v: str(v).replace("torch.", ""))


def planned(c, **kw):
    """Every group's shared tokens: the plan's third array, behind two of one int32 a sequence, each on 256 bytes."""
    ws = c.workspace(0xA5)
    assert ws.data_ptr() % 256 == 0
    c.check(c.run(workspace=ws, **kw), c.rows)
    at = 2 * (-(-4 * c.S // 256) * 256)
    return ws[at:at + 4 * c.prefix.numel()].view(torch.int32).tolist()


def most(c):
    """What may be shared: whole blocks, and no sequence's last token."""
    out, s = [], 0
    for n, p in c.groups:
        out.append(max(0, min(p, min(c.lens[s:s + n]) - 1)) // c.B * c.B if n > 1 else 0)
        s += n
    return out


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", HEADS)
def test_groups_of_all_kinds(H, Hkv, D, B, dtype):
    c = Case([(19, 40 * B), (3, B), (1, 3 * B), (7, 0), (2, 11 * B)], [1, 2, B, B + 1, 130, 17, 63, 64, 65, 300], H, Hkv,
             D, B, dtype, seed=H, anchor=True)
    got, want = planned(c), most(c)
    assert got[0] == want[0] == 40 * B and got[5] == want[5] > 0      # the group of 19, the anchor
    assert got[2] == got[3] == 0                                      # a sequence alone, no prefix
    assert all(g in (0, w) for g, w in zip(got, want))


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", HEADS[:4])
@pytest.mark.parametrize("tokens", [1, 8, 16, 33, 64, 65, 128, 129, 257, 1000])
def test_every_length(tokens, H, Hkv, D, B, dtype):
    """The group of 40 is shared at every length that has a block to share."""
    c = Case([(40, tokens), (5, tokens)], [0, 1, 2, 40, 9] if tokens > 1 else [1], H, Hkv, D, B, dtype, seed=tokens, anchor=True)
    got, want = planned(c), most(c)
    assert got[0] == want[0] == (tokens - 1) // B * B and got[2] == want[2] > 0
    assert got[1] in (0, want[1])


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("n", [1, 2, 4, 16, 17, 33, 64, 127, 130, 257])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (3, 1, 64), (2, 2, 64)])
def test_every_group_size(n, H, Hkv, D, dtype):
    c = Case([(n, 320)], [1, 30, 16, 33], H, Hkv, D, 16, dtype, seed=n, anchor=True)
    assert planned(c) == most(c) and most(c)[0] == (320 if n > 1 else 0)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B,groups,shared", [
    (32, 1, 64, 16, [(17, 800), (3, 320), (9, 640), (60, 480)], [0, 1, 2, 3]),
    (32, 8, 128, 16, [(256, 2048), (64, 512), (32, 256)], [0, 1, 2]),
    (33, 3, 128, 16, [(44, 320), (67, 1600), (132, 48), (5, 3200)], [0, 1, 2, 3]),
    (8, 8, 64, 16, [(1027, 64)], [0]), (32, 32, 128, 16, [(8, 304), (9, 320), (10, 336)] * 4, range(12))])
def test_items_of_all_sizes(H, Hkv, D, B, groups, shared, dtype):
    """Several items a group, teams of them, two kv-heads an item; groups cut anywhere."""
    c = Case(groups, [1, 3, 17], H, Hkv, D, B, dtype, seed=H + D)
    c.rows = [0, c.S // 3, c.S // 2, c.S - 1]
    got, want = planned(c), most(c)
    assert [got[g] for g in shared] == [want[g] for g in shared] and min(want[g] for g in shared) > 0


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("scale", [0.0, -0.3, 30.0, 1e-30])
def test_any_scale(scale, dtype):
    c = Case([(5, 192), (2, 64)], [5, 40, 20], 8, 2, 64, 16, dtype, seed=11, anchor=True)
    c.scale = scale
    got = planned(c)
    assert got[0] == 192 and got[2] == most(c)[2]


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_what_is_shared_by_nobody(dtype):
    """Sequences alone, no prefix, prefixes of less than a block, a prefix no longer than the shortest context allows, and
    a few sequences over short ones, which are quicker read by each for itself."""
    for groups, own in (([(1, 640)], [5]), ([(6, 0)], [700]), ([(6, 15)], [700]), ([(1, 320)] * 4, [9]),
                        ([(4, 16)], [0, 30]), ([(3, 32), (5, 48)], [40])):
        assert planned(Case(groups, own, 8, 2, 128, 16, dtype)) == [0] * len(groups)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_long_prefixes_among_sequences_of_their_own(dtype):
    """A group's length counts, not what stands beside it: half of a batch behind one prefix, the rest behind nothing."""
    c = Case([(40, 2048), (40, 0)], [100, 7, 300], 32, 8, 128, 16, dtype, seed=21)
    c.rows = [0, 39, 40, 79]
    assert planned(c) == [2048, 0]
