"""The shared-prefix decode against its definition in 64 bits, at the sizes and groupings where it can go wrong."""
import numpy as np
import pytest
import torch

from pagedattention_kv_cache_reshape_gb300 import pa

import q4_reference as R
from shared_prefix_checks import DEV, Case
from test_gpu_rope_q4 import _lib  # noqa: F401  (builds and loads the library)

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float32]
ids = dict(ids=lambda v: str(v).replace("torch.", ""))

# H, Hkv, D, B
HEADS = [(32, 8, 128, 16), (14, 2, 64, 32), (4, 4, 128, 8), (16, 1, 64, 16), (32, 1, 128, 32), (5, 5, 64, 8),
         (6, 2, 128, 16), (33, 3, 64, 16), (62, 2, 128, 8)]


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", HEADS)
def test_groups_of_all_kinds(H, Hkv, D, B, dtype):
    """A long prefix for many, a short one, a single sequence, none shared, a pair; own parts from one token on."""
    groups = [(19, 40 * B), (3, B), (1, 3 * B), (7, 0), (2, 11 * B)]
    Case(groups, [1, 2, B, B + 1, 130, 17, 63, 64, 65, 300], H, Hkv, D, B, dtype, seed=H, anchor=True).run_checked()
    Case(groups, [1, 2, B, B + 1, 130, 17, 63, 64, 65, 300], H, Hkv, D, B, dtype, seed=H).run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", HEADS[:4])
@pytest.mark.parametrize("tokens", [1, 7, 8, 15, 16, 31, 32, 63, 64, 65, 127, 128, 129, 200, 256, 257, 1000])
def test_every_length(tokens, H, Hkv, D, B, dtype):
    """Shared lengths of any kind: only whole blocks, and no sequence's last token, are computed once.  (So many sequences
    that sharing pays at every length.)"""
    own = [0, 1, 2, 40, 9] if tokens > 1 else [1]
    Case([(40, tokens), (5, tokens)], own, H, Hkv, D, B, dtype, seed=tokens, anchor=True).run_checked()
    Case([(5, tokens)], [0, 1, 2, 40, 9] if tokens > 1 else [1], H, Hkv, D, B, dtype, seed=tokens).run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("n", [1, 2, 3, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 130, 257])
@pytest.mark.parametrize("H,Hkv,D", [(8, 2, 128), (3, 1, 64), (2, 2, 64)])
def test_every_group_size(n, H, Hkv, D, dtype):
    Case([(n, 320)], [1, 30, 16, 33], H, Hkv, D, 16, dtype, seed=n, anchor=True).run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_one_sequence_one_token(dtype):
    for groups, own in (([(1, 0)], [1]), ([(1, 16)], [0]), ([(2, 0)], [1]), ([(2, 1)], [0]), ([(4, 16)], [1])):
        Case(groups, own, 8, 2, 128, 16, dtype).run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("S,NG", [(300, 1), (2000, 700), (9000, 4500)])
def test_many_sequences_and_groups(S, NG, dtype):
    """Up to more groups than the plan keeps in shared memory."""
    rng = np.random.default_rng(S)
    cuts = np.sort(rng.integers(0, S + 1, NG - 1))             # empty groups among them
    size = np.diff(np.concatenate([[0], cuts, [S]]))
    groups = [(int(n), int(p)) for n, p in zip(size, rng.integers(0, 9, NG) * 8)]
    c = Case(groups, rng.integers(1, 20, S), 4, 2, 64, 8, dtype, seed=1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.run(dev_status=st)
    assert pa.get_device_status(st) == pa.OK
    c.check(out, rows=sorted(set(rng.integers(0, S, 200).tolist()) | {0, S - 1}))


@pytest.mark.parametrize("H,Hkv,D,B,groups", [
    (32, 1, 64, 16, [(17, 800), (3, 320), (9, 640), (60, 480)]),      # 5, 1, 3 and 15 items a kv-head
    (32, 8, 128, 16, [(64 * 4, 2048), (64, 512), (32, 256)]), (32, 8, 128, 32, [(64 * 2 + 1, 1024), (64 * 3, 640), (2, 64)]),
    (16, 4, 64, 8, [(64 * 7 + 40, 400)]), (33, 3, 128, 16, [(22 * 2, 320), (22 * 3 + 1, 1600), (22 * 6, 48), (5, 3200)]),
    (8, 8, 64, 16, [(256 * 4 + 3, 64)])])
def test_teams(H, Hkv, D, B, groups):
    """Groups of several items a kv-head, which teams of CTAs share, beside others that fill no team."""
    Case(groups, [1, 3, 17], H, Hkv, D, B, torch.bfloat16, seed=H + D).run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B,n,step", [(32, 32, 128, 16, 8, 16), (32, 32, 64, 8, 3, 8), (32, 8, 128, 32, 40, 64),
                                              (15, 15, 128, 8, 5, 24), (32, 1, 64, 16, 3, 208), (16, 4, 64, 16, 70, 48)])
def test_many_pieces(H, Hkv, D, B, n, step, dtype):
    """Groups of all lengths whose items are cut anywhere: many pieces a CTA, of all kinds, again and again."""
    c = Case([(n + i % 3, 300 // B * B + step * i) for i in range(12)], [1, 30, 7, 100], H, Hkv, D, B, dtype, seed=n)
    want = c.run_checked()
    for _ in range(20):
        assert torch.equal(c.run(), want)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("H,Hkv,D,B", [(32, 8, 128, 16), (14, 2, 64, 32), (6, 6, 64, 8)])
def test_a_key_that_stands_out_is_found(H, Hkv, D, B, dtype):
    """One key after another, at the ends of blocks, tiles and parts, holds nearly all the weight of every row."""
    P, own = 16 * B + 2 * B, 2 * B + 3
    c = Case([(3, P), (2, 5 * B)], [own], H, Hkv, D, B, dtype, seed=5, anchor=True)
    c.q = torch.ones_like(c.q)
    c.k = torch.where(torch.isnan(c.k), c.k, 0.01 * c.k)
    plain = c.k.clone()
    places = sorted({0, 1, 63, 64, 65, 127, 128, 129, P - 1, P, P + 1, P + B - 1, P + B, P + own - 1, 255, 256, 2 * B - 1})
    for t in [t for t in places if t < P + own]:
        c.k.copy_(plain)
        blk = c.bt[:3, t // B].long()
        c.k[blk, t % B] = 4.0
        out = c.run()
        c.check(out, c.rows)
        want = c.v[blk, t % B].float().repeat_interleave(H // Hkv, 1)
        w = float(np.exp(-3.9 * np.sqrt(D)))                  # the other keys' weight, each, at most
        err = (out[:3].float() - want).abs()
        assert float((err / (want.abs() * 2.0 ** -7 + 16 * (P + own) * w + 1e-5)).max()) <= 1, t


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_lengths_that_do_not_go_together(dtype):
    """A prefix length beyond some sequence's context, or short of what is shared: never a wrong result."""
    for prefix in ([500, 48], [64, 40], [4096, 4096], [1, 0], [63, 65]):
        c = Case([(6, 64), (4, 48)], [1, 5, 40, 0], 8, 2, 128, 16, dtype, seed=3, anchor=True)
        c.bt = torch.cat([c.bt, torch.full((c.S, 256), -1, dtype=torch.int32, device=DEV)], 1).contiguous()
        c.prefix[:2] = torch.tensor(prefix, dtype=torch.int32)
        # tokens 64.. of the first group differ by sequence: they may only be called shared where none has them
        c.prefix[:2].clamp_(max=64)
        c.run_checked()
    c = Case([(5, 96)], [0], 8, 2, 128, 16, dtype, seed=4)        # everything shared, contexts alike
    c.prefix.fill_(96)
    c.run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("starts", [[0, 3, 2, 9], [1, 3, 5, 9], [0, 3, 5, 8], [0, 3, 5, 10], [0, -1, 5, 9],
                                    [0, 2 ** 31 - 1, 5, 9], [0, 9, 9, 8]])
def test_starts_out_of_order_share_nothing(starts, dtype):
    c = Case([(3, 64), (2, 32), (4, 160)], [5, 40], 8, 2, 128, 16, dtype, seed=6)
    c.starts.copy_(torch.tensor(starts))
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.run(dev_status=st)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    c.check(out)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31])
def test_a_prefix_length_out_of_range_shares_nothing(bad, dtype):
    c = Case([(3, 64), (2, 32), (4, 160)], [5, 40], 8, 2, 128, 16, dtype, seed=7)
    c.prefix[1] = bad
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = c.run(dev_status=st)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    c.check(out)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("bad", [0, -5, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_a_context_out_of_range_leaves_its_row(bad, dtype):
    c = Case([(4, 64), (2, 32)], [5, 40, 1], 8, 2, 128, 16, dtype, seed=8, anchor=True)
    rows = [0, 5]
    c.ctx[rows] = bad
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = torch.full_like(c.q, 7.0)
    c.run(dev_status=st, out=out)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    assert torch.all(out[rows] == 7.0)
    c.check(out, rows=[1, 2, 3, 4])
    c.ctx.fill_(bad)                                              # none is in range
    out.fill_(7.0)
    c.run(out=out)
    assert torch.all(out == 7.0)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_table_entries_are_reported(bad, dtype):
    """In the shared part, and in one sequence's own: other groups, and other sequences, keep their results."""
    c = Case([(4, 64), (3, 160)], [5, 40, 20], 8, 2, 128, 16, dtype, seed=9, anchor=True)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    c.bt[0, 2] = bad
    c.run(dev_status=st)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    c.check(c.run(), rows=[4, 5, 6])
    c = Case([(4, 64), (3, 160)], [5, 40, 20], 8, 2, 128, 16, dtype, seed=9, anchor=True)
    c.bt[1, 5] = bad
    st.zero_()
    out = c.run(dev_status=st)
    assert pa.get_device_status(st) == pa.ERR_OUT_OF_RANGE
    c.check(out, rows=[0, 2, 3, 4, 5, 6])


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_nan_and_infinities_stay_in_their_rows(dtype):
    c = Case([(6, 320), (3, 0)], [5, 40, 20], 8, 2, 128, 16, dtype, seed=10, anchor=True)
    q = c.q.clone()
    q[2, 3, 7] = float("nan")
    q[4, 0] = float("inf")
    out = c.run(q=q)
    assert torch.isnan(out[2, 3]).all() and torch.isnan(out[4, 0]).all()
    keep = torch.ones(c.S, 8, dtype=torch.bool, device=DEV)
    keep[2, 3] = keep[4, 0] = False
    want = c.run()
    assert torch.equal(out[keep], want[keep])
    # a NaN among the shared values reaches every row of its kv-head, one of a sequence's own only that sequence
    k, v = c.k.clone(), c.v.clone()
    v[c.bt[0, 3].long(), 2, 1, 9] = float("nan")
    k[c.bt[7, 0].long(), 1, 0, 3] = float("nan")
    out = c.run(k_cache=k, v_cache=v)
    bad = torch.isnan(out)
    assert bad[:6, 4:, 9].all() and bad[7, :4].all() and int(bad.sum()) == 6 * 4 + 4 * 128


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("scale", [0.0, -0.3, 30.0, 1e-30])
def test_any_scale(scale, dtype):
    """Equal weights, the smallest logits on top, one key alone on top."""
    c = Case([(5, 192), (2, 64)], [5, 40, 20], 8, 2, 64, 16, dtype, seed=11, anchor=True)
    c.scale = scale
    c.run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_logits_that_grow_along_the_keys(dtype):
    """Every tile has a new largest logit, so all that was summed before is scaled down."""
    c = Case([(70, 1024)], [200, 3], 8, 2, 128, 16, dtype, seed=12)
    for s in range(c.S):
        n = c.lens[s]
        t = torch.arange(n, device=DEV)
        blk = c.bt[s].long()[t // 16]
        for h in range(2):
            c.k[blk, t % 16, h] = (torch.ones(n, 128, device=DEV) * (t / n * 12)[:, None]).to(dtype)
    c.q = torch.ones_like(c.q) * torch.linspace(0.1, 1, c.H, device=DEV)[None, :, None].to(dtype)
    c.run_checked()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_results_do_not_depend_on_blocks_workspace_or_run(dtype):
    c = Case([(20, 640), (5, 0), (9, 96)], [5, 40, 200], 32, 8, 128, 16, dtype, seed=13, anchor=True)
    want = c.run()
    ws = c.workspace()
    for _ in range(3):
        assert torch.equal(c.run(workspace=ws), want)
    perm = torch.randperm(c.nb, device=DEV)
    k, v = torch.empty_like(c.k), torch.empty_like(c.v)
    k[perm], v[perm] = c.k, c.v
    bt = torch.where(c.bt >= 0, perm[c.bt.clamp(min=0).long()].int(), c.bt)
    assert torch.equal(c.run(k_cache=k, v_cache=v, block_tables=bt), want)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_rows_that_start_anywhere(dtype):
    """q, out and the pools one element off the 16-byte grid."""
    c = Case([(6, 192), (2, 64)], [5, 40, 20], 8, 2, 64, 16, dtype, seed=14, anchor=True)
    want = c.run_checked()

    def off(t):
        flat = torch.empty(t.numel() + 1, dtype=t.dtype, device=DEV)[1:]
        return flat.copy_(t.flatten()).view(t.shape)
    for name, t in (("q", c.q), ("k_cache", c.k), ("v_cache", c.v)):
        c.check(c.run(**{name: off(t)}), c.rows)
    out = off(torch.zeros_like(c.q))
    c.check(c.run(out=out), c.rows)
    assert out.data_ptr() % 16 and want.shape == out.shape


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_two_calls_at_once(dtype):
    """On two streams, each with a workspace and an output of its own, several calls in flight on both."""
    cases = [Case([(20, 640), (5, 0), (9, 96)], [5, 40, 200], 32, 8, 128, 16, dtype, seed=19),
             Case([(70, 1024), (3, 64)], [200, 3], 8, 2, 128, 16, dtype, seed=20)]
    want = [c.run() for c in cases]
    ws, out = [c.workspace() for c in cases], [[torch.zeros_like(c.q) for _ in range(8)] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(8):
        for j, c in enumerate(cases):
            c.run(out=out[j][i], workspace=ws[j], stream=streams[j])
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[j]) for j in range(2) for o in out[j])


@pytest.mark.parametrize("sequences", [129, 176, 257, 300, 385, 512])
@pytest.mark.parametrize("own", [1, 300, 2000])
def test_teams_whose_part_is_little_work(sequences, own):
    """A group of several items, which take a team of as many CTAs, beside so much other work that the team's own
    share of the SMs would be less than one CTA each."""
    groups = [(40, 0), (2, 90), (sequences, 83), (1, 2040), (9, 35)]
    c = Case(groups, [own, 32, 32, 1, 2, own], 2, 1, 64, 32, torch.bfloat16, seed=sequences)
    c.rows = [0, 41, 42, 43, 44, 42 + 127, 42 + 128, 42 + sequences - 1, c.S - 1]
    for ws in (c.workspace(0xFF), c.workspace(0)):
        c.run_checked(workspace=ws)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
@pytest.mark.parametrize("prefix", [0, 2048])
def test_what_comes_behind_a_call_sees_its_rows(prefix, dtype):
    """The next operation on the stream starts when all rows are written, whether or not anything was shared."""
    c = Case([(7, prefix), (3, 0)], [30000, 3, 9000], 8, 2, 128, 16, dtype, seed=18)
    want, seen = c.run(), []
    torch.cuda.synchronize()
    for _ in range(5):
        out = torch.zeros_like(c.q)
        torch.cuda.synchronize()
        seen.append(c.run(out=out).clone())
    torch.cuda.synchronize()
    assert all(torch.equal(s, want) for s in seen)


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_a_workspace_that_starts_on_any_16_bytes(dtype):
    """Its end too: what lies behind the bytes asked for stays as it was."""
    c = Case([(6, 192), (2, 64), (20, 48)], [5, 40, 20], 8, 2, 128, 16, dtype, seed=17, anchor=True)
    want, n = c.run_checked(), c.workspace().numel()
    for start in (0, 16, 32, 48, 240):
        raw = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device=DEV)
        assert raw.data_ptr() % 256 == 0
        assert torch.equal(c.run(workspace=raw[start:start + n]), want)
        assert (raw[:start] == 0xA5).all() and (raw[start + n:] == 0xA5).all()


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_far_blocks_past_32_bits(dtype):
    """Blocks whose offsets in elements pass 2^32."""
    c = Case([(3, 64)], [5, 40], 8, 2, 128, 16, dtype, seed=15, anchor=True)
    per = c.k[0].numel()
    far = (2 ** 32) // per + 3
    k = torch.zeros(far + c.nb, 16, 2, 128, dtype=dtype, device=DEV)
    v = torch.zeros_like(k)
    k[far:], v[far:] = c.k, c.v
    bt = torch.where(c.bt >= 0, c.bt + far, c.bt)
    assert torch.equal(c.run(k_cache=k, v_cache=v, block_tables=bt), c.run())


@pytest.mark.parametrize("dtype", DTYPES, **ids)
def test_a_captured_call_follows_its_buffers(dtype):
    """Lengths, groups and prefixes change between replays; two graphs with workspaces of their own, one after the
    other on streams of their own."""
    c = Case([(12, 640)], [33], 32, 8, 128, 16, dtype, seed=16)
    starts, prefix = torch.tensor([0, 12, 12, 12], device=DEV).int(), torch.tensor([640, 0, 0], device=DEV).int()
    graphs = []
    for _ in range(2):
        s, g, out = torch.cuda.Stream(), torch.cuda.CUDAGraph(), torch.zeros_like(c.q)
        ws = torch.full((pa.decode_shared_prefix_workspace_size(12, 3, 32, 8, 128, 16, c.mb),), 0xFF, dtype=torch.uint8, device=DEV)
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
            c.run(group_starts=starts, prefix_lens=prefix, out=out, workspace=ws)
        graphs.append((s, g, out, ws))
    for st, pr, ctx in (([0, 12, 12, 12], [640, 0, 0], [673] * 12), ([0, 4, 8, 12], [640, 320, 16], [650 + i for i in range(12)]),
                        ([0, 1, 11, 12], [0, 640, 640], [673 - 3 * i for i in range(12)]), ([0, 0, 0, 12], [5, 6, 639], [641] * 12),
                        ([0, 12, 12, 12], [640, 0, 0], [1] * 12)):
        starts.copy_(torch.tensor(st)), prefix.copy_(torch.tensor(pr)), c.ctx.copy_(torch.tensor(ctx))
        c.lens = ctx
        torch.cuda.synchronize()
        for s, g, out, _ in graphs:
            out.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        want = c.run(group_starts=starts, prefix_lens=prefix)
        c.check(want)
        for _, _, out, _ in graphs:
            assert torch.equal(out, want)


def test_another_stream_and_memory_of_its_own():
    c = Case([(12, 640)], [33], 8, 2, 128, 16, torch.bfloat16, seed=17)
    want = c.run()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        out = c.run(stream=stream)
        torch.cuda.current_stream().wait_stream(s)
        assert torch.equal(out, want)


def test_questions_about_one_video():
    """As a server does it: a video's tokens written once with positions on three axes, its blocks shared by the block
    manager, every request's own tokens appended, and one shared-prefix decode a step."""
    H, Hkv, D, B, n_video, S, steps = 8, 2, 128, 16, 16 * 23, 5, 4
    dtype = torch.bfloat16
    m = pa.BlockManager(128, B, 64)
    g = torch.Generator().manual_seed(20)
    tab = R.table(512, D).to(DEV)
    axis = (torch.arange(D // 2) % 3).int().to(DEV)
    kc, vc = (torch.full((128, B, Hkv, D), float("nan"), dtype=dtype, device=DEV) for _ in "kv")

    def rows(n):
        x = torch.randn(n, (H + 2 * Hkv) * D, generator=g).to(dtype).to(DEV)
        return [t.unflatten(1, (-1, D)) for t in x.split([H * D, Hkv * D, Hkv * D], 1)]

    def slots(ids, start, count):
        bt, _ = m.tables(ids, 64)
        cu = torch.arange(len(ids) + 1, dtype=torch.int32) * count
        return bt.to(DEV), pa.compute_slot_mapping(bt.to(DEV), torch.tensor(start, dtype=torch.int32, device=DEV),
                                                   cu.to(DEV), 128, count * len(ids), B)
    assert m.allocate_slots(100, n_video) == pa.OK
    t = torch.arange(n_video)
    pos = torch.stack([t // 46, t % 46 // 8, t % 8]).int().to(DEV)     # frames of 46 tokens, rows of 8
    _, slot = slots([100], [0], n_video)
    q, k, v = rows(n_video)
    pa.mrope_and_cache(q, k, v, tab, pos, axis, kc, vc, slot)
    seqs = list(range(S))
    for s in seqs:
        assert m.share_prefix(100, s, n_video) == pa.OK
    starts = torch.tensor([0, S], dtype=torch.int32, device=DEV)
    prefix = torch.tensor([n_video], dtype=torch.int32, device=DEV)
    for step in range(steps):
        assert m.allocate_slots_batch(seqs, [1] * S) == pa.OK
        bt, slot = slots(seqs, [n_video + step] * S, 1)
        q, k, v = rows(S)
        p = torch.full((3, S), 46 + step, dtype=torch.int32, device=DEV)
        qr = pa.mrope_and_cache(q, k, v, tab, p, axis, kc, vc, slot)
        ctx = torch.full((S,), n_video + step + 1, dtype=torch.int32, device=DEV)
        out = pa.decode_shared_prefix(qr, kc, vc, bt, ctx, starts, prefix, 0.088)
        c = Case.__new__(Case)
        c.H, c.Hkv, c.D, c.B, c.dtype, c.S, c.scale = H, Hkv, D, B, dtype, S, 0.088
        c.q, c.k, c.v, c.bt, c.lens = qr, kc, vc, bt, [n_video + step + 1] * S
        c.check(out)
        c.check(pa.decode(qr, kc, vc, bt, ctx, 0.088))
    m.close()
