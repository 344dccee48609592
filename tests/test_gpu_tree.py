"""Attention of drafted trees on the GPU (through the C ABI) against the float64
oracle, within the bound that the roundings allow (spec_support.close)."""

import numpy as np
import pytest
import torch

from spec_support import TreeOnDevice, close, tree_workload
from support import dev_to_bits, widen_out

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_394_b200 import pagedkv
    return pagedkv


HIST = [0, 5, 16, 40, 100, 0, 257]
NODES = [1, 17, 16, 0, 64, 33, 7]
SHAPES = [(d, bs, g, dt) for d in (64, 128) for bs in (16, 32) for g in (1, 2, 4, 8)
          for dt in ("fp16", "bf16")]


@pytest.mark.parametrize("d,bs,g,dtype", SHAPES)
def test_every_shape(pk, d, bs, g, dtype):
    t = TreeOnDevice(pk, tree_workload(HIST, NODES, 2 * g, 2, d, bs, dtype, seed=d + bs + g))
    assert t.run() == 0
    t.check()


@pytest.mark.parametrize("d,bs,g,dtype", [(128, 16, 1, "fp16"), (128, 32, 4, "bf16"),
                                          (128, 16, 8, "fp16"), (64, 16, 2, "bf16"),
                                          (64, 32, 8, "fp16"), (64, 16, 1, "bf16")])
def test_every_e4m3_shape(pk, d, bs, g, dtype):
    w = tree_workload(HIST, NODES, 2 * g, 2, d, bs, dtype, seed=7 * d + bs + g)
    t = TreeOnDevice(pk, w, scales=([0.0125, 0.02], [0.01, 0.03]))
    assert t.run() == 0
    t.check()


def some_rows(w, count, seed=0):
    """Rows at random, and each sequence's first and last."""
    rng = np.random.default_rng(seed)
    total, h = len(w.q), w.num_heads
    rows = {(int(a), int(b)) for a, b in zip(rng.integers(0, total, count),
                                             rng.integers(0, h, count))}
    for a, b in zip(w.query_start[:-1], w.query_start[1:]):
        if b > a:
            rows |= {(int(a), 0), (int(b) - 1, h - 1)}
    return rows


# units cut into several pieces, of one and of two query tiles, beside short ones
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,bs,g,dtype", SHAPES)
def test_every_shape_in_pieces(pk, d, bs, g, dtype, fp8):
    w = tree_workload([1700, 33, 64, 900, 0], [21, 0, 40, 3, 64], 2 * g, 2, d, bs, dtype,
                      seed=3 * d + bs + g)
    t = TreeOnDevice(pk, w, scales=([0.0125, 0.02], [0.01, 0.03]) if fp8 else None)
    assert t.run() == 0
    t.check(some_rows(w, 20))


# up to 64 rows a unit, cut; and more of them, whole, than there are SMs
@pytest.mark.parametrize("d,bs,g,dtype", SHAPES)
def test_every_shape_of_few_rows(pk, d, bs, g, dtype):
    most = 64 // g
    w = tree_workload([1700, 33, 64, 900, 0], [most // 2, 0, most, 3, most], 2 * g, 2, d, bs,
                      dtype, seed=5 * d + bs + g)
    t = TreeOnDevice(pk, w)
    assert t.run() == 0
    t.check(some_rows(w, 20))
    hist = [7 * i % 150 for i in range(80)]
    w = tree_workload(hist, [i % (most // 4 + 1) for i in range(80)], 2 * g, 2, d, bs, dtype,
                      seed=6 * d + bs + g)
    t = TreeOnDevice(pk, w)
    assert t.run() == 0
    t.check(some_rows(w, 20))


@pytest.mark.parametrize("fp8", [False, True])
def test_many_sequences(pk, fp8):
    """More sequences than a CTA has threads, most of one tile, some empty, one
    long (cut) or none (more units than CTAs, left whole)."""
    rng = np.random.default_rng(5)
    for extra in ([3000], []):
        hist = extra + [int(x) for x in rng.integers(0, 60, 700)]
        nodes = [int(x) for x in rng.integers(0, 5, len(hist))]
        nodes[0] = 7
        w = tree_workload(hist, nodes, 2, 1, 64, 16, "fp16", seed=41)
        t = TreeOnDevice(pk, w, scales=([0.0125], [0.01]) if fp8 else None)
        assert t.run() == 0
        t.check()


@pytest.mark.parametrize("kind", ["chain", "star", "forest"])
@pytest.mark.parametrize("g,dtype", [(1, "fp16"), (8, "bf16")])
def test_largest_trees_of_each_kind(pk, kind, g, dtype):
    w = tree_workload([70, 1000], [256, 255], 2 * g, 2, 128, 16, dtype, seed=3, kind=kind)
    t = TreeOnDevice(pk, w)
    assert t.run() == 0
    rng = np.random.default_rng(1)
    rows = {(int(a), int(b)) for a, b in zip(rng.integers(0, 511, 60), rng.integers(0, 2 * g, 60))}
    t.check(rows | {(0, 0), (255, 2 * g - 1), (256, 0), (510, 2 * g - 1)})


@pytest.mark.parametrize("hist,nodes,h,hkv,d,dtype,fp8", [
    ([9000], [8], 8, 1, 128, "bf16", False), ([12345, 31], [64, 3], 16, 2, 128, "fp16", False),
    ([6001, 4095], [33, 12], 8, 8, 64, "bf16", False), ([8191], [16], 32, 8, 128, "fp16", True),
    ([5000, 0, 64], [1, 1, 1], 4, 2, 128, "bf16", True), ([30000], [2], 1, 1, 64, "fp16", True)])
def test_long_histories(pk, hist, nodes, h, hkv, d, dtype, fp8):
    w = tree_workload(hist, nodes, h, hkv, d, 16, dtype, seed=sum(hist))
    t = TreeOnDevice(pk, w, scales=([0.0125] * hkv, [0.01] * hkv) if fp8 else None)
    assert t.run() == 0
    rng = np.random.default_rng(0)
    total = sum(nodes)
    rows = {(int(a), int(b)) for a, b in zip(rng.integers(0, total, 24), rng.integers(0, h, 24))}
    t.check(rows | {(0, 0), (total - 1, h - 1)})


def test_history_ends_at_every_place_of_a_tile(pk):
    # 64-key tiles: the tree starts and ends at each offset within one
    hist = list(range(55, 135, 3))
    w = tree_workload(hist, [9] * len(hist), 4, 2, 128, 16, "fp16", seed=8)
    t = TreeOnDevice(pk, w)
    assert t.run() == 0
    t.check()


def test_chain_is_prefill_and_one_node_is_decode(pk):
    w = tree_workload([100, 3, 700], [20, 33, 64], 8, 2, 128, 16, "fp16", seed=4, kind="chain")
    t = TreeOnDevice(pk, w)
    assert t.run() == 0
    pre = torch.empty_like(t.q)
    pk.paged_attn_prefill(pre, t.q, t.k_cache, t.v_cache, t.tables, t.lens, t.qstart, w.scale, 2,
                          16, w.max_context_len, 64, dev_err=t.err)
    ref, mag = t.reference()
    for o in (t.out, pre):
        close(widen_out(dev_to_bits(o), w), ref, mag, "fp16")
    w = tree_workload([0, 63, 64, 511, 1300], [1] * 5, 8, 2, 128, 16, "bf16", seed=5)
    t = TreeOnDevice(pk, w)
    assert t.run() == 0
    dec = torch.empty_like(t.q)
    pk.paged_attn_decode(dec, t.q, t.k_cache, t.v_cache, t.tables, t.lens, w.scale, 2, 16,
                         w.max_context_len, dev_err=t.err)
    ref, mag = t.reference()
    for o in (t.out, dec):
        close(widen_out(dev_to_bits(o), w), ref, mag, "bf16")


@pytest.mark.parametrize("hist,heads", [([70, 20], 8), ([1130, 20], 8), ([1130, 650], 2),
                                        ([70, 20], 2), ([2100, 950], 4)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("d,dtype", [(128, "bf16"), (128, "fp16"), (64, "fp16")])
def test_what_a_row_does_not_see_does_not_enter_it(pk, d, dtype, fp8, hist, heads):
    """NaN and infinities in a node's K and V reach its descendants only."""
    w = tree_workload(hist, [40, 24], heads, 2, d, 16, dtype, seed=11)
    t = TreeOnDevice(pk, w, scales=([0.0125, 0.02], [0.01, 0.03]) if fp8 else None)
    ref, mag = t.reference()
    inf, nan = ((0x7C00, 0x7E00) if dtype == "fp16" else (0x7F80, 0x7FC0)) if not fp8 else (
        0x7F, 0xFF)  # E4M3 has no infinities: two NaNs
    sees = np.zeros((64, 64), dtype=bool)
    for a, b in ((0, 40), (40, 64)):
        for j in range(b - a):
            n = j
            while n >= 0:
                sees[a + j, a + n] = True
                n = w.parents[a + n]
    bad_v, bad_k = [3, 17, 39, 41], [8, 50]
    for node in bad_v:
        s = int(w.slot_mapping[node])
        t.v_ref[s // 16, :, s % 16, ::3] = inf
        t.v_ref[s // 16, :, s % 16, 1::3] = nan
    for node in bad_k:
        s = int(w.slot_mapping[node])
        t.k_ref[s // 16, :, s % 16, :] = nan
    t.upload()
    assert t.run() == 0
    got = widen_out(dev_to_bits(t.out), w)
    bad = np.zeros(got.shape, dtype=bool)
    inf_at = np.zeros(got.shape, dtype=bool)
    for node in bad_v:
        rows = sees[:, node]
        bad[rows, :, 0::3] = True
        bad[rows, :, 1::3] = True
        inf_at[rows, :, 0::3] = not fp8
    for node in bad_k:
        bad[sees[:, node]] = True
        inf_at[sees[:, node]] = False
    assert not bad.all() and bad.any()
    ok = ~bad.any(axis=(1, 2))
    close(got[ok], ref[ok], mag[ok], dtype)                 # rows that see nothing of it
    part = bad.any(axis=(1, 2)) & ~bad.all(axis=(1, 2))     # untouched dims of the others
    close(got[part][~bad[part]], ref[part][~bad[part]], mag[part][~bad[part]], dtype)
    assert not np.isfinite(got[bad]).any()
    assert np.isposinf(got[inf_at]).all()
    assert np.isnan(got[bad & ~inf_at]).all()


def test_rows_behind_the_last_sequence_are_left_as_they_were(pk):
    w = tree_workload([40, 9], [12, 5], 4, 2, 128, 16, "fp16", seed=12)
    t = TreeOnDevice(pk, w)
    pad = 30
    q = torch.cat([t.q, torch.full((pad, 4, 128), float("nan"), dtype=t.q.dtype, device="cuda")])
    out = torch.full_like(q, 7.0)
    parents = torch.cat([t.parents, torch.full((pad,), -99, dtype=torch.int32, device="cuda")])
    # two more sequences of the padded batch have no nodes (one has no tokens at all)
    tables = torch.cat([t.tables, t.tables[:2]])
    lens = torch.cat([t.lens, torch.tensor([0, 30], dtype=torch.int32, device="cuda")])
    qs = torch.cat([t.qstart, t.qstart[-1:], t.qstart[-1:]])
    pk.paged_attn_tree(out, q, t.k_cache, t.v_cache, tables, lens, qs, parents, w.scale, 2, 16,
                       tables.shape[1] * 16, 64, dev_err=t.err)
    torch.cuda.synchronize()
    assert int(t.err.item()) == 0
    assert (out[17:] == 7.0).all()
    t.out = out[:17].contiguous()
    t.check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0])
@pytest.mark.parametrize("dtype,fp8", [("fp16", False), ("bf16", False), ("bf16", True)])
def test_other_scales(pk, scale, dtype, fp8):
    # |scale q . k| stays below 2^6 (q, k ~ N(0, 1), 64 dims, scaled down)
    w = tree_workload([30, 150], [20, 31], 4, 2, 64, 16, dtype, seed=13)
    t = TreeOnDevice(pk, w, scales=([0.01, 0.01], [0.01, 0.02]) if fp8 else None)
    if scale == 3.0:
        t.q.mul_(1 / 16)
        w.q = dev_to_bits(t.q)
    assert t.run(scale=scale) == 0
    t.check(scale=scale)


def test_errors_are_reported_and_other_sequences_stay_right(pk):
    w = tree_workload([40, 50, 60, 70], [10, 11, 12, 13], 8, 2, 128, 16, "fp16", seed=14)
    t = TreeOnDevice(pk, w)
    ref, mag = t.reference()

    def fresh():
        t.err.zero_()
        t.out.fill_(7.0)

    def rest_is_right(but):
        got = widen_out(dev_to_bits(t.out), w)
        for i in range(4):
            a, b = int(w.query_start[i]), int(w.query_start[i + 1])
            if i != but:
                close(got[a:b], ref[a:b], mag[a:b], "fp16")
        return got[int(w.query_start[but]):int(w.query_start[but + 1])]

    for bad in (5, 6, 255, -2, 2 ** 30, -2 ** 31):  # node 5's parent: itself, later, outside
        fresh()
        t.parents = torch.from_numpy(w.parents).cuda()
        t.parents[10 + 5] = bad
        assert t.run() == pk.DEVERR_BAD_TREE
        rest_is_right(1)
    t.parents = torch.from_numpy(w.parents).cuda()
    # the node is then a child of the history
    fresh()
    t.parents[10 + 5] = 77
    assert t.run() == pk.DEVERR_BAD_TREE
    kept = w.parents.copy()
    w.parents[10 + 5] = -1
    ref1, mag1 = t.reference()
    w.parents = kept
    close(widen_out(dev_to_bits(t.out), w), ref1, mag1, "fp16")
    t.parents = torch.from_numpy(w.parents).cuda()
    for length in (-1, 12, w.max_context_len + 1, 2 ** 31 - 1):   # 12 tokens < 13 nodes
        fresh()
        t.lens = torch.from_numpy(w.context_lens).cuda()
        t.lens[3] = length
        assert t.run() == pk.DEVERR_BAD_CONTEXT
        assert (rest_is_right(3) == 7.0).all()
    t.lens = torch.from_numpy(w.context_lens).cuda()
    # rows past the end of q (the last sequence's), and before its start (the first's)
    fresh()
    t.qstart = torch.tensor([0, 10, 21, 33, 47], dtype=torch.int32, device="cuda")
    assert t.run() == pk.DEVERR_BAD_CONTEXT
    assert (rest_is_right(3) == 7.0).all()
    fresh()
    t.qstart = torch.tensor([-1, 10, 21, 33, 46], dtype=torch.int32, device="cuda")
    assert t.run() == pk.DEVERR_BAD_CONTEXT
    assert (rest_is_right(0) == 7.0).all()
    t.qstart = torch.from_numpy(w.query_start).cuda()
    fresh()
    t.tables = torch.from_numpy(w.block_tables).cuda()
    t.tables[2, 1] = w.num_blocks
    assert t.run() == pk.DEVERR_BAD_BLOCK
    rest_is_right(2)


def test_bad_scale_is_reported(pk):
    w = tree_workload([40], [10], 4, 2, 128, 16, "fp16", seed=15)
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        t = TreeOnDevice(pk, w, scales=([0.01, 0.01], [0.01, 0.01]))
        t.vs[1] = bad
        assert t.run() == pk.DEVERR_BAD_SCALE


def test_offsets_past_32_bits(pk):
    """A cache of more than 2^32 bytes and 2^31 elements: the sequence's blocks lie at its end."""
    w = tree_workload([90], [20], 8, 8, 128, 16, "fp16", seed=16)
    t = TreeOnDevice(pk, w)
    blocks = (2 ** 31) // (8 * 16 * 128) + 16
    big = [torch.zeros((blocks, 8, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    tables = t.tables.clone()
    for i, b in enumerate(w.block_tables[0]):
        at = blocks - 1 - i
        big[0][at], big[1][at] = t.k_cache[int(b)], t.v_cache[int(b)]
        tables[0, i] = at
    t.k_cache, t.v_cache, t.tables = big[0], big[1], tables
    assert t.run() == 0
    t.check()


def test_side_stream_and_captured_graph(pk):
    w = tree_workload([200, 31, 900], [20, 8, 64], 16, 2, 128, 16, "bf16", seed=17)
    t = TreeOnDevice(pk, w)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    t.attend(stream=s)
    s.synchronize()
    t.check()
    # captured; replayed on new values and a shorter batch in the same buffers
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.attend()
    t.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    t.check()
    w2 = tree_workload([150, 600, 20], [19, 30, 1], 16, 2, 128, 16, "bf16", seed=18)
    t2 = TreeOnDevice(pk, w2)
    n, blocks = len(w2.q), min(w.num_blocks, w2.num_blocks)
    assert w2.num_blocks <= w.num_blocks and w2.max_context_len <= w.max_context_len
    t.out.fill_(7.0)
    t.q[:n] = t2.q
    t.parents[:n] = t2.parents
    t.k_cache[:blocks], t.v_cache[:blocks] = t2.k_cache[:blocks], t2.v_cache[:blocks]
    t.tables.fill_(-1)
    t.tables[:, :t2.tables.shape[1]] = t2.tables
    t.lens.copy_(t2.lens)
    t.qstart.copy_(t2.qstart)
    g.replay()
    torch.cuda.synchronize()
    assert int(t.err.item()) == 0 and (t.out[n:] == 7.0).all()
    t2.out = t.out[:n].contiguous()
    t2.check()


def test_two_runs_agree_bit_for_bit(pk):
    w = tree_workload([3000, 17], [40, 9], 16, 2, 128, 16, "bf16", seed=19)
    t = TreeOnDevice(pk, w)
    t.run()
    first = t.out.clone()
    for _ in range(3):
        t.out.zero_()
        t.run()
        assert torch.equal(first, t.out)



# rows and pieces are stored 32 bytes at a time where the addresses allow it
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hist", [[3000, 17], [40, 9]])   # cut; whole
def test_places_of_output_and_workspace(pk, hist, fp8):
    w = tree_workload(hist, [20, 9], 16, 2, 128, 16, "fp16", seed=29)
    t = TreeOnDevice(pk, w, scales=([0.0125, 0.02], [0.01, 0.03]) if fp8 else None)
    assert t.run() == 0
    first, n = t.out.clone(), t.out.numel()
    need = pk.tree_workspace_bytes(w.num_seqs, w.num_heads, w.num_kv_heads, w.head_dim,
                                   w.max_context_len, t.max_nodes)
    assert (need > 0) == (hist[0] > 64)
    for at in (0, 16, 32, 48):
        ws = torch.full((at + need + 64,), 0x5A, dtype=torch.uint8, device="cuda")
        room = torch.full((n + 64,), 7.0, dtype=first.dtype, device="cuda")
        t.out = room[at // 2:at // 2 + n].view_as(first)
        assert t.run(workspace=ws[at:at + need] if need else None) == 0
        assert torch.equal(first, t.out)
        assert (room[:at // 2] == 7.0).all() and (room[at // 2 + n:] == 7.0).all()
        assert (ws[:at] == 0x5A).all() and (ws[at + need:] == 0x5A).all()
    if need:
        with pytest.raises(RuntimeError):
            t.run(workspace=ws[:need - 1])
        with pytest.raises(RuntimeError):
            t.run(workspace=ws[8:8 + need])
