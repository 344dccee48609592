"""The speculative-decoding oracle against other routes to the same values, the
allocator's truncate against the oracle's block manager, and the host checks of
the C ABI (nothing here reaches a GPU)."""

import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import block_manager as OB
from oracle import speculative as OS
from paged_kv_cache_394_b200 import workloads as W
from spec_support import random_parents, tree_workload

KINDS = ("tree", "chain", "star", "forest")


def written(w):
    from oracle import cache_ops as OC
    kc, vc, bad = OC.reshape_and_cache(w.key, w.value, w.k_cache, w.v_cache, w.slot_mapping,
                                       w.block_size)
    assert not bad
    return kc, vc


def attention(w):
    return OS.tree_attention(w.q, *written(w), w.block_tables, w.context_lens, w.query_start,
                             w.parents, w.scale, w.num_kv_heads, w.block_size, w.dtype)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_tree_attention_equals_masked_attention_of_torch(kind, dtype):
    """torch's scaled_dot_product_attention in float64 with the ancestor mask, the
    mask from powers of the parent relation, on dense data laid out here."""
    w = tree_workload([5, 0, 33], [9, 4, 17], 4, 2, 64, 16, dtype, seed=2, kind=kind)
    out, (kc, vc) = attention(w), written(w)
    for i in range(3):
        a, b, c = w.query_start[i], w.query_start[i + 1], int(w.context_lens[i])
        n = b - a
        rel = np.eye(n)
        for j, p in enumerate(w.parents[a:b]):
            if p >= 0:
                rel[j, p] = 1
        mask = np.concatenate([np.ones((n, c - n)), np.linalg.matrix_power(rel, n)], axis=1) > 0
        k, v = (np.stack([OA.gather_kv(x, w.block_tables[i], c, h // 2, 16, dtype)
                          for h in range(4)]) for x in (kc, vc))
        q = OA.widen(w.q[a:b], dtype).transpose(1, 0, 2)
        ref = torch.nn.functional.scaled_dot_product_attention(
            *(torch.from_numpy(x) for x in (q, k, v)), attn_mask=torch.from_numpy(mask),
            scale=w.scale).numpy().transpose(1, 0, 2)
        assert np.abs(out[a:b] - ref).max() <= 1e-12


def test_chain_equals_prefill_and_single_nodes_equal_decode():
    w = tree_workload([5, 0, 33], [9, 4, 17], 4, 2, 64, 16, "fp16", seed=3, kind="chain")
    ref = OA.paged_attention_prefill(w.q, *written(w), w.block_tables, w.context_lens,
                                     w.query_start, w.scale, 2, 16, "fp16")
    assert np.abs(attention(w) - ref).max() <= 1e-13
    w = tree_workload([5, 0, 33], [1, 1, 1], 4, 2, 64, 16, "fp16", seed=4)
    ref = OA.paged_attention_decode(w.q, *written(w), w.block_tables, w.context_lens, w.scale, 2,
                                    16, "fp16")
    assert np.abs(attention(w) - ref).max() <= 1e-13


def test_each_branch_equals_its_own_sequence():
    """A node's row is that of the last token of the sequence history + its path."""
    w = tree_workload([20], [12], 2, 1, 64, 16, "fp16", seed=5)
    out, (kc, vc) = attention(w), written(w)
    for j in range(12):
        path = OS.path_to(w.parents, j)
        t = list(range(20)) + [20 + n for n in path]
        k, v = (OS.cached_rows(x, w.block_tables[0], t, 0, 16, "fp16") for x in (kc, vc))
        for h in range(2):
            assert np.abs(OA.attend(OA.widen(w.q[j, h], "fp16"), k, v, w.scale)
                          - out[j, h]).max() <= 1e-13


def test_planted_mistakes_in_the_mask_are_caught():
    w = tree_workload([20], [12], 2, 1, 64, 16, "fp16", seed=5)
    out = attention(w)
    for wrong in (np.arange(-1, 11), np.full(12, -1), np.r_[-1, w.parents[:-1]]):
        bad = tree_workload([20], [12], 2, 1, 64, 16, "fp16", seed=5)
        bad.parents = wrong.astype(np.int32)
        assert np.abs(attention(bad) - out).max() > 1e-2


def exact_marginals(parents, target, draft):
    """The distribution of the tokens that follow the root, exactly: every drafted
    tree weighed by its probability, every outcome of the uniforms by theirs.
    One level of children; the walk is carried out on probabilities."""
    vocab, kids = len(target), len(parents) - 1
    out = np.zeros(vocab)
    for toks in itertools.product(range(vocab), repeat=kids):
        weight = np.prod([draft[t] for t in toks]) if draft is not None else 1.0 / vocab ** kids
        r, left = target.copy(), 1.0
        for t in toks:
            q = draft if draft is not None else np.eye(vocab)[t]
            accept = min(1.0, r[t] / q[t]) if q[t] > 0 else 1.0
            out[t] += weight * left * accept
            left *= 1 - accept
            r = np.maximum(r - q, 0) if draft is not None else r * (1 - q)
            if left <= 0 or r.sum() <= 0:
                left = 0.0
                break
            r = r / r.sum()
        out += weight * left * r
    return out


@pytest.mark.parametrize("kids", [1, 2, 3])
@pytest.mark.parametrize("with_draft", [True, False])
def test_speculative_sampling_keeps_the_target_distribution(kids, with_draft):
    rng = np.random.default_rng(kids)
    target, draft = rng.dirichlet(np.ones(4)), rng.dirichlet(np.ones(4))
    got = exact_marginals([-1] + [0] * kids, target, draft if with_draft else None)
    assert np.abs(got - target).max() <= 1e-12


@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_follows_its_probabilities(with_draft):
    """verify_one on a fine grid of uniforms: the share of the outcomes equals the
    probabilities that exact_marginals sums, up to the grid's step."""
    rng = np.random.default_rng(9)
    target, draft = rng.dirichlet(np.ones(3)), rng.dirichlet(np.ones(3))
    grid, m = (np.arange(40) + 0.5) / 40, 40
    for toks in itertools.product(range(3), repeat=2):
        r, left, want = target.copy(), 1.0, np.zeros(3)
        for t in toks:
            q = draft if with_draft else np.eye(3)[t]
            a = min(1.0, r[t] / q[t])
            want[t] += left * a
            left *= 1 - a
            r = np.maximum(r - q, 0) if with_draft else r * (1 - q)
            if r.sum() > 0:
                r = r / r.sum()
        want += left * r
        got = np.zeros(3)
        p = np.stack([target] * 3)
        for u1, u2, un in itertools.product(grid, grid, grid):
            kept, nxt = OS.verify_one([-1, 0, 0], [0, *toks], p,
                                      np.stack([draft] * 3) if with_draft else None,
                                      [0, u1, u2], un)
            got[toks[kept[1] - 1] if len(kept) > 1 else nxt] += 1 / m ** 3
        # three thresholds, each off by at most half a step of the grid
        assert np.abs(got - want).max() <= 3 * 0.5 / m


def test_verify_hand_worked():
    p = np.array([[0.5, 0.5, 0], [0, 1, 0], [0.2, 0.3, 0.5]])
    q = np.array([[1, 0, 0], [0, 0.5, 0.5], [0, 0, 1.0]])
    # u q = 0.4 < 0.5: node 1 kept; then u q = 0.9 * 0.5 < 1 for token 1: node 2 kept
    assert OS.verify_one([-1, 0, 1], [9, 0, 1], p, q, [0, 0.4, 0.9], 0.1) == ([0, 1, 2], 0)
    # 0.6 >= 0.5: rejected, the residual of (0.5, 0.5, 0) - (1, 0, 0) is token 1's
    assert OS.verify_one([-1, 0, 1], [9, 0, 1], p, q, [0, 0.6, 0.0], 0.99) == ([0], 1)
    # certain draft: kept with the target's own 0.5; rejected, token 0 has no weight left
    assert OS.verify_one([-1, 0], [9, 0], p[:2], None, [0, 0.49], 0.3) == ([0, 1], 1)
    assert OS.verify_one([-1, 0], [9, 0], p[:2], None, [0, 0.5], 0.0) == ([0], 1)
    # the same token again is rejected too; the second token is certain by then
    assert OS.verify_one([-1, 0, 0, 0], [9, 0, 0, 1], np.stack([p[0]] * 4), None,
                         [0, 0.5, 0.0, 0.99], 0.9) == ([0, 3], 1)


def test_compaction_reads_before_it_writes():
    w = tree_workload([20, 3], [8, 5], 2, 2, 64, 16, "fp16", seed=6)
    kc, vc = written(w)
    acc = np.array([[1, 2, 3, 7, -1], [0, 2, -1, -1, -1]], dtype=np.int32)
    k2, v2 = OS.compact(kc, vc, w.block_tables, w.context_lens, w.query_start, acc, [4, 2], 16)
    for old, new in ((kc, k2), (vc, v2)):
        for i, (hist, path) in enumerate(((20, [1, 2, 3, 7]), (3, [0, 2]))):
            row = w.block_tables[i]
            for d, a in enumerate(path):
                s, t = hist + a, hist + d
                assert np.array_equal(new[row[t // 16], :, t % 16], old[row[s // 16], :, s % 16])
            for t in range(hist):
                assert np.array_equal(new[row[t // 16], :, t % 16], old[row[t // 16], :, t % 16])


# ---- allocator ----------------------------------------------------------------
@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_394_b200 import pagedkv
    return pagedkv


def test_truncate_equals_the_oracle_on_random_traces(pk):
    for seed in range(6):
        rng = np.random.default_rng(seed)
        order = rng.permutation(40)
        a, o = pk.BlockAllocator(40, 4, order), OB.BlockManager(40, 4, order)
        live, nid = [], 0
        for _ in range(400):
            op = rng.integers(0, 6)
            both = []
            for m in (a, o):
                r = np.random.default_rng(nid * 7 + int(op))
                try:
                    if op == 0:
                        both.append(m.add_seq(nid, int(r.integers(0, 20))))
                    elif op == 1 and live:
                        both.append(m.fork(live[int(r.integers(len(live)))], nid))
                    elif op == 2 and live:
                        toks = list(r.integers(0, 2, int(r.integers(0, 16))))
                        both.append(m.add_seq_cached(nid, toks))
                    elif op == 3 and live:
                        s = live[int(r.integers(len(live)))]
                        both.append(m.append_slots([s] * int(r.integers(1, 9))))
                    elif op == 4 and live:
                        s = live[int(r.integers(len(live)))]
                        n = m.seq_len(s)
                        both.append(m.truncate(s, int(r.integers(0, n + 1))))
                    elif live:
                        both.append(m.free_seq(live[int(r.integers(len(live)))]))
                    else:
                        both.append("nothing")
                except Exception as e:
                    both.append(type(e).__name__ and "failed")
            ids = [s for s in range(nid + 1) if s in o.seqs]
            assert (both[0] == "failed") == (both[1] == "failed")
            if op == 3 and both[0] not in ("failed", "nothing"):
                assert list(both[0][0]) == list(both[1][0]) and both[0][1] == both[1][1]
            nid += 1
            live = ids
            assert a.num_free() == o.num_free()
            assert a.context_lens(ids) == [o.seq_len(s) for s in ids]
            tables = a.block_table(ids, 40) if ids else []
            assert [[b for b in row if b >= 0] for row in tables] == [o.seq_blocks(s) for s in ids]
            assert [a.refcount(b) for b in range(40)] == o.refcount


def test_truncate_refusals_and_cached_blocks(pk):
    a = pk.BlockAllocator(10, 4)
    a.add_seq(1, 10)
    for sid, n in ((1, 11), (1, -1), (2, 0)):
        with pytest.raises(pk.PagedKVError):
            a.truncate(sid, n)
    assert a.seq_len(1) == 10 and a.num_free() == 7
    a.truncate(1, 8)
    assert a.seq_num_blocks(1) == 2 and a.num_free() == 8
    a.truncate(1, 0)
    assert a.seq_num_blocks(1) == 0 and a.num_free() == 10
    # a cached block that is cut back into and written again is found no more
    a = pk.BlockAllocator(10, 4)
    toks = [1, 2, 3, 4, 5, 6, 7, 8]
    assert a.add_seq_cached(1, toks) == 0
    a.truncate(1, 6)
    a.append_slot(1)
    assert a.add_seq_cached(2, toks) == 4


# ---- host checks of the C ABI -------------------------------------------------
GOOD, BAD, ODD = ctypes.c_void_p(0x1000), ctypes.c_void_p(0x1008), ctypes.c_void_p(0x1002)


def tree_call(pk, fp8=False, **over):
    a = dict(out=GOOD, q=GOOD, k=GOOD, v=GOOD, tables=GOOD, lens=GOOD, qs=GOOD, parents=GOOD,
             scale=1.0, ks=GOOD, vs=GOOD, num_seqs=2, num_tokens=8, heads=8, kv=2, d=128, bs=16,
             mb=8, mctx=100, mq=4, nb=20, dt=0, ws=GOOD, ws_bytes=1 << 40, err=None, stream=None)
    a.update(over)
    if not fp8:
        a.pop("ks"), a.pop("vs")
    return (pk._paged_attn_tree_fp8 if fp8 else pk._paged_attn_tree)(*a.values())


@pytest.mark.parametrize("fp8", [False, True])
def test_tree_refusals(pk, fp8):
    inv, uns = pk.ERR_INVALID_ARG, pk.ERR_UNSUPPORTED
    for name in ("out", "q", "k", "v", "tables", "lens", "qs", "parents"):
        assert tree_call(pk, fp8, **{name: None}) == inv, name
    for name in ("out", "q", "k", "v"):
        assert tree_call(pk, fp8, **{name: BAD}) == inv, name
    for name in ("tables", "lens", "qs", "parents", "err") + (("ks", "vs") if fp8 else ()):
        assert tree_call(pk, fp8, **{name: ODD}) == inv, name
    for over in (dict(num_seqs=-1), dict(num_tokens=-1), dict(heads=0), dict(kv=0), dict(mb=0),
                 dict(mctx=-1), dict(mq=-1), dict(nb=0), dict(dt=2), dict(dt=3), dict(dt=9),
                 dict(heads=7), dict(scale=float("nan")), dict(scale=float("inf")), dict(mq=101),
                 dict(mctx=129, mq=4)):
        assert tree_call(pk, fp8, **over) == inv, over
    for over in (dict(d=96), dict(d=256), dict(bs=8), dict(bs=64), dict(heads=6), dict(heads=32),
                 dict(mq=257, mctx=300, mb=20)):
        assert tree_call(pk, fp8, **over) == uns, over
    for over in (dict(num_seqs=0), dict(num_tokens=0), dict(mq=0)):
        assert tree_call(pk, fp8, **over) == pk.OK, over
    long = dict(mctx=6000, mb=400)    # short contexts need no workspace
    assert pk.tree_workspace_bytes(2, 8, 2, 128, 100, 4) == 0
    assert pk.tree_workspace_bytes(2, 8, 2, 128, 6000, 4) > 0
    for over in (dict(ws=None), dict(ws=BAD), dict(ws_bytes=0), dict(ws_bytes=16)):
        assert tree_call(pk, fp8, **over, **long) == pk.ERR_WORKSPACE, over
    if fp8:
        assert tree_call(pk, True, ks=None) == inv and tree_call(pk, True, vs=None) == inv


def verify_call(pk, **over):
    a = dict(acc=GOOD, cnt=GOOD, nxt=GOOD, p=GOOD, ps=100, q=GOOD, qstr=100, tok=GOOD, par=GOOD,
             qs=GOOD, u=GOOD, un=GOOD, num_seqs=2, num_tokens=8, mq=4, vocab=100, dt=3, err=None,
             stream=None)
    a.update(over)
    return pk._verify_draft(*a.values())


def test_verify_refusals(pk):
    inv, uns = pk.ERR_INVALID_ARG, pk.ERR_UNSUPPORTED
    for name in ("acc", "cnt", "nxt", "p", "tok", "par", "qs", "u", "un"):
        assert verify_call(pk, **{name: None}) == inv, name
    for name in ("acc", "cnt", "nxt", "p", "q", "tok", "par", "qs", "u", "un", "err"):
        assert verify_call(pk, **{name: ODD}) == inv, name
    for over in (dict(num_seqs=-1), dict(num_tokens=-1), dict(mq=-1), dict(vocab=0), dict(dt=2),
                 dict(dt=4), dict(ps=99), dict(qstr=99), dict(p=ctypes.c_void_p(0x1002)),
                 dict(q=ctypes.c_void_p(0x1002)), dict(dt=0, p=ctypes.c_void_p(0x1001))):
        assert verify_call(pk, **over) == inv, over
    assert verify_call(pk, mq=257) == uns
    assert verify_call(pk, vocab=2 ** 30 + 1, ps=2 ** 31, qstr=2 ** 31) == uns
    assert verify_call(pk, num_seqs=0) == pk.OK


def compact_call(pk, **over):
    a = dict(k=GOOD, v=GOOD, tables=GOOD, lens=GOOD, qs=GOOD, acc=GOOD, cnt=GOOD, num_seqs=2,
             mq=4, kv=2, d=128, bs=16, mb=8, nb=20, dt=0, err=None, stream=None)
    a.update(over)
    return pk._compact_accepted(*a.values())


def test_compact_refusals(pk):
    inv, uns = pk.ERR_INVALID_ARG, pk.ERR_UNSUPPORTED
    for name in ("k", "v", "tables", "lens", "qs", "acc", "cnt"):
        assert compact_call(pk, **{name: None}) == inv, name
    for name in ("tables", "lens", "qs", "acc", "cnt", "err"):
        assert compact_call(pk, **{name: ODD}) == inv, name
    for over in (dict(k=BAD), dict(v=BAD), dict(num_seqs=-1), dict(mq=-1), dict(kv=0), dict(mb=0),
                 dict(nb=0), dict(dt=3), dict(dt=-1)):
        assert compact_call(pk, **over) == inv, over
    for over in (dict(d=96), dict(bs=64), dict(mq=257)):
        assert compact_call(pk, **over) == uns, over
    for over in (dict(num_seqs=0), dict(mq=0)):
        assert compact_call(pk, **over) == pk.OK, over


def test_binding_refuses_host_tensors_and_mixed_types(pk):
    t = torch.zeros((2, 2, 128), dtype=torch.float16)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        pk.paged_attn_tree(t, t, t, t, i, i, i, i, 1.0, 2, 16, 16, 2)
    with pytest.raises(ValueError):
        pk.verify_draft(i, i, i, t, i, i, i, i, i, 2)
    with pytest.raises(ValueError):
        pk.compact_accepted(t, t, i, i, i, i, i)


def test_tree_helpers():
    rng = np.random.default_rng(0)
    for kind in KINDS:
        p = random_parents(rng, 20, kind)
        assert all(-1 <= x < j for j, x in enumerate(p))
    with pytest.raises(ValueError):
        OS.path_to([-1, 1], 1)
    assert OS.path_to([-1, 0, 1, 0], 2) == [0, 1, 2]
    assert W.NAMES
