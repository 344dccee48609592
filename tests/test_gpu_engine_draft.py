"""Drafted steps of the continuous-batching driver: trees attended, verified and
compacted one after the other, replayed step by step through the oracle.

Every step's slots and copy-on-write pairs, kept nodes and next tokens equal the
oracle's, the tree attention lies within the bound that the roundings allow, and
after every step the two pools are identical bit for bit.
"""

import numpy as np
import pytest
import torch

from oracle import attention as OA
from oracle import cache_ops as OC
from oracle import speculative as OS
from oracle.block_manager import BlockManager
from paged_kv_cache_394_b200 import workloads as W
from spec_support import close
from support import ATOL, RTOL, dev_to_bits

pytestmark = pytest.mark.gpu


def widened(t, dtype="fp16"):
    from oracle.dtypes import widen
    return widen(dev_to_bits(t), dtype)


class Draws:
    """Peaked target and draft distributions on the host, children drawn from the draft's."""

    def __init__(self, seed, vocab, certain=False):
        self.rng, self.vocab, self.certain = np.random.default_rng(seed), vocab, certain

    def __call__(self, parents, query_start):
        rng, v = self.rng, self.vocab
        par, qs = parents.cpu().numpy(), query_start.cpu().numpy()
        t = len(par)
        logits = 3.0 * rng.standard_normal((t, v))
        both = [logits, logits + 0.7 * rng.standard_normal((t, v))]
        target, draft = ((e / e.sum(axis=1, keepdims=True)).astype(np.float32)
                         for e in (np.exp(x - x.max(axis=1, keepdims=True)) for x in both))
        tokens = np.zeros(t, dtype=np.int32)
        for a, b in zip(qs[:-1], qs[1:]):
            for j in range(a + 1, b):
                c = np.cumsum(draft[a + par[j]].astype(np.float64))
                tokens[j] = min(np.searchsorted(c, rng.random() * c[-1]), v - 1)
        u, u_next = rng.random(t).astype(np.float32), rng.random(len(qs) - 1).astype(np.float32)
        self.last = (par, qs, target, None if self.certain else draft, tokens, u, u_next)
        dev = lambda x: None if x is None else torch.from_numpy(x).cuda()  # noqa: E731
        return tuple(dev(x) for x in self.last[2:])


@pytest.mark.parametrize("certain,bs,d,hkv,g", [(False, 16, 64, 2, 2), (True, 32, 128, 1, 8)])
def test_drafted_batching_matches_oracle_replay(certain, bs, d, hkv, g):
    from paged_kv_cache_394_b200 import engine as E

    h, nb = hkv * g, 96
    rng = np.random.default_rng(3)
    order = rng.permutation(nb)
    draws = Draws(7, 211, certain)
    given = {}

    def values(kind, shape):
        bits = W._normal_bits(rng, shape, "fp16")
        given[kind] = bits
        return torch.from_numpy(bits.view(np.int16)).cuda().view(torch.float16)

    b = E.ContinuousBatcher(nb, bs, h, hkv, d, max_num_seqs=6, max_num_batched_tokens=260,
                            max_model_len=256, free_order=order, values=values,
                            drafter=E.tree_drafter(2, 18), max_draft=18, draws=draws)
    trace = E.synthetic_trace(5, 9, mean_interarrival=1.0, prompt_median=40,
                              output_range=(2, 30), max_prompt=100)
    trace[3].samples = 3
    for r in trace:
        b.submit(r)
    ref = BlockManager(nb, bs, free_order=order)
    kc = np.zeros((nb, hkv, bs, d), np.uint16)
    vc = np.zeros_like(kc)
    steps = cows = moved = kept = nodes = 0
    while not b.idle():
        given.clear()
        rec = b.step()
        steps += 1
        assert steps < 200
        slots, pairs = [], []
        for sid, plen in rec.admitted:
            ref.add_seq(sid, plen)
            row = ref.seq_blocks(sid)
            slots += [row[t // bs] * bs + t % bs for t in range(plen)]
        hist = [ref.seq_len(s) for s in rec.decoded]
        for sid, tree in zip(rec.decoded, rec.parents):
            for _ in tree:
                slot, a, c = ref.append_slot(sid)
                slots.append(slot)
                if a >= 0:
                    pairs.append((a, c))
        assert slots == list(rec.slots)
        assert pairs == [tuple(x) for x in rec.cow_pairs]
        cows += len(pairs)
        if pairs:
            OC.copy_blocks(kc, vc, np.array(pairs), inplace=True)
        if slots:
            OC.reshape_and_cache(given["key"], given["value"], kc, vc, np.array(slots), bs,
                                 inplace=True)
        if rec.admitted:
            ids = [sid for sid, _ in rec.admitted]
            lens = np.array([pl for _, pl in rec.admitted])
            got = widened(b.last_outputs["prefill"][2])
            want = OA.paged_attention_prefill(
                given["q_prefill"], kc, vc, np.array(ref.block_table(ids, b.max_blocks),
                                                     dtype=np.int32),
                lens, np.concatenate([[0], np.cumsum(lens)]), b.scale, hkv, bs, "fp16")
            assert (np.abs(got - want) <= ATOL + RTOL * np.abs(want)).all()
        if rec.decoded:
            par, qs, target, draft, tokens, u, u_next = draws.last
            tables = np.array(ref.block_table(rec.decoded, b.max_blocks), dtype=np.int32)
            lens = np.array([ref.seq_len(s) for s in rec.decoded])
            args = (tables, lens, qs, par, b.scale, hkv, bs, "fp16")
            want = OS.tree_attention(given["q_tree"], kc, vc, *args)
            mag = OS.tree_attention(given["q_tree"], kc, vc & np.uint16(0x7FFF), *args)
            close(widened(b.last_outputs["tree"][2]), want, mag, "fp16")
            width = max(len(t) for t in rec.parents)
            acc, count, nxt = OS.verify(qs, par, tokens, target.astype(np.float64),
                                        None if draft is None else draft.astype(np.float64), u,
                                        u_next, width)
            assert rec.kept == count.tolist() and rec.next_tokens == nxt.tolist()
            assert np.array_equal(b.last_outputs["tree"][6].cpu().numpy(), acc)
            kc, vc = OS.compact(kc, vc, tables, lens, qs, acc, count, bs)
            moved += sum(int((acc[i, :c] != np.arange(c)).sum()) for i, c in enumerate(count))
            kept += int(count.sum())
            nodes += len(par)
            for sid, n, c in zip(rec.decoded, hist, count):
                ref.truncate(sid, n + int(c))
        for sid in rec.finished:
            ref.free_seq(sid)
        for parent, child in rec.forked:
            ref.fork(parent, child)
        assert b.alloc.num_free() == ref.num_free()
        live = [s for s in b.running]
        assert b.alloc.context_lens(live) == [ref.seq_len(s) for s in live]
        assert np.array_equal(dev_to_bits(b.k_cache), kc)
        assert np.array_equal(dev_to_bits(b.v_cache), vc)
    assert cows >= 2 and moved > 0 and nodes > kept > 2 * len(trace)
    assert b.alloc.num_free() == nb and ref.num_free() == nb


def test_synthetic_drafts_run_to_the_end():
    from paged_kv_cache_394_b200 import engine as E

    b = E.ContinuousBatcher(400, 16, 8, 2, 128, dtype=torch.bfloat16, max_num_seqs=16,
                            max_model_len=300, vocab_size=1000, max_draft=9,
                            drafter=lambda sid, n: [-1] + list(range(8)))
    for r in E.synthetic_trace(1, 12, mean_interarrival=0.3, prompt_median=60,
                               output_range=(20, 60), max_prompt=200):
        b.submit(r)
    kept = drafted = 0
    while not b.idle():
        rec = b.step()
        assert all(1 <= k <= len(t) for k, t in zip(rec.kept, rec.parents))
        kept, drafted = kept + sum(rec.kept), drafted + len(rec.kept)
    assert kept > drafted > 0            # more than a token a step: the draft is near the target
    assert b.alloc.num_free() == 400


def test_drafter_refusals():
    from paged_kv_cache_394_b200 import engine as E

    for tree in ([], [-1] * 2, [0], [-1, 1], [-1, 0, 3], [-1] + [0] * 4):
        b = E.ContinuousBatcher(40, 16, 4, 2, 64, max_draft=4, vocab_size=50,
                                drafter=lambda sid, n, tree=tree: tree)
        b.submit(E.Request(0, 5, 5))
        b.step()
        with pytest.raises(ValueError):
            b.step()
    for n in (0, 257):
        with pytest.raises(ValueError):
            E.ContinuousBatcher(40, 16, 4, 2, 64, max_draft=n, drafter=lambda sid, n: [-1])


def test_one_captured_step_of_all_three(graph_steps=4):
    """Tree attention, verification and compaction captured into one graph and
    replayed on new inputs in the same buffers; the outputs equal the calls' own."""
    from paged_kv_cache_394_b200 import pagedkv as pk
    from spec_support import TreeOnDevice, tree_workload

    w = tree_workload([70, 300, 9], [12, 20, 5], 8, 2, 128, 16, "bf16", seed=31)
    t = TreeOnDevice(pk, w)
    n, v, width = len(w.q), 500, 20
    draws = Draws(9, v)
    state = [x.clone() for x in draws(t.parents, t.qstart)]
    out = [torch.zeros((3, width), dtype=torch.int32, device="cuda"),
           torch.zeros(3, dtype=torch.int32, device="cuda"),
           torch.zeros(3, dtype=torch.int32, device="cuda")]

    def step():
        t.attend()
        pk.verify_draft(*out, state[0], state[2], t.parents, t.qstart, state[3], state[4], width,
                        draft_probs=state[1], dev_err=t.err)
        pk.compact_accepted(t.k_cache, t.v_cache, t.tables, t.lens, t.qstart, out[0], out[1],
                            dev_err=t.err)

    before = [t.k_cache.clone(), t.v_cache.clone()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(graph_steps):
        for x, y in zip(state, draws(t.parents, t.qstart)):
            x.copy_(y)
        t.q.normal_()
        results = []
        for run in (step, g.replay):
            t.k_cache.copy_(before[0])
            t.v_cache.copy_(before[1])
            for x in (t.out, *out):
                x.zero_()
            run()
            torch.cuda.synchronize()
            results.append([x.clone() for x in (t.out, *out, t.k_cache, t.v_cache)])
        assert int(t.err.item()) == 0
        for a, b in zip(*results):
            assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
        assert n == int(t.qstart[-1]) and results[0][2].min() >= 1
