"""Verification of drafted trees and compaction of the accepted path on the GPU
against the oracle: whole numbers and copies, so equal exactly."""

import numpy as np
import pytest
import torch

from oracle import speculative as OS
from spec_support import TreeOnDevice, random_parents, tree_workload
from support import dev_to_bits

pytestmark = pytest.mark.gpu
DT = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pk():
    from paged_kv_cache_394_b200 import pagedkv
    return pagedkv


class Case:
    """A batch of trees with peaked target and draft distributions, children drawn
    from the draft's."""

    def __init__(self, nodes, vocab, dtype, draft, seed, kind="tree", sharp=4.0, pad=0):
        rng = np.random.default_rng(seed)
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.qs = np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)
        t = int(self.qs[-1])
        self.parents = np.concatenate(
            [random_parents(rng, n, kind) for n in nodes] + [np.zeros(0)]).astype(np.int32)
        logits = torch.randn((t, vocab + pad), generator=gen, device="cuda") * sharp
        noise = torch.randn((t, vocab + pad), generator=gen, device="cuda")
        self.target = torch.softmax(logits[:, :vocab], dim=1).to(DT[dtype])
        d = torch.softmax((logits + 0.8 * noise)[:, :vocab], dim=1).to(DT[dtype])
        if pad:   # rows further apart than the vocabulary, at any alignment
            wide = [torch.full((t, vocab + pad), float("nan"), dtype=DT[dtype], device="cuda")
                    for _ in range(2)]
            wide[0][:, :vocab], wide[1][:, 1:vocab + 1] = self.target, d
            self.target, d = wide[0][:, :vocab], wide[1][:, 1:vocab + 1]
        c = np.cumsum(d.double().cpu().numpy(), axis=1)
        self.tokens = np.zeros(t, dtype=np.int32)
        for a, b in zip(self.qs[:-1], self.qs[1:]):
            for j in range(a + 1, b):
                row = c[a + max(self.parents[j], 0)]
                self.tokens[j] = min(np.searchsorted(row, rng.random() * row[-1]), vocab - 1)
        self.draft = d if draft else None
        self.u = rng.random(t).astype(np.float32)
        self.u_next = rng.random(len(nodes)).astype(np.float32)
        self.width = max([1, *nodes])
        self.err = torch.zeros(1, dtype=torch.int32, device="cuda")

    def run(self, pk, width=None, **more):
        s, width = len(self.qs) - 1, width or self.width
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()  # noqa: E731
        self.accepted = torch.full((s, width), 99, dtype=torch.int32, device="cuda")
        self.count = torch.full((s,), 99, dtype=torch.int32, device="cuda")
        self.next = torch.full((s,), 99, dtype=torch.int32, device="cuda")
        self.inputs = [dev(self.tokens), dev(self.parents), dev(self.qs), dev(self.u),
                       dev(self.u_next)]
        torch.cuda.synchronize()
        pk.verify_draft(self.accepted, self.count, self.next, self.target, *self.inputs, width,
                        draft_probs=self.draft, dev_err=self.err, **more)
        torch.cuda.synchronize()
        return int(self.err.item())

    def reference(self, width=None):
        wide = lambda x: x.double().cpu().numpy()  # noqa: E731
        return OS.verify(self.qs, self.parents, self.tokens, wide(self.target),
                         None if self.draft is None else wide(self.draft), self.u, self.u_next,
                         width or self.width)

    def check(self, width=None):
        a, c, n = self.reference(width)
        assert np.array_equal(self.count.cpu().numpy(), c)
        assert np.array_equal(self.accepted.cpu().numpy(), a)
        assert np.array_equal(self.next.cpu().numpy(), n)
        return c


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("dtype", ["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 256, 1000, 4099, 32000])
def test_trees_and_chains(pk, vocab, dtype, draft):
    kept = []
    for seed, kind in enumerate(("tree", "chain", "star", "forest")):
        c = Case([8, 1, 0, 33, 16, 5], vocab, dtype, draft, 100 * seed + vocab, kind)
        assert c.run(pk) == 0
        kept += list(c.check())
    assert vocab < 100 or max(kept) > 1      # something is accepted


@pytest.mark.parametrize("vocab,pad", [(1000, 24), (1001, 7), (4096, 1), (151, 3)])
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
def test_strided_rows(pk, vocab, pad, dtype):
    c = Case([8, 20, 3], vocab, dtype, True, vocab, pad=pad)
    assert not c.target.is_contiguous() and c.target.stride(0) == vocab + pad
    assert c.run(pk) == 0
    c.check()


@pytest.mark.parametrize("draft", [True, False])
def test_large_vocabulary_and_batch(pk, draft):
    c = Case([9] * 40, 160001, "fp32", draft, 5)
    assert c.run(pk) == 0
    c.check()
    c = Case([256, 200], 3001, "fp32", draft, 6, kind="star")
    assert c.run(pk) == 0
    c.check()


def test_uniforms_at_their_ends(pk):
    for u in (0.0, np.nextafter(np.float32(1), np.float32(0))):
        for un in (0.0, np.nextafter(np.float32(1), np.float32(0))):
            for draft in (True, False):
                c = Case([8, 12, 1], 500, "fp32", draft, 7)
                c.u[:], c.u_next[:] = u, un
                assert c.run(pk) == 0
                c.check()


def test_one_hot_targets_and_zero_weights(pk):
    # a certain target: the drafted token is kept if and only if it is the target's
    c = Case([6, 6, 6], 300, "fp32", False, 8, kind="star")
    t = torch.zeros_like(c.target)
    t[:, 17] = 1.0
    c.target = t
    c.tokens[:] = [0, 3, 17, 4, 17, 5] + [0, 17, 17, 17, 1, 2] + [0, 1, 2, 3, 4, 5]
    assert c.run(pk) == 0
    assert list(c.check()) == [2, 2, 1]
    assert c.next.tolist() == [17, 17, 17]
    # the draft equal to the target: everything tried first is kept
    c = Case([9, 9], 300, "fp32", True, 9, kind="chain")
    c.draft = c.target.clone()
    c.tokens[:] = [int(x) for x in c.target.argmax(dim=1).roll(1)]
    assert c.run(pk) == 0
    assert list(c.check()) == [9, 9]
    # nothing left of the residual: the target's own distribution again
    c = Case([3], 8, "fp32", False, 10, kind="star")
    c.target = torch.zeros_like(c.target)
    c.target[0, 5] = 0.25
    c.tokens[:], c.u[:] = [0, 5, 5], 0.9
    assert c.run(pk) == 0
    assert list(c.check()) == [1] and c.next.tolist() == [5]


def test_negative_and_nan_weights_count_as_nothing(pk):
    c = Case([6, 6], 400, "fp32", True, 11)
    c.target[:, 5:60] = -1.0
    c.target[:, 80:90] = float("nan")
    c.draft[:, 200:230] = float("nan")
    assert c.run(pk) == 0
    c.check()


def test_errors(pk):
    c = Case([6, 5, 7], 400, "fp32", True, 12, kind="chain")
    good = c.reference()
    c.parents[6 + 2] = 4          # after its node: never reached, and reported
    err = c.run(pk)
    assert err & pk.DEVERR_BAD_TREE and not err & ~(pk.DEVERR_BAD_TREE)
    for i in (0, 2):
        assert c.next[i].item() == good[2][i] and c.count[i].item() == good[1][i]
    c = Case([6, 5, 7], 400, "fp32", True, 12, kind="star")
    for bad in (400, -1, 2 ** 30):
        c.err.zero_()
        c.u[:] = 0.999999        # nothing before it is kept
        c.tokens[7] = bad
        assert c.run(pk) == pk.DEVERR_BAD_DRAFT
        assert c.next.min().item() >= 0
    c = Case([6, 5, 7], 400, "fp32", True, 12)
    for rows in ([0, 6, 4, 18], [0, 6, 11, 19], [-1, 6, 11, 18]):
        c.err.zero_()
        c.qs = np.array(rows, dtype=np.int32)
        assert c.run(pk, width=8) == pk.DEVERR_BAD_CONTEXT
    c = Case([6], 400, "fp32", True, 13)
    assert c.run(pk, width=5) == pk.DEVERR_BAD_CONTEXT
    assert c.count.tolist() == [0] and c.next.tolist() == [-1]
    assert c.accepted.tolist() == [[-1] * 5]
    for value in (0.0, float("inf")):
        c = Case([6], 400, "fp32", False, 14)
        c.target[:] = value
        if value == 0.0:
            c.u[:] = 0.5
        assert c.run(pk) == pk.DEVERR_BAD_DRAFT
        assert c.next.tolist() == [-1] and c.count[0].item() >= 1


def test_wider_than_needed_and_empty(pk):
    c = Case([3, 0, 5], 50, "fp16", True, 15)
    assert c.run(pk, width=256) == 0
    c.check(width=256)
    c = Case([0, 0], 50, "fp32", True, 16)
    assert c.run(pk) == 0
    assert c.count.tolist() == [0, 0] and c.next.tolist() == [-1, -1]


def test_verify_on_a_side_stream_and_captured(pk):
    c = Case([8, 9, 30], 5000, "fp32", True, 17)
    s = torch.cuda.Stream()
    assert c.run(pk, stream=s) == 0
    c.check()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pk.verify_draft(c.accepted, c.count, c.next, c.target, *c.inputs, c.width,
                        draft_probs=c.draft, dev_err=c.err)
    c.u = np.random.default_rng(3).random(len(c.u)).astype(np.float32)
    c.inputs[3].copy_(torch.from_numpy(c.u))
    for _ in range(2):
        c.accepted.zero_()
        g.replay()
        torch.cuda.synchronize()
        c.check()


def test_accepted_tokens_follow_the_target(pk):
    """What speculative sampling promises: the first token after the root is
    distributed as the target's.  20000 trees of one shape over 6 tokens: each
    frequency within 5 standard deviations."""
    n, vocab = 20000, 6
    target = torch.tensor([0.4, 0.3, 0.15, 0.1, 0.05, 0.0])
    draft = torch.tensor([0.1, 0.2, 0.3, 0.1, 0.1, 0.2])
    gen = torch.Generator().manual_seed(4)
    for kids in (1, 3):
        w = 1 + kids
        tok = torch.multinomial(draft.expand(n, -1), w, replacement=True, generator=gen)
        par = torch.tensor([-1] + [0] * kids).repeat(n).int().cuda()
        out = [torch.empty((n, w), dtype=torch.int32, device="cuda"),
               torch.empty(n, dtype=torch.int32, device="cuda"),
               torch.empty(n, dtype=torch.int32, device="cuda")]
        rows = lambda p: p.expand(n * w, -1).contiguous().cuda()  # noqa: E731
        pk.verify_draft(*out, rows(target), tok.reshape(-1).int().cuda(), par,
                        torch.arange(0, n * w + 1, w, dtype=torch.int32, device="cuda"),
                        torch.rand(n * w, generator=gen).cuda(),
                        torch.rand(n, generator=gen).cuda(), w, draft_probs=rows(draft))
        acc, cnt, nxt = (x.cpu() for x in out)
        assert cnt.max() <= 2
        first = torch.where(cnt == 2, tok.gather(1, acc[:, 1:2].clamp(min=0).long())[:, 0],
                            nxt.long())
        freq = torch.bincount(first, minlength=vocab).double() / n
        sd = (target.double() * (1 - target.double()) / n).sqrt()
        assert ((freq - target.double()).abs() <= 5 * sd + 1e-12).all(), freq


# ---- compaction --------------------------------------------------------------
def paths(rng, nodes, kind="random"):
    width = max([1, *nodes])
    acc = np.full((len(nodes), width), -1, dtype=np.int32)
    count = np.zeros(len(nodes), dtype=np.int32)
    for i, n in enumerate(nodes):
        k = {"random": int(rng.integers(0, n + 1)), "all": n, "none": 0,
             "last": min(n, 1)}[kind]
        rise = np.sort(rng.permutation(n)[:k]) if kind != "last" else np.arange(n)[-1:]
        acc[i, :k], count[i] = rise, k
    return acc, count


@pytest.mark.parametrize("kind", ["random", "all", "none", "last"])
@pytest.mark.parametrize("d,bs,hkv,dtype,fp8", [
    (128, 16, 2, "fp16", False), (64, 32, 1, "bf16", False), (128, 32, 8, "bf16", True),
    (64, 16, 5, "fp16", True), (128, 16, 32, "fp16", False)])
def test_compaction_is_exact(pk, d, bs, hkv, dtype, fp8, kind):
    nodes = [1, 17, 16, 0, 64, 33, 256]
    w = tree_workload([0, 5, 16, 40, 100, 0, 250], nodes, hkv, hkv, d, bs, dtype, seed=21)
    t = TreeOnDevice(pk, w, scales=([0.01] * hkv, [0.01] * hkv) if fp8 else None)
    acc, count = paths(np.random.default_rng(d + bs + hkv), nodes, kind)
    pk.compact_accepted(t.k_cache, t.v_cache, t.tables, t.lens, t.qstart,
                        torch.from_numpy(acc).cuda(), torch.from_numpy(count).cuda(),
                        dev_err=t.err)
    torch.cuda.synchronize()
    assert int(t.err.item()) == 0
    ref = OS.compact(t.k_ref, t.v_ref, w.block_tables, w.context_lens, w.query_start, acc, count,
                     bs)
    for got, want in zip((t.k_cache, t.v_cache), ref):
        got = got.cpu().numpy() if fp8 else dev_to_bits(got)
        assert np.array_equal(got, want)


def test_compaction_errors_leave_the_sequence_alone(pk):
    nodes = [10, 11, 12]
    w = tree_workload([40, 50, 60], nodes, 2, 2, 64, 16, "fp16", seed=22)
    t = TreeOnDevice(pk, w)
    acc = np.tile(np.array([0, 2, 5, 9] + [-1] * 8, dtype=np.int32), (3, 1))
    count = np.full(3, 4, dtype=np.int32)

    def run(acc, count, lens=None, tables=None):
        t.upload()
        t.err.zero_()
        pk.compact_accepted(t.k_cache, t.v_cache, t.tables if tables is None else tables,
                            t.lens if lens is None else lens, t.qstart,
                            torch.from_numpy(acc).cuda(), torch.from_numpy(count).cuda(),
                            dev_err=t.err)
        torch.cuda.synchronize()
        return int(t.err.item())

    def check(acc, count):
        ref = OS.compact(t.k_ref, t.v_ref, w.block_tables, w.context_lens, w.query_start, acc,
                         count, 16)
        assert np.array_equal(dev_to_bits(t.k_cache), ref[0])
        assert np.array_equal(dev_to_bits(t.v_cache), ref[1])

    rest = np.array([4, 0, 4], dtype=np.int32)
    for bad in ([0, 2, 2, 9], [0, 5, 2, 9], [0, 2, 5, 11], [-1, 2, 5, 9], [0, 2, 5, 2 ** 30]):
        a = acc.copy()
        a[1, :4] = bad
        assert run(a, count) == pk.DEVERR_BAD_TREE
        check(acc, rest)
    for n in (-1, 12, 2 ** 30):
        assert run(acc, np.array([4, n, 4], dtype=np.int32)) == pk.DEVERR_BAD_TREE
        check(acc, rest)
    for length in (-1, 10, 10 ** 6):
        lens = t.lens.clone()
        lens[1] = length
        assert run(acc, count, lens=lens) == pk.DEVERR_BAD_CONTEXT
        check(acc, rest)
    tables = t.tables.clone()
    tables[1, 3] = w.num_blocks     # tokens 48 .. 63: every source and destination but the first
    assert run(acc, count, tables=tables) == pk.DEVERR_BAD_BLOCK


def test_compaction_on_a_side_stream_captured_and_past_32_bits(pk):
    nodes = [40, 12]
    w = tree_workload([70, 9], nodes, 8, 8, 128, 16, "fp16", seed=23)
    t = TreeOnDevice(pk, w)
    acc, count = paths(np.random.default_rng(5), nodes)
    acc_d, count_d = torch.from_numpy(acc).cuda(), torch.from_numpy(count).cuda()
    blocks = (2 ** 31) // (8 * 16 * 128) + 16
    big = [torch.zeros((blocks, 8, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    tables, at = t.tables.clone(), blocks - 1
    spot = {}
    for i in range(2):
        for k, b in enumerate(w.block_tables[i]):
            if b >= 0:
                big[0][at], big[1][at] = t.k_cache[int(b)], t.v_cache[int(b)]
                tables[i, k], spot[int(b)] = at, at
                at -= 1
    ref = OS.compact(t.k_ref, t.v_ref, w.block_tables, w.context_lens, w.query_start, acc, count,
                     16)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        pk.compact_accepted(big[0], big[1], tables, t.lens, t.qstart, acc_d, count_d,
                            dev_err=t.err)
    g.replay()
    torch.cuda.synchronize()
    for cache, want in zip(big, ref):
        for b, where in spot.items():
            assert np.array_equal(dev_to_bits(cache[where]), want[b])
