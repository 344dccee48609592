"""Draft verification by clusters of CTAs: a CTA's shared memory is written by
another one only after it has started.  The order is held to in the source, as
no run can show a store that came too early; clusters of every size are run
with calls close behind one another, so that their CTAs start at odd times."""

import os
import re

import pytest
import torch

import paged_kv_cache_394_b200

KERNEL = os.path.join(os.path.dirname(paged_kv_cache_394_b200.__file__), "csrc",
                      "verify_draft.cu")


def test_every_cta_is_known_to_run_before_a_remote_store():
    with open(KERNEL) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    body = text[text.index("verify_draft_kernel(const VerifyParams"):]
    first = body.index("map_shared_rank")
    arrive, wait = (body.find("cluster_%s_started()" % w) for w in ("arrive", "wait"))
    assert 0 <= arrive < body.index("grid_dependency_wait()") < wait < first
    # no CTA leaves, and none waits for less, between the two halves
    assert "return" not in body[arrive:first]
    assert not re.search(r"if \(rank\b[^)]*\)[^}]*cluster_(arrive|wait)_started", body[:first])


@pytest.mark.gpu
@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("vocab", [1500, 5000, 9001, 40000])   # clusters of 1, 2, 4 and 8 CTAs
def test_calls_close_behind_one_another(vocab, draft):
    from paged_kv_cache_394_b200 import pagedkv as pk

    from test_gpu_verify import Case

    # 37 sequences: 37 times 8 CTAs are all that fit at once, so that a call's
    # clusters start as the ones before them leave
    c = Case([256, 1, 9, 0, 30] * 7 + [5, 80], vocab, "bf16", draft, vocab)
    assert c.run(pk) == 0
    first = [x.clone() for x in (c.accepted, c.count, c.next)]
    c.check()
    outs = [[torch.full_like(x, 77) for x in first] for _ in range(24)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for o in outs:
            pk.verify_draft(*o, c.target, *c.inputs, c.width, draft_probs=c.draft, dev_err=c.err)
    for replay in range(2):
        for o in outs:
            for x in o:
                x.fill_(77)
        g.replay()
        torch.cuda.synchronize()
        assert int(c.err.item()) == 0
        for o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, first))
    # the same calls without a graph
    for o in outs:
        pk.verify_draft(*o, c.target, *c.inputs, c.width, draft_probs=c.draft, dev_err=c.err)
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, first))
