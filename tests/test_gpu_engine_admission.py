"""Admission beside drafted steps: blocks kept for the trees of what was just
admitted, a drafter that fails, and the token budget."""

import pytest

pytestmark = pytest.mark.gpu


def chain(n):
    return [-1] + list(range(n - 1))


def batcher(num_blocks, drafter, **more):
    from paged_kv_cache_394_b200 import engine as E

    return E.ContinuousBatcher(num_blocks, 16, 4, 2, 64, vocab_size=50, drafter=drafter, **more)


def request(arrival, prompt, output, samples=1):
    from paged_kv_cache_394_b200 import engine as E

    return E.Request(0, prompt, output, arrival=arrival, samples=samples)


# two requests of a block each, whose trees take two blocks more each: 6 blocks in all
@pytest.mark.parametrize("blocks,together", [(5, False), (6, False), (8, True)])
def test_a_tight_pool_keeps_blocks_for_the_first_trees(blocks, together):
    b = batcher(blocks, lambda sid, n: chain(32), max_draft=32, max_model_len=64)
    for _ in range(2):
        b.submit(request(0, 16, 8))
    at_once = 0
    for _ in range(40):
        rec = b.step()
        at_once = max(at_once, len(rec.decoded))
        if b.idle():
            break
    assert b.idle() and b.alloc.num_free() == blocks
    assert at_once == (2 if together else 1)


def test_blocks_are_kept_for_every_sample():
    # the first trees of 4 sequences may take 3 blocks each, and 13 are free, 2 of them
    # for the second prompt
    b = batcher(15, lambda sid, n: chain(32), max_draft=32, max_model_len=64)
    b.submit(request(0, 20, 6, samples=3))
    b.submit(request(0, 20, 6))
    first = b.step()
    assert len(first.admitted) == 1 and len(first.forked) == 2
    for _ in range(40):
        b.step()
        if b.idle():
            break
    assert b.idle() and b.alloc.num_free() == 15


@pytest.mark.parametrize("bad", [[0], [-1, 1], [], [-1] + [0] * 40, None])
def test_a_failing_drafter_loses_no_request(bad):
    state = {"bad": False}

    def drafter(sid, n):
        if state["bad"]:
            if bad is None:
                raise ValueError("no draft")
            return bad
        return chain(3)

    b = batcher(40, drafter, max_draft=8, max_model_len=64)
    b.submit(request(0, 10, 30))
    b.submit(request(2, 10, 5))
    b.step()
    b.step()
    free, lens = b.alloc.num_free(), b.alloc.context_lens(list(b.running))
    state["bad"] = True
    for _ in range(2):
        with pytest.raises(ValueError):
            b.step()
        assert len(b.waiting) == 1 and b.next_seq == 1 and b.step_index == 2
        assert b.alloc.num_free() == free
        assert b.alloc.context_lens(list(b.running)) == lens
    state["bad"] = False
    rec = b.step()
    assert [sid for sid, _ in rec.admitted] == [1]
    while not b.idle():
        b.step()
    assert b.alloc.num_free() == 40


@pytest.mark.parametrize("budget,most", [(40, 5), (8, 1), (6, 1), (400, 16)])
def test_trees_keep_to_the_token_budget(budget, most):
    b = batcher(200, lambda sid, n: chain(16), max_draft=16, max_num_batched_tokens=budget,
                max_model_len=64)
    for _ in range(8):
        b.submit(request(0, 5, 12))
    eight = 0
    while not b.idle():
        rec = b.step()
        if len(rec.decoded) == 8:
            eight += 1
            assert [len(t) for t in rec.parents] == [most] * 8
        if rec.decoded:
            drafted = sum(len(t) for t in rec.parents)
            assert drafted <= max(budget, len(rec.decoded))
            assert drafted + rec.prefill_tokens <= max(budget, len(rec.decoded))
        assert all(1 <= k <= len(t) for k, t in zip(rec.kept, rec.parents))
    assert eight > 0 or budget < 40
    assert b.alloc.num_free() == 200
