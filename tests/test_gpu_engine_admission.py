"""Admission beside drafted steps: a drafter that fails."""

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
