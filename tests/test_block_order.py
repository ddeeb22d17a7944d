"""What the tcgen05 block attention's barriers order, modelled on the CPU: nothing that a step leaves for another role may be
overwritten by a later step before that role is known to have read it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "kv_cache_decode_flash_gb300", "csrc")
STEPS = 24


def _constant(name):
    src = open(os.path.join(CSRC, "k_cross_tc.cu")).read()
    return int(re.search(r"constexpr int %s = (\d+);" % name, src).group(1))


def _before(wide):
    """after[e]: every event that is known to be over when e happens."""
    jobs = 2 * STEPS if wide else STEPS
    step = (lambda i: i >> 1) if wide else (lambda i: i)
    last = (lambda s: 2 * s + 1) if wide else (lambda s: s)  # a step's last job
    dep = {}

    def need(e, *others):
        dep.setdefault(e, set()).update(o for o in others if o is not None)

    # the issuing thread: scores of two jobs ahead; a barrier that it commits to is reached when all it issued before is done
    order = [("qk", 0), ("qk", 1)]
    for i in range(jobs):
        order.append(("pv", i))
        if i + 2 < jobs:
            order.append(("qk", i + 2))
    for a, b in zip(order, order[1:]):
        need(b, a)
    for i in range(jobs):
        need(("qk", i), ("k", step(i)))
        need(("softmax", i), ("qk", i), ("softmax", i - 2) if i >= 2 else None, ("vexp", step(i)))
        need(("pv", i), ("softmax", i), ("v", step(i)))
    # the loaders: two stages each; a step's factor is written as soon as the step before it is stored
    for tile, word, product in (("k", "kfac", "qk"), ("v", "vexp", "pv")):
        for s in range(STEPS):
            need((tile, s), (word, s), (product, last(s - 2)) if s >= 2 else None)
            need((word, s), (tile, s - 1) if s else None)
    after = {}

    def walk(e):
        stack = [e]
        while stack:
            x = stack[-1]
            todo = [d for d in dep.get(x, ()) if d not in after]
            if todo:
                stack.extend(todo)
                continue
            after[x] = set().union(*[after[d] | {d} for d in dep.get(x, ())]) if dep.get(x) else set()
            stack.pop()
        return after[e]

    for e in list(dep):
        walk(e)
    return after, [[i for i in range(jobs) if step(i) == s] for s in range(STEPS)]


@pytest.mark.parametrize("wide", [False, True], ids=["one half", "two halves"])
@pytest.mark.parametrize("word,slots", [("kfac", "KFACS"), ("vexp", "SLOTS")])
def test_a_slot_is_written_after_its_last_reader(word, slots, wide):
    n = _constant(slots)
    after, jobs = _before(wide)
    for s in range(n, STEPS):
        for i in jobs[s - n]:
            assert ("softmax", i) in after[(word, s)], "step %d's %s may overwrite step %d's before job %d has read it" % (
                s, word, s - n, i)


def test_the_model_sees_a_slot_too_few():
    after, jobs = _before(False)
    assert all(("softmax", s - 5) in after[("kfac", s)] for s in range(5, STEPS))
    assert any(("softmax", s - 4) not in after[("kfac", s)] for s in range(4, STEPS))
