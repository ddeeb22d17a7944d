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


def _before(wide, parts, tiles):
    """after[e]: every event that is known to be over when e happens.  A step's K is `parts` tiles, which take `tiles` places
    in turn; V's tiles have two."""
    jobs = 2 * STEPS if wide else STEPS
    step = (lambda i: i >> 1) if wide else (lambda i: i)
    last = (lambda s: 2 * s + 1) if wide else (lambda s: s)  # a step's last job
    dep = {}

    def need(e, *others):
        dep.setdefault(e, set()).update(o for o in others if o is not None)

    # the issuing thread: scores of two jobs ahead; a barrier that it commits to is reached when all it issued before is done
    qk = lambda i: [("qk", i, part) for part in range(parts)]  # noqa: E731
    order = qk(0) + qk(1)
    for i in range(jobs):
        order.append(("pv", i))
        if i + 2 < jobs:
            order += qk(i + 2)
    for a, b in zip(order, order[1:]):
        need(b, a)
    for i in range(jobs):
        for part in range(parts):
            need(("qk", i, part), ("k", step(i) * parts + part))
        need(("softmax", i), ("qk", i, parts - 1), ("softmax", i - 2) if i >= 2 else None, ("vexp", step(i)))
        need(("pv", i), ("softmax", i), ("v", step(i)))
    # the loaders: a step's factor is written as soon as the step before it is stored
    for s in range(STEPS):
        need(("kfac", s), ("k", s * parts - 1) if s else None)
        for n in range(s * parts, (s + 1) * parts):
            old = n - tiles  # the tile whose place it takes
            need(("k", n), ("kfac", s), ("k", n - 1) if n else None,
                 ("qk", last(old // parts), old % parts) if old >= 0 else None)
        need(("v", s), ("vexp", s), ("pv", last(s - 2)) if s >= 2 else None)
        need(("vexp", s), ("v", s - 1) if s else None)
    after = {}

    def walk(e):
        stack = [e]
        while stack:
            assert len(stack) < 100000, "something waits for itself"
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
@pytest.mark.parametrize("parts,tiles", [(1, 2), (2, 2), (2, 3), (2, 4)])
@pytest.mark.parametrize("word,slots", [("kfac", "KFACS"), ("vexp", "SLOTS")])
def test_a_slot_is_written_after_its_last_reader(word, slots, parts, tiles, wide):
    n = _constant(slots)
    after, jobs = _before(wide, parts, tiles)
    for s in range(n, STEPS):
        for i in jobs[s - n]:
            assert ("softmax", i) in after[(word, s)], "step %d's %s may overwrite step %d's before job %d has read it" % (
                s, word, s - n, i)


def test_the_model_sees_a_slot_too_few():
    after, jobs = _before(False, 1, 2)
    assert all(("softmax", s - 5) in after[("kfac", s)] for s in range(5, STEPS))
    assert any(("softmax", s - 4) not in after[("kfac", s)] for s in range(4, STEPS))


@pytest.mark.parametrize("wide", [False, True], ids=["one half", "two halves"])
@pytest.mark.parametrize("parts,tiles", [(1, 2), (2, 2), (2, 3), (2, 4)])
def test_no_role_waits_for_itself(parts, tiles, wide):
    """What a K or V tile waits for does not wait for that tile."""
    after, _ = _before(wide, parts, tiles)
    assert all(e not in before for e, before in after.items())
    assert {e[1] for e in after if e[0] == "pv"} == set(range(2 * STEPS if wide else STEPS))
