"""The ring of K tiles of mk_attn_mass (csrc/ops/mk_attn_mass.cu) as a model, on
the CPU: a producer and two warps of MMAs that wait for every tile, of which each
takes every second one.  All orders in which they can run are gone through.

A wait asks for a parity, so it passes if the barrier has completed one phase
more than the waiter has seen, and never again once it has completed two."""
import os
import re

import pytest

SRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "moe_decode_megakernel_gb300", "csrc", "ops",
                   "mk_attn_mass.cu")


def overtaken(stages, tiles, count, both):
    """Whether some order of events completes a phase of `full` twice behind a warp's back.  count: arrivals that free a
    stage; both: a warp arrives for the other's tiles, too (once its wait has passed), not only for its own (once
    their MMAs are done, which may be any time later)."""
    # tiles that were filled, each warp's next tile, and of its own tiles before that the first one not yet handed back
    start = (0, 0, 0, 0, 1)
    seen, todo = {start}, [start]
    while todo:
        filled, at0, at1, done0, done1 = state = todo.pop()
        at, done = (at0, at1), (done0, done1)

        def arrivals(t):
            n = sum(1 for w in range(2) if t % 2 == w and done[w] > t)
            return n + (sum(1 for w in range(2) if t % 2 != w and at[w] > t) if both else 0)

        nexts = []
        if filled < tiles and (filled < stages or arrivals(filled - stages) >= count):
            nexts.append((filled + 1, *state[1:]))
        for w in range(2):
            t = at[w]
            if t < tiles:
                phases = (filled - 1 - t % stages) // stages + 1 if filled > t % stages else 0  # of full[t % stages]
                if phases > t // stages + 1:
                    return True
                if phases == t // stages + 1:
                    nexts.append((filled, *(x + (i == w) for i, x in enumerate(at)), *done))
            if done[w] < at[w]:
                nexts.append((filled, *at, *(x + 2 * (i == w) for i, x in enumerate(done))))
        if not nexts and (filled, at0, at1) != (tiles, tiles, tiles):
            raise AssertionError(f"nothing can go on from {state}")
        for s in nexts:
            if s not in seen:
                seen.add(s)
                todo.append(s)
    return False


def kernel():
    """(arrivals that free a stage, whether a warp hands back the other group's tiles) of the kernel."""
    with open(SRC) as f:
        src = f.read()
    count = int(re.search(r"mbar_init\(&c\.empty\[i\], (\d+)\)", src)[1])
    body = src[src.index("bool issue_mmas("):src.index("bool sum_slots(")]
    loop = body[body.index("wait(c, &c.full[k.stage], k.phase, a.status)"):]
    own = loop.index("commit_if(lead, empty + k.stage * 8)")
    other = re.search(r"\}\s*else\s*\{\s*arrive_if\(lead, empty \+ k\.stage \* 8\);", loop)
    assert 0 < own < loop.index("k.advance")
    return count, other is not None and other.start() > own


@pytest.mark.parametrize("stages", [3, 4, 5, 6, 8])
def test_no_warp_is_overtaken(stages):
    count, both = kernel()
    assert not overtaken(stages, 3 * stages + 2, count, both)


def test_the_model_sees_a_warp_overtaken():
    # a stage freed by its tile's own warp alone
    assert all(overtaken(stages, 3 * stages + 2, 1, False) for stages in (3, 4, 5, 6, 8))
