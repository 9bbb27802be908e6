"""The order of waits in pages_resize (csrc/pages.hip), read off its source: a schedule that goes
wrong without them cannot be asked for, so no run shows that one is missing."""
import os
import re

import draft_sampling_lossless_amd as dsl

SOURCE = os.path.join(os.path.dirname(dsl.LIB_PATH), "csrc", "pages.hip")


def body(name):
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    text = text[text.index(f"void {name}("):]
    return text[:text.index("\n}\n")]


def test_everyone_waits_for_its_loads():
    """`everyone` is a wait for a wave's own loads and atomics, then the barrier."""
    text = body("pages_resize_all")
    wait = text[text.index("auto everyone"):]
    wait = wait[:wait.index("};")]
    assert 0 < wait.index("s_waitcnt vmcnt(0)") < wait.index("__syncthreads()")


def test_counts_asked_for_are_there_before_shared_pages_are_counted_off():
    """A count passes through 0 where all who share a page leave it; counts that any wave has asked
    for before have to be there by then."""
    text = body("pages_resize_all")
    off = text.index("atomicSub(a.refs + shared")
    asked = text.rindex("first_counts();", 0, off)
    branch = text.rindex("__syncthreads_or(any)", asked, off)
    assert "everyone();" in text[branch:off]


def test_every_step_of_shared_counts_is_waited_for():
    """Between any two of: counted off, read, the last one found, read, set."""
    text = body("pages_resize_all")
    steps = [m.start() for m in re.finditer(
        r"atomicSub\(a\.refs \+ shared|count_of\(shared\[e\]\) == 0|atomicMax\(a\.refs|count_of\(shared\[e\]\) == b0|__hip_atomic_store\(a\.refs", text)]
    steps = [s for s in steps if s >= text.index("atomicSub(a.refs + shared")]
    assert len(steps) == 5
    for a, b in zip(steps, steps[1:]):
        assert "everyone();" in text[a:b]
