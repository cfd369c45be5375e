"""The exchanges between the four softmax warps of the single-token attention kernel (csrc/gdn_attn_decode.cu), read from
its source: each warp writes its part of an array in shared memory and reads all four parts, and the four run freely
between their barriers. So between a warp's read of an array and anyone's next write of it there has to be a barrier of
the four, and between a write and a read as well. The steps of the role are taken from the source in its order
(the loop over a unit's tiles with the branch that moves the maximum taken or not, then the unit's end) and walked for
units of one, two and three tiles after one another."""
import itertools
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_linear_gdn_gb300",
                      "csrc", "gdn_attn_decode.cu")
BARRIER = r"any_of_128\(|sync_128\("


def events(text):
    """('barrier',), ('write', array), ('read', array) in the order of the text."""
    out = []
    for line in text.splitlines():
        line = line.split("//")[0]
        if re.search(BARRIER, line):
            out.append(("barrier", None))
        for array in ("s_red", "s_sum"):
            if re.search(array + r"\[warp \* 16 \+ h\] = ", line):
                out.append(("write", array))
            elif array + "[" in line:
                out.append(("read", array))
    return out


def role():
    """(steps of a tile before the branch, of the branch, of a unit's end)."""
    src = open(SOURCE).read()
    src = src[src.index("---- softmax: thread = key of the tile"):]
    src = src[:src.index("if (s_fail)")]
    branch, end = src.index("if (any_of_128(above"), src.index("the unit's sums, then its rows")
    after = src.index("split_off(a0, a1)")
    return events(src[:branch]), events(src[branch:after]), events(src[end:])


def hazards(steps):
    """Accesses that two warps may make in either order: a write after a read, or a read after a write, of one array with
    no barrier between."""
    last = {}
    for what, array in steps:
        if what == "barrier":
            last = {}
            continue
        before = last.get(array, set())
        if what == "write" and "read" in before or what == "read" and "write" in before:
            yield what, array
        last.setdefault(array, set()).add(what)


def test_the_role_is_found():
    before, branch, end = role()
    assert before == []
    assert branch[0] == ("barrier", None) and ("write", "s_red") in branch and ("read", "s_red") in branch
    assert [w for w, _ in end if w != "barrier"].count("write") == 1 and ("barrier", None) in end


@pytest.mark.parametrize("units", list(itertools.product([1, 2, 3], repeat=2)))
def test_every_exchange_has_its_barriers(units):
    before, branch, end = role()
    vote = branch[:1]            # the vote of every tile is a barrier
    stop = branch[1:]            # (where the maximum moves, a second vote and an exchange)
    for moved in itertools.product([False, True], repeat=sum(units)):
        steps, i = [], 0
        for tiles in units:
            for _ in range(tiles):
                steps += before + vote + (stop if moved[i] else [])
                i += 1
            steps += end
        assert list(hazards(steps)) == []


def test_a_shared_array_without_a_barrier_is_found():
    before, branch, end = role()
    one = [(w, "s_red" if a else a) for w, a in before + branch + end]
    assert list(hazards(one)) == [("write", "s_red")]
