"""The order that the barriers of the tensor-core tree kernel leave open (CPU: a model of its
roles, gone through in every interleaving).

The value warp notes in a flag that a unit's values were cleaned, the softmax warps read it
when they write the unit's rows.  Units follow one another in a ring of flags, whose number of
places is read from the kernel's source."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "context_paged_decode_gb300", "csrc", "dcp_tree_tc.cu")
UNITS = 6


def programs(tiles):
    """Each role's steps: ("wait", event), ("post", event), ("write" | "read", unit)."""
    values, products = [], []
    softmax = [[], []]                         # two of the eight warps, which may drift apart
    for i in range(UNITS):
        if i:
            values.append(("wait", ("qfree", i - 1)))
        values += [("post", ("q", i)), ("write", i), ("post", ("vok", i))]
        products.append(("wait", ("q", i)))
        for k in range(tiles + 1):
            if k < tiles:
                products.append(("post", ("s", i, k)))
                if k == tiles - 1:
                    products.append(("post", ("qfree", i)))
            if k == 1 and i:
                products += [("wait", ("ofree", i - 1, w)) for w in (0, 1)]
            if k:
                products.append(("wait", ("vok", i)))
                products += [("wait", ("p", i, k - 1, w)) for w in (0, 1)]
        products.append(("post", ("o", i)))
        for w, own in enumerate(softmax):
            for k in range(tiles):
                own += [("wait", ("s", i, k)), ("post", ("p", i, k, w))]
            own += [("wait", ("o", i)), ("post", ("here", i, w)), ("wait", ("here", i, 1 - w)),
                    ("read", i), ("post", ("ofree", i, w))]
    return [values, products, *softmax]


def lost(tiles, places):
    """Units whose flag a softmax warp may find overwritten."""
    roles = programs(tiles)
    posts = [[("post" == s[0]) and s[1] for s in r] for r in roles]
    where = {e: (r, n) for r, steps in enumerate(posts) for n, e in enumerate(steps) if e}
    bad, seen, todo = set(), set(), [(0,) * len(roles)]
    while todo:
        at = todo.pop()
        for r, steps in enumerate(roles):
            if at[r] == len(steps):
                continue
            kind, what = steps[at[r]]
            if kind == "wait" and at[where[what][0]] <= where[what][1]:
                continue
            if kind == "read":
                written = [s[1] for s in roles[0][:at[0]] if s[0] == "write"]
                if [u for u in written if u % places == what % places][-1] != what:
                    bad.add(what)
            nxt = at[:r] + (at[r] + 1,) + at[r + 1:]
            if nxt not in seen:
                seen.add(nxt)
                todo.append(nxt)
    assert tuple(map(len, roles)) in seen      # every role comes to its end
    return bad


@pytest.mark.parametrize("tiles", [1, 2, 3])
def test_no_flag_is_overwritten_before_it_is_read(tiles):
    text = open(SOURCE).read()
    places = int(re.search(r"constexpr int kTtFlags = (\d+);", text).group(1))
    assert not lost(tiles, places)
    assert text.count("item % kTtFlags]") == 2     # the write and the read


def test_two_places_are_too_few_for_units_of_a_tile():
    assert lost(1, 2) and not lost(1, 3)
