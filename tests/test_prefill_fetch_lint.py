"""Static check, on the CPU, of how the prefill attention's fetch warp hands a 4-bit tile over (fetch_unit).

The word that says which keys of a tile have no page is an ordinary store; an asynchronous copy's arrival on a barrier
(cp.async.mbarrier.arrive.noinc) releases the copies and no ordinary store.  So
  F1  between the store and the arrivals of the tile's copies its lane makes a plain arrival, which releases it, on every path;
  F2  raw_full is initialised with what arrives on it: that one, and either each lane's (lane 0's with the bytes to expect) or
      each lane's copies'.
"""
from __future__ import annotations

import re

import pytest

from test_attn_fence_lint import body, source

LANES = 32
PLAIN = r"(?<!\w)mbar_arrive\(bar\)"
STORE = r"sm\.gone\[[^\]]*\] = gone;"


def split(b: str):
    """(what precedes the branch on `whole` from the wait for room on, its whole branch, the other one)."""
    start = b.index("sm.raw_empty[to]")
    at = b.index("if (whole) {", start)
    other = b.index("} else {", at)
    end = b.index("cp.async.mbarrier.arrive", other)
    return b[start:at], b[at:other], b[other:b.index("\n", end)]


def problems(src: str):
    out = []
    before, whole, ragged = split(body(src, "fetch_unit"))
    stores = list(re.finditer(STORE, before))
    if len(stores) != 1 or len(re.findall(STORE, whole + ragged)):
        return ["F1"]
    # one block of lane 0: the store where the tile begins, then the arrival
    if not re.search(r"if \(lane == 0\) \{\s*if \(kv == 0\) " + STORE + r"\s*" + PLAIN + r";\s*\}", before):
        out.append("F1")
    first = 1 if re.search(PLAIN, before) else 0
    by_lanes = LANES if re.search(r"if \(lane == 0\) mbar_arrive_expect_tx\(bar, [^;]*;\s*else " + PLAIN, whole) else 0
    by_copies = LANES if re.search(r"cp\.async\.mbarrier\.arrive\.noinc", ragged) and not re.search(PLAIN, ragged) else 0
    count = re.search(r"mbar_init\(&sm\.raw_full\[i\], (\d+)\)", src)
    if not count or by_lanes != LANES or by_copies != LANES or int(count.group(1)) != first + LANES:
        out.append("F2")
    return out


def test_missing_pages_are_told_by_a_release():
    assert problems(source()) == []


@pytest.mark.parametrize("was,now,rule", [("mbar_arrive(bar);\n            }", "}", "F1"), ("mbar_init(&sm.raw_full[i], 33)", "mbar_init(&sm.raw_full[i], 32)", "F2"),
                                          ("else mbar_arrive(bar);", "", "F2")])
def test_what_is_missing_is_found(was, now, rule):
    """Planted in copies of the text."""
    src = source()
    assert src.count(was) == 1
    assert rule in problems(src.replace(was, now))
