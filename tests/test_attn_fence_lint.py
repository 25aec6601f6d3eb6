"""Static check, on the CPU, of the prefill attention's roles: how they hand tensor memory and shared-memory operands
to one another.

tcgen05 operations and the async proxy are ordered between threads by fences around every hand-over:
  A1  a tensor-memory load, and an MMA issue, has a fence_after_sync between it and the wait before it;
  A2  an arrival that says that tensor memory was read or written (p_full) comes after tcgen05.wait::st and
      fence_before_sync, in this order, since the last store;
  A3  operands that threads write to shared memory (converted codes, queries, cp.async) cross into the async
      proxy (fence_smem_to_async) between the writes and the arrival that hands them over.
Function bodies are read as straight-line text; the issuing lambda counts where it is called.
"""
from __future__ import annotations

import os
import re

import pytest

from test_tcgen05_fence_lint import CSRC, function_bodies, strip_comments

PATH = os.path.join(CSRC, "kda_attn_prefill.cu")
WAIT = r"\bwait_warp\s*\(|\bslot_wait\s*\(|\bsoftmax_sync\s*\("
AFTER, BEFORE, PROXY = r"fence_after_sync\s*\(", r"fence_before_sync\s*\(", r"fence_smem_to_async\s*\("
ROLES = ("issue_products", "softmax_unit", "load_unit")


def source() -> str:
    return strip_comments(open(PATH).read())


def body(src: str, name: str) -> str:
    """The function's body without the bodies of its lambdas that issue (their calls count instead)."""
    found = [b for n, b, _ in function_bodies(src, r"__device__[^;{}()]*\b%s\s*\(" % name)]
    assert len(found) == 1, name
    b = found[0]
    m = re.search(r"auto qk = \[&\]\([^)]*\)\s*\{", b)
    if m:
        depth, i = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(b[i], 0)
            i += 1
        b = b[:m.start()] + b[i:]
    m = re.search(r"auto slot_wait = [^\n]*\n", b)   # the wait itself
    return b if not m else b[:m.start()] + b[m.end():]


def events(text: str, kinds):
    got = [(m.start(), kind) for kind, pat in kinds for m in re.finditer(pat, text)]
    return [k for _, k in sorted(got)]


def problems(src: str):
    out = []
    for name in ROLES:
        b = body(src, name)
        # A1
        last = None
        for k in events(b, (("wait", WAIT), ("after", AFTER), ("use", r"\btmem_ld32(?:_async)?\s*\(|\bqk\s*\(|\bmma_ts\s*\(|\btc::mma\s*\("))):
            if k == "use" and last != "after":
                out.append(("A1", name))
            elif k != "use":
                last = k
        # A2
        state = None
        for k in events(b, (("store", r"\btmem_st32\s*\("), ("done", r"\btmem_wait_st\s*\("), ("before", BEFORE), ("hand", r"mbar_arrive\s*\(&sm\.p_full"))):
            if k == "hand":
                if state != "before":
                    out.append(("A2", name))
                state = None
            elif k == "before":
                state = "before" if state == "done" else "early"
            else:
                state = k
    # A3: in the loaders, writes by threads and their hand-over
    b = body(src, "load_unit")
    written = False
    for k in events(b, (("write", r"cp_async_wait_all\s*\(|\*reinterpret_cast<uint4 \*>\(sm\.(?:kv|q)\["), ("proxy", PROXY),
                        ("proxy", r"return true;"),   # (the end of a branch: its hand-over has the rule to itself)
                        ("hand", r"mbar_arrive\s*\(&sm\.(?:full|q_full)"))):
        if k == "write":
            written = True
        elif k == "proxy":
            written = False
        elif written:
            out.append(("A3", "load_unit"))
            written = False
    return out


def test_roles_hand_over_behind_fences():
    src = source()
    assert problems(src) == []
    for name, pat, least in (("issue_products", r"\bmma_ts\s*\(", 1), ("issue_products", r"\bqk\s*\(", 2), ("softmax_unit", r"\btmem_ld32", 3),
                             ("softmax_unit", r"mbar_arrive\s*\(&sm\.p_full", 1), ("load_unit", PROXY, 3)):
        assert len(re.findall(pat, body(src, name))) >= least, (name, pat)   # there is something to check


def removals(name: str, pat: str):
    """The source without one of the matches in this function, for each of them."""
    src = source()
    start = src.index(function_bodies(src, r"__device__[^;{}()]*\b%s\s*\(" % name)[0][1])
    end = start + len(function_bodies(src, r"__device__[^;{}()]*\b%s\s*\(" % name)[0][1])
    for m in re.finditer(pat, src[start:end]):
        yield src[:start + m.start()] + src[start + m.end():]


@pytest.mark.parametrize("name,pat,rule", [("issue_products", r"tc::fence_after_sync\(\);", "A1"), ("softmax_unit", r"tc::fence_after_sync\(\);", "A1"),
                                           ("softmax_unit", r"tc::fence_before_sync\(\);", "A2"), ("softmax_unit", r"tmem_wait_st\(\);", "A2"),
                                           ("load_unit", r"tc::fence_smem_to_async\(\);", "A3")])
def test_a_missing_fence_is_found(name, pat, rule):
    """Planted in copies of the text: each of the function's fences taken out in turn."""
    n = 0
    for src in removals(name, pat):
        n += 1
        assert (rule, name) in problems(src), (name, pat, n)
    assert n
