"""The way out of the few-row attention's clusters when a copy is lost, on the
CPU: a model of the order of events, and that the kernel's source keeps it.

A CTA that waits for its K/V copy gives up after one wait's limit, waits as
long again for each copy in flight, and only then sends its shares to the
other CTAs, which began to wait for them as long before.  A store to a CTA
that has left is undefined, so none may leave before all shares have landed: a
CTA that gave up waiting for them stays until every other has sent."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = os.path.join(ROOT, "speculative_decoding_verification_81_gb300", "csrc", "sv_chunk_few.cu")
LIMIT = 1.0


def play(lost, depth, flight, closing):
    """Exit time of each CTA, and when each share lands at it; lost: copies that never land, by CTA."""
    sent = [0.01 + (LIMIT * (1 + depth) if x else 0.0) for x in lost]  # the wait, and one for each copy in flight
    landed = [s + flight for s in sent]
    out = []
    for own in sent:
        everything = max(landed)
        joined = everything <= own + LIMIT
        end = max(own, everything) if joined else own + LIMIT
        out.append((end, joined))
    if closing:  # a CTA that gave up stands at the barrier until the others stand there or have left, after their sends
        there = max(max(s, end) for s, (end, _) in zip(sent, out))
        out = [(end, True) if joined else (min(max(there, everything), there + LIMIT), False) for end, joined in out]
    out = [end for end, _ in out]
    return out, landed


@pytest.mark.parametrize("n", [2, 4, 16])
@pytest.mark.parametrize("depth", [2, 4])
@pytest.mark.parametrize("flight", [0.0, 1e-6, 0.5])
def test_no_share_is_sent_to_a_cta_that_has_left(n, depth, flight):
    for which in ([], [0], [n - 1], list(range(n)), list(range(1, n))):
        lost = [i in which for i in range(n)]
        ends, landed = play(lost, depth, flight, closing=True)
        assert min(ends) >= max(landed)
    ends, landed = play([True] + [False] * (n - 1), depth, flight, closing=False)
    assert min(ends) < max(landed)  # without the closing barrier the others had left


def kernel_body():
    s = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    at = s.index("chunk_few_kernel(const FewParams p) {")
    depth, i = 0, s.index("{", at)
    for j in range(i, len(s)):
        depth += {"{": 1, "}": -1}.get(s[j], 0)
        if depth == 0:
            return s[i + 1:j]


def test_the_kernel_has_one_way_out_behind_its_sends():
    body = kernel_body()
    sends = [m.start() for m in re.finditer(r"\bsend_f2\(", body)]
    begun = [m.start() for m in re.finditer(r"\bcluster_wait\(\)", body)]
    joined = body.index("late = !warp_wait_bounded(&joined, 0)")
    assert len(sends) == 2 and len(begun) == 1 and begun[0] < min(sends) and max(sends) < joined
    # no return but those of the lambdas, which return to the body
    assert not re.search(r"\breturn\b", re.sub(r"= \[&\].*?\n    +\};", "", body, flags=re.S))
    # the end of the body, in no other block: a warp that gave up stays
    assert re.search(r"\n    if \(late\) \{\s*cluster_sync_any\(\);\s*warp_wait_bounded\(&joined, 0\);\s*\}\s*$", body)


def test_copies_in_flight_are_waited_for_from_the_lost_one_on():
    body = kernel_body()
    lost = body[body.index("lost = true;"):]
    loop = re.match(r"lost = true;\s*for \(int k = i; k < min\(n, i \+ kDepth\); \+\+k\) \{\s*warp_wait_bounded", lost)
    assert loop, lost[:300]
