"""A chunk attention call's number, its arrival counters and the report of a wait
that gave up, compiled for the host from the kernels' header: calls of any
grids over one workspace, their CTAs in any order, some of them giving up.

A cut item's CTAs each count one arrival; the one that reads nc - 1 merges.  A
CTA that gives up counts none for the items left to it."""
import ctypes
import itertools
import os
import random
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_81_gb300", "csrc")
SRC = r"""
#include "sv_chunk_call.h"
using namespace sv::chunk;
typedef unsigned long long u64;
extern "C" u64 c_share(int cta, int grid) { return call_share(cta, grid); }
extern "C" u64 c_number(u64 shares) { return call_number(shares); }
extern "C" u64 c_tag(u64 call) { return call_tag(call); }
extern "C" int c_counters(u64 call, int grid, int cta) { return counters_of(call, grid, cta); }
extern "C" int c_max_grid() { return kCallShares; }
extern "C" int c_bytes(int grid) { return kCallBytes + 2 * grid * kCtaCounters * (int)sizeof(int); }
"""


@pytest.fixture(scope="module")
def C(tmp_path_factory):
    d = tmp_path_factory.mktemp("chunk_call")
    (d / "shim.cpp").write_text(SRC)
    subprocess.check_call(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-fsanitize=undefined",
                           "-fno-sanitize-recover", "-static-libubsan", f"-I{CSRC}", str(d / "shim.cpp"),
                           "-o", str(d / "shim.so")])
    L = ctypes.CDLL(str(d / "shim.so"))
    u64 = ctypes.c_ulonglong
    L.c_share.restype = L.c_number.restype = L.c_tag.restype = u64
    L.c_number.argtypes = L.c_tag.argtypes = [u64]
    L.c_counters.argtypes = [u64, ctypes.c_int, ctypes.c_int]
    return L


def test_every_cta_of_a_call_reads_its_number(C):
    rng = random.Random(1)
    word = 0
    for call in range(400):
        grid = rng.choice([1, 2, 3, 16, 128, 151, 152, C.c_max_grid() - 1, C.c_max_grid()])
        ctas = list(range(grid))
        rng.shuffle(ctas)
        for c in ctas:  # each reads the word as it adds its share
            assert C.c_number(word) == call
            word += C.c_share(c, grid)
    assert word == 400 * C.c_max_grid()


def test_numbers_do_not_wrap(C):
    """A call every microsecond for a century is below 2^52 calls."""
    word = (1 << 52) * C.c_max_grid() - C.c_max_grid()
    assert C.c_number(word) == (1 << 52) - 1 and C.c_number(word + 1) == (1 << 52) - 1


def test_the_zeroed_part_holds_everything(C):
    assert C.c_bytes(152) <= 64 * 1024 and C.c_bytes(1020) <= 64 * 1024 < C.c_bytes(1021)


def items(rng, grid):
    """Cut items as a call's ranges make them: from CTA c_first on, over nc CTAs, each starting where none other does."""
    out, c = [], 0
    while c < grid - 1:
        nc = rng.randint(1, min(5, grid - c))
        if nc > 1:
            out.append((c, nc))
        c += nc - rng.randint(0, 1) if nc > 1 else 1
    return [x for i, x in enumerate(out) if x[0] not in {y[0] for y in out[:i]}]


def play_call(rng, cut, grid, counters, base_of, reset, gone):
    """One call's arrivals in any order; returns the items that were merged, each with how many had arrived."""
    merged = []
    todo = [(c_first + i, n) for n, (c_first, nc) in enumerate(cut) for i in range(nc)]
    rng.shuffle(todo)
    arrived = [0] * len(cut)
    for cta, n in todo:
        if cta in gone:
            continue
        c_first, nc = cut[n]
        at = base_of(c_first) + 3  # one of its eight
        before, counters[at] = counters[at], counters[at] + 1
        arrived[n] += 1
        if before == nc - 1:
            merged.append((n, arrived[n]))
            if reset:
                counters[at] = 0
    return merged


@pytest.mark.parametrize("sets", [True, False])
def test_a_call_after_one_that_gave_up_merges_right(C, sets):
    """With a set for each parity every item of a sound call is merged once, by
    its last arrival.  With one set that the last arrival resets, as it was
    before, calls after one that gave up merge early or never."""
    rng = random.Random(2)
    grid = 24
    counters = [0] * (2 * grid * 8)
    wrong = 0
    for call in range(600):
        cut = items(rng, grid)
        gone = set(rng.sample(range(grid), rng.randint(1, 3))) if rng.random() < 0.2 else set()
        if sets:
            own = C.c_counters(call, grid, 0)
            assert not any(counters[own:own + grid * 8])  # zeros when it begins
            for c in range(grid):  # (at any time of the call: nobody counts in that set)
                at = C.c_counters(call + 1, grid, c)
                counters[at:at + 8] = [0] * 8
            base = lambda c: C.c_counters(call, grid, c)
        else:
            base = lambda c: c * 8
        merged = play_call(rng, cut, grid, counters, base, not sets, gone)
        if not gone:
            wrong += sorted(merged) != [(n, nc) for n, (_, nc) in enumerate(cut)]
    assert (wrong == 0) == sets


def test_the_sets_of_a_call_do_not_overlap(C):
    for grid in (1, 5, 152):
        at = [C.c_counters(p, grid, c) for p in (0, 1) for c in range(grid)]
        assert sorted(at) == list(range(0, 2 * grid * 8, 8))
        assert [C.c_counters((1 << 52) + p, grid, c) for p in (0, 1) for c in range(grid)] == at


@pytest.mark.parametrize("looks", [True, False])
def test_a_timeout_is_the_last_word(C, looks):
    """The two writers of a status in every order of their steps, a sequence's
    warp (status, then a look at gave_up) and a CTA that gives up (gave_up,
    then every status): the status is TIMEOUT in the end.  Without the look it
    may be OK."""
    tag = C.c_tag(7)

    def writer(m):
        m["status"] = "OK"
        yield
        seen = looks and m["gave_up"] == tag
        yield
        if seen:
            m["status"] = "TIMEOUT"
        yield

    def quitter(m):
        m["gave_up"] = tag
        yield
        m["status"] = "TIMEOUT"
        yield

    ends = set()
    for order in set(itertools.permutations("www" "qq")):
        m = {"status": "of an earlier call", "gave_up": C.c_tag(6)}  # the call before gave up too
        who = {"w": writer(m), "q": quitter(m)}
        for x in order:
            next(who[x])
        ends.add(m["status"])
    assert ends == ({"TIMEOUT"} if looks else {"OK", "TIMEOUT"})


def test_an_earlier_calls_timeout_is_not_this_ones(C):
    assert len({C.c_tag(k) for k in range(100)} | {0}) == 101  # 0: none ever
