"""What a wait that gave up leaves and says: every sequence of the call is
reported, and the workspace serves the next call as it is.  No wait is made to
run out: the host sets what such a call would have left in the workspace.

The workspace begins with two 64-bit words for each of the two forms (4096 for
each call of the form that has begun; the number + 1 of its last call in which a
wait gave up), and from byte 256 on has two sets of arrival counters, 8 for
each SM, which calls of the general form use in turn."""
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv
from test_gpu_chunk import Case, near

pytestmark = pytest.mark.gpu
EMPTY = [(0, 0)] * 33  # more sequences than the form for few rows takes
FORMS = {
    "few rows": ([(300, 2), (40, 3), (0, 1)], dict(hq=8, hkv=2)),
    "cut items": ([(9000, 70), (20, 1)], dict(hq=8, hkv=1)),
    "cut items of few rows": ([(20000, 1), (700, 1)] + EMPTY, dict(hq=32, hkv=8, page_size=64)),
    "whole items": ([(5, 1)] * 60, dict(hq=8, hkv=2, d=64)),
}


def workspace(c):
    n = sv.sv_workspace_size(sv.SV_OP_CHUNK_ATTENTION, 0, 0, Hq=c.q.shape[1], Hkv=c.k.shape[1], D=c.q.shape[2])
    ws = torch.full((n,), 0xa5, dtype=torch.uint8, device="cuda")
    ws[:1 << 16].zero_()
    return ws


@pytest.mark.parametrize("calls", [0, 1, 2, 7])
@pytest.mark.parametrize("form", FORMS)
def test_every_sequence_is_reported_and_the_next_call_is_right(form, calls):
    lens, kw = FORMS[form]
    c = Case(lens, seed=50, **kw)
    ws, want = workspace(c), c.want()
    few = form == "few rows"
    words = ws[16 * few:16 * few + 16].view(torch.int64)
    for _ in range(calls):
        c.run(ws=ws)
    assert words.tolist() == [4096 * calls, 0]
    words[1] = calls + 1  # a CTA of the coming call has given up
    st = torch.full((len(lens),), -7, dtype=torch.int32, device="cuda")
    c.run(ws=ws, seq_status=st)
    assert (st == sv.SV_ERR_TIMEOUT).all()
    near(*c.check(ws=ws), want)  # (its statuses are OK)
    assert words.tolist() == [4096 * (calls + 2), calls + 1]


@pytest.mark.parametrize("calls", [1, 2, 3, 8])
@pytest.mark.parametrize("left", [1, -1, 3, 1 << 20])
@pytest.mark.parametrize("form", ["cut items", "cut items of few rows"])
def test_arrivals_that_a_call_left_do_not_count_in_the_next(form, left, calls):
    lens, kw = FORMS[form]
    c = Case(lens, seed=51, **kw)
    ws = workspace(c)
    for _ in range(calls):
        c.run(ws=ws)
    n = 8 * torch.cuda.get_device_properties(0).multi_processor_count
    counters = ws[256:256 + 8 * n].view(torch.int32).view(2, n)
    counters[(calls - 1) & 1] = left  # the set of the last call, as if it had stopped anywhere
    ws[:16].view(torch.int64)[1] = calls
    for _ in range(3):
        c.check(ws=ws)


def test_both_forms_and_head_sizes_take_turns_on_one_workspace():
    cases = [Case(*FORMS[f][:1], seed=52 + i, **FORMS[f][1]) for i, f in enumerate(FORMS)]
    ws = max((workspace(c) for c in cases), key=len)
    want = [c.run() for c in cases]
    order = [0, 1, 1, 2, 3, 0, 0, 2, 1, 3, 3, 2, 2, 0, 1, 0, 1, 1, 1, 2]
    for i in order:
        out, lse = cases[i].run(ws=ws)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])
    few = order.count(0)
    assert ws[:32].view(torch.int64).tolist() == [4096 * (len(order) - few), 0, 4096 * few, 0]
