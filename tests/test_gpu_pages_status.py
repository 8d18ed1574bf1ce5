"""Which page ids the table call looks at: those that it hands out, and the held
ones that new rows fall into."""
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("bad", [-1, 10, 1 << 30])
def test_a_bad_page_without_new_rows_is_not_reported(bad):
    """Sequence 0 is idle with its prefix ending inside the bad page; the rows of
    1 fall into a bad page, those of 2 into the page after one, and 3 is idle
    at a page's end."""
    past, new, held = [20, 20, 32, 32], [0, 3, 5, 0], [2, 2, 3, 2]
    table = i32([[0, bad, -1], [1, bad, -1], [2, bad, 3], [bad, 4, -1]])
    st = i32([-7] * 4)
    before = table.clone()
    starts, slots, counts, free = sv.sv_build_block_tables(i32(past), i32(new), i32(held), table,
                                                           i32([9, 8, 7, 6, 5, -1, -1, -1, -1, -1]), i32([5]), 16, 9,
                                                           seq_status=st)
    torch.cuda.synchronize()
    assert st.tolist() == [sv.SV_OK, sv.SV_ERR_BAD_INPUT, sv.SV_OK, sv.SV_OK]
    assert starts.tolist() == [0, 0, 3, 8, 8] and counts.tolist() == held and free.tolist() == [5]
    assert slots.tolist() == [-1] * 3 + [3 * 16 + i for i in range(5)] + [-1]
    assert torch.equal(table, before)
