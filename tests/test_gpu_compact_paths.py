"""A path whose later positions climb from below 0 is reported, and no page of a slot below the
sequence's first is looked up for it."""
import numpy as np
import pytest
import torch

import speculative_decoding_verification_81_gb300 as sv

pytestmark = pytest.mark.gpu


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device="cuda")


def test_a_path_that_climbs_from_below_zero():
    gen = torch.Generator(device="cuda").manual_seed(1)
    k = torch.randn((9, 2, 8, 64), generator=gen, device="cuda").to(torch.bfloat16)
    v = torch.randn((9, 2, 8, 64), generator=gen, device="cuda").to(torch.bfloat16)
    before = [k.clone(), v.clone()]
    table, prefix = i32([[3, 1, 5, 8], [0, 2, 4, 7]]), i32([20, 10])
    path = i32([[0, -40, -30, 5], [0, 2, 5, -1]])
    st = i32([-7, -7])
    lens = sv.sv_compact_kv_paged(k, v, table, prefix, i32([3, 2]), path, seq_status=st)
    torch.cuda.synchronize()
    assert lens.tolist() == [20, 13] and st.tolist() == [sv.SV_ERR_BAD_INPUT, sv.SV_OK]
    for now, old in zip((k, v), before):
        for page in (3, 1, 5, 8):
            assert torch.equal(now[page], old[page])
        flat = [t[table[1].long()].transpose(1, 2).reshape(32, 2, 64) for t in (now, old)]
        assert torch.equal(flat[0][11], flat[1][12]) and torch.equal(flat[0][12], flat[1][15])
